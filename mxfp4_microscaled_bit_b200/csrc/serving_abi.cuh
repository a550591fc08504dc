// serving_abi.cuh -- the C ABI of the serving operators (include/fp4lin_serving.h): host-side
// argument checks and launches.  Part of the library's one translation unit (fp4lin.cu includes it
// last); it uses that file's host helpers.
#pragma once

#include "../../include/fp4lin_serving.h"
#include "kv_paged.cuh"
#include "kv_paged_attention.cuh"
#include "kv_paged_prefill.cuh"
#include "matvec.cuh"
#include "rmsnorm.cuh"

namespace {

// log2 of a page size, or -1 where it is none of 16, 32, 64, 128.
int page_shift(int page)
{
    return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1;
}

// Raise a kernel's dynamic shared memory once per device.
template <typename Kernel>
int raise_smem(Kernel *kern, bool *done, size_t bytes)
{
    std::lock_guard<std::mutex> lk(g_mutex);
    if (!*done) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
            cudaGetLastError();
            return FP4LIN_ERR_CUDA;
        }
        *done = true;
    }
    return FP4LIN_OK;
}

inline int launched(cudaError_t e)
{
    if (e == cudaSuccess)
        return FP4LIN_OK;
    cudaGetLastError();
    return FP4LIN_ERR_CUDA;
}

// ------------------------------------------------------------------ norm
// As many CTAs as are resident together at 128 registers a thread; they walk the rows.  8192 x 4096
// with 4 / 8 / 12 / 16 / all CTAs of 128 threads an SM: 39.2 / 39.9 / 40.9 / 40.9 / 47 us.
unsigned norm_grid(int64_t ctas, int threads, int sms)
{
    return (unsigned)std::min<int64_t>(ctas, (int64_t)sms * std::max(1, 512 / threads));
}

template <int HAD>
cudaError_t launch_norm(const NormShape &a, int sms, cudaStream_t s)
{
    const int lanes = (a.cols / 32 + 31) / 32 * 32;
    if (lanes == 32)
        return launch_pdl(rmsnorm_mxfp8_kernel<HAD, 128>, dim3(norm_grid((a.rows_pad + 3) / 4, 128, sms)), dim3(128), 0, s, a);
    const dim3 grid(norm_grid(a.rows_pad, lanes, sms));
    if (lanes <= 512)
        return launch_pdl(rmsnorm_mxfp8_kernel<HAD, 512>, grid, dim3(lanes), 0, s, a);
    return launch_pdl(rmsnorm_mxfp8_kernel<HAD, 1024>, grid, dim3(lanes), 0, s, a);
}

// ------------------------------------------------------------------ attention
// Requests of at most KVP_SPLIT_ROWS (token, head) rows are the split kernel's, which streams the
// cache at HBM speed; the others the tensor-core kernel's.  With 32 or 64 in its place, which makes the
// split kernel read the cache once for every 16 rows (us for 16 / 32 / 64; 8 kv heads, D = 128):
// 32 requests of 32 rows over 4096 keys 158 / 234 / 234, 64 of 20 rows 303 / 433 / 433, one of 32 rows
// over 32768 keys 51 / 81 / 81, 16 of 32 rows over 600 keys 28 / 58 / 58; only one of 32 rows over
// 2048 keys is better off there, 25 / 15 / 15.
constexpr int KVP_SPLIT_ROWS = 16;

struct KvPagedPlan {
    int nt, rows, tiles, chunk, S, max_rows;
    int64_t prefill_tiles;  // 0: no request can have more than KVP_SPLIT_ROWS rows
    size_t split_bytes, ws_bytes;  // the split kernel's share, and all
};

// Keys a CTA: enough CTAs for several on every SM, in multiples of a step of the CTA's warps, at most
// KVP_MAX_CHUNK (32 ragged requests of up to 32768 keys, 8 heads: 300 us with 1024, 278 with 2048, 287 with
// 4096).
KvPagedPlan plan_paged(int B, int H, int G, int max_new, int64_t max_len, int D, int sms)
{
    KvPagedPlan p{};
    const int64_t all = (int64_t)max_new * G, most = std::min<int64_t>(all, KVP_SPLIT_ROWS);
    p.max_rows = KVP_SPLIT_ROWS;
    p.prefill_tiles = all > KVP_SPLIT_ROWS ? (all + KPP_ROWS - 1) / KPP_ROWS * B * H : 0;
    // 8 rows a tile where none has more.  Next to longer requests the split kernel sees single tokens mostly,
    // of G rows: 63 of 1000 keys, 8 heads of 4, beside a prompt take 64 us so, 145 in tiles of 16.
    p.nt = (p.prefill_tiles ? G : most) <= 8 ? 1 : 2;
    p.rows = 8 * p.nt;
    p.tiles = (int)((most + p.rows - 1) / p.rows);
    const int64_t units = (int64_t)B * H * p.tiles;
    int64_t chunk = (max_len * units + (int64_t)sms * 12 - 1) / ((int64_t)sms * 12);
    chunk = (chunk + 127) / 128 * 128;
    chunk = std::min<int64_t>(std::max<int64_t>(chunk, 128), KVP_MAX_CHUNK);
    // a cluster joins up to 8 splits at once: longer splits are better than a second launch.  One request, 8
    // heads, D = 128: 2000 keys 8.1 us, with a second launch 11.9; 3900 keys 10.3 and 15.8; 16000 keys 24
    // and 51; the other way round are 16 requests of 3900 keys, 42.5 and 39.5.
    const int64_t joined = (max_len + 8 * 128 - 1) / (8 * 128) * 128;
    if (joined <= KVP_MAX_CHUNK)
        chunk = std::max(chunk, joined);
    else  // 1 / 4 requests of 32768 keys: from 256 / 512 / 1024 / 2048 on 28 / 26 / 20 / 27 and 62 / 63 / 63 / 69 us
        chunk = std::max<int64_t>(chunk, 1024);
    p.chunk = (int)chunk;
    p.S = (int)((max_len + chunk - 1) / chunk);
    // up to 8 splits are one cluster, joined in the kernel; more leave their parts in the workspace
    p.split_bytes = p.S > 8 ? (size_t)units * p.S * p.rows * (D + 4) * sizeof(float) : 0;
    p.ws_bytes = p.split_bytes;
    if (p.prefill_tiles)
        p.ws_bytes += kpp_workspace(p.prefill_tiles, sms, D);
    return p;
}

bool g_prefill_attr[kMaxDevices][2] = {};

bool paged_sizes_ok(int B, int H, int G, int D, int max_new, int64_t max_len)
{
    return B >= 1 && H >= 1 && G >= 1 && G <= 16 && (D == 64 || D == 128) && max_new >= 1 && max_len >= 1 &&
           max_len <= 0x7FFFFFFF - KVP_MAX_CHUNK && (int64_t)B * H <= 65535 && (int64_t)max_new * G <= 65535 * 8;
}

template <int D>
cudaError_t launch_paged(const KvPagedShape &a, const KvPagedPlan &p, cudaStream_t s)
{
    if (a.prefill_most) {
        cudaError_t e = launch_pdl(kv_paged_plan_kernel, dim3(1), dim3(KPP_PLAN_THREADS), 0, s, a);
        if (e == cudaSuccess)
            e = launch_pdl(kv_paged_prefill_kernel<D>, dim3((unsigned)kpp_grid(a.prefill_most, a.sms)), dim3(KPP_THREADS),
                           kpp_smem(D), s, a);
        if (e == cudaSuccess && a.max_len > KPP_MIN_BLOCKS * KPP_KEYS)  // else no tile is shared
            e = launch_pdl(kv_paged_prefill_merge_kernel<D>,
                           dim3(a.prefill_most * 9 <= a.sms ? KPP_ROWS : KPP_ROWS / KVP_WARPS,  // more than 8 parts, or not
                                (unsigned)std::min(a.prefill_most, 2 * a.sms / 3)),
                           dim3(KVP_THREADS), 0, s, a);
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.S, (unsigned)(a.B * a.H), (unsigned)p.tiles);
    cfg.blockDim = dim3(KVP_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.joined ? 2 : 1;
    const cudaError_t e = p.nt == 1 ? cudaLaunchKernelEx(&cfg, kv_paged_split_kernel<D, 1>, a)
                                    : cudaLaunchKernelEx(&cfg, kv_paged_split_kernel<D, 2>, a);
    if (e != cudaSuccess || p.S <= 8)
        return e;
    const dim3 mgrid((unsigned)std::min<int64_t>((int64_t)a.max_new * a.G, p.max_rows), (unsigned)(a.B * a.H));
    return launch_pdl(kv_paged_merge_kernel<D>, mgrid, dim3(KVP_THREADS), 0, s, a, p.rows);
}

// ------------------------------------------------------------------ matvec
// CTAs a row tile (a cluster's size): as many as fit the GPU together, two CTAs an SM.  At 32 tiles and
// 56 chunks of K, 8 / 7 / 6 / 4 CTAs a tile take 13.0 / 14.4 / 17.3 / 17.8 us (NVFP4, 5 rows); at 112
// tiles and 16 chunks, where 2 fit, 1 / 2 / 3 / 4 take 28.9 / 22.2 / 32.1 / 25.7 us (MXFP4, 16 rows).
int matvec_ranks(int64_t tiles, int nchunks, int sms)
{
    int best = 1;
    for (int r = 2; r <= 8 && tiles * r <= 2 * (int64_t)sms; ++r) {
        const int per = (nchunks + r - 1) / r;
        if ((nchunks + per - 1) / per == r)  // no CTA has nothing to do
            best = r;
    }
    return best;
}

bool g_matvec_attr[kMaxDevices][16] = {};

template <bool NV, bool X8, int HAD, int NT>
int launch_matvec(const MatvecShape &a, int tiles, int ranks, int slot, cudaStream_t s)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return FP4LIN_ERR_CUDA;
    auto *kern = matvec_kernel<NV, X8, HAD, NT>;
    const int st = raise_smem(kern, &g_matvec_attr[dev][slot], mv_smem(MV_MAX_M, MV_SEG, 1) + 1024);
    if (st != FP4LIN_OK)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * ranks));
    cfg.blockDim = dim3(MV_THREADS);
    cfg.dynamicSmemBytes = mv_smem(a.M, std::min(a.per_cta, MV_SEG), ranks);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched(cudaLaunchKernelEx(&cfg, kern, a));
}

template <bool NV, int NT>
int launch_matvec_x(const MatvecShape &a, int hadamard, int tiles, int ranks, cudaStream_t s)
{
    constexpr int base = (NV ? 0 : 6) + (NT - 1) * 3;
    if (a.xs)
        return launch_matvec<NV, true, 0, NT>(a, tiles, ranks, base, s);
    if (hadamard)
        return launch_matvec<NV, false, NV ? 16 : 32, NT>(a, tiles, ranks, base + 1, s);
    return launch_matvec<NV, false, 0, NT>(a, tiles, ranks, base + 2, s);
}

int matvec_entry(bool nv, const void *x, const uint8_t *xs, int64_t M, int64_t K, int64_t ld_x, int hadamard,
                 const uint8_t *w, const uint8_t *ws, const float *g, void *y, int64_t N, int64_t ldy, void *stream)
{
    if (!x || !w || !ws || !y || (nv && !g))
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (M < 1 || N < 1 || K < 1 || ld_x < K || ldy < N)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (hadamard != 0 && (xs || hadamard != (nv ? 16 : 32)))
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (M > MV_MAX_M || K % 64 != 0 || ld_x % (xs ? 16 : 8) != 0 || K > (1 << 24) || N > (1 << 27))
        return FP4LIN_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(ws, 16) || !aligned(y, 2) || (xs && !aligned(xs, 16)) ||
        (nv && !aligned(g, 4)))
        return FP4LIN_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    const int st = current_device(&dev);
    if (st != FP4LIN_OK)
        return st;
    MatvecShape a{};
    a.x = x;
    a.xs = xs;
    a.w = w;
    a.ws = ws;
    a.g = g;
    a.y = reinterpret_cast<__nv_bfloat16 *>(y);
    a.ld_x = ld_x;
    a.ldy = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.katoms_w = (K / (nv ? 16 : 32) + 3) / 4;
    a.katoms_x = (K / 32 + 3) / 4;
    a.nchunks = (int)((K + MV_CHUNK - 1) / MV_CHUNK);
    const int tiles = (int)((N + MV_ROWS - 1) / MV_ROWS);
    const int ranks = matvec_ranks(tiles, a.nchunks, dev->sms);
    a.mp_shift = M > 4 ? 3 : M > 2 ? 2 : M > 1 ? 1 : 0;
    a.per_cta = (a.nchunks + ranks - 1) / ranks;
    a.wide_w = aligned(w, 32);
    cudaStream_t s = as_stream(stream);
    if (nv)
        return M <= 8 ? launch_matvec_x<true, 1>(a, hadamard, tiles, ranks, s)
                      : launch_matvec_x<true, 2>(a, hadamard, tiles, ranks, s);
    return M <= 8 ? launch_matvec_x<false, 1>(a, hadamard, tiles, ranks, s)
                  : launch_matvec_x<false, 2>(a, hadamard, tiles, ranks, s);
}

bool g_table_attr[kMaxDevices] = {};

}  // namespace

extern "C" {

int rmsnorm_mxfp8(const void *x, int64_t ld_x, const void *residual, int64_t ld_r, const void *weight, float eps,
                  int hadamard, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scales, void *summed,
                  int64_t ld_s, void *stream)
{
    if (!x || !weight || !codes || !scales || (residual == nullptr) != (summed == nullptr))
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (rows < 1 || cols < 1 || ld_x < cols || (residual && (ld_r < cols || ld_s < cols)) || !(eps >= 0.0f) ||
        eps > 3.4e38f)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (hadamard != 0 && hadamard != 16 && hadamard != 32)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (cols % 32 != 0 || cols > NORM_MAX_COLS || rows > (1 << 30) || ld_x % 8 != 0 ||
        (residual && (ld_r % 8 != 0 || ld_s % 8 != 0)))
        return FP4LIN_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(codes, 16) || !aligned(scales, 16) ||
        (residual && (!aligned(residual, 16) || !aligned(summed, 16))))
        return FP4LIN_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    const int st = current_device(&dev);
    if (st != FP4LIN_OK)
        return st;
    NormShape a{};
    a.x = reinterpret_cast<const __nv_bfloat16 *>(x);
    a.r = reinterpret_cast<const __nv_bfloat16 *>(residual);
    a.w = reinterpret_cast<const __nv_bfloat16 *>(weight);
    a.s = reinterpret_cast<__nv_bfloat16 *>(summed);
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.rows_pad = (rows + 127) / 128 * 128;
    a.cols = (int)cols;
    a.ld_x = ld_x;
    a.ld_r = ld_r;
    a.ld_s = ld_s;
    a.katoms = (cols / 32 + 3) / 4;
    a.eps = eps;
    a.inv_cols = 1.0f / (float)cols;
    a.wide_x = aligned(x, 32) && ld_x % 16 == 0;
    a.wide_r = residual && aligned(residual, 32) && ld_r % 16 == 0;
    a.wide_s = residual && aligned(summed, 32) && ld_s % 16 == 0;
    a.wide_w = aligned(weight, 32);
    a.wide_c = aligned(codes, 32);
    cudaStream_t s = as_stream(stream);
    return launched(hadamard == 16   ? launch_norm<16>(a, dev->sms, s)
                    : hadamard == 32 ? launch_norm<32>(a, dev->sms, s)
                                     : launch_norm<0>(a, dev->sms, s));
}

int nvfp4_matvec(const void *x, const uint8_t *x_scales, int64_t M, int64_t K, int64_t ld_x, int hadamard,
                 const uint8_t *w_codes, const uint8_t *w_scales, const float *g_w, void *y, int64_t N, int64_t ldy,
                 void *stream)
{
    return matvec_entry(true, x, x_scales, M, K, ld_x, hadamard, w_codes, w_scales, g_w, y, N, ldy, stream);
}

int mxfp4_matvec(const void *x, const uint8_t *x_scales, int64_t M, int64_t K, int64_t ld_x, int hadamard,
                 const uint8_t *w_codes, const uint8_t *w_scales, void *y, int64_t N, int64_t ldy, void *stream)
{
    return matvec_entry(false, x, x_scales, M, K, ld_x, hadamard, w_codes, w_scales, nullptr, y, N, ldy, stream);
}

int kv_block_tables(int32_t *table, int64_t ld_table, int width, const int32_t *lens, const int32_t *new_lens, int B,
                    const int32_t *free_pages, int num_free, const int32_t *free_head, int page, int max_tokens,
                    int32_t *cu_new, int32_t *slots, int32_t *next_head, void *stream)
{
    if (!table || !lens || !new_lens || !free_pages || !free_head || !cu_new || !slots || !next_head)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (B < 1 || width < 1 || ld_table < width || num_free < 1 || max_tokens < 1 || free_head == next_head)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    const int shift = page_shift(page);
    if (shift < 0 || B > TABLE_MAX_REQUESTS || max_tokens > (1 << 30) || ((int64_t)width << shift) > 0x7FFFFFFF)
        return FP4LIN_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) ||
        !aligned(free_head, 4) || !aligned(cu_new, 4) || !aligned(slots, 4) || !aligned(next_head, 4))
        return FP4LIN_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    int st = current_device(&dev);
    if (st != FP4LIN_OK)
        return st;
    int ordinal = 0;
    if (cudaGetDevice(&ordinal) != cudaSuccess)
        return FP4LIN_ERR_CUDA;
    st = raise_smem(kv_table_kernel, &g_table_attr[ordinal], table_smem(TABLE_MAX_REQUESTS));
    if (st != FP4LIN_OK)
        return st;
    TableShape a{};
    a.table = table;
    a.lens = lens;
    a.new_lens = new_lens;
    a.free_list = free_pages;
    a.head = free_head;
    a.cu = cu_new;
    a.slots = slots;
    a.next_head = next_head;
    a.ld = ld_table;
    a.B = B;
    a.width = width;
    a.F = num_free;
    a.max_tokens = max_tokens;
    a.shift = shift;
    const int64_t items = std::max<int64_t>(max_tokens, (int64_t)(max_tokens >> shift) + B + 1);
    const int64_t grid = std::min<int64_t>((items + TABLE_THREADS - 1) / TABLE_THREADS, dev->sms);
    return launched(launch_pdl(kv_table_kernel, dim3((unsigned)grid), dim3(TABLE_THREADS), table_smem(B),
                               as_stream(stream), a));
}

int kv_fp8_store(const void *k_new, int64_t ld_k, const void *v_new, int64_t ld_v, const int32_t *slots, int T,
                 uint8_t *k_codes, uint8_t *k_scales, uint8_t *v_codes, uint8_t *v_scales, int num_pages, int H,
                 int page, int D, void *stream)
{
    if (!k_new || !v_new || !slots || !k_codes || !k_scales || !v_codes || !v_scales)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (T < 1 || H < 1 || D < 1 || num_pages < 1 || ld_k < (int64_t)H * D || ld_v < (int64_t)H * D)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    const int shift = page_shift(page);
    if (shift < 0 || (D != 64 && D != 128) || ld_k % 8 != 0 || ld_v % 8 != 0 || H > 32767 || T > 65535 * APPEND_TOKENS ||
        ((int64_t)num_pages << shift) > 0x7FFFFFFF)
        return FP4LIN_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) ||
        !aligned(slots, 4))
        return FP4LIN_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    const int st = current_device(&dev);
    if (st != FP4LIN_OK)
        return st;
    AppendShape a{};
    a.k = reinterpret_cast<const __nv_bfloat16 *>(k_new);
    a.v = reinterpret_cast<const __nv_bfloat16 *>(v_new);
    a.slots = slots;
    a.kc = k_codes;
    a.ks = k_scales;
    a.vc = v_codes;
    a.vs = v_scales;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.slots_end = (int64_t)num_pages << shift;
    a.T = T;
    a.H = H;
    a.shift = shift;
    // fewer tokens a CTA while there are fewer CTAs than the SMs hold, down to a token a warp
    a.per_cta = APPEND_TOKENS;
    while (a.per_cta > APPEND_WARPS && (int64_t)((T + a.per_cta - 1) / a.per_cta) * H * 2 < (int64_t)dev->sms * 3)
        a.per_cta /= 2;
    const dim3 grid((unsigned)(2 * H), (unsigned)((T + a.per_cta - 1) / a.per_cta));
    cudaStream_t s = as_stream(stream);
    return launched(D == 64 ? launch_pdl(kv_append_kernel<64>, grid, dim3(APPEND_THREADS), 0, s, a)
                            : launch_pdl(kv_append_kernel<128>, grid, dim3(APPEND_THREADS), 0, s, a));
}

size_t kv_fp8_attention_workspace_bytes(int B, int H, int G, int max_new, int64_t max_len, int D)
{
    if (!paged_sizes_ok(B, H, G, D, max_new, max_len))
        return 0;
    int sms = 148, dev = 0, v = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
        sms = v;
    else
        cudaGetLastError();
    return plan_paged(B, H, G, max_new, max_len, D, sms).ws_bytes;
}

int kv_fp8_attention(const void *q, int64_t ld_q, int T, const uint8_t *k_codes, const uint8_t *k_scales,
                     const uint8_t *v_codes, const uint8_t *v_scales, int num_pages, int page, const int32_t *table,
                     int64_t ld_table, int width, const int32_t *lens, const int32_t *cu_new, int max_new,
                     int64_t max_len, float scale, void *out, int B, int H, int G, int D, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !table || !lens || !cu_new || !out)
        return FP4LIN_ERR_INVALID_ARGUMENT;
    if (B < 1 || H < 1 || G < 1 || D < 1 || T < 1 || num_pages < 1 || width < 1 || ld_table < width || max_new < 1 ||
        max_len < 1 || ld_q < (int64_t)H * G * D || !(scale >= -3.4e38f && scale <= 3.4e38f))
        return FP4LIN_ERR_INVALID_ARGUMENT;
    const int shift = page_shift(page);
    if (shift < 0 || !paged_sizes_ok(B, H, G, D, max_new, max_len) || ld_q % 8 != 0 ||
        ((int64_t)num_pages << shift) > 0x7FFFFFFF)
        return FP4LIN_ERR_UNSUPPORTED_SHAPE;
    if (max_len > ((int64_t)width << shift))
        return FP4LIN_ERR_INVALID_ARGUMENT;  // the table cannot hold max_len rows
    if (!aligned(q, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(out, 16) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(cu_new, 4) || (workspace && !aligned(workspace, 16)))
        return FP4LIN_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    const int st = current_device(&dev);
    if (st != FP4LIN_OK)
        return st;
    const KvPagedPlan p = plan_paged(B, H, G, max_new, max_len, D, dev->sms);
    if (p.ws_bytes && (!workspace || workspace_bytes < p.ws_bytes))
        return FP4LIN_ERR_WORKSPACE;
    KvPagedShape a{};
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a.kc = k_codes;
    a.ks = k_scales;
    a.vc = v_codes;
    a.vs = v_scales;
    a.table = table;
    a.lens = lens;
    a.cu = cu_new;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    a.ws = reinterpret_cast<float *>(workspace);
    a.ld_q = ld_q;
    a.ld_t = ld_table;
    a.qscale = scale * 1.4426950408889634f;
    a.B = B;
    a.H = H;
    a.G = G;
    a.T = T;
    a.NP = num_pages;
    a.shift = shift;
    a.max_new = max_new;
    a.max_len = (int)max_len;
    a.chunk = p.chunk;
    a.S = p.S;
    a.tiles = p.tiles;
    a.max_rows = p.max_rows;
    a.joined = p.S > 1 && p.S <= 8;
    a.sms = dev->sms;
    a.prefill_ws = reinterpret_cast<int4 *>(reinterpret_cast<uint8_t *>(workspace) + p.split_bytes);
    if (p.prefill_tiles)
        a.prefill_jobs = reinterpret_cast<KppJob *>(a.prefill_ws + kpp_jobs_at(p.prefill_tiles, dev->sms, D));
    // no more tiles than T tokens can make: rows / 256, and a started one for each request of many rows
    const int64_t q_rows = (int64_t)T * G, many = std::min<int64_t>(B, q_rows / (KVP_SPLIT_ROWS + 1));
    a.prefill_most = (int)std::min(p.prefill_tiles, (q_rows / KPP_ROWS + many) * H);
    if (a.prefill_most) {
        int ordinal = 0;
        if (cudaGetDevice(&ordinal) != cudaSuccess)
            return FP4LIN_ERR_CUDA;
        const int ready = D == 64 ? raise_smem(kv_paged_prefill_kernel<64>, &g_prefill_attr[ordinal][0], kpp_smem(64))
                                  : raise_smem(kv_paged_prefill_kernel<128>, &g_prefill_attr[ordinal][1], kpp_smem(128));
        if (ready != FP4LIN_OK)
            return ready;
    }
    cudaStream_t s = as_stream(stream);
    return launched(D == 64 ? launch_paged<64>(a, p, s) : launch_paged<128>(a, p, s));
}

}  // extern "C"
