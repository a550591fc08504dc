// kv_paged_prefill.cuh -- kv_paged_attention.cuh's attention for requests with many new tokens: the
// same mathematics on tcgen05.
//
// 4 D flops and one exponential a score: at D = 128 a 256 x 128 block of scores is ~2050 cycles of the
// exponential unit and ~2100 of the tensor cores, and takes ~5400.  Each is busy for two fifths of the time:
// what sets the pace is the chain from a block's keys through its scores and weights to its values, which a
// block with one live tile takes as long for.  Two prompts of up to 2048 tokens behind contexts of up to
// 8191, 8 kv heads of 4 query heads, D = 128 (539 GFLOP): 593 us, 909 TFLOP/s, 55% of the measured bf16
// rate.  One CTA an SM takes 256 (token, head) rows of one kv head, as two tiles of 128: while the
// softmax of one runs, the tensor cores work on the other, and every key block that is converted serves
// both.
//   warps 0-3, 4-7   softmax of tile 0, 1: a thread owns a row.  Reads 64 of the row's scores from TMEM,
//                    applies both scales in one multiply-add, writes the f16 weights over the scores
//                    in TMEM; meanwhile the next 64 are computed into the tile's other buffer (with
//                    one buffer of 128 the kernel took 799 us).  The output is rescaled only when the
//                    maximum has grown by more than 2^KPP_LAZY, which is rare; the weights start at
//                    2^KPP_BIAS, so that they stay in f16 and lose only what is 2^-31 of a row's largest.
//   warps 8-11       load 128 keys of K and V from their pages, a block ahead in registers, and
//                    write them as f16 (exact) in the 128-byte-swizzled operand layout.
//   warp 13          waits for what warp 12 needs next and meets it at a named barrier, which costs the
//                    issue far less than a wait of its own (723 us).
//   warp 12          issues the MMAs: S = Q K^T (both in shared memory, K-major) and O += P V (P from
//                    TMEM, V as an MN-major operand: its rows are keys, as in the cache).
// TMEM: scores and weights of the tiles in columns 0 and 128 (two buffers of 64 keys each), outputs in
// 256 and 256 + D.
//
// Which tiles there are is known on the device only: kv_paged_plan_kernel lists them, and this kernel's
// grid has as many CTAs as T tokens can need.  (A grid over every request's longest case spent 130 us
// more where one prompt of 2048 tokens came with 63 decoding requests.)  Where there are few tiles, and at
// the end of many, CTAs share a tile's keys (kpp_split) and leave their sums to
// kv_paged_prefill_merge_kernel: one request of 32 rows over 32768 keys takes 51 us instead of 512.
#pragma once

#include <algorithm>
#include <type_traits>

#include "kv_paged_attention.cuh"

namespace fp4lin {

constexpr int KPP_THREADS = 512;
constexpr int KPP_KEYS = 128;          // keys a block
constexpr int KPP_ROWS = 256;          // rows a CTA
constexpr int KPP_SLOTS = 4;           // blocks whose page factors are held at once
constexpr int KPP_MIN_BLOCKS = 4;      // blocks of keys to a CTA, at least (one request of 512 rows over 4096
                                       // keys: 2 / 3 / 4 / 8 / 16 take 38 / 34 / 36 / 43 / 61 us)
constexpr int KPP_LAZY = 8;            // log2 growth of the maximum that is let pass
constexpr int KPP_SCAN = 1 << 20;      // pages among which a page of zeros looks for others (a wait ends in 1 s)
constexpr int KPP_BIAS = KVP_BIAS - KPP_LAZY;  // how far below the maximum M is put

struct KppCtrl {
    uint64_t kfull[2], kfree[2], vfull[2], vfree[2], sfull[2][2], pfull[2][2], odone[2], drain;
    alignas(16) float kf[KPP_SLOTS][8], xv[KPP_SLOTS][8], c[KPP_SLOTS][8];
    uint32_t tmem;
    int abort, nan;
};

// How `alive` tiles become CTAs: the last `tail` of them are `parts` CTAs each.  Up to half a GPU's worth
// is shared so that it fills the GPU, up to two thirds by three; one to a CTA leaves less than a third
// idle above that; of more than a GPU's worth, a quarter of that by four, which evens out the last wave
// (464 tiles of 52 to 80 blocks of keys: 683 us without).
struct KppSplit {
    int tail, parts;
};

__host__ __device__ inline KppSplit kpp_split(int alive, int sms)
{
    if (alive <= sms / 2)
        return {alive, alive ? sms / alive : 1};
    if (alive <= 2 * sms / 3)
        return {alive, 3};
    if (alive <= sms)
        return {0, 1};
    return {sms / 4, 4};
}

// The most CTAs that up to `most` tiles can become, and of them those that share a tile.  Neither falls as
// `most` grows: a call's tokens may allow fewer tiles than its workspace was sized for.
inline int64_t kpp_grid(int64_t most, int sms)
{
    return most <= sms / 2 ? sms : std::max<int64_t>(2 * sms, most + 3 * (sms / 4));
}
inline int64_t kpp_parts(int64_t most, int sms) { return most <= sms / 2 ? sms : 2 * (int64_t)sms; }

// A CTA's work: head bh's rows from row0 on (of a request with `len` rows in the cache and its first
// token at `first`), `blocks` blocks of keys from key0 on; sums: its place among the sums where the tile
// is shared, else -1.
struct alignas(16) KppJob {
    int bh, row0, key0, blocks, sums, len, first, live;
};

// Workspace, in units of 16 bytes: a header (jobs, tail tiles, parts); for each shared tile its bh, first
// row, rows and number of splits; the sums [tile, part, row, D + 4]; the jobs.
inline int64_t kpp_jobs_at(int64_t most, int sms, int D)
{
    return 1 + sms + kpp_parts(most, sms) * KPP_ROWS * (D + 4) / 4;
}
inline size_t kpp_workspace(int64_t most, int sms, int D)
{
    return 16 * (size_t)kpp_jobs_at(most, sms, D) + sizeof(KppJob) * (size_t)kpp_grid(most, sms);
}

constexpr size_t kpp_smem(int D) { return 1024 + (size_t)(KPP_ROWS + 4 * KPP_KEYS) * D * 2 + sizeof(KppCtrl); }

// One lane of a converged warp issues a whole batch, so that little stands between the MMAs (the warp
// shares its scheduler with a softmax's): D[128 x N] = sum over D/16 steps of A[128 x 16] B[N x 16]^T,
// f16 operands in shared memory (descriptors of their first steps; 32 bytes a step, the next 64
// dimensions 16 KB on).  Then `bar` hears of it, and at once of what this warp has waited for.
template <int D>
__device__ __forceinline__ void kpp_issue_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t *bar)
{
    if constexpr (D == 128)
        asm volatile("{\n\t.reg .pred e, on, off;\n\t.reg .b64 x, y;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "setp.eq.u32 on, %3, %3;\n\tsetp.ne.u32 off, %3, %3;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, off;\n\t"
                 "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 1024;\n\tadd.s64 y, %2, 1024;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 1026;\n\tadd.s64 y, %2, 1026;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 1028;\n\tadd.s64 y, %2, 1028;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 1030;\n\tadd.s64 y, %2, 1030;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
                 "@e mbarrier.arrive.release.cta.shared::cta.b64 _, [%4];\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(smem_u32(bar))
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred e, on, off;\n\t.reg .b64 x, y;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "setp.eq.u32 on, %3, %3;\n\tsetp.ne.u32 off, %3, %3;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, off;\n\t"
                 "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, on;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
                 "@e mbarrier.arrive.release.cta.shared::cta.b64 _, [%4];\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(smem_u32(bar))
                     : "memory");
}

// The same for D[128 x N] (+)= P V over 64 keys: P in TMEM (8 columns a step), V MN-major (2 KB a step).
__device__ __forceinline__ void kpp_issue_values(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, uint32_t acc,
                                                 uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred e, on, first;\n\t.reg .b64 y;\n\t.reg .b32 t;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "setp.eq.u32 on, %3, %3;\n\tsetp.ne.u32 first, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, first;\n\t"
                 "add.u32 t, %1, 8;\n\tadd.s64 y, %2, 128;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t], y, %3, on;\n\t"
                 "add.u32 t, %1, 16;\n\tadd.s64 y, %2, 256;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t], y, %3, on;\n\t"
                 "add.u32 t, %1, 24;\n\tadd.s64 y, %2, 384;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t], y, %3, on;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
                 "@e mbarrier.arrive.release.cta.shared::cta.b64 _, [%4];\n\t}" ::"r"(d),
                 "r"(p), "l"(v), "r"(idesc), "r"(smem_u32(bar)), "r"(acc)
                 : "memory");
}

// MN-major operand, 128-byte swizzle: rows (k) of 128 bytes = 64 values along MN, 8-row groups 1024
// bytes apart (stride byte offset), the next 64 values `lbo` bytes on (leading byte offset).
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t saddr, uint32_t lbo)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor of kind::f16: binary32 accumulator, f16 operands, M = 128.
constexpr uint32_t kpp_idesc(int N, bool b_mn_major)
{
    return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(N / 8) << 17) | ((128u / 16u) << 24);
}

// 64 columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%2"
                 "5,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%4"
                 "8,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
                   "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
                   "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]),
                   "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
                   "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
                   "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]),
                   "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]),
                   "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
                 : "memory");
}

// 8 columns, loaded, scaled by f and stored back.
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f)
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 codes of (row, 16-byte chunk cc of the row) as f16 into the operand layout at `base`: blocks of
// 128 rows x 128 bytes, one for each 64 dimensions; 16-byte chunk x of row r sits at x ^ (r % 8).
template <int D>
__device__ __forceinline__ void kpp_convert(uint8_t *base, int row, int cc, uint4 u)
{
    uint32_t f[8];
    e4m3x4_to_f16(u.x, f[0], f[1]);
    e4m3x4_to_f16(u.y, f[2], f[3]);
    e4m3x4_to_f16(u.z, f[4], f[5]);
    e4m3x4_to_f16(u.w, f[6], f[7]);
    uint8_t *p = base + (cc >> 2) * (KPP_KEYS * 128) + row * 128;
    const int c0 = 2 * (cc & 3), sw = row & 7;
    // lanes of the upper dimensions store their odd chunk first: a quarter warp then meets each bank once
    const bool odd = cc >> 2;
    *reinterpret_cast<uint4 *>(p + (((c0 + odd) ^ sw) << 4)) =
        odd ? make_uint4(f[4], f[5], f[6], f[7]) : make_uint4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<uint4 *>(p + (((c0 + !odd) ^ sw) << 4)) =
        odd ? make_uint4(f[0], f[1], f[2], f[3]) : make_uint4(f[4], f[5], f[6], f[7]);
}

// The factor from a score's dot product to log2 units: 2^Xk times the row's.  Kept above 0, so that
// the -inf of a masked score stays one.
__device__ __forceinline__ float kpp_factor(float kf, float qs) { return fmaxf(kf * qs, 1.17549435e-38f); }

// The CTAs' work from the requests' lengths.  One CTA: a thread counts the tiles of a range of requests,
// the block adds them up, and then each thread looks up its jobs' requests.
constexpr int KPP_PLAN_THREADS = 1024;

__global__ void __launch_bounds__(KPP_PLAN_THREADS) kv_paged_plan_kernel(KvPagedShape a)
{
    __shared__ int upto_of[KPP_PLAN_THREADS], warp_sum[KPP_PLAN_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const int per = (a.B + KPP_PLAN_THREADS - 1) / KPP_PLAN_THREADS;
    auto tiles_of = [&](int r) {
        const int n = kvp_request(a, r).n * a.G;
        return n > a.max_rows ? (n + KPP_ROWS - 1) / KPP_ROWS * a.H : 0;
    };
    int upto = 0;
    for (int r = tid * per; r < min(tid * per + per, a.B); ++r)
        upto += tiles_of(r);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        upto += lane >= o ? y : 0;
    }
    if (lane == 31)
        warp_sum[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w)
        upto += warp_sum[w];
    upto_of[tid] = upto;
    __syncthreads();
    // more than prefill_most only where offsets fall, which is an error anyway
    const int alive = min(upto_of[KPP_PLAN_THREADS - 1], a.prefill_most);
    const KppSplit sp = kpp_split(alive, a.sms);
    const int alone = alive - sp.tail, jobs = alone + sp.tail * sp.parts;
    if (tid == 0)
        a.prefill_ws[0] = make_int4(jobs, sp.tail, sp.parts, 0);
    for (int j = tid; j < jobs; j += KPP_PLAN_THREADS) {
        const int shared = j < alone ? -1 : (j - alone) / sp.parts, parts = shared < 0 ? 1 : sp.parts;
        const int part = shared < 0 ? 0 : j - alone - shared * parts;
        int t = shared < 0 ? j : alone + shared;
        int lo = 0, hi = KPP_PLAN_THREADS - 1;  // the first range that ends behind t
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (upto_of[mid] > t)
                hi = mid;
            else
                lo = mid + 1;
        }
        t -= lo ? upto_of[lo - 1] : 0;
        int b = lo * per;
        for (int n; (n = tiles_of(b)) <= t; ++b)
            t -= n;
        const KvPagedRequest rq = kvp_request(a, b);
        const int rows = rq.n * a.G, of_head = (rows + KPP_ROWS - 1) / KPP_ROWS, h = t / of_head;
        KppJob job;
        job.bh = b * a.H + h;
        job.row0 = (of_head - 1 - (t - h * of_head)) * KPP_ROWS;  // longest first
        job.live = min(KPP_ROWS, rows - job.row0);
        job.len = rq.len;
        job.first = rq.first;
        // the blocks of keys that the tile's last row sees, and this CTA's share of them
        const int blocks = (rq.len + (job.row0 + job.live - 1) / a.G + KPP_KEYS) / KPP_KEYS;
        const int chunk = max((blocks + parts - 1) / parts, KPP_MIN_BLOCKS);
        job.key0 = part * chunk * KPP_KEYS;
        job.blocks = max(0, min(blocks - part * chunk, chunk));
        job.sums = blocks > chunk ? shared * parts + part : -1;
        if (shared >= 0 && part == 0)
            a.prefill_ws[1 + shared] = make_int4(job.bh, job.row0, job.live, (blocks + chunk - 1) / chunk);
        a.prefill_jobs[j] = job;
    }
}

template <int D>
__global__ void __launch_bounds__(KPP_THREADS, 1) kv_paged_prefill_kernel(KvPagedShape a)
{
    extern __shared__ uint8_t kpp_raw[];
    uint8_t *sm = kpp_raw + ((1024u - (smem_u32(kpp_raw) & 1023u)) & 1023u);
    constexpr int TILE = 128 * D * 2;  // bytes of an operand tile
    uint8_t *s_q = sm, *s_k = sm + 2 * TILE, *s_v = sm + 4 * TILE;
    KppCtrl &ct = *reinterpret_cast<KppCtrl *>(sm + 6 * TILE);
    volatile int *abort = &ct.abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    KppJob job = a.prefill_jobs[blockIdx.x];
    // one value for the warp: the compiler may keep them, and addresses made of them, in uniform registers
    job.bh = __reduce_min_sync(0xffffffffu, job.bh);
    job.row0 = __reduce_min_sync(0xffffffffu, job.row0);
    job.key0 = __reduce_min_sync(0xffffffffu, job.key0);
    if ((int)blockIdx.x >= a.prefill_ws[0].x || job.blocks == 0)
        return;
    const int b = job.bh / a.H, h = job.bh - b * a.H, row0 = job.row0, live = job.live, len = job.len;
    const int key0 = job.key0, blocks = job.blocks;
    const int tiles = live > 128 ? 2 : 1;
    const int kend = len + (row0 + live - 1) / a.G + 1;  // keys that the last row sees
    const int all = len + row0 / a.G;                    // last key that every row sees
    const int P1 = (1 << a.shift) - 1;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.kfull[i], 128);
            mbar_init(&ct.kfree[i], 1);
            mbar_init(&ct.vfull[i], 128);
            mbar_init(&ct.vfree[i], 1);
            for (int half = 0; half < 2; ++half) {
                mbar_init(&ct.sfull[i][half], 2);
                mbar_init(&ct.pfull[i][half], 128);
            }
            mbar_init(&ct.odone[i], 2);
        }
        mbar_init(&ct.drain, 1);
        ct.abort = 0;
        ct.nan = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ct.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // q: a thread's own row, to f16 (kv_paged_attention.cuh), into the operand layout
    float qs = 0.0f;
    const int tile = warp >> 2, trow = tid & 127;
    const int rho = row0 + tid, tok = rho / a.G, head = rho - tok * a.G;
    const bool mine = tid < live;
    if (warp < 8) {
        const __nv_bfloat16 *src =
            a.q + (int64_t)(job.first + (mine ? tok : 0)) * a.ld_q + (int64_t)(h * a.G + (mine ? head : 0)) * D;
        float m = 0.0f;
        for (int i = 0; i < D / 8; ++i) {
            float f[8];
            bf16x8_to_f32(mine ? ld_nc_v4(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = fmaxf(m, finite_abs(f[j]));
        }
        const uint32_t e = kvp_q_exponent(m);
        // a negative scale turns q around, so that the row's factor is not negative
        const float inv = copysignf(kvp_q_inverse(e), a.qscale);
        qs = kvp_q_scale(e) * fabsf(a.qscale);
        for (int i = 0; i < D / 8; ++i) {
            float f[8];
            bf16x8_to_f32(mine ? ld_nc_v4(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u), f);
            uint4 v;
            v.x = cvt_f16x2(f[0] * inv, f[1] * inv);
            v.y = cvt_f16x2(f[2] * inv, f[3] * inv);
            v.z = cvt_f16x2(f[4] * inv, f[5] * inv);
            v.w = cvt_f16x2(f[6] * inv, f[7] * inv);
            *reinterpret_cast<uint4 *>(s_q + tile * TILE + (i >> 3) * (128 * 128) + trow * 128 +
                                       (((i & 7) ^ (trow & 7)) << 4)) = v;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct.tmem;

    if (warp < 8) {
        if (tile < tiles) {
            const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
            const uint32_t t_s = tmem + lanes + tile * 128, t_o = tmem + lanes + 256 + tile * D;
            const int lim = mine ? len + tok : -1;
            float M = -INFINITY, den = 0.0f;
            bool ok = true;
#pragma unroll 1
            for (int step = 0; step < 2 * blocks; ++step) {  // 64 keys each
                const int half = step & 1, i = step >> 1, slot = i & (KPP_SLOTS - 1), k0 = key0 + 64 * step;
                ok = warp_wait(&ct.sfull[tile][half], i & 1, abort, lane);
                if (!ok)
                    break;
                tc_fence_after();
                const float4 kf = *reinterpret_cast<const float4 *>(&ct.kf[slot][4 * half]);
                const float4 xv = *reinterpret_cast<const float4 *>(&ct.xv[slot][4 * half]);
                const float4 cv = *reinterpret_cast<const float4 *>(&ct.c[slot][4 * half]);
                uint32_t s[64];
                tmem_ld64(t_s + 64 * half, s);
                if (k0 + 63 > all || live < KPP_ROWS) {
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (k0 + j > lim)
                            s[j] = 0xFF800000u;
                }
                // the largest s' = f s + Xv: f is positive and one for 16 keys, so it is that of the largest s
                const float f[4] = {kpp_factor(kf.x, qs), kpp_factor(kf.y, qs), kpp_factor(kf.z, qs), kpp_factor(kf.w, qs)};
                const float x[4] = {xv.x, xv.y, xv.z, xv.w}, c[4] = {cv.x, cv.y, cv.z, cv.w};
                float m = -INFINITY;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float t0 = max3f(__uint_as_float(s[16 * g]), __uint_as_float(s[16 * g + 1]), __uint_as_float(s[16 * g + 2]));
                    float t1 = max3f(__uint_as_float(s[16 * g + 3]), __uint_as_float(s[16 * g + 4]), __uint_as_float(s[16 * g + 5]));
#pragma unroll
                    for (int j = 6; j < 14; j += 4) {
                        t0 = max3f(t0, __uint_as_float(s[16 * g + j]), __uint_as_float(s[16 * g + j + 1]));
                        t1 = max3f(t1, __uint_as_float(s[16 * g + j + 2]), __uint_as_float(s[16 * g + j + 3]));
                    }
                    t0 = max3f(t0, __uint_as_float(s[16 * g + 14]), __uint_as_float(s[16 * g + 15]));
                    m = fmaxf(m, fmaf(fmaxf(t0, t1), f[g], x[g]));
                }
                float corr = 1.0f;
                if (m - M > (float)KVP_BIAS) {  // NaN while no key was seen
                    corr = ex2(M - (m - KPP_BIAS));  // 0 for the first keys
                    M = m - KPP_BIAS;
                }
                // The last product is waited for before the output is scaled, and always before the last
                // weights are given out: the wait after the loop then has one phase only to mean.
                const bool grown = __any_sync(0xffffffffu, corr != 1.0f);
                if (step > 0 && (grown || step + 1 == 2 * blocks)) {
                    ok = warp_wait(&ct.odone[tile], (step - 1) & 1, abort, lane);
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; grown && k < D / 8; ++k)
                        tmem_scale8(t_o + 8 * k, corr);
                }
                den *= corr;
                const float base = M == -INFINITY ? 0.0f : M;
                // weights 2^(s' - M), over the scores' columns
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t w[16];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float ff = f[2 * q + g], xx = x[2 * q + g] - base;
                        const uint64_t f2 = f2_pack(ff, ff), x2 = f2_pack(xx, xx);
                        uint64_t sum = 0ull;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const int e = 32 * q + 16 * g + j;
                            float a0, a1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), f2, x2), a0, a1);
                            const float w0 = ex2(a0), w1 = ex2(a1);
                            sum = f2_add(sum, f2_pack(w0, w1));
                            w[8 * g + j / 2] = cvt_f16x2_finite(w0, w1);
                        }
                        float s0, s1;
                        f2_unpack(sum, s0, s1);
                        den = fmaf(s0 + s1, c[2 * q + g], den);
                    }
                    tmem_st16(t_s + 64 * half + 16 * q, w);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&ct.pfull[tile][half]);
            }
            if (ok && warp_wait(&ct.odone[tile], 1, abort, lane)) {
                tc_fence_after();
                const bool whole = job.sums < 0;
                // the sums without the bias: den has none, the products do
                const float inv =
                    pow2_const(-KPP_BIAS) * (!whole ? 1.0f : den > 0.0f ? __fdiv_rn(1.0f, den) : den == 0.0f ? 0.0f : den);
                __nv_bfloat16 *dst =
                    a.out + (int64_t)(job.first + (mine ? tok : 0)) * a.H * a.G * D + (int64_t)(h * a.G + (mine ? head : 0)) * D;
                float *sums = reinterpret_cast<float *>(a.prefill_ws + 1 + a.sms) +
                              ((int64_t)job.sums * KPP_ROWS + tid) * (D + 4);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    float o[32];
                    tmem_ld32(t_o + 32 * k, o);
                    if (mine && whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                                    : "=r"(y[e])
                                    : "f"(o[j + 2 * e + 1] * inv), "f"(o[j + 2 * e] * inv));
                            st_v4(dst + 32 * k + j, make_uint4(y[0], y[1], y[2], y[3]));
                        }
                    } else if (mine) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4 *>(sums + 32 * k + j) =
                                make_float4(o[j] * inv, o[j + 1] * inv, o[j + 2] * inv, o[j + 3] * inv);
                    }
                }
                if (mine && !whole)
                    *reinterpret_cast<float2 *>(sums + D) = make_float2(M, den);
                if (ct.nan && mine) {  // a NaN value code among the keys that not every row sees
                    const int last = min(lim, key0 + blocks * KPP_KEYS - 1);
                    for (int key = max(all + 1, key0); key <= last; ++key) {
                        const int page = a.table[b * a.ld_t + (key >> a.shift)];
                        if (page < 0 || page >= a.NP)
                            continue;
                        const uint8_t *v = a.vc + ((((int64_t)page * a.H + h) << a.shift) + (key & P1)) * D;
                        for (int d = 0; d < D; ++d)
                            if ((v[d] & 127) == 127) {
                                if (whole)
                                    dst[d] = __ushort_as_bfloat16(0x7FC0);
                                else
                                    sums[d] = __int_as_float(0x7fc00000);
                            }
                    }
                }
            }
        }
    } else if (warp < 12) {
        constexpr int CPR = D / 16, RPP = 128 / CPR, PASSES = KPP_KEYS / RPP;  // 16-byte chunks a row, rows a pass
        const int u = tid - 256, cc = u % CPR, r0 = u / CPR;
        const int32_t *table = a.table + b * a.ld_t;
        // Every thread reads the table entries of its own rows (the same for all threads, or two halves
        // of them), two blocks ahead, and the codes one block ahead, so that no load waits for another
        // within a block.  Nothing is exchanged: a shuffle would wait its turn behind the operands that
        // the tensor cores read from shared memory.
        auto entries_of = [&](int i, int *e) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int key = key0 + i * KPP_KEYS + ((r0 + p * RPP) & ~15);
                e[p] = key < kend ? table[key >> a.shift] : -1;
            }
        };
        auto load = [&](const uint8_t *codes, int i, const int *e, uint4 *x) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int row = r0 + p * RPP;
                x[p] = ld_nc_v4_if(codes + ((((int64_t)e[p] * a.H + h) << a.shift) + (row & P1)) * D + 16 * cc,
                                   (uint32_t)e[p] < (uint32_t)a.NP && key0 + i * KPP_KEYS + row < kend);
            }
        };
        // lane g < 8 of the first of these warps: the page of keys 16 g .. and its scale bytes
        const bool scales = warp == 8 && lane < 8;
        auto page_of = [&](int i) {
            const int key = key0 + i * KPP_KEYS + 16 * lane;
            if (!scales || key >= kend)
                return -1;
            const int page = table[key >> a.shift];
            if (page >= 0 && page < a.NP)
                return page;
            report_error(FP4LIN_ERR_OUT_OF_RANGE);
            return -1;
        };
        uint4 xk[PASSES], xv[PASSES];
        int then[PASSES];
        entries_of(0, then);
        load(a.kc, 0, then, xk);
        load(a.vc, 0, then, xv);
        entries_of(1, then);
        int page = page_of(0);
        uint32_t kbyte = page >= 0 ? a.ks[(int64_t)page * a.H + h] : 0u;
        uint32_t vbyte = page >= 0 ? a.vs[(int64_t)page * a.H + h] : 0u;
        // a page of zeros (kv_paged_attention.cuh): on the first one, warp 8 looks through the job's pages
        float zero_x = INFINITY;
        auto find_zero_x = [&]() {
            float low = INFINITY;
            const uint32_t end = min(kend, key0 + blocks * KPP_KEYS);
            uint32_t key = key0 + (lane << a.shift);  // may pass 2^31 behind the end
#pragma unroll 4
            for (int n = 0; n < KPP_SCAN / 32; ++n, key += 32 << a.shift) {
                if (key >= end)
                    break;
                const int p = table[key >> a.shift];
                const uint32_t byte = p >= 0 && p < a.NP ? a.vs[(int64_t)p * a.H + h] : 0u;
                low = byte ? fminf(low, (float)((int)byte - 127)) : low;
            }
            return kvp_zero_exponent(warp_min(low));
        };
        for (int i = 0; i < blocks; ++i) {
            const int next = page_of(i + 1);
            const int st = i & 1, par = ((i >> 1) & 1) ^ 1;
            if (i >= 2 && !warp_wait(&ct.kfree[st], par, abort, lane))
                break;
            if (warp == 8 && zero_x == INFINITY && __any_sync(0xffffffffu, page >= 0 && vbyte == 0u))
                zero_x = find_zero_x();
            if (scales) {
                const int slot = i & (KPP_SLOTS - 1);
                const float x = vbyte ? (float)((int)vbyte - 127) : zero_x;
                ct.kf[slot][lane] = mxfp8_scale(kbyte);
                ct.xv[slot][lane] = page >= 0 ? x : -INFINITY;
                ct.c[slot][lane] = page >= 0 ? ex2(-x) * pow2_const(-KPP_BIAS) : 0.0f;
            }
            kbyte = next >= 0 ? a.ks[(int64_t)next * a.H + h] : 0u;
            vbyte = next >= 0 ? a.vs[(int64_t)next * a.H + h] : 0u;
#pragma unroll
            for (int p = 0; p < PASSES; ++p)
                kpp_convert<D>(s_k + st * TILE, r0 + p * RPP, cc, xk[p]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(&ct.kfull[st]);
            if (i + 1 < blocks)
                load(a.kc, i + 1, then, xk);
            if (i >= 2 && !warp_wait(&ct.vfree[st], par, abort, lane))
                break;
            if (key0 + (i + 1) * KPP_KEYS - 1 > all) {  // keys that some rows do not see: weight 0 must stay 0
                bool nan = false;
#pragma unroll
                for (int p = 0; p < PASSES; ++p)
                    if (key0 + i * KPP_KEYS + r0 + p * RPP > all)
                        nan |= drop_nan_codes(xv[p].x) | drop_nan_codes(xv[p].y) | drop_nan_codes(xv[p].z) |
                               drop_nan_codes(xv[p].w);
                if (nan)
                    ct.nan = 1;
            }
#pragma unroll
            for (int p = 0; p < PASSES; ++p)
                kpp_convert<D>(s_v + st * TILE, r0 + p * RPP, cc, xv[p]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(&ct.vfull[st]);
            if (i + 1 < blocks)
                load(a.vc, i + 1, then, xv);
            entries_of(i + 2, then);
            page = next;
        }
    } else {
        if (warp == 12) {
            constexpr uint32_t IQK = kpp_idesc(64, false), IPV = kpp_idesc(D, true);
            const uint64_t dq = desc_sw128(smem_u32(s_q)), dk = desc_sw128(smem_u32(s_k));
            const uint64_t dv = desc_sw128_mn(smem_u32(s_v), KPP_KEYS * 128);
            // 64 keys: half a stage, 8 KB into each of its 64-dimension blocks
            auto scores = [&](int j, int half, int i) {
                kpp_issue_scores<D>(tmem + j * 128 + half * 64, dq + j * (TILE >> 4),
                                    dk + ((i & 1) * TILE + half * 64 * 128 >> 4), IQK, &ct.sfull[j][half]);
            };
            auto values = [&](int j, int half, int i) {
                kpp_issue_values(tmem + 256 + j * D, tmem + j * 128 + half * 64,
                                 dv + ((i & 1) * TILE + half * 64 * 128 >> 4), IPV, i > 0 || half > 0, &ct.odone[j]);
            };
            bool ok = !meet_or(false);
            if (ok) {
                tc_fence_after();
                for (int half = 0; half < 2; ++half)
                    for (int j = 0; j < tiles; ++j)
                        scores(j, half, 0);
                tc_commit_w(&ct.kfree[0]);
            }
            for (int i = 0; ok && i < blocks; ++i) {
                const bool more = i + 1 < blocks;
#pragma unroll 1
                for (int turn = 0; turn < 2 * tiles; ++turn) {
                    const int half = tiles == 2 ? turn >> 1 : turn, j = tiles == 2 ? turn & 1 : 0;
                    ok = !meet_or(false);
                    if (!ok)
                        break;
                    tc_fence_after();
                    values(j, half, i);
                    if (more)
                        scores(j, half, i + 1);
                }
                if (ok) {
                    tc_commit_w(&ct.vfree[i & 1]);
                    if (more)
                        tc_commit_w(&ct.kfree[(i + 1) & 1]);
                }
            }
            // nothing may be in flight when TMEM goes and the shared memory with it
            tc_commit_w(&ct.drain);
            if (lane == 0)
                wait_bounded(&ct.drain, 0, abort, false);
            __syncwarp();
        } else if (warp == 13) {
            // the waits of the issuing warp, in its order and a step ahead of it
            bool ok = warp_poll(&ct.kfull[0], 0, abort, lane);
            ok = !meet_or(!ok);
            for (int i = 0; ok && i < blocks; ++i) {
                ok = warp_poll(&ct.vfull[i & 1], (i >> 1) & 1, abort, lane);
                if (ok && i + 1 < blocks)
                    ok = warp_poll(&ct.kfull[(i + 1) & 1], ((i + 1) >> 1) & 1, abort, lane);
#pragma unroll 1
                for (int turn = 0; turn < 2 * tiles; ++turn) {
                    const int half = tiles == 2 ? turn >> 1 : turn, j = tiles == 2 ? turn & 1 : 0;
                    ok = ok && warp_poll(&ct.pfull[j][half], i & 1, abort, lane);
                    ok = !meet_or(!ok);
                    if (!ok)
                        break;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Rows of the shared tile blockIdx.y, 1 or KVP_WARPS to a CTA: a warp each, or, where few tiles have many
// parts, the whole CTA for one after the other.
template <int D>
__global__ void __launch_bounds__(KVP_THREADS) kv_paged_prefill_merge_kernel(KvPagedShape a)
{
    pdl_wait();
    const int4 head = a.prefill_ws[0], t = a.prefill_ws[1 + blockIdx.y];
    if ((int)blockIdx.y >= head.y || t.w < 2)
        return;
    const int b = t.x / a.H, h = t.x - b * a.H;
    const int64_t first = a.cu[b];
    auto join = [&](auto cta, int r) {
        if (r >= t.z)
            return;
        const int rho = t.y + r, i = rho / a.G, j = rho - i * a.G;
        const float *src = reinterpret_cast<const float *>(a.prefill_ws + 1 + a.sms) +
                           ((int64_t)blockIdx.y * head.z * KPP_ROWS + r) * (D + 4);
        kvp_merge_row<D, decltype(cta)::value>(src, (int64_t)KPP_ROWS * (D + 4), t.w,
                                               a.out + ((first + i) * a.H * a.G + h * a.G + j) * D);
    };
    const int per = KPP_ROWS / gridDim.x, r = blockIdx.x * per;
    if (per == KVP_WARPS && t.w <= 8)
        join(std::false_type{}, r + (threadIdx.x >> 5));
    else
        for (int k = 0; k < per; ++k)
            join(std::true_type{}, r + k);
}

}  // namespace fp4lin
