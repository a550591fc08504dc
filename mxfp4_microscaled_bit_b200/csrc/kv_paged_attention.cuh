// kv_paged_attention.cuh -- causal attention of a ragged batch's new tokens over the paged 8-bit
// cache (kv_paged.cuh): request b has len_b rows in the cache before this step and n_b = cu[b+1] -
// cu[b] new tokens whose rows are in it too; new token i sees positions 0 .. len_b + i.  Query head
// j uses kv head j / G.  With codes k, v and page exponents Xk, Xv:
//   s_l = scale * 2^Xk * (q . k_l),  o = sum_l softmax(s)_l * 2^Xv * v_l.
//
// The value scale rides in the exponent: with s'_l = log2(e) s_l + Xv(l) and M near max s',
//   w_l = 2^(s'_l - M),  o = (sum_l w_l v_l) / (sum_l w_l 2^-Xv(l)),
// so one running maximum and one exponential a score serve both sums, the weights that meet the
// value codes have one bound whatever the pages' scales, and one fused multiply-add applies both
// scales.  A page whose value byte is 0 (all codes zero) takes part in the second sum only, under any
// exponent.  Its keys should not move M, nor vanish beside it: it gets KVP_ZERO_GAP less than the least
// of a CTA's other pages.  (A constant, -8, put M 2^29 above pages of values near 2^-37.)
//
// Scores, maxima, sums and outputs are binary32.  K and V codes are exact in f16; q is scaled by a
// power of two to [2^14, 2^15) at its row's maximum, exact down to 2^-31 of it (2^-17 with the maximum at
// 1, where a channel that no key uses could spoil the others).  The weights that meet the value codes
// are rounded to f16: to 2^-11 of themselves against bf16 outputs, and below f16's normals to half its
// smallest step, 2^-25.  So they are kept high in f16, at most 2^KVP_BIAS and a binade or two above where
// scores pass 2^23: M is that far below the maximum, and the split kernel loses only what is 2^-39 of
// a row's largest (2^-25 with the largest at 1, where all keys beside one of 18 more were lost).  The
// second sum leaves the factor out, with its 2^-Xv, so that values of any magnitude keep their room in
// binary32; the first leaves it out at its end.
#pragma once

#include <cooperative_groups.h>

#include "gemm_sm100.cuh"
#include "kv_attention.cuh"  // mma_16816x
#include "mxfp8.cuh"

namespace fp4lin {

constexpr int KVP_THREADS = 128;
constexpr int KVP_WARPS = KVP_THREADS / 32;
constexpr int KVP_MAX_CHUNK = 2048;    // keys a CTA
constexpr int KVP_STEP = 32;           // keys a warp takes at a time
constexpr float KVP_ZERO_GAP = 24.0f;
constexpr float KVP_ZERO_X = -8.0f;    // pages of zeros where there are no others
constexpr int KVP_BIAS = 14;           // log2 of the largest weight

// 2^k for a constant k.
__host__ __device__ constexpr float pow2_const(int k) { return k < 0 ? 0.5f * pow2_const(k + 1) : k ? 2.0f * pow2_const(k - 1) : 1.0f; }

struct KppJob;

struct KvPagedShape {
    const __nv_bfloat16 *q;  // [T, H*G, D], token stride ld_q
    const uint8_t *kc, *ks, *vc, *vs;
    const int32_t *table, *lens, *cu;
    __nv_bfloat16 *out;      // [T, H*G, D]
    float *ws;               // [B*H, tiles, S, rows, D + 4], where S > 1 and not joined
    int64_t ld_q, ld_t;
    float qscale;            // scale * log2(e)
    int B, H, G, T, NP, shift, max_new, max_len;
    int chunk, S, tiles;
    bool joined;             // the S splits of a tile are one cluster
    int max_rows;            // requests of more rows are the tensor-core kernel's (kv_paged_prefill.cuh)
    int4 *prefill_ws;        // its workspace
    KppJob *prefill_jobs;
    int prefill_most, sms;   // its tiles, at most
};

// One request as a CTA sees it; ok is false where the lengths cannot be what the caller promised
// (the request is skipped and reported).
struct KvPagedRequest {
    int len, first, n;
    bool ok;
};

__device__ __forceinline__ KvPagedRequest kvp_request(const KvPagedShape &a, int b)
{
    KvPagedRequest r;
    r.len = a.lens[b];
    r.first = a.cu[b];
    const int64_t n = (int64_t)a.cu[b + 1] - r.first;
    r.ok = r.len >= 0 && r.first >= 0 && n >= 0 && n <= a.max_new && r.first + n <= a.T &&
           (int64_t)r.len + n <= a.max_len;
    r.n = r.ok ? (int)n : 0;
    return r;
}

// The exponent of a page of zeros beside others whose least is `low` (infinite: there are none).
__device__ __forceinline__ float kvp_zero_exponent(float low)
{
    return low == INFINITY ? KVP_ZERO_X : fmaxf(low - KVP_ZERO_GAP, -126.0f);
}

__device__ __forceinline__ float warp_min(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = fminf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// f16x2 of two weights; one that passes f16 (from 2^14 by the scores' own rounding) stays finite.
__device__ __forceinline__ uint32_t cvt_f16x2_finite(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Transpose of an 8 x 8 f16 fragment.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The exponent byte of a row of q's maximum, kept where the power of two that takes it to [2^14, 2^15) and
// its inverse are both normal.
__device__ __forceinline__ uint32_t kvp_q_exponent(float m) { return m > 0.0f ? min(max(__float_as_uint(m) >> 23, 15u), 253u) : 141u; }
__device__ __forceinline__ float kvp_q_inverse(uint32_t e) { return __uint_as_float((268u - e) << 23); }
__device__ __forceinline__ float kvp_q_scale(uint32_t e) { return __uint_as_float((e - 14u) << 23); }

// Row `rho` of a tile as f16 B fragments: this lane's D/4 values (d = t*D/4 ..) in the order the
// key codes are used, under kvp_q_exponent's power of two.  Returns its inverse.
template <int D>
__device__ __forceinline__ float kvp_load_q(const __nv_bfloat16 *p, bool live, uint32_t (*qb)[2])
{
    uint4 u[D / 32];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        u[i] = live ? ld_nc_v4(p + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        float f[8];
        bf16x8_to_f32(u[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = fmaxf(m, finite_abs(f[j]));
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t e = kvp_q_exponent(m);
    const float inv = kvp_q_inverse(e);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        float f[8];
        bf16x8_to_f32(u[i], f);
        qb[2 * i][0] = cvt_f16x2(f[0] * inv, f[1] * inv);
        qb[2 * i][1] = cvt_f16x2(f[2] * inv, f[3] * inv);
        qb[2 * i + 1][0] = cvt_f16x2(f[4] * inv, f[5] * inv);
        qb[2 * i + 1][1] = cvt_f16x2(f[6] * inv, f[7] * inv);
    }
    return kvp_q_scale(e);
}

// Split form: CTA (s, b*H + h, z) takes keys [s*chunk, (s+1)*chunk) for rows z*8*NT .. of the
// request's n*G (token, head) rows.  HBM bound for single tokens: every K and V byte is loaded once,
// straight into registers as tensor-core fragments -- no shared memory, no exchange between warps
// until the end.  A warp takes 32 keys at a time (its next K and V rows are in flight while it works).
// Scores^T = K q^T by mma_16816x (A: 16 keys x 16 dimensions, B: 8 rows of q): a lane needs rows
// g and g+8 of the keys, whichever dimensions, as long as q uses the same: it takes D/4 contiguous
// bytes.  O^T += V^T w^T: the lane needs the same dimension of keys 2t, 2t+1 in one register, two
// byte permutes of two rows' words; it takes D/8 contiguous dimensions (those of all D/16 M tiles).
// The weights change from the score layout to B fragments by an 8 x 8 transpose in registers.
// 32 requests of 16384 to 32768 keys, 8 kv heads of 4, D = 128 (1.52 GB): 260 to 278 us with the merge,
// 5.5 to 5.9 TB/s, 85 to 90% of a plain copy's rate; one request of 1000 keys 6.7 us.
template <int D, int NT>
__global__ void __launch_bounds__(KVP_THREADS, NT == 1 ? 3 : 2) kv_paged_split_kernel(KvPagedShape a)
{
    constexpr int R = 8 * NT, KW = D / 16, VW = D / 32;  // rows, 32-bit words a lane needs of a K / V row
    __shared__ int s_page[KVP_MAX_CHUNK / 16];
    __shared__ float s_kf[KVP_MAX_CHUNK / 16], s_xv[KVP_MAX_CHUNK / 16];
    __shared__ float s_m[KVP_WARPS][R], s_den[KVP_WARPS][R];
    __shared__ float s_o[KVP_WARPS][R][D + 4];
    __shared__ float s_cm[R], s_cden[R];  // of the whole CTA
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int bh = blockIdx.y, b = bh / a.H, h = bh - b * a.H;
    pdl_wait();
    const KvPagedRequest rq = kvp_request(a, b);
    if (!rq.ok && blockIdx.x == 0 && blockIdx.z == 0 && tid == 0)
        report_error(FP4LIN_ERR_OUT_OF_RANGE);
    const int rows = rq.n * a.G, row0 = blockIdx.z * R;
    if (row0 >= rows || rows > a.max_rows)
        return;
    const int imin = row0 / a.G, imax = (min(row0 + R, rows) - 1) / a.G;
    const int k0 = blockIdx.x * a.chunk, kend = rq.len + imax + 1;  // keys the tile's last row sees
    if (k0 >= kend && !a.joined)
        return;
    const int k1 = min(kend, k0 + a.chunk);  // rows behind len + n hold anything, and are not read
    const int P1 = (1 << a.shift) - 1;

    const int groups = max(0, k1 - k0 + 15) / 16;  // of 16 keys, which lie in one page
    for (int i = tid; i < groups; i += KVP_THREADS) {
        const int page = a.table[b * a.ld_t + ((k0 + 16 * i) >> a.shift)];
        const bool ok = page >= 0 && page < a.NP;
        if (!ok)
            report_error(FP4LIN_ERR_OUT_OF_RANGE);
        s_page[i] = ok ? page : -1;
    }
    uint32_t qb[NT][KW][2];
    float qs[NT][2];
    int lim[NT][2];  // last key that this lane's rows (columns 2t, 2t+1 of the scores) see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int rho = row0 + 8 * nt + g, i = rho / a.G, j = rho - i * a.G;
        const bool live = rho < rows;
        const float s = kvp_load_q<D>(a.q + (int64_t)(rq.first + (live ? i : 0)) * a.ld_q + (h * a.G + (live ? j : 0)) * D +
                                          t * (D / 4),
                                      live, qb[nt]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            qs[nt][c] = __shfl_sync(0xffffffffu, s, (2 * t + c) * 4) * a.qscale;
            const int r = row0 + 8 * nt + 2 * t + c;
            lim[nt][c] = r < rows ? rq.len + r / a.G : -1;
        }
    }
    __syncthreads();

    uint32_t kr[2][2][KW], vr[2][4][VW];
    // A group of 16 keys is in one page: its rows lie together, and in bounds even where the request
    // ends within them (scores of keys behind it are masked, its values dropped below).
    auto group = [&](int key, bool &go) {
        const int page = key < k1 ? s_page[(key - k0) >> 4] : -1;
        go = page >= 0;
        return ((((int64_t)page * a.H + h) << a.shift) + (key & P1)) * D;
    };
    auto load_k = [&](int kb) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bool go;
            const uint8_t *p = a.kc + group(kb + 16 * u, go) + g * D + t * (D / 4);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int w = 0; w < KW; w += 4) {
                    const uint4 x = ld_nc_v4_if(p + 8 * e * D + 4 * w, go);
                    kr[u][e][w] = x.x;
                    kr[u][e][w + 1] = x.y;
                    kr[u][e][w + 2] = x.z;
                    kr[u][e][w + 3] = x.w;
                }
        }
    };
    auto load_v = [&](int kb) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bool go;
            const uint8_t *p = a.vc + group(kb + 16 * u, go) + 2 * t * D + g * (D / 8);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = (e & 1) + 8 * (e >> 1);
                if constexpr (VW == 4) {
                    const uint4 x = ld_nc_v4_if(p + row * D, go);
                    vr[u][e][0] = x.x;
                    vr[u][e][1] = x.y;
                    vr[u][e][2] = x.z;
                    vr[u][e][3] = x.w;
                } else {
                    const uint2 x = ld_nc_v2_if(p + row * D, go);
                    vr[u][e][0] = x.x;
                    vr[u][e][1] = x.y;
                }
            }
        }
    };

    float o[NT][D / 16][4], den[NT][2], M[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        M[nt][0] = M[nt][1] = -INFINITY;
        den[nt][0] = den[nt][1] = 0.0f;
#pragma unroll
        for (int u = 0; u < D / 16; ++u)
            o[nt][u][0] = o[nt][u][1] = o[nt][u][2] = o[nt][u][3] = 0.0f;
    }
    bool nan = false;
    int kb = k0 + warp * KVP_STEP;
    load_k(kb);
    load_v(kb);
    bool zeros = false;
    for (int i = tid; i < groups; i += KVP_THREADS) {  // the scales, while the first rows are on their way
        const int page = s_page[i];
        const bool ok = page >= 0;
        const uint32_t kbyte = ok ? a.ks[(int64_t)page * a.H + h] : 0u, vbyte = ok ? a.vs[(int64_t)page * a.H + h] : 0u;
        s_kf[i] = mxfp8_scale(kbyte);
        // no page: weight 0; a page of zeros: infinite for now
        s_xv[i] = ok ? (vbyte ? (float)((int)vbyte - 127) : INFINITY) : -INFINITY;
        zeros |= ok && !vbyte;
    }
    if (__syncthreads_or(zeros)) {
        float low = INFINITY;
        for (int i = lane; i < groups; i += 32)
            low = fminf(low, s_xv[i] == -INFINITY ? INFINITY : s_xv[i]);
        low = kvp_zero_exponent(warp_min(low));
        __syncthreads();
        for (int i = tid; i < groups; i += KVP_THREADS)
            s_xv[i] = s_xv[i] == INFINITY ? low : s_xv[i];
        __syncthreads();
    }
    for (; kb < k1; kb += KVP_WARPS * KVP_STEP) {
        const bool more = kb + KVP_WARPS * KVP_STEP < k1;
        float s[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16(kr[u][0][w], a0, a2);
                e4m3x4_to_f16(kr[u][1][w], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_16816x(s[u][nt], a0, a1, a2, a3, qb[nt][w][0], qb[nt][w][1]);
            }
        }
        if (more)
            load_k(kb + KVP_WARPS * KVP_STEP);
        float xv[2], c[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = (kb + 16 * u - k0) >> 4;
            const bool in = kb + 16 * u < k1;
            const float kf = in ? s_kf[i] : 0.0f;
            xv[u] = in ? s_xv[i] : -INFINITY;
            c[u] = ex2(-xv[u]) * pow2_const(-KVP_BIAS);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[u][nt][e] = fmaf(s[u][nt][e] * qs[nt][e & 1], kf, xv[u]);
        }
        if (kb + KVP_STEP - 1 > rq.len + imin || row0 + R > rows) {  // some row does not see some key
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (kb + 16 * u + g + 8 * (e >> 1) > lim[nt][e & 1])
                            s[u][nt][e] = -INFINITY;
        }
        uint32_t wb[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float corr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                m = fmaxf(m - KVP_BIAS, M[nt][e]);
                const float base = m == -INFINITY ? 0.0f : m;
                corr[e] = ex2(M[nt][e] - base);
                M[nt][e] = m;
                float add = 0.0f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float w0 = ex2(s[u][nt][e] - base), w1 = ex2(s[u][nt][e + 2] - base);
                    s[u][nt][e] = w0;
                    s[u][nt][e + 2] = w1;
                    add = xv[u] == -INFINITY ? add : fmaf(w0 + w1, c[u], add);
                }
                den[nt][e] = fmaf(den[nt][e], corr[e], add);
            }
            if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {
                    o[nt][u][0] *= corr[0];
                    o[nt][u][1] *= corr[1];
                    o[nt][u][2] *= corr[0];
                    o[nt][u][3] *= corr[1];
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                wb[u][nt][0] = movmatrix(cvt_f16x2_finite(s[u][nt][0], s[u][nt][1]));
                wb[u][nt][1] = movmatrix(cvt_f16x2_finite(s[u][nt][2], s[u][nt][3]));
            }
        }
        if (kb + KVP_STEP - 1 > rq.len + imin) {
            // a weight of 0 must stay 0: rows behind the end hold anything, and a NaN code among the keys
            // that not every row sees is dropped here and put in where it is seen at the end
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = kb + 16 * u + 2 * t + (e & 1) + 8 * (e >> 1);
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        if (key >= k1)
                            vr[u][e][w] = 0u;
                        else if (key > rq.len + imin)
                            nan |= drop_nan_codes(vr[u][e][w]);
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t sel = x ? 0x7362u : 0x5140u;
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16(__byte_perm(vr[u][0][w], vr[u][1][w], sel), a0, a1);
                    e4m3x4_to_f16(__byte_perm(vr[u][2][w], vr[u][3][w], sel), a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816x(o[nt][2 * w + x], a0, a1, a2, a3, wb[u][nt][0], wb[u][nt][1]);
                }
        if (more)
            load_v(kb + KVP_WARPS * KVP_STEP);
    }

    // the warps' shares: lane (g, t) holds dimensions g*D/8 + 2u, +1 of rows 2t, 2t+1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float d = den[nt][e];
            d += __shfl_xor_sync(0xffffffffu, d, 4);
            d += __shfl_xor_sync(0xffffffffu, d, 8);
            d += __shfl_xor_sync(0xffffffffu, d, 16);
            const int r = 8 * nt + 2 * t + e;
            if (g == 0) {
                s_m[warp][r] = M[nt][e];
                s_den[warp][r] = d;
            }
#pragma unroll
            for (int u = 0; u < D / 16; ++u)
                *reinterpret_cast<float2 *>(&s_o[warp][r][g * (D / 8) + 2 * u]) = make_float2(o[nt][u][e], o[nt][u][e + 2]);
        }
    const bool any_nan = __syncthreads_or(nan);
    const int live_rows = min(R, rows - row0);
    const int64_t part = ((int64_t)bh * a.tiles + blockIdx.z) * a.S + blockIdx.x;
    auto write_out = [&](int r, int d, float sum, const float *v) {
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : sum == 0.0f ? 0.0f : sum;
        const int rho = row0 + r, tok = rho / a.G, j = rho - tok * a.G;
        uint2 y;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.x) : "f"(v[1] * inv), "f"(v[0] * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.y) : "f"(v[3] * inv), "f"(v[2] * inv));
        *reinterpret_cast<uint2 *>(a.out + ((int64_t)(rq.first + tok) * a.H * a.G + h * a.G + j) * D + d) = y;
    };
    for (int i = tid; i < live_rows * (D / 4); i += KVP_THREADS) {
        const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        float m = s_m[0][r];
#pragma unroll
        for (int w = 1; w < KVP_WARPS; ++w)
            m = fmaxf(m, s_m[w][r]);
        const float base = m == -INFINITY ? 0.0f : m;
        float sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < KVP_WARPS; ++w) {
            const float f = ex2(s_m[w][r] - base);
            sum = fmaf(f, s_den[w][r], sum);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = fmaf(f * pow2_const(-KVP_BIAS), s_o[w][r][d + j], v[j]);
        }
        if (any_nan) {
            const int last = min(k1 - 1, rq.len + (row0 + r) / a.G);
            for (int key = max(k0, rq.len + imin + 1); key <= last; ++key) {
                const int page = s_page[(key - k0) >> 4];
                const uint8_t *p = a.vc + ((((int64_t)page * a.H + h) << a.shift) + (key & P1)) * D + d;
                for (int j = 0; page >= 0 && j < 4; ++j)
                    if ((p[j] & 127) == 127)
                        v[j] = __int_as_float(0x7fc00000);
            }
        }
        if (a.S == 1) {
            write_out(r, d, sum, v);
        } else if (a.joined) {
            *reinterpret_cast<float4 *>(&s_o[0][r][d]) = make_float4(v[0], v[1], v[2], v[3]);  // read by this thread alone
            if (d == 0) {
                s_cm[r] = m;
                s_cden[r] = sum;
            }
        } else {
            float *dst = a.ws + (part * R + r) * (D + 4);
            *reinterpret_cast<float4 *>(dst + d) = make_float4(v[0], v[1], v[2], v[3]);
            if (d == 0)
                *reinterpret_cast<float2 *>(dst + D) = make_float2(m, sum);
        }
    }
    if (!a.joined)
        return;
    // the splits of the cluster, each CTA a share of the outputs
    cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
    cl.sync();
    for (int i = tid * a.S + (int)blockIdx.x; i < live_rows * (D / 4); i += KVP_THREADS * a.S) {
        const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        float m[8], den[8], v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float4 o4[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int from = q < a.S ? q : 0;
            m[q] = q < a.S ? *cl.map_shared_rank(&s_cm[r], from) : -INFINITY;
            den[q] = *cl.map_shared_rank(&s_cden[r], from);
            o4[q] = *reinterpret_cast<const float4 *>(cl.map_shared_rank(&s_o[0][r][d], from));
        }
        float top = m[0], sum = 0.0f;
#pragma unroll
        for (int q = 1; q < 8; ++q)
            top = fmaxf(top, m[q]);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < a.S) {
                const float f = ex2(m[q] - base);
                sum = fmaf(f, den[q], sum);
                v[0] = fmaf(f, o4[q].x, v[0]);
                v[1] = fmaf(f, o4[q].y, v[1]);
                v[2] = fmaf(f, o4[q].z, v[2]);
                v[3] = fmaf(f, o4[q].w, v[3]);
            }
        }
        write_out(r, d, sum, v);
    }
    cl.sync();  // no CTA leaves while it is read
}

// Joins a row's splits: o = sum_s 2^(M_s - M) o_s / sum_s 2^(M_s - M) den_s, by one warp, or, where there
// are many, by the CTA, whose warps take every KVP_WARPS-th and then meet.  src: the row's first split,
// `step` floats from one to the next.
template <int D, bool CTA>
__device__ __forceinline__ void kvp_merge_row(const float *src, int64_t step, int splits, __nv_bfloat16 *dst)
{
    constexpr int V = D / 32, W = CTA ? KVP_WARPS : 1;
    __shared__ float part[KVP_WARPS][D + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s0 = CTA ? warp : 0;
    float M = -INFINITY, den = 0.0f, v[V] = {};
    for (int s = s0 + W * lane; s < splits; s += 32 * W)
        M = fmaxf(M, src[s * step + D]);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll 4
    for (int s = s0; s < splits; s += W) {
        const float *p = src + s * step;
        const float2 md = *reinterpret_cast<const float2 *>(p + D);
        const float f = ex2(md.x - base);
        den = fmaf(f, md.y, den);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 x = *reinterpret_cast<const float2 *>(p + lane * V + k);
            v[k] = fmaf(f, x.x, v[k]);
            v[k + 1] = fmaf(f, x.y, v[k + 1]);
        }
    }
    auto inverse = [](float d) { return d > 0.0f ? __fdiv_rn(1.0f, d) : d == 0.0f ? 0.0f : d; };
    if constexpr (!CTA) {
        const float inv = inverse(den);
#pragma unroll
        for (int k = 0; k < V; k += 2)
            *reinterpret_cast<__nv_bfloat162 *>(dst + lane * V + k) = __floats2bfloat162_rn(v[k] * inv, v[k + 1] * inv);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            part[warp][lane * V + k] = v[k];
        if (lane == 0) {
            part[warp][D] = M;
            part[warp][D + 1] = den;
        }
        __syncthreads();
        float f[KVP_WARPS], top = -INFINITY;
#pragma unroll
        for (int w = 0; w < KVP_WARPS; ++w)
            top = fmaxf(top, part[w][D]);
        den = 0.0f;
#pragma unroll
        for (int w = 0; w < KVP_WARPS; ++w) {
            f[w] = ex2(part[w][D] - (top == -INFINITY ? 0.0f : top));
            den = fmaf(f[w], part[w][D + 1], den);
        }
        const float inv = inverse(den);
        for (int d = threadIdx.x; d < D; d += KVP_THREADS) {
            float o = 0.0f;
#pragma unroll
            for (int w = 0; w < KVP_WARPS; ++w)
                o = fmaf(f[w], part[w][d], o);
            dst[d] = __float2bfloat16_rn(o * inv);
        }
        __syncthreads();
    }
}

template <int D>
__global__ void __launch_bounds__(KVP_THREADS) kv_paged_merge_kernel(KvPagedShape a, int R)
{
    const int bh = blockIdx.y, b = bh / a.H, h = bh - b * a.H, rho = blockIdx.x;
    pdl_wait();
    const KvPagedRequest rq = kvp_request(a, b);
    const int rows = rq.n * a.G;
    if (rho >= rows || rows > a.max_rows)
        return;
    const int z = rho / R, r = rho - z * R, i = rho / a.G, j = rho - i * a.G;
    const int imax = (min((z + 1) * R, rows) - 1) / a.G;
    const int splits = (rq.len + imax + a.chunk) / a.chunk;  // ceil((len + imax + 1) / chunk)
    const float *src = a.ws + (((int64_t)bh * a.tiles + z) * a.S * R + r) * (D + 4);
    kvp_merge_row<D, true>(src, (int64_t)R * (D + 4), splits,
                           a.out + ((int64_t)(rq.first + i) * a.H * a.G + h * a.G + j) * D);
}

}  // namespace fp4lin
