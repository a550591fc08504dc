// matvec.cuh -- y[m, n] = sum_k x[m, k] W[n, k] for a few rows of 16- or 8-bit activations and the
// library's 4-bit weights (codes [N, K/2], block scales in the tensor-core layout).
//
//   NVFP4: W = g * e2m1(code) * e4m3(sf), blocks of 16;  MXFP4: W = e2m1(code) * 2^(sf - 127), of 32.
//   x: bf16 (rotated on the way in by H_b / sqrt(b) when the weights are), or MXFP8 (mxfp8.cuh).
//
// Bound by HBM: 0.5 + 1/16 (1/32) bytes a weight, each read once; 2 M flops a weight.  A weight
// goes from a 256-bit load to a tensor-core fragment in registers: E2M1 times its scale is exact
// in f16 (at most 6 bits), so the scale costs one f16x2 multiply a pair and the product accumulates
// in binary32 over the whole slice of K.  Exponents that f16 cannot hold are taken out first:
//   x: scaled by a power of two (a row's largest magnitude in the slice lands in [2^14, 2^15));
//      what is below 2^-39 of that maximum is lost, less than binary32 sums resolve;
//   MXFP4 scales: relative to the row's largest in the segment; blocks more than 2^24 below it
//      lose bits that the sum could not hold either.
// Rotated activations are rounded to f16 once (2^-11 relative steps, against bf16 outputs).
//
// A CTA takes 128 weight rows and a slice of K; the CTAs of one row tile form a cluster (at most 8)
// and add their sums through distributed shared memory in a fixed order: one launch, no workspace,
// the same bits every time.
#pragma once

#include <cooperative_groups.h>

#include "kv_attention.cuh"  // mma_16816x, f16x2_bits
#include "mxfp8.cuh"
#include "quantize.cuh"

namespace fp4lin {

constexpr int MV_THREADS = 256;
constexpr int MV_ROWS = 128;       // weight rows a CTA: 8 warps x 16
constexpr int MV_CHUNK = 256;      // k a warp step: 64 consecutive values a lane and row
constexpr int MV_SEG = 8;          // chunks a segment: x and the scales are normalised once per segment
constexpr int MV_MAX_M = 16;

struct MatvecShape {
    const void *x;                 // bf16 [M, K] or E4M3 [M, K]
    const uint8_t *xs;             // E8M0, tensor-core layout of [M, K/32] (MXFP8 x)
    const uint8_t *w, *ws;
    const float *g;
    __nv_bfloat16 *y;
    int64_t ld_x, ldy, katoms_w, katoms_x;
    int M, N, K, nchunks, per_cta; // per_cta: chunks a CTA of the cluster takes
    bool wide_w, wide_x;
};

// Shared memory: a segment's x as B fragments (16 bytes for 8 consecutive k of one row), the
// per-row exponents, and the CTA's sums.
constexpr size_t mv_smem(int M, int chunks)
{
    return (size_t)chunks * MV_CHUNK * M * 2 + MV_MAX_M * 4 + (size_t)MV_ROWS * M * 4;
}

// 32 consecutive values of row m at column k as binary32, rotated where asked.
template <bool X8, int HAD>
__device__ __forceinline__ void mv_load_x(const MatvecShape &a, int m, int k, float *v)
{
    if constexpr (X8) {
        const uint8_t *p = static_cast<const uint8_t *>(a.x) + m * a.ld_x + k;
        const float s = mxfp8_scale(a.xs[tc_offset(m, k / 32, a.katoms_x)]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + 16 * i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t lo, hi;
                e4m3x4_to_f16(w[j], lo, hi);
                const float2 p0 = half2_to_float2(lo), p1 = half2_to_float2(hi);
                v[16 * i + 4 * j] = p0.x * s;
                v[16 * i + 4 * j + 1] = p0.y * s;
                v[16 * i + 4 * j + 2] = p1.x * s;
                v[16 * i + 4 * j + 3] = p1.y * s;
            }
        }
    } else {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.x) + m * a.ld_x + k;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            bf16x8_to_f32(*reinterpret_cast<const uint4 *>(p + 8 * i), v + 8 * i);
        if constexpr (HAD == 16) {
            fwht_scaled_packed<16>(v, 0.25f);
            fwht_scaled_packed<16>(v + 16, 0.25f);
        } else if constexpr (HAD == 32) {
            fwht_scaled_packed<32>(v, __uint_as_float(0x3E3504F3u));
        }
    }
}

// Eight E2M1 codes times the f16x2 scale `s` (both halves): four f16x2, exact.
__device__ __forceinline__ void mv_weights(uint32_t w, uint32_t s, uint32_t *h)
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 t0, t1, t2, t3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 t0, b0;\n\tcvt.rn.f16x2.e2m1x2 t1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 t2, b2;\n\tcvt.rn.f16x2.e2m1x2 t3, b3;\n\t"
        "mul.rn.f16x2 %0, t0, %5;\n\tmul.rn.f16x2 %1, t1, %5;\n\t"
        "mul.rn.f16x2 %2, t2, %5;\n\tmul.rn.f16x2 %3, t3, %5;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w), "r"(s));
}

// f16x2 of 2^-d for d >= 0: 0 from 25 on.
__device__ __forceinline__ uint32_t mv_pow2_neg(uint32_t d)
{
    const uint32_t h = d <= 14u ? (15u - d) << 10 : d <= 24u ? 1u << (24u - d) : 0u;
    return h | (h << 16);
}

// One warp: 16 weight rows.  MMA row p (0..15) is the tile's row 32 q + 4 warp + i with i = p % 4 and
// q = 2 (p/4 % 2) + p/8: a lane's two rows (p = g and g + 8) then have neighbouring words in a scale
// atom, and the warp's scale bytes fill whole 64-byte runs.
template <bool NV, bool X8, int HAD, int NT>
__global__ void __launch_bounds__(MV_THREADS, 2) matvec_kernel(MatvecShape a)
{
    extern __shared__ __align__(16) uint8_t mv_dyn[];
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
    const int tile = blockIdx.x / ranks;
    const int c0 = rank * a.per_cta, c1 = min(c0 + a.per_cta, a.nchunks);
    uint4 *s_x = reinterpret_cast<uint4 *>(mv_dyn);
    const int seg_chunks = min(a.per_cta, MV_SEG);
    float *s_scale = reinterpret_cast<float *>(mv_dyn + (size_t)seg_chunks * MV_CHUNK * a.M * 2);
    float *s_y = s_scale + MV_MAX_M;  // [M][128]

    const int q0 = 2 * (g >> 2), in_tile = 4 * warp + (g & 3);
    const int rowA = tile * MV_ROWS + 32 * q0 + in_tile, rowB = rowA + 32;
    const uint8_t *wA = a.w + (int64_t)rowA * (a.K / 2), *wB = a.w + (int64_t)rowB * (a.K / 2);
    const bool liveA = rowA < a.N, liveB = rowB < a.N;
    // this lane's two scale words: atom (tile, ct), row in_tile, words q0 and q0 + 1
    const uint8_t *sc = a.ws + (int64_t)tile * a.katoms_w * 512 + in_tile * 16 + q0 * 4;

    // The scale bytes of 64 values from k on, rows A and B (MXFP4: in the low 16 bits, as 64 values are
    // half of an atom's 4 columns).  Through L1: the neighbouring lanes' words share its sectors.
    auto ld_scales = [&](int k, bool in) {
        uint2 s = make_uint2(0u, 0u);
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t@q ld.global.nc.v2.u32 {%0,%1}, [%2];\n\t}"
                     : "+r"(s.x), "+r"(s.y)
                     : "l"(sc + (int64_t)(k / (NV ? 64 : 128)) * 512), "r"((uint32_t)in));
        return s;
    };
    auto half_of = [&](uint2 s) { return NV || !(t & 1) ? s : make_uint2(s.x >> 16, s.y >> 16); };
    auto load_w = [&](int c, uint32_t *ra, uint32_t *rb, uint2 &s) {
        const int k = c * MV_CHUNK + 64 * t;
        const bool in = c < c1 && k < a.K;
        ld_nc_32B_if(wA + k / 2, a.wide_w, in && liveA, ra);
        ld_nc_32B_if(wB + k / 2, a.wide_w, in && liveB, rb);
        s = ld_scales(k, in);
    };

    float tot[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        tot[nt][0] = tot[nt][1] = tot[nt][2] = tot[nt][3] = 0.0f;
    pdl_wait();
    const float gw = NV ? *a.g : 1.0f;
    for (int sb = c0; sb < c1; sb += MV_SEG) {
        const int se = min(sb + MV_SEG, c1);
        uint32_t wa[2][8], wb[2][8];
        uint2 ws[2];
        load_w(sb, wa[0], wb[0], ws[0]);
        // stage x: largest magnitude per row, then f16 fragments
        const int kb = sb * MV_CHUNK, kn = min(se * MV_CHUNK, a.K) - kb, blocks = kn / 32;
        __syncthreads();  // the previous segment's fragments are done with
        for (int m = warp; m < a.M; m += MV_THREADS / 32) {
            float top = 0.0f;
            for (int i = lane; i < blocks; i += 32) {
                float v[32];
                mv_load_x<X8, HAD>(a, m, kb + 32 * i, v);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    top = fmaxf(top, finite_abs(v[j]));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // 2^(14 - e), e the exponent of `top`; both it and its inverse stay normal
            const uint32_t e = top > 0.0f ? min(max(__float_as_uint(top) >> 23, 15u), 253u) : 141u;
            const float inv = __uint_as_float((268u - e) << 23);
            if (lane == 0)
                s_scale[m] = __uint_as_float((e - 14u) << 23);
            for (int i = lane; i < (se - sb) * (MV_CHUNK / 32); i += 32) {
                float v[32];
                if (i < blocks)
                    mv_load_x<X8, HAD>(a, m, kb + 32 * i, v);
                else
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = 0.0f;
                // chunk i/8, lane slot t = (i/2)%4, words 4*(i%2) .. +3
                const int c = i >> 3, tt = (i >> 1) & 3, w0 = 4 * (i & 1);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint4 f;
                    f.x = f16x2_bits(v[8 * w] * inv, v[8 * w + 1] * inv);
                    f.y = f16x2_bits(v[8 * w + 2] * inv, v[8 * w + 3] * inv);
                    f.z = f16x2_bits(v[8 * w + 4] * inv, v[8 * w + 5] * inv);
                    f.w = f16x2_bits(v[8 * w + 6] * inv, v[8 * w + 7] * inv);
                    s_x[((c * 8 + w0 + w) * a.M + m) * 4 + tt] = f;
                }
            }
        }
        uint32_t refA = 0u, refB = 0u;  // MXFP4: the rows' largest scale bytes in the segment
        if constexpr (!NV) {
            for (int c = sb; c < se; ++c) {
                const int k = c * MV_CHUNK + 64 * t;
                const uint2 s = half_of(ld_scales(k, k < a.K));
                refA = max(refA, max(s.x & 255u, (s.x >> 8) & 255u));
                refB = max(refB, max(s.y & 255u, (s.y >> 8) & 255u));
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                refA = max(refA, __shfl_xor_sync(0xffffffffu, refA, o));
                refB = max(refB, __shfl_xor_sync(0xffffffffu, refB, o));
            }
        }
        __syncthreads();
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
        auto multiply = [&](int c, const uint32_t *va, const uint32_t *vb, uint2 raw) {
            const uint2 sw = half_of(raw);
            uint32_t sA[4], sB[4];  // f16x2 scales of the lane's 16-value quarters
            if constexpr (NV) {
                uint32_t a01, a23, b01, b23;
                e4m3x4_to_f16(sw.x, a01, a23);
                e4m3x4_to_f16(sw.y, b01, b23);
                sA[0] = __byte_perm(a01, a01, 0x1010);
                sA[1] = __byte_perm(a01, a01, 0x3232);
                sA[2] = __byte_perm(a23, a23, 0x1010);
                sA[3] = __byte_perm(a23, a23, 0x3232);
                sB[0] = __byte_perm(b01, b01, 0x1010);
                sB[1] = __byte_perm(b01, b01, 0x3232);
                sB[2] = __byte_perm(b23, b23, 0x1010);
                sB[3] = __byte_perm(b23, b23, 0x3232);
            } else {
                sA[0] = sA[1] = mv_pow2_neg(refA - (sw.x & 255u));
                sA[2] = sA[3] = mv_pow2_neg(refA - ((sw.x >> 8) & 255u));
                sB[0] = sB[1] = mv_pow2_neg(refB - (sw.y & 255u));
                sB[2] = sB[3] = mv_pow2_neg(refB - ((sw.y >> 8) & 255u));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t ha[4], hb[4];
                mv_weights(va[i], sA[i >> 1], ha);
                mv_weights(vb[i], sB[i >> 1], hb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int m = 8 * nt + g;
                    const uint4 f = m < a.M ? s_x[(((c - sb) * 8 + i) * a.M + m) * 4 + t] : make_uint4(0u, 0u, 0u, 0u);
                    mma_16816x(acc[nt], ha[0], hb[0], ha[1], hb[1], f.x, f.y);
                    mma_16816x(acc[nt], ha[2], hb[2], ha[3], hb[3], f.z, f.w);
                }
            }
        };
        for (int c = sb; c < se; c += 2) {
            if (c + 1 < se)
                load_w(c + 1, wa[1], wb[1], ws[1]);
            multiply(c, wa[0], wb[0], ws[0]);
            if (c + 1 < se) {
                if (c + 2 < se)
                    load_w(c + 2, wa[0], wb[0], ws[0]);
                multiply(c + 1, wa[1], wb[1], ws[1]);
            }
        }
        const float fA = NV ? gw : mxfp8_scale(refA), fB = NV ? gw : mxfp8_scale(refB);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // columns 2t, 2t+1 of the token tile
                const int m = 8 * nt + 2 * t + e;
                const float xs = m < a.M ? s_scale[m] : 0.0f;
                tot[nt][e] = fmaf(acc[nt][e] * xs, fA, tot[nt][e]);
                tot[nt][e + 2] = fmaf(acc[nt][e + 2] * xs, fB, tot[nt][e + 2]);
            }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = 8 * nt + 2 * t + e;
            if (m < a.M) {
                s_y[m * MV_ROWS + 32 * q0 + in_tile] = tot[nt][e];
                s_y[m * MV_ROWS + 32 * q0 + 32 + in_tile] = tot[nt][e + 2];
            }
        }
    cl.sync();
    // this CTA's share of the tile's outputs: rows rank, rank + ranks, .. of M * 128 / 32 groups of 32
    for (int i = rank * 32 + (tid & 31) + (tid >> 5) * 32 * ranks; i < a.M * MV_ROWS; i += ranks * MV_THREADS) {
        float sum = 0.0f;
        for (int r = 0; r < ranks; ++r)
            sum += *cl.map_shared_rank(s_y + i, r);
        const int m = i / MV_ROWS, n = tile * MV_ROWS + (i - m * MV_ROWS);
        if (n < a.N)
            a.y[m * a.ldy + n] = __float2bfloat16_rn(sum);
    }
    cl.sync();  // no CTA leaves while its sums are read
}

}  // namespace fp4lin
