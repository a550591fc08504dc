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
//   x, bf16: scaled by a power of two (a row's largest magnitude in 256 values lands in [2^14, 2^15));
//      what is below 2^-39 of that maximum is lost, less than binary32 sums resolve where that value
//      meets a weight;
//   x, MXFP8: the row's largest scale in 256 values becomes 2^MV_X8_TOP, so that codes reach 28672.
//      Exact for blocks whose scale is down to 2^-21 of it, the others are rounded to 2^-30 of it (with
//      the largest at 1, codes of a block 2^16 below it lost bits and from 2^25 on all of them, which is
//      the whole answer where the larger block meets zero weights);
//   MXFP4 scales: the row's largest in 256 values becomes 2^MV_W4_TOP, so that weights reach 49152.  Exact
//      for blocks whose scale is down to 2^-36 of it, rounded at 2^-37, zero below (with the largest at 1
//      blocks 2^24 below it lost bits, all there is where x is zero under the larger one).
// Rotated activations are rounded to f16 once (2^-11 relative steps, against bf16 outputs).
//
// What it takes to come near HBM's rate with so few bytes is little to wait for before the weights are
// asked for, and little to do for each.  A CTA takes 128 weight rows, 16 a warp, and a slice of K; the
// CTAs that share rows form a cluster (at most 8) along K.  The partial sums of a row go to one CTA of
// the cluster through distributed shared memory and are added in a fixed order: one launch, no
// workspace, the same bits every time.  Between launches of a graph, weights from HBM: NVFP4,
// one rotated row, 4096 x 4096 4.9 us; five rows, 4096 x 14336 14.0 us (2.4 TB/s); MXFP4, sixteen 8-bit rows,
// 14336 x 4096 19.5 us, of which ~9 us are the weights' loads alone (two chunks of each warp in flight), the
// rest the conversions, scales and products of 16 warps an SM.
#pragma once

#include <cooperative_groups.h>

#include "kv_attention.cuh"  // mma_16816x
#include "kv_paged.cuh"      // f16x2_pow2
#include "mxfp8.cuh"
#include "quantize.cuh"

namespace fp4lin {

constexpr int MV_THREADS = 256;
constexpr int MV_WARPS = MV_THREADS / 32;
constexpr int MV_ROWS = 128;       // rows of the scale layout's tiles: 8 groups of 16
constexpr int MV_CHUNK = 256;      // k a warp step: 64 consecutive values a lane and row
constexpr int MV_SEG = 8;          // chunks of x that a CTA holds at a time
constexpr int MV_DEPTH = 2;        // chunks of weights that a warp has in flight
constexpr int MV_MAX_M = 16;
constexpr int MV_X8_TOP = 6;       // log2 of the largest MXFP8 scale in f16: 448 times that is below 2^15
constexpr int MV_W4_TOP = 13;      // of the largest MXFP4 scale: 6 times that is below 2^16

struct MatvecShape {
    const void *x;                 // bf16 [M, K] or E4M3 [M, K]
    const uint8_t *xs;             // E8M0, tensor-core layout of [M, K/32] (MXFP8 x)
    const uint8_t *w, *ws;
    const float *g;
    __nv_bfloat16 *y;
    int64_t ld_x, ldy, katoms_w, katoms_x;
    int M, N, K, nchunks, per_cta; // per_cta: chunks a CTA of the cluster takes
    int mp_shift;                  // 1 << mp_shift: M rounded up to a power of two, at most 8
    bool wide_w;
};

// Rows of x from one word of a lane's 64 values to the next in shared memory.  Odd, and lane slot t of word
// i sits at t ^ (i / 2): eight lanes that write one row's words, or read eight rows' word, meet each bank
// once (with a stride of 16 and no exchange the writes took 32 cycles a warp, and 16 rows of 14336 x 4096
// MXFP4 weights 20.2 us instead of 17.8).
__host__ __device__ constexpr int mv_stride(int M) { return M | 1; }

// Shared memory: a segment's x as B fragments (16 bytes for 8 consecutive k of one row) with the
// scale of each (chunk, row), and the partial sums that the cluster's warps send this CTA.
constexpr size_t mv_smem(int M, int chunks, int ranks)
{
    return (size_t)chunks * MV_CHUNK * mv_stride(M) * 2 + MV_SEG * MV_MAX_M * 4 + (size_t)ranks * M * ((MV_ROWS + ranks - 1) / ranks) * 4;
}

// A lane's share of a (row, chunk) of x: 8 consecutive values, raw.
struct MvRaw {
    uint4 v;        // bf16; MXFP8: codes in x, y
    uint32_t byte;  // MXFP8: the block's scale
};

// x and xs point at this lane's share of chunk 0.
template <bool X8>
__device__ __forceinline__ MvRaw mv_load_x(const uint8_t *x, const uint8_t *xs, int c, bool go)
{
    MvRaw r;
    r.byte = 0u;
    if constexpr (X8) {
        const uint2 v = ld_nc_v2_if(x + c * MV_CHUNK, go);
        r.v = make_uint4(v.x, v.y, 0u, 0u);
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.nc.u8 %0, [%1];\n\t}"
                     : "+r"(r.byte)
                     : "l"(xs + c * 1024), "r"((uint32_t)go));  // 8 columns of the scale layout are two atoms
    } else {
        r.v = ld_nc_v4_if(x + c * (MV_CHUNK * 2), go);
    }
    return r;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The power of two that takes a magnitude with these binary32 bits to [2^14, 2^15), and its inverse;
// both stay normal.
__device__ __forceinline__ uint32_t mv_exponent(uint32_t top) { return top ? min(max(top >> 23, 15u), 253u) : 141u; }
__device__ __forceinline__ float mv_inverse(uint32_t top) { return __uint_as_float((268u - mv_exponent(top)) << 23); }
__device__ __forceinline__ float mv_scale(uint32_t top) { return __uint_as_float((mv_exponent(top) - 14u) << 23); }

// A (row, chunk) of x, 8 values a lane, as f16 fragments (f) under one power of two (returned).  The
// whole warp calls it.  MXFP8: the codes relative to the chunk's largest scale.
// bf16: relative to the largest magnitude, rotated first where asked (a rotation's block is 2 or 4
// lanes' values).
template <bool X8, int HAD>
__device__ __forceinline__ float mv_stage(const MvRaw &r, int lane, uint4 &f)
{
    if constexpr (X8) {
        const uint32_t ref = __reduce_max_sync(0xffffffffu, r.byte);
        // two factors: the first leaves every code exact (2^-9 * 2^-14 is a subnormal f16), the second,
        // where the block is further down, rounds once
        const int k = (int)(ref - r.byte), near = min(k, MV_X8_TOP + 14);
        const uint32_t s = f16x2_pow2(MV_X8_TOP - near);
        uint32_t h[4];
        e4m3x4_to_f16(r.v.x, h[0], h[1]);
        e4m3x4_to_f16(r.v.y, h[2], h[3]);
        f = make_uint4(mul_f16x2(h[0], s), mul_f16x2(h[1], s), mul_f16x2(h[2], s), mul_f16x2(h[3], s));
        if (k > near) {
            const uint32_t s2 = f16x2_pow2(near - k);
            f = make_uint4(mul_f16x2(f.x, s2), mul_f16x2(f.y, s2), mul_f16x2(f.z, s2), mul_f16x2(f.w, s2));
        }
        return mxfp8_scale(ref) * (1.0f / (1 << MV_X8_TOP));
    } else {
        float v[8];
        bf16x8_to_f32(r.v, v);
        uint32_t top;
        if constexpr (HAD == 0) {
            const uint32_t m = 0x7FFF7FFFu;  // magnitudes; a NaN is passed over
            const uint32_t t2 = max_bf16x2(max_bf16x2(r.v.x & m, r.v.y & m), max_bf16x2(r.v.z & m, r.v.w & m));
            top = max(t2 << 16, t2 & 0xFFFF0000u);
        } else {
            fwht<8>(v);
#pragma unroll
            for (int o = 1; o < HAD / 8; o <<= 1)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float w = __shfl_xor_sync(0xffffffffu, v[j], o);
                    v[j] = lane & o ? __fsub_rn(w, v[j]) : __fadd_rn(v[j], w);
                }
            float t = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __fmul_rn(v[j], HAD == 16 ? 0.25f : __uint_as_float(0x3E3504F3u));
                t = fmaxf(t, fabsf(v[j]));
            }
            top = __float_as_uint(t);
        }
        top = __reduce_max_sync(0xffffffffu, top);  // bits in order, as no magnitude is negative
        const float inv = mv_inverse(top);
        f = make_uint4(cvt_f16x2(v[0] * inv, v[1] * inv), cvt_f16x2(v[2] * inv, v[3] * inv),
                       cvt_f16x2(v[4] * inv, v[5] * inv), cvt_f16x2(v[6] * inv, v[7] * inv));
        return mv_scale(top);
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

// n / d for n * d < 2^20 by a reciprocal (n up to 2048 here, d up to 128): 2^20/d rounded up is off by
// less than d/2^20 of 1/d.
struct SmallDiv {
    uint32_t inv;
    __device__ __forceinline__ explicit SmallDiv(int d) : inv((1u << 20) / (uint32_t)d + 1u) {}
    __device__ __forceinline__ int operator()(int n) const { return (int)(((uint32_t)n * inv) >> 20); }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// One warp: 16 weight rows.  MMA row p (0..15) of row group w is the 128-row tile's row 32 q + 4 w + i
// with i = p % 4 and q = 2 (p/4 % 2) + p/8: a lane's two rows (p = g and g + 8) then have neighbouring
// words in a scale atom, and the warp's scale bytes fill whole 64-byte runs.
template <bool NV, bool X8, int HAD, int NT>
__global__ void __launch_bounds__(MV_THREADS, 2) matvec_kernel(MatvecShape a)
{
    extern __shared__ __align__(16) uint8_t mv_dyn[];
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
    const int tile = blockIdx.x / ranks;
    const SmallDiv by_ranks(ranks);
    const int c0 = rank * a.per_cta, c1 = min(c0 + a.per_cta, a.nchunks);
    const int seg_chunks = min(a.per_cta, MV_SEG), ms = mv_stride(a.M);
    uint4 *s_x = reinterpret_cast<uint4 *>(mv_dyn);
    float *s_xs = reinterpret_cast<float *>(mv_dyn + (size_t)seg_chunks * MV_CHUNK * ms * 2);  // [chunk][MV_MAX_M]
    float *s_y = s_xs + MV_SEG * MV_MAX_M;           // [source rank][M][rows of this rank]
    const int own = (MV_ROWS + ranks - 1) / ranks;  // the CTA's row n is rank n % ranks'

    const int q0 = 2 * (g >> 2), in_tile = 4 * warp + (g & 3);
    const int rowA = tile * MV_ROWS + 32 * q0 + in_tile, rowB = rowA + 32;
    const uint8_t *wA = a.w + (int64_t)rowA * (a.K / 2), *wB = a.w + (int64_t)rowB * (a.K / 2);
    const bool liveA = rowA < a.N, liveB = rowB < a.N;
    // this lane's two scale words: atom (tile, ct), row in_tile, words q0 and q0 + 1
    const uint8_t *sc = a.ws + (int64_t)tile * a.katoms_w * 512 + in_tile * 16 + q0 * 4;

    // s: the scale bytes of 64 values of rows A and B (MXFP4: two of an atom's 4 columns).  Through L1,
    // as the neighbouring lanes' words share its sectors.
    auto load_w = [&](int c, bool go, uint32_t *ra, uint32_t *rb, uint2 &s) {
        const int k = c * MV_CHUNK + 64 * t;
        go = go && k < a.K;
        ld_nc_32B_if(wA + k / 2, a.wide_w, go && liveA, ra);
        ld_nc_32B_if(wB + k / 2, a.wide_w, go && liveB, rb);
        s = make_uint2(0u, 0u);
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t@q ld.global.nc.v2.u32 {%0,%1}, [%2];\n\t}"
                     : "+r"(s.x), "+r"(s.y)
                     : "l"(sc + (int64_t)(k / (NV ? 64 : 128)) * 512), "r"((uint32_t)go));
    };

    // the row of x that this lane's fragments come from: one behind the last repeats it (its sums are dropped)
    int xrow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        xrow[nt] = min(8 * nt + g, a.M - 1);
    float tot[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        tot[nt][0] = tot[nt][1] = tot[nt][2] = tot[nt][3] = 0.0f;
    pdl_wait();
    cluster_arrive();  // completed before a CTA writes into another: by then all have started
    for (int sb = c0; sb < c1; sb += MV_SEG) {
        const int se = min(sb + MV_SEG, c1);
        // Stage x while the weights are on their way.  A warp has a row of x (two where M > 8) and every
        // 8/Mp-th chunk of it, Mp = M rounded up to a power of two, at most 8; BATCH chunks are loaded
        // together.  A chunk's largest magnitude is the warp's own business.
        constexpr int BATCH = 4;
        const int xm = warp & ((1 << a.mp_shift) - 1), xc = warp >> a.mp_shift, xstep = MV_WARPS >> a.mp_shift;
        const int chunks = se - sb, xk = sb * MV_CHUNK + 8 * lane;
        MvRaw raw[BATCH];
        auto load_x = [&](int m, int c) {
            const uint8_t *x = static_cast<const uint8_t *>(a.x) + (m * a.ld_x + xk) * (X8 ? 1 : 2);
            const uint8_t *xs = X8 ? a.xs + tc_offset(m, xk / 32, a.katoms_x) : nullptr;
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int cb = c + b * xstep;
                raw[b] = mv_load_x<X8>(x, xs, cb, m < a.M && cb < chunks && xk + cb * MV_CHUNK < a.K);
            }
        };
        load_x(xm, xc);
        uint32_t wa[MV_DEPTH][8], wb[MV_DEPTH][8];
        uint2 ws[MV_DEPTH];
#pragma unroll
        for (int d = 0; d < MV_DEPTH; ++d)
            load_w(sb + d, sb + d < se, wa[d], wb[d], ws[d]);
        __syncthreads();  // the last segment's fragments are done with
#pragma unroll 1
        for (int m = xm; m < a.M; m += 8) {
            // word i = lane % 8 of lane slot t = lane / 8
            uint4 *to = s_x + ((lane & 7) * ms + m) * 4 + ((lane >> 3) ^ ((lane & 7) >> 1));
#pragma unroll 1
            for (int c = xc; c < chunks; c += BATCH * xstep) {
                if (m != xm || c != xc)
                    load_x(m, c);
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const int cb = c + b * xstep;
                    if (cb < chunks) {
                        uint4 f;
                        const float scale = mv_stage<X8, HAD>(raw[b], lane, f);
                        to[cb * 32 * ms] = f;
                        if (lane == 0)
                            s_xs[cb * MV_MAX_M + m] = NV ? scale : scale * (1.0f / (1 << MV_W4_TOP));
                    }
                }
            }
        }
        __syncthreads();
        auto multiply = [&](int c, const uint32_t *va, const uint32_t *vb, uint2 sw) {
            uint32_t sA[4], sB[4];  // f16x2 scales of the lane's 16-value quarters
            float fA = 1.0f, fB = 1.0f;
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
                if (t & 1) {  // 64 values are half of an atom's 4 columns
                    sw.x >>= 16;
                    sw.y >>= 16;
                }
                const uint32_t a0 = sw.x & 255u, a1 = (sw.x >> 8) & 255u, b0 = sw.y & 255u, b1 = (sw.y >> 8) & 255u;
                uint32_t refA = max(a0, a1), refB = max(b0, b1);  // the rows' largest in the chunk
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) {
                    refA = max(refA, __shfl_xor_sync(0xffffffffu, refA, o));
                    refB = max(refB, __shfl_xor_sync(0xffffffffu, refB, o));
                }
                sA[0] = sA[1] = f16x2_pow2(MV_W4_TOP + (int)(a0 - refA));
                sA[2] = sA[3] = f16x2_pow2(MV_W4_TOP + (int)(a1 - refA));
                sB[0] = sB[1] = f16x2_pow2(MV_W4_TOP + (int)(b0 - refB));
                sB[2] = sB[3] = f16x2_pow2(MV_W4_TOP + (int)(b1 - refB));
                fA = mxfp8_scale(refA);
                fB = mxfp8_scale(refB);
            }
            // two sums side by side (four: 5% slower, the warps of an SM hide an MMA's latency already)
            constexpr int CHAINS = 2 / NT;
            float acc[CHAINS][NT][4];
#pragma unroll
            for (int q = 0; q < CHAINS; ++q)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    acc[q][nt][0] = acc[q][nt][1] = acc[q][nt][2] = acc[q][nt][3] = 0.0f;
            const uint4 *xc = s_x + (c - sb) * 32 * ms;
            const int step = 4 * ms;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t ha[4], hb[4];
                mv_weights(va[i], sA[i >> 1], ha);
                mv_weights(vb[i], sB[i >> 1], hb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 f = xc[i * step + 4 * xrow[nt] + (t ^ (i >> 1))];
                    mma_16816x(acc[(2 * i) % CHAINS][nt], ha[0], hb[0], ha[1], hb[1], f.x, f.y);
                    mma_16816x(acc[(2 * i + 1) % CHAINS][nt], ha[2], hb[2], ha[3], hb[3], f.z, f.w);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // columns 2t, 2t+1 of the token tile; rows A, A, B, B
                    float sum = acc[0][nt][e];
                    if constexpr (CHAINS == 2)
                        sum += acc[1][nt][e];
                    const float xs = s_xs[(c - sb) * MV_MAX_M + 8 * nt + 2 * t + (e & 1)];
                    tot[nt][e] = NV ? fmaf(sum, xs, tot[nt][e]) : fmaf(sum * xs, e < 2 ? fA : fB, tot[nt][e]);
                }
        };
#pragma unroll 1
        for (int c = sb; c < se; c += MV_DEPTH) {
#pragma unroll
            for (int d = 0; d < MV_DEPTH; ++d) {
                if (c + d < se) {
                    multiply(c + d, wa[d], wb[d], ws[d]);
                    if (c + d + MV_DEPTH < se)
                        load_w(c + d + MV_DEPTH, true, wa[d], wb[d], ws[d]);
                }
            }
        }
    }
    // each row's share goes to the CTA that sums it
    cluster_wait();
    {
        const int nA = 16 * warp + g, nB = nA + 8;  // rows in the CTA's own order: a warp's 16 MMA rows
        const int slot = rank * a.M * own;
        float *toA = cl.map_shared_rank(s_y, nA - by_ranks(nA) * ranks) + slot + by_ranks(nA);
        float *toB = cl.map_shared_rank(s_y, nB - by_ranks(nB) * ranks) + slot + by_ranks(nB);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = 8 * nt + 2 * t + e;
                if (m < a.M) {
                    toA[m * own] = tot[nt][e];
                    toB[m * own] = tot[nt][e + 2];
                }
            }
    }
    cluster_arrive();
    cluster_wait();
    const float gw = NV ? *a.g : 1.0f;
    const SmallDiv by_own(own);
    for (int i = tid; i < a.M * own; i += MV_THREADS) {
        const int m = by_own(i), n = (i - m * own) * ranks + rank;
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            sum += r < ranks ? s_y[r * a.M * own + i] : 0.0f;
        const int p = n & 15, row = tile * MV_ROWS + 32 * (2 * ((p >> 2) & 1) + (p >> 3)) + 4 * (n >> 4) + (p & 3);
        if (n < MV_ROWS && row < a.N)
            a.y[m * a.ldy + row] = __float2bfloat16_rn(sum * gw);
    }
}

}  // namespace fp4lin
