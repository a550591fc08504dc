// rmsnorm.cuh -- RMS norm with the residual's addition in front and an MXFP8 output behind.
//
//   s = bf16(x + r);  n = (s * (1 / sqrt(mean(s^2) + eps))) * w;  n' = H_b n / sqrt(b);
//   each 32 values of n': E8M0 byte and E4M3 codes as mxfp8.cuh defines them.
//
// Bound by HBM: 2 (x) + 2 (r) + 2 (s) + 1 (codes) + 1/32 (scales) bytes a value, read and written
// once: a lane holds one whole 32-value block of its row in registers from the load to the codes,
// so the row is read once, the rotation and the block maximum need no shuffles, and the only
// exchange is the row's sum of squares.  A row of up to 1024 values is one warp's, a longer one
// takes one CTA of cols/32 lanes.  Sums and the norm are binary32.
#pragma once

#include "mxfp8.cuh"
#include "quantize.cuh"  // fwht_scaled_packed, tc_offset

namespace fp4lin {

constexpr int NORM_MAX_COLS = 32768;

struct NormShape {
    const __nv_bfloat16 *x, *r, *w;  // r may be null
    __nv_bfloat16 *s;                // null when r is null
    uint8_t *codes, *scales;
    int64_t rows, ld_x, ld_r, ld_s, katoms;
    int64_t rows_pad;                // rows of the scale layout (a multiple of 128)
    int cols;
    float eps, inv_cols;
    bool wide_x, wide_r, wide_s, wide_w, wide_c;  // 256-bit accesses are aligned
};

// 32 bytes through the coherent path: s may be x's or r's own memory, so these are not .nc loads.
__device__ __forceinline__ void ld_32B(const void *p, bool wide, uint32_t *r)
{
    if (wide) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p)
                     : "memory");
    } else {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%8];\n\t"
                     "ld.global.L1::no_allocate.v4.b32 {%4,%5,%6,%7}, [%8+16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p)
                     : "memory");
    }
}

// 32 consecutive bf16.
__device__ __forceinline__ void load_bf16x32(const __nv_bfloat16 *p, bool wide, uint32_t *raw)
{
    ld_32B(p, wide, raw);
    ld_32B(p + 16, wide, raw + 8);
}

__device__ __forceinline__ void st_32B(void *p, bool wide, const uint32_t *v)
{
    if (wide) {
        st_v8(p, v);
    } else {
        st_v4(p, make_uint4(v[0], v[1], v[2], v[3]));
        st_v4(static_cast<uint8_t *>(p) + 16, make_uint4(v[4], v[5], v[6], v[7]));
    }
}

// THREADS 128: each of the CTA's four warps has a row of its own (cols <= 1024); else the CTA, of
// cols/32 threads rounded up to whole warps and at most THREADS, has one row.  The grid walks the
// rows: the weights stay in registers, and the next row is on its way while this one is reduced.
// 8192 x 4096 with residual and rotation: 39.4 us, 6.0 TB/s, 93% of a plain copy's rate.  One row: 2.1 us
// between launches of a graph.
template <int HAD, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_mxfp8_kernel(NormShape a)
{
    constexpr bool WARP_ROWS = THREADS == 128;
    constexpr int RPC = WARP_ROWS ? 4 : 1;  // rows a CTA
    constexpr bool AHEAD = THREADS <= 512;  // else there are no registers for a second row
    __shared__ float s_part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blk = WARP_ROWS ? lane : (int)threadIdx.x, nblk = a.cols / 32;
    const bool live = blk < nblk;
    const int64_t step = (int64_t)gridDim.x * RPC;
    int64_t row = (int64_t)blockIdx.x * RPC + (WARP_ROWS ? warp : 0);
    uint32_t wr[16], xr[16], rr[16];
    auto load = [&](int64_t at) {
        if (live && at < a.rows) {
            load_bf16x32(a.x + at * a.ld_x + blk * 32, a.wide_x, xr);
            if (a.r)
                load_bf16x32(a.r + at * a.ld_r + blk * 32, a.wide_r, rr);
        }
    };
    pdl_wait();
    if (AHEAD)
        load(row);
    if (live)
        load_bf16x32(a.w + blk * 32, a.wide_w, wr);
    for (int turn = 0; row < a.rows_pad; row += step, turn ^= 1) {  // the same rows for a whole warp (CTA)
        const int64_t word = tc_offset(row, blk, a.katoms) & ~(int64_t)3;
        if (row >= a.rows) {  // padding rows of the scale layout
            if ((blk & 3) == 0 && blk < 4 * a.katoms)
                *reinterpret_cast<uint32_t *>(a.scales + word) = 0u;
            continue;
        }
        if (!AHEAD)
            load(row);
        float v[32], sum = 0.0f;
        if (live) {
            if (a.r) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float lo = __fadd_rn(__uint_as_float(xr[i] << 16), __uint_as_float(rr[i] << 16));
                    const float hi = __fadd_rn(__uint_as_float(xr[i] & 0xFFFF0000u), __uint_as_float(rr[i] & 0xFFFF0000u));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(xr[i]) : "f"(hi), "f"(lo));
                }
                st_32B(a.s + row * a.ld_s + blk * 32, a.wide_s, xr);
                st_32B(a.s + row * a.ld_s + blk * 32 + 16, a.wide_s, xr + 8);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[2 * i] = __uint_as_float(xr[i] << 16);
                v[2 * i + 1] = __uint_as_float(xr[i] & 0xFFFF0000u);
            }
            float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s4[i & 3] = fmaf(v[i], v[i], s4[i & 3]);
            sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        }
        if (AHEAD)
            load(row + step);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (!WARP_ROWS) {
            if (lane == 0)
                s_part[turn][warp] = sum;
            __syncthreads();
            const int warps = (int)blockDim.x >> 5;
            sum = lane < warps ? s_part[turn][lane] : 0.0f;
#pragma unroll
            for (int o = 16; o; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float rs = __frsqrt_rn(fmaf(sum, a.inv_cols, a.eps));
        uint32_t byte = 0u;
        if (live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[2 * i] = __fmul_rn(__fmul_rn(v[2 * i], rs), __uint_as_float(wr[i] << 16));
                v[2 * i + 1] = __fmul_rn(__fmul_rn(v[2 * i + 1], rs), __uint_as_float(wr[i] & 0xFFFF0000u));
            }
            if constexpr (HAD == 16) {
                fwht_scaled_packed<16>(v, 0.25f);
                fwht_scaled_packed<16>(v + 16, 0.25f);
            } else if constexpr (HAD == 32) {
                fwht_scaled_packed<32>(v, __uint_as_float(0x3E3504F3u));
            }
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                amax = fmaxf(amax, block_abs(v[i]));
            byte = mxfp8_scale_byte(amax);
            const float inv = mxfp8_inverse(byte);
            uint32_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                c[i] = pack_e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
            st_32B(a.codes + row * a.cols + blk * 32, a.wide_c, c);
        }
        // four lanes' bytes make one word of the scale layout (zero in padding columns)
        uint32_t sw = byte << (8 * (lane & 3));
        sw |= __shfl_xor_sync(0xffffffffu, sw, 1);
        sw |= __shfl_xor_sync(0xffffffffu, sw, 2);
        if ((lane & 3) == 0 && blk < 4 * a.katoms)
            *reinterpret_cast<uint32_t *>(a.scales + word) = sw;
    }
}

}  // namespace fp4lin
