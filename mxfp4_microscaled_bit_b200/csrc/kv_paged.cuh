// kv_paged.cuh -- the paged 8-bit KV cache: block tables and slots from request lengths, and the
// append of new K and V rows.
//
// A cache is codes [num_pages, H, P, D] E4M3 and scales [num_pages, H] E8M0 (mxfp8.cuh): the P rows
// of one page and head share one power-of-two scale and are one contiguous P * D bytes.
#pragma once

#include "mxfp8.cuh"

namespace fp4lin {

// ------------------------------------------------------------------ block tables and slots
// For request b with len_b rows in the cache and new_b to come, P rows a page:
//   had = ceil(len/P), need = ceil((len + new)/P), cu = exclusive sum of new,
//   table[b, had + i] = free[head + (exclusive sum of need - had)_b + i],
//   slot(cu_b + i) = table[b, p / P] * P + p % P with p = len_b + i.
// A few KB in and out: bound by launch and latency.  One launch: every CTA sums all requests'
// lengths itself (from L2, at most TABLE_MAX_REQUESTS of them) and then takes its share of the new
// table entries and of the tokens, finding a token's request by bisection in shared memory; a slot
// on a page that this call hands out is computed from the free list, so no CTA waits for another.
// 509 requests with ~40,000 new tokens: 3.8 us between launches of a graph.
constexpr int TABLE_THREADS = 512;
constexpr int TABLE_MAX_REQUESTS = 8192;

struct TableShape {
    int32_t *table;  // [B, ld]
    const int32_t *lens, *new_lens, *free_list, *head;
    int32_t *cu, *slots, *next_head;
    int64_t ld;
    int B, width, F, max_tokens, shift;  // P = 1 << shift
};

constexpr size_t table_smem(int B) { return ((size_t)2 * (B + 1) + 64) * 4; }

// Both sums stop growing past `cap` tokens, so garbage lengths cannot wrap them.
struct TableSums {
    uint32_t tokens, pages;
};

__device__ __forceinline__ TableSums table_add(TableSums a, TableSums b, uint32_t cap)
{
    return {min(a.tokens + b.tokens, cap), min(a.pages + b.pages, 0x7FFFFFFFu)};
}

// Request b's new tokens and pages; bad: a negative length, or more rows than its table row holds.
__device__ __forceinline__ TableSums table_request(const TableShape &a, int b, bool &bad)
{
    const int len = a.lens[b], nw = a.new_lens[b];
    if (len < 0 || nw < 0) {
        bad = true;
        return {0u, 0u};
    }
    const int64_t rows = (int64_t)a.width << a.shift;
    const int64_t end = (int64_t)len + nw;
    bad |= end > rows;
    const int64_t P1 = (1 << a.shift) - 1;
    const int64_t had = (min((int64_t)len, rows) + P1) >> a.shift, need = (min(end, rows) + P1) >> a.shift;
    return {(uint32_t)nw, (uint32_t)(need - had)};
}

// Largest b with first[b] <= v, given first[0] = 0 <= v < first[B].
__device__ __forceinline__ int table_find(const uint32_t *first, int B, uint32_t v)
{
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(TABLE_THREADS) kv_table_kernel(TableShape a)
{
    extern __shared__ uint32_t tb_smem[];
    uint32_t *s_tok = tb_smem, *s_page = tb_smem + a.B + 1, *s_warp = s_page + a.B + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t cap = (uint32_t)a.max_tokens + 1u;
    pdl_wait();
    const int head = *a.head;
    const int per = (a.B + TABLE_THREADS - 1) / TABLE_THREADS;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    bool bad = false;
    TableSums mine = {0u, 0u};
    for (int b = b0; b < b1; ++b)
        mine = table_add(mine, table_request(a, b, bad), cap);
    TableSums run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const TableSums up = {__shfl_up_sync(0xffffffffu, run.tokens, o), __shfl_up_sync(0xffffffffu, run.pages, o)};
        if (lane >= o)
            run = table_add(run, up, cap);
    }
    if (lane == 31) {
        s_warp[2 * warp] = run.tokens;
        s_warp[2 * warp + 1] = run.pages;
    }
    __syncthreads();
    TableSums before = {0u, 0u};
    for (int w = 0; w < warp; ++w)
        before = table_add(before, TableSums{s_warp[2 * w], s_warp[2 * w + 1]}, cap);
    const TableSums left = {__shfl_up_sync(0xffffffffu, run.tokens, 1), __shfl_up_sync(0xffffffffu, run.pages, 1)};
    if (lane > 0)
        before = table_add(before, left, cap);
    for (int b = b0; b < b1; ++b) {
        s_tok[b] = before.tokens;
        s_page[b] = before.pages;
        before = table_add(before, table_request(a, b, bad), cap);
    }
    if (b0 < b1 && b1 == a.B) {
        s_tok[a.B] = before.tokens;
        s_page[a.B] = before.pages;
    }
    __syncthreads();
    const uint32_t all_tokens = s_tok[a.B], pages = s_page[a.B];
    const uint32_t tokens = min(all_tokens, (uint32_t)a.max_tokens);
    const bool head_ok = head >= 0 && head <= a.F;
    const int64_t left_free = head_ok ? (int64_t)a.F - head : 0;
    bad |= all_tokens > (uint32_t)a.max_tokens || !head_ok || (int64_t)pages > left_free;
    const int first = blockIdx.x * TABLE_THREADS + tid, stride = gridDim.x * TABLE_THREADS;
    for (int b = first; b <= a.B; b += stride)
        a.cu[b] = (int32_t)min(s_tok[b], tokens);
    if (first == 0)
        *a.next_head = head_ok ? (int32_t)(head + min((int64_t)pages, left_free)) : head;
    const int P1 = (1 << a.shift) - 1;
    for (int64_t e = first; e < (int64_t)pages; e += stride) {  // new table entries
        const int b = table_find(s_page, a.B, (uint32_t)e);
        const int64_t col = (min((int64_t)a.lens[b], (int64_t)a.width << a.shift) + P1) >> a.shift;
        a.table[b * a.ld + col + (e - s_page[b])] = e < left_free ? a.free_list[head + e] : -1;
    }
    for (int64_t t = first; t < a.max_tokens; t += stride) {  // slots
        int32_t slot = -1;
        if (t < (int64_t)tokens) {
            const int b = table_find(s_tok, a.B, (uint32_t)t);
            const int64_t len = a.lens[b], p = len + (t - s_tok[b]), col = p >> a.shift;
            const int64_t had = (len + P1) >> a.shift;
            if (col < a.width) {
                int page = -1;
                if (col < had)
                    page = a.table[b * a.ld + col];
                else if (s_page[b] + (col - had) < left_free)
                    page = a.free_list[head + s_page[b] + (col - had)];
                if (page >= 0 && page <= (0x7FFFFFFF >> a.shift))
                    slot = (page << a.shift) + (int)(p & P1);
                else
                    bad = true;
            }
        }
        a.slots[t] = slot;
    }
    if (bad)
        report_error(FP4LIN_ERR_OUT_OF_RANGE);
}

// ------------------------------------------------------------------ append
// New rows arrive as runs: consecutive tokens whose slots follow one another within a page (as
// kv_table_kernel lays them out).  A run that begins at row 0 starts its page afresh; a later one
// finds the page's older rows under its old scale: the larger of the two exponents is the page's
// new one, and when it grew the older rows are re-encoded to it.
//   2 (in) + 1 (out) bytes a value, for K and V.  Latency bound: a CTA's slots, rows and codes wait for one
// another, and prompts' bytes take half of its time at HBM's rate.  A CTA owns the runs that begin in its `per_cta` tokens, for one head of K or of V; the
// CTAs of a token's heads are neighbours, so that its row is read together.  A warp takes up to 16
// rows, all loads in flight and the values in registers between the maximum and the encoding;
// P/16 warps are a group that takes a run.  With many runs, as in decoding, each warp takes a run
// for itself, row by row.
// 7 prompts of up to 2041 tokens, 8 heads of 128: 15.3 us, 3.5 TB/s; 64 single tokens 2.9 us.
constexpr int APPEND_THREADS = 256;
constexpr int APPEND_WARPS = APPEND_THREADS / 32;
constexpr int APPEND_TOKENS = 128;  // most tokens a CTA looks at

struct AppendShape {
    const __nv_bfloat16 *k, *v;  // [T, H, D], token strides ld_k, ld_v
    const int32_t *slots;
    uint8_t *kc, *ks, *vc, *vs;
    int64_t ld_k, ld_v, slots_end;  // slots_end = num_pages * P
    int T, H, shift, per_cta;
};

// Largest block_abs of eight bf16.
__device__ __forceinline__ float bf16x8_amax(uint4 u)
{
    float f[8], m = 0.0f;
    bf16x8_to_f32(u, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, block_abs(f[i]));
    return m;
}

__device__ __forceinline__ uint2 bf16x8_encode(uint4 u, float inv)
{
    float f[8];
    bf16x8_to_f32(u, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = __fmul_rn(f[i], inv);
    return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

// f16x2 of 2^k for k <= 15 (0 below f16's least, 2^-24).
__device__ __forceinline__ uint32_t f16x2_pow2(int k)
{
    const uint32_t h = k >= -14 ? (uint32_t)(15 + k) << 10 : k >= -24 ? 1u << (24 + k) : 0u;
    return h | (h << 16);
}

// The warps of a group meet (named barrier 1 + group).
__device__ __forceinline__ void append_meet(int group, int warps)
{
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
}

template <int D>
__global__ void __launch_bounds__(APPEND_THREADS, 3) kv_append_kernel(AppendShape a)
{
    constexpr int LPR = D / 8;         // lanes a row (8 values each)
    constexpr int RPW = 32 / LPR;      // rows a warp pass
    constexpr int PASSES = 16 / RPW;   // of a warp's 16 rows
    __shared__ int s_t[APPEND_TOKENS], s_slot[APPEND_TOKENS], s_n[APPEND_TOKENS], s_runs;
    __shared__ float s_max[APPEND_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << a.shift, h = blockIdx.x >> 1;
    const bool is_v = blockIdx.x & 1;
    const __nv_bfloat16 *x = (is_v ? a.v : a.k) + (int64_t)h * D;
    const int64_t ld = is_v ? a.ld_v : a.ld_k;
    uint8_t *codes = is_v ? a.vc : a.kc, *scales = is_v ? a.vs : a.ks;
    pdl_wait();
    if (warp == 0) {  // the runs that begin here
        const int t0 = blockIdx.y * a.per_cta, t1 = min(t0 + a.per_cta, a.T);
        int slot[APPEND_TOKENS / 32], prev[APPEND_TOKENS / 32], runs = 0;
#pragma unroll
        for (int k = 0; k < APPEND_TOKENS / 32; ++k) {
            const int t = t0 + 32 * k + lane;
            slot[k] = t < t1 ? a.slots[t] : -1;
            prev[k] = t < t1 && t > 0 ? a.slots[t - 1] : -2;
        }
#pragma unroll
        for (int k = 0; k < APPEND_TOKENS / 32; ++k) {
            const bool range = slot[k] >= 0 && slot[k] < a.slots_end;
            if (slot[k] != -1 && !range)
                report_error(FP4LIN_ERR_OUT_OF_RANGE);
            const bool lead = range && ((slot[k] & (P - 1)) == 0 || prev[k] != slot[k] - 1);
            const uint32_t leads = __ballot_sync(0xffffffffu, lead);
            if (lead) {
                const int i = runs + __popc(leads & ((1u << lane) - 1u));
                s_t[i] = t0 + 32 * k + lane;
                s_slot[i] = slot[k];
            }
            runs += __popc(leads);
        }
        if (lane == 0)
            s_runs = runs;
    }
    __syncthreads();
    const int runs = s_runs;
    // run lengths: at most to the page's end
    for (int i = warp; i < runs; i += APPEND_WARPS) {
        const int t = s_t[i], slot = s_slot[i], most = min(P - (slot & (P - 1)), a.T - t);
        int n = 1;
        for (int base = 1; base < most; base += 32) {
            const int j = base + lane;
            const bool go = j < most && a.slots[t + j] == slot + j;
            const uint32_t same = __ballot_sync(0xffffffffu, go);
            const int c = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
            n += c;
            if (c < 32)
                break;
        }
        if (lane == 0)
            s_n[i] = n;
    }
    __syncthreads();
    const int sub = lane / LPR, col = (lane % LPR) * 8;
    const bool by_warp = runs >= APPEND_WARPS;
    const int warps = by_warp ? 1 : P / 16, group = warp / warps, in_group = warp - group * warps;
    for (int i = group; i < runs; i += APPEND_WARPS / warps) {
        const int t = s_t[i], slot = s_slot[i], n = s_n[i], off = slot & (P - 1);
        const int64_t page_head = (int64_t)(slot >> a.shift) * a.H + h;
        uint8_t *dst = codes + page_head * P * D + col;
        const __nv_bfloat16 *src = x + (int64_t)t * ld + col;
        const uint32_t old = off ? scales[page_head] : 0u;
        const int first = 16 * in_group + sub, step = 16 * warps;
        uint4 held[PASSES];  // the warp's first 16 rows
        float m = 0.0f;
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            held[p] = ld_nc_v4_if(src + (int64_t)(first + p * RPW) * ld, first + p * RPW < n);
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            m = fmaxf(m, bf16x8_amax(held[p]));
        for (int r0 = first + step; r0 < n; r0 += step)  // a warp alone with a longer run
            for (int r = r0; r < min(r0 + 16, n); r += RPW)
                m = fmaxf(m, bf16x8_amax(ld_nc_v4(src + (int64_t)r * ld)));
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // in order, as none is negative
        if (warps > 1) {
            if (lane == 0)
                s_max[warp] = m;
            append_meet(group, warps);
            for (int w = 0; w < warps; ++w)
                m = fmaxf(m, s_max[group * warps + w]);
        }
        const uint32_t byte = max(mxfp8_scale_byte(m), old);
        const float inv = mxfp8_inverse(byte);
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            if (first + p * RPW < n)
                *reinterpret_cast<uint2 *>(dst + (off + first + p * RPW) * D) = bf16x8_encode(held[p], inv);
        for (int r0 = first + step; r0 < n; r0 += step)
            for (int r = r0; r < min(r0 + 16, n); r += RPW)
                *reinterpret_cast<uint2 *>(dst + (off + r) * D) = bf16x8_encode(ld_nc_v4(src + (int64_t)r * ld), inv);
        if (off && byte > old && old) {  // older rows (all zero codes under byte 0) to the larger exponent
            const uint32_t f = f16x2_pow2((int)(old - byte));  // 0: codes times that are below half an E4M3 step
            for (int r = in_group * RPW + sub; r < off; r += warps * RPW) {
                uint2 *c = reinterpret_cast<uint2 *>(dst + r * D);
                const uint2 v = *c;
                *c = make_uint2(e4m3x4_shift(v.x, f), e4m3x4_shift(v.y, f));
            }
        }
        append_meet(group, warps);  // every warp has read the old scale and s_max
        if (in_group == 0 && lane == 0)
            scales[page_head] = (uint8_t)byte;
    }
}

}  // namespace fp4lin
