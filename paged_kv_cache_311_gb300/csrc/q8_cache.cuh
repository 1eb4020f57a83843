// q8_cache.cuh -- the 8-bit cache's writers: append_cache_q8_kernel (new
// tokens' K and V into e4m3 blocks with one scale per block and kv head) and
// summarize_blocks_kernel (per block and kv head, each key dimension's
// smallest and largest value).
//
// The cache.  A block's rows of one kv head are e4m3 values v with one scale
// 2^e: the row's numbers are v * 2^e.  e is the smallest exponent (>= -126)
// with max|x| <= 448 * 2^e over the block's rows.  A power of two costs a
// floating 8-bit type no precision (its relative step is 2^-3 of the leading
// bit whatever the scale) and makes a later, larger scale harmless: the rows
// already held are divided by a power of two, which is exact until a value
// falls below 2^-6 of the new scale and loses low bits to the subnormal grid.
//
// Work units.  A call appends n_s tokens to each sequence s; a unit is one
// (block touched by the call, kv head).  A token leads its unit when it is the
// sequence's first new token or opens a block: exactly one warp then owns the
// block's rows and scale of that head, so nothing is shared between warps and
// the result does not depend on any order.  A CTA looks at a run of tokens, a
// thread each, lists the leaders in shared memory and deals (leader, head) to
// its warps: in a prompt only one token in block_size leads, and a warp for
// every token spent its time finding that out (216 us for 12.8K tokens of 40
// heads, 12.8K x 80 warps, where the bytes need 57).
//
// What bounds them: HBM.  Those tokens are written in 59 to 67 us (84 to 96 %
// of a copy's rate), the blocks of prompts of 4K to 16K tokens summarised
// from the 8-bit cache in 36 to 42 us (31 needed).  A decode step of 256
// requests is a launch and a chain of loads: 3.7 us and 2.7.
#pragma once

#include <cuda_fp8.h>

#include "pkv_device.cuh"

namespace pkv {

// The kernels below are launched as programmatic dependents of whatever runs
// before them on the stream: their CTAs may come up while that drains, and
// wait here before they touch memory.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Floats between two blocks' scales: the kv heads, rounded up so that a
// block's scales are whole 16-byte pieces (copy_blocks and swap_blocks move
// them as they move blocks).
inline int q8_scale_stride(int num_kv_heads) { return (num_kv_heads + 3) / 4 * 4; }

struct AppendParams {
    const void *key;
    const void *value;
    uint8_t *k_cache;
    uint8_t *v_cache;
    float *k_scales;
    float *v_scales;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;   // null: token t is sequence t's only new token
    uint32_t *status;
    int64_t num_blocks;
    int num_seqs, num_tokens, num_kv_heads, max_blocks_per_seq, scale_stride;
    int tokens_per_cta;           // at most kUnitTokens
};

struct SummarizeParams {
    const void *k_cache;
    const float *k_scales;        // null: 16-bit cache
    void *summaries;              // [NB, Hk, 2, D]
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;
    uint32_t *status;
    int64_t num_blocks;
    int num_seqs, num_tokens, num_kv_heads, max_blocks_per_seq, scale_stride;
    int tokens_per_cta;           // at most kUnitTokens
};

// A unit's rows: rows [row0, row1) of physical block `block` are the call's
// tokens t, t + 1, ...; the block holds `row1` rows after the call.
struct AppendUnit {
    int t, row0, row1, block;
};

constexpr int kUnitWarps = 8;
constexpr int kUnitThreads = kUnitWarps * 32;
constexpr int kUnitTokens = 64;   // tokens a CTA looks at, at most

// Whether token t leads a unit (false also for padding and for what is refused).
template <int BS, typename P>
__device__ __forceinline__ bool append_unit(const P &p, int t, AppendUnit &u)
{
    int s = t, q0 = t, q1 = t + 1;
    if (p.query_start) {
        // the largest s with query_start[s] <= t
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.query_start[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        s = lo;
        q0 = p.query_start[s];
        q1 = p.query_start[s + 1];
        if (t < q0 || t >= q1)
            return false;   // a padding token
    }
    const int L = p.context_lens[s];
    const int n = q1 - q0;
    if (!p.query_start && L == 0)
        return false;       // a padding sequence
    if (q0 < 0 || q1 > p.num_tokens || L < n || (int64_t)L > (int64_t)p.max_blocks_per_seq * BS) {
        report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
        return false;
    }
    const int pos = L - n + (t - q0);
    u.t = t;
    u.row0 = pos % BS;
    if (u.row0 != 0 && t != q0)
        return false;
    u.row1 = min(BS, u.row0 + (q1 - t));
    u.block = p.block_tables[(int64_t)s * p.max_blocks_per_seq + pos / BS];
    if (u.block < 0 || (int64_t)u.block >= p.num_blocks) {
        report(p.status, PKV_DEV_BAD_BLOCK);
        return false;
    }
    return true;
}

// Lists the units that this CTA's tokens lead (blockIdx.x * tokens ..) in
// shared memory and returns their number.  All threads call it.
template <int BS, typename P>
__device__ __forceinline__ int list_units(const P &p, AppendUnit *list, int *count)
{
    if (threadIdx.x == 0)
        *count = 0;
    __syncthreads();
    wait_for_stream();
    const int64_t t = (int64_t)blockIdx.x * p.tokens_per_cta + threadIdx.x;
    AppendUnit u;
    if ((int)threadIdx.x < p.tokens_per_cta && t < p.num_tokens && append_unit<BS>(p, (int)t, u))
        list[atomicAdd(count, 1)] = u;   // the order decides which warp works, not what it writes
    __syncthreads();
    return *count;
}

// |x| of a pair of 16-bit values, and packed minima / maxima.
template <typename T> struct Pair16;
template <> struct Pair16<__half> {
    using V = __half2;
};
template <> struct Pair16<__nv_bfloat16> {
    using V = __nv_bfloat162;
};
template <typename T>
__device__ __forceinline__ typename Pair16<T>::V as_pair(uint32_t w)
{
    return *reinterpret_cast<typename Pair16<T>::V *>(&w);
}
template <typename V>
__device__ __forceinline__ uint32_t as_word(V v)
{
    return *reinterpret_cast<uint32_t *>(&v);
}

// The exponent of the scale that `amax` (finite, >= 0) needs: the smallest e
// >= -126 with amax <= 448 * 2^e, from its bits (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exponent(float amax)
{
    const uint32_t b = __float_as_uint(amax);
    const int x = (int)(b >> 23) - 127;   // amax = m * 2^x, 1 <= m < 2 (subnormals end at -126)
    return max(-126, x - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0));
}

// Two fp32 values -> two e4m3 bytes (nearest even; the lower byte is `lo`).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two e4m3 bytes -> two f16 values (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t two)
{
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
    return d;
}

__device__ __forceinline__ float2 float2_of_e4m3(uint32_t two)
{
    const uint32_t w = f16x2_of_e4m3(two);
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Eight 16-bit values -> eight e4m3 bytes of x * inv.  `odd`: the unit holds
// an infinity; those become NaN (NaN converts to NaN by itself).
template <typename T>
__device__ __forceinline__ uint2 quantize8(uint4 w, float inv, bool odd)
{
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = Unpack<T>::pair(in[i]);
        f.x *= inv;
        f.y *= inv;
        if (odd) {
            f.x = isinf(f.x) ? NAN : f.x;
            f.y = isinf(f.y) ? NAN : f.y;
        }
        o[i] = e4m3x2(f.x, f.y);
    }
    return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

// One unit's rows of one kv head, K or V, by one warp.
template <typename T, int D, int BS>
__device__ __forceinline__ void append_rows(const AppendParams &p, const AppendUnit &u, int h, bool is_v, int lane)
{
    constexpr int LPR = D / 8;        // lanes per row (16 bytes of input each)
    constexpr int RPL = 32 / LPR;     // rows a warp holds per load
    constexpr int NL = BS / RPL;      // loads of a full block
    const uint4 *src = reinterpret_cast<const uint4 *>(is_v ? p.value : p.key);
    uint8_t *blk = (is_v ? p.v_cache : p.k_cache) + ((int64_t)u.block * p.num_kv_heads + h) * (BS * D);
    float *scale = (is_v ? p.v_scales : p.k_scales) + (int64_t)u.block * p.scale_stride + h;
    const int r = lane / LPR, c = lane % LPR;
    const int n = u.row1 - u.row0;

    uint4 x[NL];
    uint32_t m = 0;   // the largest magnitude, as an ordered pattern of |x| in fp32
    bool odd = false;
    typename Pair16<T>::V mx = as_pair<T>(0u);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int row = i * RPL + r;
        x[i] = make_uint4(0, 0, 0, 0);
        if (row < n)
            x[i] = src[((int64_t)(u.t + row) * p.num_kv_heads + h) * LPR + c];
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        // |x| by clearing the sign bits; a NaN operand loses to a number
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mx = __hmax2(mx, as_pair<T>(w[k] & 0x7fff7fffu));
    }
    {
        const float2 f = Unpack<T>::pair(as_word(mx));
        m = __float_as_uint(fmaxf(f.x, f.y));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (m >= 0x7f800000u) {
        // an infinity: the finite values set the scale
        odd = true;
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = Unpack<T>::pair(w[k] & 0x7fff7fffu);
                a = f.x < INFINITY ? fmaxf(a, f.x) : a;
                a = f.y < INFINITY ? fmaxf(a, f.y) : a;
            }
        }
        m = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
    }
    int e = scale_exponent(__uint_as_float(m));
    if (u.row0 > 0) {
        // rows already held: the scale never shrinks; when it grows they are
        // written again, divided by the power of two
        const int old = (int)((__float_as_uint(*scale) >> 23) & 0xffu) - 127;
        if (old >= e) {
            e = old;
        } else {
            const float down = __uint_as_float((uint32_t)max(old - e + 127, 0) << 23);
            uint2 *rows = reinterpret_cast<uint2 *>(blk);
            for (int i = lane; i < u.row0 * LPR; i += 32) {
                const uint2 v = rows[i];
                const float2 a = float2_of_e4m3(v.x & 0xffffu), b = float2_of_e4m3(v.x >> 16);
                const float2 f = float2_of_e4m3(v.y & 0xffffu), g = float2_of_e4m3(v.y >> 16);
                rows[i] = make_uint2(e4m3x2(a.x * down, a.y * down) | e4m3x2(b.x * down, b.y * down) << 16,
                                     e4m3x2(f.x * down, f.y * down) | e4m3x2(g.x * down, g.y * down) << 16);
            }
        }
    }
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int row = i * RPL + r;
        if (row < n)
            *reinterpret_cast<uint2 *>(blk + (u.row0 + row) * D + c * 8) = quantize8<T>(x[i], inv, odd);
    }
    __syncwarp();
    if (lane == 0)
        *scale = __uint_as_float((uint32_t)(e + 127) << 23);
}

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kUnitThreads)
append_cache_q8_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ AppendUnit list[kUnitTokens];
    __shared__ int count;
    const int units = 2 * p.num_kv_heads;
    const int items = list_units<BS>(p, list, &count) * units;
    for (int i = blockIdx.y * kUnitWarps + (threadIdx.x >> 5); i < items; i += gridDim.y * kUnitWarps)
        append_rows<T, D, BS>(p, list[i / units], (i % units) >> 1, i & 1, threadIdx.x & 31);
}

// One block's rows of one kv head by one warp: load() issues the loads,
// finish() writes the minima and maxima.  A lane keeps to its own 4 or 8
// bytes of every row, so that rows meet in registers: with 16 bytes per lane
// and several rows to a load, the shuffles that joined the rows cost more
// than the comparisons.  T: the cache's 16-bit type, or for an e4m3 cache
// (Q8) the summaries' type.
template <typename T, int D, int BS, bool Q8>
struct BlockRange {
    using E = typename std::conditional<Q8, __half, T>::type;
    using V = typename Pair16<E>::V;
    static constexpr int ROW = D * (Q8 ? 1 : 2);            // bytes of a row
    static constexpr int LW = ROW == 256 ? 2 : 1;           // words a lane holds of a row
    static constexpr int LPR = ROW / (4 * LW);              // lanes per row
    static constexpr int RPL = 32 / LPR;                    // rows per load
    static constexpr int NL = BS / RPL;
    static constexpr int NP = LW * (Q8 ? 2 : 1);            // pairs of values a lane holds of a row
    static constexpr int U = NL * LW <= 8 ? 4 : NL * LW <= 16 ? 2 : 1;   // blocks a warp has in flight
    uint32_t x[NL][LW];
    float scale;

    __device__ __forceinline__ void load(const SummarizeParams &p, const AppendUnit &u, int h, int lane)
    {
        const uint32_t *blk = reinterpret_cast<const uint32_t *>(p.k_cache) +
                              ((int64_t)u.block * p.num_kv_heads + h) * (BS * ROW / 4) + (lane % LPR) * LW;
        const int r = lane / LPR;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            // lanes without a row of their own repeat row 0
            const int row = i * RPL + r;
            const uint32_t *src = blk + (row < u.row1 ? row : 0) * (ROW / 4);
            if constexpr (LW == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(src);
                x[i][0] = v.x;
                x[i][1] = v.y;
            } else {
                x[i][0] = *src;
            }
        }
        if constexpr (Q8)
            scale = p.k_scales[(int64_t)u.block * p.scale_stride + h];
    }

    __device__ __forceinline__ void finish(const SummarizeParams &p, const AppendUnit &u, int h, int lane) const
    {
        V lo[NP], hi[NP];
#pragma unroll
        for (int i = 0; i < NL; ++i) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                V v;
                if constexpr (Q8)
                    v = as_pair<E>(f16x2_of_e4m3((k & 1) ? x[i][k >> 1] >> 16 : x[i][k >> 1] & 0xffffu));
                else
                    v = as_pair<E>(x[i][k]);
                // NaN stays: a block with a NaN key says so
                lo[k] = i ? __hmin2_nan(lo[k], v) : v;
                hi[k] = i ? __hmax2_nan(hi[k], v) : v;
            }
        }
        if constexpr (RPL == 2) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                lo[k] = __hmin2_nan(lo[k], as_pair<E>(__shfl_xor_sync(0xffffffffu, as_word(lo[k]), LPR)));
                hi[k] = __hmax2_nan(hi[k], as_pair<E>(__shfl_xor_sync(0xffffffffu, as_word(hi[k]), LPR)));
            }
        }
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.summaries) +
                        ((int64_t)u.block * p.num_kv_heads + h) * D + (lane % LPR) * NP;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t o[NP];
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                o[k] = as_word(r ? hi[k] : lo[k]);
                if constexpr (Q8) {
                    const float2 f = __half22float2(as_pair<__half>(o[k]));
                    o[k] = Mma<T>::pack(f.x * scale, f.y * scale);
                }
            }
            if (lane < LPR) {
                if constexpr (NP == 2)
                    *reinterpret_cast<uint2 *>(dst + r * (D / 2)) = make_uint2(o[0], o[1]);
                else
                    dst[r * (D / 2)] = o[0];
            }
        }
    }
};

template <typename T, int D, int BS, bool Q8>
__global__ void __launch_bounds__(kUnitThreads)
summarize_blocks_kernel(const __grid_constant__ SummarizeParams p)
{
    using R = BlockRange<T, D, BS, Q8>;
    __shared__ AppendUnit list[kUnitTokens];
    __shared__ int count;
    const int lane = threadIdx.x & 31, Hk = p.num_kv_heads;
    const int items = list_units<BS>(p, list, &count) * Hk;
    const int step = gridDim.y * kUnitWarps;
    for (int i0 = blockIdx.y * kUnitWarps + (threadIdx.x >> 5); i0 < items; i0 += step * R::U) {
        R b[R::U];
#pragma unroll
        for (int k = 0; k < R::U; ++k) {
            const int i = i0 + k * step;
            if (i < items)
                b[k].load(p, list[i / Hk], i % Hk, lane);
        }
#pragma unroll
        for (int k = 0; k < R::U; ++k) {
            const int i = i0 + k * step;
            if (i < items)
                b[k].finish(p, list[i / Hk], i % Hk, lane);
        }
    }
}

}  // namespace pkv
