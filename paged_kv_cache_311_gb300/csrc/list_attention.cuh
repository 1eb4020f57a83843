// list_attention.cuh -- single-query attention over a list of a sequence's
// blocks: all of them in an e4m3 cache (paged_attention_decode_q8), or the
// selected ones of a 16-bit or an e4m3 cache (paged_attention_decode_selected).
//
//   out[s, h] = sum_i softmax_i(scale * ks_b(i) * q[s, h] . k_i) * vs_b(i) * v_i
// over the tokens i of the listed blocks, ks and vs the block's scales (1 in a
// 16-bit cache).
//
// One CTA per (partition of the list, kv head, sequence); it owns the kv
// head's G query heads, so each K/V byte is read once.  With more than one
// partition the CTAs write (max, sum, unnormalised sum of values) and
// list_merge_kernel combines them.
#pragma once

#include "pa_decode.cuh"
#include "q8_cache.cuh"

namespace pkv {

struct ListParams {
    void *out;
    const void *q;
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const float *k_scales;       // null: 16-bit cache
    const float *v_scales;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *selected;     // null: every block; else [B, Hk, num_selected]
    float *ws_ml;                // [B][H][np][2], np > 1
    float *ws_acc;               // [B][H][np][D]
    uint32_t *status;
    int64_t num_blocks;
    int num_seqs, num_kv_heads, group, max_blocks_per_seq, max_context_len;
    int num_selected, scale_stride;
    int part_blocks;             // list entries per partition
    int np;                      // partitions
    int out_dtype, q_dtype;
    float qscale;                // softmax scale * log2(e)
};

constexpr int kListWarps = 4;
constexpr int kListMaxGroup = 8;
constexpr int kListCap = 1024;   // list entries one CTA stages

// The list entries of one CTA, staged in shared memory.
struct ListStage {
    int32_t phys[kListCap];
    float ks[kListCap];
    float vs[kListCap];
};

// Stages entries [e0, e0 + part_blocks) of a (sequence, kv head) row's list:
// physical block ids and scales.  Returns the number of tokens they hold (the
// sequence's last block, always the list's last entry, may be partial), or -1
// if the row is refused.  All threads of the CTA call it; ends with a barrier.
//
// A selected list is refused unless it is strictly ascending and inside the
// sequence's blocks, with -1 only behind its last entry: so no block counts
// twice and only the last entry can be partial.
template <int BS>
__device__ __forceinline__ int stage_list(const ListParams &p, ListStage *st, int seq, int kvh, int part, int L)
{
    const int nblk = (L + BS - 1) / BS;
    const int total = p.selected ? p.num_selected : nblk;
    const int e0 = part * p.part_blocks, e1 = min(e0 + p.part_blocks, total);
    const int32_t *sel = p.selected ? p.selected + ((int64_t)seq * p.num_kv_heads + kvh) * p.num_selected : nullptr;
    const int32_t *table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
    int bad = 0, tokens = 0;
    for (int e = e0 + (int)threadIdx.x; e < e1; e += kListWarps * 32) {
        int j = e;
        if (sel) {
            const int before = e > 0 ? sel[e - 1] : -1;
            j = sel[e];
            if (j < 0 && j != -1)
                bad = 1;
            if (j < 0)
                continue;
            if (j >= nblk || (e > 0 && (before < 0 || before >= j))) {
                bad = 1;
                continue;
            }
        }
        int b = table[j];
        if (b < 0 || (int64_t)b >= p.num_blocks) {
            bad = 1;
            b = 0;
        }
        st->phys[e - e0] = b;
        if (p.k_scales) {
            st->ks[e - e0] = p.k_scales[(int64_t)b * p.scale_stride + kvh];
            st->vs[e - e0] = p.v_scales[(int64_t)b * p.scale_stride + kvh];
        }
        tokens = max(tokens, (e - e0) * BS + min(BS, L - j * BS));
    }
    __shared__ int most[kListWarps];
    tokens = __reduce_max_sync(0xffffffffu, tokens);
    if ((threadIdx.x & 31) == 0)
        most[threadIdx.x >> 5] = tokens;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0)
            report(p.status, PKV_DEV_BAD_BLOCK);
        return -1;
    }
#pragma unroll
    for (int w = 0; w < kListWarps; ++w)
        tokens = max(tokens, most[w]);
    return tokens;
}

// A row that has no result: zeros, or a partial that says so (sum -1) or that
// holds nothing (sum 0).
template <int D>
__device__ __forceinline__ void write_empty(const ListParams &p, int seq, int kvh, int part, bool refused)
{
    for (int i = threadIdx.x; i < p.group * D; i += kListWarps * 32) {
        const int64_t sh = ((int64_t)seq * p.num_kv_heads + kvh) * p.group + i / D;
        if (p.np == 1) {
            store_out(p.out, p.out_dtype, sh * D + i % D, 0.f);
        } else if (i % D == 0) {
            const int64_t slot = sh * p.np + part;
            p.ws_ml[slot * 2 + 0] = -INFINITY;
            p.ws_ml[slot * 2 + 1] = refused ? -1.f : 0.f;
        }
    }
}

__device__ __forceinline__ float load_q(const ListParams &p, int64_t i)
{
    return p.q_dtype == PKV_F16 ? to_float(static_cast<const __half *>(p.q)[i])
                                : to_float(static_cast<const __nv_bfloat16 *>(p.q)[i]);
}

// D / 32 consecutive values of one row, from the cache's type to fp32.
template <typename T, int N>
__device__ __forceinline__ void load_row(const uint8_t *row, int lane, float (&x)[N])
{
    if constexpr (std::is_same<T, uint8_t>::value) {
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const float2 f = float2_of_e4m3(*reinterpret_cast<const uint16_t *>(row + lane * N + k));
            x[k] = f.x;
            x[k + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const float2 f = Unpack<T>::pair(reinterpret_cast<const uint32_t *>(row)[(lane * N + k) / 2]);
            x[k] = f.x;
            x[k + 1] = f.y;
        }
    }
}

// T: __half, __nv_bfloat16, or uint8_t for an e4m3 cache.  One warp takes a
// token at a time, a lane D / 32 of its dimensions.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kListWarps * 32)
list_attention_kernel(const __grid_constant__ ListParams p)
{
    constexpr bool Q8 = std::is_same<T, uint8_t>::value;
    constexpr int N = D / 32;
    constexpr int MG = kListMaxGroup;
    __shared__ ListStage st;
    __shared__ float s_m[kListWarps][MG], s_l[kListWarps][MG];
    __shared__ float s_acc[kListWarps][MG][D];
    const int part = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = p.context_lens[seq];
    if (L < 0 || L > p.max_context_len) {
        if (part == 0 && kvh == 0 && threadIdx.x == 0)
            report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
        write_empty<D>(p, seq, kvh, part, true);
        return;
    }
    const int tokens = stage_list<BS>(p, &st, seq, kvh, part, L);
    if (tokens <= 0) {
        write_empty<D>(p, seq, kvh, part, tokens < 0);
        return;
    }
    const int64_t head0 = ((int64_t)seq * p.num_kv_heads + kvh) * p.group;
    float q[MG][N], acc[MG][N], m[MG], l[MG];
#pragma unroll
    for (int g = 0; g < MG; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            q[g][k] = g < p.group ? load_q(p, (head0 + g) * D + lane * N + k) * p.qscale : 0.f;
            acc[g][k] = 0.f;
        }
    }
    constexpr int ROW = D * (Q8 ? 1 : 2);
    for (int t = warp; t < tokens; t += kListWarps) {
        const int64_t row = ((int64_t)st.phys[t / BS] * p.num_kv_heads + kvh) * BS + t % BS;
        float k[N], v[N];
        load_row<T, N>(p.k_cache + row * ROW, lane, k);
        load_row<T, N>(p.v_cache + row * ROW, lane, v);
        const float ks = Q8 ? st.ks[t / BS] : 1.f, vs = Q8 ? st.vs[t / BS] : 1.f;
#pragma unroll
        for (int g = 0; g < MG; ++g) {
            if (g < p.group) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    s = fmaf(q[g][i], k[i], s);
#pragma unroll
                for (int off = 1; off < 32; off <<= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, off);
                s *= ks;
                const float mn = fmaxf(m[g], s);
                const float a = mn == -INFINITY ? 1.f : exp2f(m[g] - mn);
                // a NaN score stays one, also before any number has come
                const float e = s == -INFINITY ? 0.f : exp2f(s - (mn == -INFINITY ? 0.f : mn));
                m[g] = mn;
                l[g] = l[g] * a + e;
                const float ev = e * vs;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[g][i] = acc[g][i] * a + ev * v[i];
            }
        }
    }
#pragma unroll
    for (int g = 0; g < MG; ++g) {
        if (lane == 0) {
            s_m[warp][g] = m[g];
            s_l[warp][g] = l[g];
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            s_acc[warp][g][lane * N + i] = acc[g][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.group * D; i += kListWarps * 32) {
        const int g = i / D, d = i % D;
        float M = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < kListWarps; ++w)
            M = fmaxf(M, s_m[w][g]);
#pragma unroll
        for (int w = 0; w < kListWarps; ++w) {
            if (s_m[w][g] != -INFINITY || s_l[w][g] != 0.f) {
                const float f = exp2f(s_m[w][g] - M);
                num += f * s_acc[w][g][d];
                den += f * s_l[w][g];
            }
        }
        if (p.np == 1) {
            store_out(p.out, p.out_dtype, (head0 + g) * D + d, den == 0.f ? 0.f : num / den);
        } else {
            const int64_t slot = (head0 + g) * p.np + part;
            p.ws_acc[slot * D + d] = num;
            if (d == 0) {
                p.ws_ml[slot * 2 + 0] = M;
                p.ws_ml[slot * 2 + 1] = den;
            }
        }
    }
}

// One CTA per (sequence, head), a thread per dimension: the log-sum-exp merge
// of the np partials.  A sum of -1 marks a refused partition: the row is zero.
template <int D>
__global__ void __launch_bounds__(D)
list_merge_kernel(const __grid_constant__ ListParams p)
{
    const int64_t sh = blockIdx.x;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml) + sh * p.np;
    const float *acc = p.ws_acc + sh * p.np * D + threadIdx.x;
    float M = -INFINITY;
    bool refused = false;
    for (int k = 0; k < p.np; ++k) {
        const float2 t = ml[k];
        M = fmaxf(M, t.x);
        refused |= t.y < 0.f;
    }
    float num = 0.f, den = 0.f;
    for (int k = 0; k < p.np; ++k) {
        const float2 t = ml[k];
        if (t.y != 0.f) {
            const float f = exp2f(t.x - M);
            num += f * acc[(int64_t)k * D];
            den += f * t.y;
        }
    }
    store_out(p.out, p.out_dtype, sh * D + threadIdx.x, refused || den == 0.f ? 0.f : num / den);
}

}  // namespace pkv
