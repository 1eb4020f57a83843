// q4_attention.cuh -- single-query attention over a 4-bit cache
// (paged_attention_decode_q4):
//   out[s, h] = sum_t softmax_t(scale * q[s, h] . k_t) * v_t,
// a row's numbers s u + m for each group of 64 dimensions (see q4_cache.cuh).
#pragma once

#include "list_attention.cuh"
#include "q4_cache.cuh"

namespace pkv {

struct Q4Params {
    void *out;
    const void *q;
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    uint32_t *status;
    int64_t num_blocks, q_stride;
    int num_kv_heads, group, max_blocks_per_seq, max_context_len, out_dtype;
    float qscale;                // softmax scale * log2(e)
};

constexpr int kQ4Warps = 4;

// One CTA per (kv head, sequence), a warp per token, D / 32 dimensions a lane.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kQ4Warps * 32)
q4_attention_kernel(const __grid_constant__ Q4Params p)
{
    using R = Q4Row<D>;
    constexpr int N = D / 32, GM = kListMaxGroup;
    __shared__ float s_m[kQ4Warps][GM], s_l[kQ4Warps][GM], s_o[kQ4Warps][GM][D];
    const int kvh = blockIdx.x, seq = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int d0 = lane * N, j = d0 / kQ4Group, i = d0 % kQ4Group / 8, shift = d0 % 8 * 4;
    wait_for_stream();
    const int L = p.context_lens[seq];
    const int32_t *table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
    bool bad = L < 0 || L > p.max_context_len;
    if (bad) {
        if (threadIdx.x == 0)
            report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    } else {
        int wrong = 0;
        for (int k = threadIdx.x; k < (L + BS - 1) / BS; k += kQ4Warps * 32)
            wrong |= table[k] < 0 || table[k] >= p.num_blocks;
        bad = __syncthreads_or(wrong);
        if (bad && threadIdx.x == 0)
            report(p.status, PKV_DEV_BAD_BLOCK);
    }
    float q[GM][N], o[GM][N], m[GM], l[GM];
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            o[g][n] = 0.f;
            q[g][n] = g < p.group ? to_float(static_cast<const T *>(p.q)[(int64_t)seq * p.q_stride + (kvh * p.group + g) * D + d0 + n]) * p.qscale : 0.f;
        }
    }
    auto numbers = [&](const uint8_t *rec, int row, float (&x)[N]) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + R::word(row, R::GROUPS * i + j)) >> shift;
        const float2 f = Unpack<T>::pair(*reinterpret_cast<const uint32_t *>(rec + R::template pair<BS>(row, j)));
#pragma unroll
        for (int n = 0; n < N; ++n)
            x[n] = fmaf((float)((w >> (4 * n)) & 15u), f.x, f.y);
    };
    for (int t = warp; !bad && t < L; t += kQ4Warps) {
        const int64_t at = ((int64_t)table[t / BS] * p.num_kv_heads + kvh) * R::template record<BS>;
        float k[N], v[N];
        numbers(p.k_cache + at, t % BS, k);
        numbers(p.v_cache + at, t % BS, v);
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            if (g < p.group) {
                float x = 0.f;
#pragma unroll
                for (int n = 0; n < N; ++n)
                    x = fmaf(q[g][n], k[n], x);
#pragma unroll
                for (int w = 16; w; w >>= 1)
                    x += __shfl_xor_sync(0xffffffffu, x, w);
                const float mn = fmaxf(m[g], x), ref = reference_of(mn);
                const float f = exp2f(m[g] - ref), e = exp2f(x - ref);
                m[g] = mn;
                l[g] = l[g] * f + e;
#pragma unroll
                for (int n = 0; n < N; ++n)
                    o[g][n] = fmaf(o[g][n], f, e * v[n]);
            }
        }
    }
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        if (lane == 0) {
            s_m[warp][g] = m[g];
            s_l[warp][g] = l[g];
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
            s_o[warp][g][d0 + n] = o[g][n];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < p.group * D; k += kQ4Warps * 32) {
        const int g = k / D, d = k % D;
        float mx = -INFINITY, num = 0.f, den = 0.f;
        for (int w = 0; w < kQ4Warps; ++w)
            mx = fmaxf(mx, s_m[w][g]);
        for (int w = 0; w < kQ4Warps; ++w) {
            const float f = exp2f(s_m[w][g] - reference_of(mx));
            num += f * s_o[w][g][d];
            den += f * s_l[w][g];
        }
        store_out(p.out, p.out_dtype, ((int64_t)seq * p.num_kv_heads * p.group + kvh * p.group + g) * D + d, den == 0.f ? 0.f : num / den);
    }
}

}  // namespace pkv
