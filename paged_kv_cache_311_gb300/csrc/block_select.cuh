// block_select.cuh -- select_blocks_kernel: for every (sequence, kv head) the
// blocks whose keys can matter most to the head's query group.
//
// A block's summary holds each key dimension's smallest and largest value, so
// sum_d max(q_d lo_d, q_d hi_d) bounds q . k from above for every key of the
// block.  The score is that bound summed over the group's G heads; with
// Q+ = sum_g max(q_g, 0) and Q- = sum_g max(-q_g, 0) it is one product of
// length 2 D:  score = Q+ . hi - Q- . lo.
//
// One cluster of C CTAs serves a (sequence, kv head): CTA c scores the
// consecutive blocks [c * chunk, (c + 1) * chunk) into its shared memory, and
// the selection runs over the cluster's shared memories, so scores never
// touch HBM and one launch does it all.
//
// Exactness.  Which blocks are selected is a set of whole numbers, so it must
// not depend on how a sum was rounded.  The fp32 scores carry an error bound
// eps = 2^-18 * S, S = sum_d (Q+ + Q-)_d * max|summary|_d over the CTA's
// blocks (see kScoreErr).  A radix selection finds the m-th largest fp32
// score T; scores above T + 2 eps are in, those below T - 2 eps are out, and
// only if what lies between does not fit are those blocks scored again in
// fp64 and selected by (score, then lowest block).
#pragma once

#include <cooperative_groups.h>

#include "pkv_device.cuh"

namespace pkv {

struct SelectParams {
    int32_t *selected;            // [B, Hk, K]
    const void *q;
    const void *summaries;        // [NB, Hk, 2, D]
    const int32_t *block_tables;
    const int32_t *context_lens;
    uint32_t *status;
    int64_t num_blocks;
    int num_seqs, num_kv_heads, group, max_blocks_per_seq, max_context_len, block_size;
    int num_selected, keep_first, keep_last;
    int chunk;                    // blocks per CTA
    int q_dtype;
};

constexpr int kSelectThreads = 256;

// Error of an fp32 score relative to S: each Q+- carries (G - 1) <= 7
// roundings, a product one, a lane's sum of 8 products 8, the sum over lanes
// 5: at most 21 roundings of 2^-24 each, so 2^-19 S bounds it; doubled for
// the rounding of S itself.
constexpr float kScoreErr = 1.0f / (1 << 18);

// A float's bits as an unsigned number of the same order; NaN counts as +inf.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x)
        x = INFINITY;
    x += 0.f;   // -0 -> +0
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_key64(double x)
{
    if (x != x)
        x = INFINITY;
    x += 0.0;
    const unsigned long long b = (unsigned long long)__double_as_longlong(x);
    return b >> 63 ? ~b : b | 1ull << 63;
}

// Shared memory of one CTA, before its `chunk` entries of each array.
struct SelectShared {
    uint32_t hist[2][256];   // read by the whole cluster, alternating rounds
    uint32_t scan[kSelectThreads / 32];
    uint32_t scan2[kSelectThreads / 32];
    float bound;             // this CTA's eps
    uint32_t count[4];       // this CTA's counts, read by the whole cluster
    uint32_t pick[2];        // the round's bin and what is left in it
    int bad;
};

// Exclusive sum of v over the CTA's threads; *total receives the sum.
__device__ __forceinline__ uint32_t cta_exclusive(uint32_t v, uint32_t *warp_sums, uint32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off)
            x += y;
    }
    __syncthreads();   // the sums of an earlier call are read
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w < warp)
            before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + x - v;
}

// The m-th largest (m >= 1) of the cluster's keys: key(i) of the entries i in
// [0, n) of each CTA for which live(i).  Four rounds of eight bits; *left =
// how many of the entries equal to the result are among the m largest.
template <typename Key, typename Live>
__device__ uint32_t cluster_kth(SelectShared *sh, int n, uint32_t m, Key key, Live live, int *round,
                                uint32_t *left)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, C = (int)cluster.num_blocks();
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        uint32_t *hist = sh->hist[*round & 1];
        ++*round;
        hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kSelectThreads) {
            if (live(i)) {
                const uint32_t k = key(i);
                if ((k & mask) == prefix)
                    atomicAdd(&hist[k >> shift & 255u], 1u);
            }
        }
        cluster.sync();
        // bins from the highest: thread t looks at bin 255 - t
        const int bin = 255 - tid;
        uint32_t v = 0;
        for (int c = 0; c < C; ++c)
            v += cluster.map_shared_rank(hist, c)[bin];
        uint32_t total;
        const uint32_t above = cta_exclusive(v, sh->scan, &total);
        if (above < m && m <= above + v) {
            sh->pick[0] = (uint32_t)bin;
            sh->pick[1] = m - above;
        }
        __syncthreads();
        prefix |= sh->pick[0] << shift;
        mask |= 255u << shift;
        m = sh->pick[1];
        __syncthreads();
    }
    *left = m;
    return prefix;
}

// The sum over the cluster's CTAs of count[slot] (all may call), and the sum
// over the CTAs before this one.
__device__ __forceinline__ uint32_t cluster_sum(SelectShared *sh, int slot, uint32_t *before)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    uint32_t all = 0, b = 0;
    for (int c = 0; c < C; ++c) {
        const uint32_t v = cluster.map_shared_rank(&sh->count[slot], c)[0];
        all += v;
        b += c < me ? v : 0u;
    }
    *before = b;
    return all;
}

template <typename T, int D>
__global__ void __launch_bounds__(kSelectThreads)
select_blocks_kernel(const __grid_constant__ SelectParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int HALF = D / 8;              // lanes that hold one of the two rows
    constexpr int LPB = 2 * HALF;            // lanes per block
    constexpr int BPW = 32 / LPB;            // blocks a warp scores side by side
    constexpr int NW = kSelectThreads / 32;
    extern __shared__ uint8_t smem[];
    SelectShared *sh = reinterpret_cast<SelectShared *>(smem);
    uint32_t *key = reinterpret_cast<uint32_t *>(smem + sizeof(SelectShared));
    uint32_t *key_lo = key + p.chunk;
    int32_t *phys = reinterpret_cast<int32_t *>(key_lo + p.chunk);
    float *qsum = reinterpret_cast<float *>(phys + p.chunk);   // Q+ [D], Q- [D]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int me = (int)cluster.block_rank();
    const int kvh = blockIdx.y, seq = blockIdx.z;
    int32_t *out = p.selected + ((int64_t)seq * p.num_kv_heads + kvh) * p.num_selected;
    const int K = p.num_selected;
    const int L = p.context_lens[seq];
    const bool bad_len = L < 0 || L > p.max_context_len;
    if (bad_len && kvh == 0 && me == 0 && tid == 0)
        report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    const int n = bad_len ? 0 : (L + p.block_size - 1) / p.block_size;
    const int b0 = min(me * p.chunk, n);
    const int mine = min(p.chunk, n - b0);
    const int32_t *table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq + b0;

    // ---- block ids; every CTA of the cluster learns whether one is bad
    int bad = 0;
    for (int i = tid; i < mine; i += kSelectThreads) {
        int b = table[i];
        if (b < 0 || (int64_t)b >= p.num_blocks) {
            bad = 1;
            b = 0;
        }
        phys[i] = b;
    }
    for (int d = tid; d < D; d += kSelectThreads) {
        float up = 0.f, down = 0.f;
        for (int g = 0; g < p.group; ++g) {
            const int64_t at = ((int64_t)seq * p.num_kv_heads * p.group + kvh * p.group + g) * D + d;
            const float x = p.q_dtype == PKV_F16 ? to_float(static_cast<const __half *>(p.q)[at])
                                                 : to_float(static_cast<const __nv_bfloat16 *>(p.q)[at]);
            // NaN goes into both sums
            up += x < 0.f ? 0.f : x;
            down += x > 0.f ? 0.f : -x;
        }
        qsum[d] = up;
        qsum[D + d] = down;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        sh->bad = bad;
        sh->bound = 0.f;
    }
    cluster.sync();
    for (int c = 0; c < (int)cluster.num_blocks(); ++c)
        bad |= *cluster.map_shared_rank(&sh->bad, c);
    if (bad || n <= K) {
        // a refused row selects nothing; a short one selects everything
        if (bad && me == 0 && tid == 0)
            report(p.status, PKV_DEV_BAD_BLOCK);
        const int have = bad ? 0 : n;
        for (int i = me * kSelectThreads + tid; i < K; i += (int)cluster.num_blocks() * kSelectThreads)
            out[i] = i < have ? i : -1;
        cluster.sync();   // no CTA leaves while another reads its shared memory
        return;
    }

    // ---- scores
    const bool is_lo = (lane % LPB) < HALF;
    const int c8 = (lane % HALF) * 8;
    float w[8];   // this lane's weights: -Q- on the minima, Q+ on the maxima
    float biggest[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        w[k] = is_lo ? -qsum[D + c8 + k] : qsum[c8 + k];
        biggest[k] = 0.f;
    }
    const uint4 *sums = reinterpret_cast<const uint4 *>(p.summaries);
    for (int i0 = warp * BPW; i0 < mine; i0 += NW * BPW) {
        const int i = i0 + lane / LPB;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (i < mine)
            x = sums[((int64_t)phys[i] * p.num_kv_heads + kvh) * LPB + lane % LPB];
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = Unpack<T>::pair(in[k]);
            s = fmaf(w[2 * k], f.x, s);
            s = fmaf(w[2 * k + 1], f.y, s);
            biggest[2 * k] = fmaxf(biggest[2 * k], fabsf(f.x));
            biggest[2 * k + 1] = fmaxf(biggest[2 * k + 1], fabsf(f.y));
        }
#pragma unroll
        for (int off = 1; off < LPB; off <<= 1)
            s += __shfl_xor_sync(0xffffffffu, s, off);
        if (i < mine && lane % LPB == 0)
            key[i] = order_key(s);
    }
    {
        float S = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            S += fabsf(w[k]) * biggest[k];
#pragma unroll
        for (int off = 1; off < LPB; off <<= 1)
            S += __shfl_xor_sync(0xffffffffu, S, off);
        if (lane % LPB == 0)   // NaN and infinite bounds order above every number
            atomicMax(reinterpret_cast<uint32_t *>(&sh->bound), __float_as_uint(S) & 0x7fffffffu);
    }
    cluster.sync();
    float S = 0.f;
    for (int c = 0; c < (int)cluster.num_blocks(); ++c) {
        const float x = *cluster.map_shared_rank(&sh->bound, c);
        S = !(x <= 3.0e38f) ? INFINITY : fmaxf(S, x);
    }
    const float eps = S * kScoreErr;

    // ---- the m-th largest score of the blocks that are not always selected
    const int first = min(p.keep_first, n), last = max(first, n - p.keep_last);
    const uint32_t m = (uint32_t)(K - (first + n - last));
    auto open = [&](int i) { const int j = b0 + i; return j >= first && j < last; };
    int round = 0;
    uint32_t left = 0;
    uint32_t tie_hi = 0, tie_lo = 0, ties = 0;   // which of the doubtful blocks are in
    float hi_edge = 0.f, lo_edge = 0.f;
    bool resolve = false;
    if (m > 0) {
        const uint32_t kth = cluster_kth(sh, mine, m, [&](int i) { return key[i]; }, open, &round, &left);
        const float t = key_value(kth);
        hi_edge = t + 2.f * eps;
        lo_edge = t - 2.f * eps;
        // an infinite bound or threshold decides nothing: all are doubtful
        if (!(fabsf(t) < INFINITY && eps < INFINITY)) {
            hi_edge = INFINITY;
            lo_edge = -INFINITY;
        }
    }
    // sure: above every doubt; doubtful: between the edges
    auto sure = [&](int i) { return m > 0 && key_value(key[i]) > hi_edge; };
    auto doubt = [&](int i) { return m > 0 && !(key_value(key[i]) > hi_edge) && !(key_value(key[i]) < lo_edge); };
    uint32_t doubt_total = 0, sure_total = 0, before;
    {
        uint32_t a = 0, b = 0, ta, tb;
        for (int i = tid; i < mine; i += kSelectThreads) {
            if (open(i)) {
                a += sure(i);
                b += doubt(i);
            }
        }
        cta_exclusive(a, sh->scan, &ta);
        cta_exclusive(b, sh->scan2, &tb);
        if (tid == 0) {
            sh->count[0] = ta;
            sh->count[1] = tb;
        }
        cluster.sync();
        sure_total = cluster_sum(sh, 0, &before);
        doubt_total = cluster_sum(sh, 1, &before);
    }
    resolve = m > 0 && sure_total + doubt_total > m;
    // what a block is: 0 out, 1 in, 2 in if its place among the ties allows
    auto state = [&](int i) -> int {
        const int j = b0 + i;
        if (j < first || j >= last)
            return 1;
        if (m == 0)
            return 0;
        if (!resolve)
            return sure(i) || doubt(i) ? 1 : 0;
        return (int)(key_lo[i]);
    };
    if (resolve) {
        // fp64 scores of the doubtful blocks; key / key_lo become their
        // high and low words, and then what each block is
        const uint32_t want = m - sure_total;
        for (int i = tid; i < mine; i += kSelectThreads)
            key_lo[i] = open(i) ? (sure(i) ? 1u : doubt(i) ? 2u : 0u) : 1u;
        __syncthreads();
        for (int i = warp; i < mine; i += NW) {
            if (key_lo[i] != 2u)
                continue;
            double s = 0.0;
            for (int k = lane; k < 2 * D; k += 32) {
                const int d = k % D;
                double wgt = 0.0;
                for (int g = 0; g < p.group; ++g) {
                    const int64_t at = ((int64_t)seq * p.num_kv_heads * p.group + kvh * p.group + g) * D + d;
                    const float x = p.q_dtype == PKV_F16 ? to_float(static_cast<const __half *>(p.q)[at])
                                                         : to_float(static_cast<const __nv_bfloat16 *>(p.q)[at]);
                    wgt += k < D ? (x > 0.f ? 0.f : x) : (x < 0.f ? 0.f : x);
                }
                const T v = static_cast<const T *>(p.summaries)[((int64_t)phys[i] * p.num_kv_heads + kvh) * 2 * D + k];
                s += wgt * (double)to_float(v);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, off);
            const unsigned long long kk = order_key64(s);
            if (lane == 0) {
                key[i] = (uint32_t)(kk >> 32);
                phys[i] = (int32_t)(uint32_t)kk;   // the id is not needed again
            }
        }
        __syncthreads();
        auto doubtful = [&](int i) { return key_lo[i] == 2u; };
        uint32_t left_hi;
        tie_hi = cluster_kth(sh, mine, want, [&](int i) { return key[i]; }, doubtful, &round, &left_hi);
        tie_lo = cluster_kth(sh, mine, left_hi, [&](int i) { return (uint32_t)phys[i]; },
                             [&](int i) { return key_lo[i] == 2u && key[i] == tie_hi; }, &round, &ties);
        __syncthreads();
        for (int i = tid; i < mine; i += kSelectThreads) {
            if (key_lo[i] == 2u) {
                const uint32_t a = key[i], b = (uint32_t)phys[i];
                key_lo[i] = a > tie_hi || (a == tie_hi && b > tie_lo) ? 1u : a == tie_hi && b == tie_lo ? 2u : 0u;
            }
        }
    }
    __syncthreads();

    // ---- emission in ascending order: each thread owns a run of blocks
    const int per = (mine + kSelectThreads - 1) / kSelectThreads;
    const int i0 = min(tid * per, mine), i1 = min(i0 + per, mine);
    uint32_t ins = 0, maybe = 0, total_in, total_maybe, in_before, maybe_before;
    for (int i = i0; i < i1; ++i) {
        const int s = state(i);
        ins += s == 1;
        maybe += s == 2;
    }
    uint32_t in_at = cta_exclusive(ins, sh->scan, &total_in);
    uint32_t maybe_at = cta_exclusive(maybe, sh->scan2, &total_maybe);
    if (tid == 0) {
        sh->count[2] = total_in;
        sh->count[3] = total_maybe;
    }
    cluster.sync();
    (void)cluster_sum(sh, 2, &in_before);
    (void)cluster_sum(sh, 3, &maybe_before);
    in_at += in_before;
    maybe_at += maybe_before;
    for (int i = i0; i < i1; ++i) {
        const int s = state(i);
        // the lowest `ties` of the equal scores are in
        const bool in = s == 1 || (s == 2 && maybe_at < ties);
        if (in)
            out[in_at + min(maybe_at, ties)] = b0 + i;
        in_at += s == 1;
        maybe_at += s == 2;
    }
    cluster.sync();   // no CTA leaves while another reads its shared memory
}

}  // namespace pkv
