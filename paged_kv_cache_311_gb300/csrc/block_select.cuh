// block_select.cuh -- select_blocks_kernel: for every (sequence, kv head) the
// blocks whose keys can matter most to the head's query group.
//
// A block's summary holds each key dimension's smallest and largest value, so
// sum_d max(q_d lo_d, q_d hi_d) bounds q . k from above for every key of the
// block.  The score is that bound summed over the group's G heads; with
// Q+ = sum_g max(q_g, 0) and Q- = sum_g max(-q_g, 0) it is one product of
// length 2 D:  score = Q+ . hi - Q- . lo.
//
// One cluster of C CTAs serves a (sequence, kv head).  CTA c scores the
// consecutive blocks [c * chunk, (c + 1) * chunk), a warp eight at a time, and
// stores the scores into the shared memory of CTA 0, which selects: scores
// never touch HBM, and one launch does it all.
//
// Exactness.  Which blocks are selected is a set of whole numbers, so it must
// not depend on how a sum was rounded.  The fp32 scores carry an error bound
// eps = 14 2^-24 S, S >= sum_d (Q+ + Q-)_d * max|summary|_d (see kScoreErr).
// CTA 0 finds the m-th largest fp32 score T; scores above T + 2 eps are in,
// those below T - 2 eps are out, and only if what lies between does not fit
// are those blocks scored again in fp64 and selected by (score, then lowest
// block).
#pragma once

#include <cooperative_groups.h>

#include "pkv_device.cuh"
#include "q8_cache.cuh"

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
    int most;                     // blocks of max_context_len
    int q_dtype;
};

constexpr int kSelectThreads = 256;

// Error of an fp32 score relative to S, in roundings of 2^-24: each Q+- sums
// its G <= 8 terms in a tree (3), a lane adds 8 products in two chains (4 + 1),
// the sum over lanes takes at most 5: 13; one more covers the rounding of S
// and of the edges T +- 2 eps.
constexpr float kScoreErr = 14.0f / (1 << 24);

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

constexpr int kSelectBins = 2048;
constexpr int kSelectCluster = 8;   // CTAs per cluster, at most
constexpr int kSelectList = 256;

// CTA 0's shared memory before its arrays.
struct SelectShared {
    uint32_t hist[kSelectBins];
    uint32_t list[kSelectList];
    uint32_t scan[kSelectThreads / 32];
    uint32_t pick[4];
    float bound[kSelectCluster];   // written by the cluster's CTAs
    int bad[kSelectCluster];
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

// The m-th largest (1 <= m <= number of live entries) of key[i], i in [0, n),
// live(i); *left = how many of the entries equal to it are among the m
// largest.  Each round spreads what is left over 2048 bins between its
// smallest and largest key -- scores of one row share their leading bits, and
// bins of fixed bits would put them all into a few, whose atomics then queue
// -- and keeps the bin of the m-th; once at most 256 keys are left, each is
// ranked against all.
template <typename Live>
__device__ uint32_t kth_largest(SelectShared *sh, const uint32_t *key, int n, uint32_t m, Live live, uint32_t *left)
{
    const int tid = threadIdx.x;
    uint32_t lo = 0xffffffffu, hi = 0;
    for (int i = tid; i < n; i += kSelectThreads) {
        if (live(i)) {
            lo = min(lo, key[i]);
            hi = max(hi, key[i]);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    __syncthreads();
    if (tid == 0) {
        sh->pick[0] = 0xffffffffu;
        sh->pick[1] = 0;
    }
    __syncthreads();
    if ((tid & 31) == 0) {
        atomicMin(&sh->pick[0], lo);
        atomicMax(&sh->pick[1], hi);
    }
    __syncthreads();
    lo = sh->pick[0];
    hi = sh->pick[1];
    for (;;) {
        // keys in [lo, hi] hold the m-th largest of themselves
        if (lo == hi) {
            *left = m;
            return lo;
        }
        const uint32_t span = hi - lo;
        const int shift = max(0, 32 - __clz(span) - 11);   // span >> shift < 2048
#pragma unroll
        for (int k = 0; k < kSelectBins / kSelectThreads; ++k)
            sh->hist[k * kSelectThreads + tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kSelectThreads) {
            if (live(i)) {
                const uint32_t k = key[i];
                if (k >= lo && k <= hi)
                    atomicAdd(&sh->hist[(k - lo) >> shift], 1u);
            }
        }
        __syncthreads();
        // thread t adds up bins [first, first + 8), from the highest down
        constexpr int BPT = kSelectBins / kSelectThreads;
        const int first = kSelectBins - BPT * (tid + 1);
        uint32_t h[BPT], sum = 0, total;
#pragma unroll
        for (int k = 0; k < BPT; ++k) {
            h[k] = sh->hist[first + k];
            sum += h[k];
        }
        uint32_t above = cta_exclusive(sum, sh->scan, &total);
        if (above < m && m <= above + sum) {
#pragma unroll
            for (int k = BPT - 1; k >= 0; --k) {
                if (above < m && m <= above + h[k]) {
                    sh->pick[0] = (uint32_t)(first + k);
                    sh->pick[1] = m - above;
                    sh->pick[2] = h[k];
                }
                above += h[k];
            }
            sh->pick[3] = 0;
        }
        __syncthreads();
        const uint32_t bin = sh->pick[0], inside = sh->pick[2];
        m = sh->pick[1];
        const uint32_t base = lo + (bin << shift);
        hi = base + min(hi - base, (1u << shift) - 1u);
        lo = base;
        if (shift == 0) {
            *left = m;
            return lo;
        }
        if (inside > kSelectList) {
            __syncthreads();   // pick is read
            continue;
        }
        for (int i = tid; i < n; i += kSelectThreads) {
            if (live(i)) {
                const uint32_t k = key[i];
                if (k >= lo && k <= hi)
                    sh->list[atomicAdd(&sh->pick[3], 1u)] = k;   // equal keys are alike: their order does not matter
            }
        }
        __syncthreads();
        if (tid < (int)inside) {
            const uint32_t k = sh->list[tid];
            uint32_t more = 0, same = 0;
            for (uint32_t j = 0; j < inside; ++j) {
                more += sh->list[j] > k;
                same += sh->list[j] == k;
            }
            if (more < m && m <= more + same) {
                sh->pick[0] = k;
                sh->pick[1] = m - more;
            }
        }
        __syncthreads();
        *left = sh->pick[1];
        return sh->pick[0];
    }
}

__device__ __forceinline__ float select_q(const SelectParams &p, int64_t i)
{
    return p.q_dtype == PKV_F16 ? to_float(static_cast<const __half *>(p.q)[i])
                                : to_float(static_cast<const __nv_bfloat16 *>(p.q)[i]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kSelectThreads)
select_blocks_kernel(const __grid_constant__ SelectParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int HALF = D / 8;              // lanes that hold one of a summary's two rows
    constexpr int LPB = 2 * HALF;            // lanes per block
    constexpr int BPW = 32 / LPB;            // blocks of one load
    constexpr int U = 8;                     // loads in flight
    constexpr int NW = kSelectThreads / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    SelectShared *sh = reinterpret_cast<SelectShared *>(smem);
    float *qsum = reinterpret_cast<float *>(smem + sizeof(SelectShared));   // Q+ [D], Q- [D]
    int32_t *phys = reinterpret_cast<int32_t *>(qsum + 2 * D);              // [chunk]
    uint32_t *key = reinterpret_cast<uint32_t *>(phys + p.chunk);           // [most], CTA 0's in use
    uint32_t *in = key + p.most;                                            // bit i: block i is selected
    uint32_t *pend = in + (p.most + 31) / 32;                               // bit i: block i is in doubt

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int me = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
    const int kvh = blockIdx.y, seq = blockIdx.z;
    cluster.barrier_arrive();   // CTA 0 has started once this completes: its memory may be written
    const int L = p.context_lens[seq];
    const bool bad_len = L < 0 || L > p.max_context_len;
    if (bad_len && kvh == 0 && me == 0 && tid == 0)
        report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    const int n = bad_len ? 0 : (L + p.block_size - 1) / p.block_size;
    const int K = p.num_selected;
    const int b0 = min(me * p.chunk, n);
    const int mine = min(p.chunk, n - b0);
    const int32_t *table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
    const int64_t q0 = ((int64_t)seq * p.num_kv_heads + kvh) * p.group * D;

    int bad = 0;
    for (int i = tid; i < mine; i += kSelectThreads) {
        int b = table[b0 + i];
        if (b < 0 || (int64_t)b >= p.num_blocks) {
            bad = 1;
            b = 0;
        }
        phys[i] = b;
    }
    if (n > K && tid < D) {
        float up[8], down[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const float x = g < p.group ? select_q(p, q0 + (int64_t)g * D + tid) : 0.f;
            // NaN goes into both sums
            up[g] = x < 0.f ? 0.f : x;
            down[g] = x > 0.f ? 0.f : -x;
        }
#pragma unroll
        for (int k = 4; k >= 1; k >>= 1) {
#pragma unroll
            for (int g = 0; g < k; ++g) {
                up[g] += up[g + k];
                down[g] += down[g + k];
            }
        }
        qsum[tid] = up[0];
        qsum[D + tid] = down[0];
    }
    bad = __syncthreads_or(bad);
    cluster.barrier_wait();

    // ---- scores, into CTA 0's shared memory
    float S = 0.f;
    if (n > K && !bad) {
        uint32_t *keys = cluster.map_shared_rank(key, 0) + b0;
        const bool is_lo = (lane % LPB) < HALF;
        const int c8 = (lane % HALF) * 8;
        float w[8];   // this lane's weights: -Q- on the minima, Q+ on the maxima
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = is_lo ? -qsum[D + c8 + k] : qsum[c8 + k];
        using V = typename Pair16<T>::V;
        V biggest[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            biggest[k] = as_pair<T>(0u);
        const uint4 *sums = reinterpret_cast<const uint4 *>(p.summaries) + kvh * LPB + lane % LPB;
        const int64_t stride = (int64_t)p.num_kv_heads * LPB;
        for (int i0 = warp * U * BPW; i0 < mine; i0 += NW * U * BPW) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * BPW + lane / LPB;
                x[u] = make_uint4(0, 0, 0, 0);
                if (i < mine)
                    x[u] = __ldg(sums + phys[i] * stride);
            }
            float s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t word[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                float2 two = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    two = ffma2(make_float2(w[2 * k], w[2 * k + 1]), Unpack<T>::pair(word[k]), two);
                    biggest[k] = __hmax2(biggest[k], as_pair<T>(word[k] & 0x7fff7fffu));
                }
                s[u] = two.x + two.y;
            }
            // sums over a block's lanes: the halves of the lanes take halves
            // of the blocks until each lane has one, then add up the rest
            int u0 = 0;
#pragma unroll
            for (int k = U / 2, off = LPB / 2; k >= 1; k >>= 1, off >>= 1) {
                const bool up = lane & off;
#pragma unroll
                for (int u = 0; u < k; ++u) {
                    const float give = up ? s[u] : s[u + k];
                    const float keep = up ? s[u + k] : s[u];
                    s[u] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
                u0 += up ? k : 0;
            }
#pragma unroll
            for (int off = LPB / 2 / U; off >= 1; off >>= 1)
                s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
            const int i = i0 + u0 * BPW + lane / LPB;
            if (i < mine && lane % (LPB / U) == 0)
                keys[i] = order_key(s[0]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = Unpack<T>::pair(as_word(biggest[k]));
            S += fabsf(w[2 * k]) * f.x;
            S += fabsf(w[2 * k + 1]) * f.y;
        }
#pragma unroll
        for (int off = 1; off < LPB; off <<= 1)
            S += __shfl_xor_sync(0xffffffffu, S, off);
        // NaN and infinity order above every number
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(S) & 0x7fffffffu);
        if (lane == 0)
            sh->scan[warp] = most;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int k = 0; k < NW; ++k)
            all = max(all, sh->scan[k]);
        S = __uint_as_float(all);
    }
    if (tid == 0) {
        SelectShared *to = cluster.map_shared_rank(sh, 0);
        to->bound[me] = S;
        to->bad[me] = bad;
    }
    cluster.sync();
    if (me != 0)
        return;

    // ---- CTA 0 selects
    S = 0.f;
    for (int c = 0; c < C; ++c) {
        S = !(sh->bound[c] <= 3.0e38f) ? INFINITY : fmaxf(S, sh->bound[c]);
        bad |= sh->bad[c];
    }
    int32_t *out = p.selected + ((int64_t)seq * p.num_kv_heads + kvh) * K;
    if (bad || n <= K) {
        // a refused row selects nothing; a short one selects everything
        if (bad && tid == 0)
            report(p.status, PKV_DEV_BAD_BLOCK);
        const int have = bad ? 0 : n;
        for (int i = tid; i < K; i += kSelectThreads)
            out[i] = i < have ? i : -1;
        return;
    }
    const int first = min(p.keep_first, n), last = max(first, n - p.keep_last);
    const uint32_t m = (uint32_t)(K - (first + n - last));   // places for blocks [first, last)
    const int words = (n + 31) / 32;
    uint32_t ties = 0;   // of the blocks in doubt, the lowest `ties` are in
    float hi_edge = INFINITY, lo_edge = INFINITY;
    if (m > 0) {
        const float eps = S * kScoreErr;
        uint32_t left;
        const float t = key_value(kth_largest(sh, key, n, m, [&](int i) { return i >= first && i < last; }, &left));
        const bool finite = fabsf(t) < INFINITY && eps < INFINITY;   // else all are in doubt
        hi_edge = finite ? t + 2.f * eps : INFINITY;
        lo_edge = finite ? t - 2.f * eps : -INFINITY;
    }
    uint32_t sure = 0, doubt = 0;
    for (int i = tid; i < words * 32; i += kSelectThreads) {   // a warp's 32 blocks are one word
        bool a = i < n, b = false;
        if (i >= first && i < last) {
            const float s = key_value(key[i]);
            a = m > 0 && s > hi_edge;
            b = m > 0 && !a && !(s < lo_edge);
            sure += a;
            doubt += b;
        }
        const uint32_t wa = __ballot_sync(0xffffffffu, a), wb = __ballot_sync(0xffffffffu, b);
        if (lane == 0) {
            in[i / 32] = wa;
            pend[i / 32] = wb;
        }
    }
    uint32_t sure_total, doubt_total;
    (void)cta_exclusive(sure, sh->scan, &sure_total);
    (void)cta_exclusive(doubt, sh->scan, &doubt_total);
    ties = m - sure_total;
    if (doubt_total > ties && S > 0.f) {
        // The blocks in doubt by their fp64 scores.
        auto exact = [&](int i) -> unsigned long long {   // by a warp
            double s = 0.0;
            const int64_t at = ((int64_t)table[i] * p.num_kv_heads + kvh) * 2 * D;
            double wgt[2 * D / 32], v[2 * D / 32];
#pragma unroll
            for (int k = 0; k < 2 * D / 32; ++k) {
                v[k] = (double)to_float(static_cast<const T *>(p.summaries)[at + k * 32 + lane]);
                wgt[k] = 0.0;
            }
            for (int g = 0; g < p.group; ++g) {
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const float x = select_q(p, q0 + (int64_t)g * D + k * 32 + lane);
                    wgt[k] += x > 0.f ? 0.f : x;
                    wgt[k + D / 32] += x < 0.f ? 0.f : x;
                }
            }
#pragma unroll
            for (int k = 0; k < 2 * D / 32; ++k)
                s += wgt[k] * v[k];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, off);
            return order_key64(s);
        };
        if (doubt_total <= kSelectList) {
            // a few (two, mostly): listed in ascending order, ranked against each other
            const int per = (words + kSelectThreads - 1) / kSelectThreads;
            const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
            uint32_t c = 0, total;
            for (int k = w0; k < w1; ++k)
                c += __popc(pend[k]);
            c = cta_exclusive(c, sh->scan, &total);
            for (int k = w0; k < w1; ++k)
                for (uint32_t w = pend[k]; w; w &= w - 1)
                    sh->list[c++] = k * 32 + __ffs(w) - 1;
            __syncthreads();
            unsigned long long *score = reinterpret_cast<unsigned long long *>(sh->hist);
            for (uint32_t e = warp; e < doubt_total; e += NW) {
                const unsigned long long kk = exact((int)sh->list[e]);
                if (lane == 0)
                    score[e] = kk;
            }
            for (int k = tid; k < words; k += kSelectThreads)
                pend[k] = 0;
            __syncthreads();
            if (tid < (int)doubt_total) {
                const unsigned long long mine64 = score[tid];
                uint32_t rank = 0;
                for (uint32_t e = 0; e < doubt_total; ++e)
                    rank += score[e] > mine64 || (score[e] == mine64 && e < (uint32_t)tid);
                if (rank < ties)
                    atomicOr(&in[sh->list[tid] / 32], 1u << (sh->list[tid] % 32));
            }
            ties = 0;
        } else
        // many: by their high words and then, among equals, by their low words
        for (int half = 0; half < 2; ++half) {
            for (int i = warp; i < n; i += NW) {
                if (!(pend[i / 32] >> (i % 32) & 1u))
                    continue;
                const unsigned long long kk = exact(i);
                if (lane == 0)
                    key[i] = half ? (uint32_t)kk : (uint32_t)(kk >> 32);
            }
            __syncthreads();
            uint32_t left;
            const uint32_t t = kth_largest(sh, key, n, ties, [&](int i) { return (pend[i / 32] >> (i % 32) & 1u) != 0; }, &left);
            __syncthreads();
            uint32_t still = 0;
            for (int i = tid; i < words * 32; i += kSelectThreads) {
                const uint32_t old = pend[i / 32];
                const bool is = i < n && (old >> lane & 1u);
                const uint32_t k = is ? key[i] : 0u;
                const uint32_t wa = __ballot_sync(0xffffffffu, is && k > t);
                const uint32_t wb = __ballot_sync(0xffffffffu, is && k == t);
                if (lane == 0) {
                    in[i / 32] |= wa;
                    pend[i / 32] = wb;
                }
                still += is && k == t;
            }
            ties = left;
            uint32_t total;
            (void)cta_exclusive(still, sh->scan, &total);
            if (total == ties)
                break;
        }
    }
    __syncthreads();

    // ---- emission in ascending order: thread t owns words [w0, w1)
    const int per = (words + kSelectThreads - 1) / kSelectThreads;
    const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
    uint32_t c = 0, total;
    for (int k = w0; k < w1; ++k)
        c += __popc(pend[k]);
    uint32_t seen = cta_exclusive(c, sh->scan, &total);
    c = 0;
    for (int k = w0; k < w1; ++k) {
        // the lowest `ties` blocks in doubt are in
        uint32_t w = pend[k], kept = 0;
        const uint32_t here = (uint32_t)__popc(w);
        if (seen + here <= ties) {
            kept = w;
        } else {
            for (uint32_t left = seen < ties ? ties - seen : 0u; left > 0; --left) {
                kept |= w & (0u - w);
                w &= w - 1;
            }
        }
        seen += here;
        in[k] |= kept;
        c += __popc(in[k]);
    }
    uint32_t at = cta_exclusive(c, sh->scan, &total);
    for (int k = w0; k < w1; ++k) {
        for (uint32_t w = in[k]; w; w &= w - 1)
            out[at++] = k * 32 + __ffs(w) - 1;
    }
}

}  // namespace pkv
