// block_select.cuh -- select_blocks_kernel: for every (sequence, kv head) the
// blocks whose keys can matter most to the head's query group.
//
// A block's summary holds each key dimension's smallest and largest value, so
// sum_d max(q_d lo_d, q_d hi_d) bounds q . k from above for every key of the
// block.  The score is that bound summed over the group's G heads; with
// Q+ = sum_g max(q_g, 0) and Q- = sum_g max(-q_g, 0) it is one product of
// length 2 D:  score = Q+ . hi - Q- . lo.
//
// The scores are a matrix product on the tensor cores (m16n8k16, fp32 sums):
// 16 blocks' summaries are A; B's columns hold the row's weights in three parts
// of the summaries' type, 24 bits in all, and a fourth column |weights|, which
// with |A| gives each block's error bound.  (In fp32 arithmetic a warp spent 65
// instructions on a block -- unpacking, sums over lanes, the bound -- and 34 us
// on 101 MB.)  A warp streams its tiles of 16 blocks through a ring of bulk
// copies, one per summary (512 bytes at head_dim 128, in rows padded by 16
// bytes so that ldmatrix meets no bank twice), whose first leave as soon as
// the ids are there, before the weights are computed.  (With the tiles in
// registers the CTAs of a wave computed weights together and waited together:
// 30 us.)  select_row then finds the row's selection.  Two ways to run them:
//   one launch (select_blocks_kernel): a cluster of C CTAs per row, whose
//     warps store their scores into the shared memory of CTA 0, which selects;
//   two (score_blocks_kernel, select_rows_kernel): scores go through the
//     workspace, for calls whose clusters would not fill the SMs evenly
//     (128 rows of up to 2048 blocks as clusters of four: some SMs got six CTAs
//     and some none).
//
// What bounds it: 16 x 8 rows of 1024 to 2048 blocks (101 MB of summaries, 15 us
// at the HBM's rate) take 29.5 to 32 us, some 23 for the scores -- a plain load
// kernel takes 21.5 for as much -- and 8 for the second launch, whose code runs
// once.  4 x 8 rows of 128 to 512 blocks take 8 us, latencies throughout.
//
// Exactness.  Which blocks are selected is a set of whole numbers, so it must
// not depend on how a sum was rounded.  A score carries an error of at most
// eps = 2^-17.5 S, S the largest sum_d |weight_d summary_d| of the row's blocks
// (see kScoreErr).  select_row finds the m-th largest score T; scores above
// T + 2 eps are in, those below T - 2 eps are out, and only if what lies
// between does not fit are those blocks (a few) scored again in pairs of fp32
// numbers and selected by (score, then lowest block).  Pairs hold 48 bits: some
// 20 operations, each off by a few 2^-47 of its operands, leave a score
// within 2^-42 of the sum of its terms' magnitudes.
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
    int chunk;                    // blocks a CTA scores
    int most;                     // blocks of max_context_len
    int key_stride;               // keys of a row, whole 16-byte pieces
    int bounds;                   // warps that score a row
    uint32_t *ws_keys;            // two launches: [B * Hk][key_stride] scores' keys
    float *ws_bound;              // [B * Hk][bounds]: score_blocks' results
    int q_dtype;
};

// Threads of a selecting CTA (NT below): 256, or 128 where the rows are more
// than the CTAs of 256 threads that an SM holds, two in one launch and four in
// two.  (256 against 128 threads, us, one launch: 256 rows of 128 blocks 8.9
// and 10.1, 512 17.2 and 13.0, 1584 of 32 28.6 and 16.9; two: 128 of 2048 29.2
// and 31.4, 680 of 432 25.2 and 22.6, 1024 of 256 36 and 32.8.)
constexpr int kSelectThreads = 256;
// Two launches: warps of a scoring CTA, tiles in flight and tiles of 16 blocks
// per warp.  (Stages, tiles: 2, 8 took 30 us on 16 x 8 rows of up to 2048
// blocks, so did 1, 4; 2, 6 34; 2, 16 34.3; 3, 4 34.5; 1, 8 31.7.)
constexpr int kScoreWarps = 4;
constexpr int kScoreStages = 2;
constexpr int kScoreTiles = 8;

// Error of a score relative to S.  A step on the tensor cores adds 16 exact
// products and the running sum, aligned to the largest of them and cut off
// (taken as) at one unit in its last place, 2^-23.  Eight chains of two steps
// each: 2 x 17 x 2^-23 of what the chain adds up.  Joining the chains and the
// three parts takes 5 roundings of 2^-24, the weights another 4 and the edges
// T +- 2 eps two.  Together 40 x 2^-23; 44 are taken.  How many bits the tensor
// cores keep of a sum is not documented: one unit of 2^-23 per product is what
// this rests on.  Measured on sums made to lose all that a cut can take: 8 x
// 2^-23 of the terms at head_dim 128, 4 x 2^-23 at 64 (a cut at 2^-25).
//
// Three parts of a weight w leave out at most 2^-24 |w| in bfloat16 (one of
// the four above).  In f16 they leave out 2^-33 |w|, but not less than half of
// f16's last bit, 2^-25, however small w is: kWeightPad, which every |w| in S
// is raised by, makes eps cover it, 44 x 2^-23 x 2^-7 = 2^-24.5.
constexpr float kScoreErr = 44.0f / (1 << 23);
template <typename T> constexpr float kWeightPad = std::is_same<T, __half>::value ? 0x1p-7f : 0x1p-9f;

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
constexpr int kSelectBins = 2048;
constexpr int kSelectCluster = 8;   // CTAs per cluster, at most
constexpr int kSelectList = 256;

// h + l with |l| at most half a unit of h: 48 bits.  Each operation is off by
// a few 2^-47 of its operands.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair pair_add(Pair a, Pair b)
{
    // the sum of the high parts and its exact rounding error, then the rest
    const float s = a.h + b.h, t = s - a.h;
    const float e = (a.h - (s - t)) + (b.h - t) + (a.l + b.l);
    const float h = s + e;
    return Pair{h, e - (h - s)};
}
__device__ __forceinline__ Pair pair_mul(Pair a, float b)
{
    const float p = a.h * b, e = fmaf(a.l, b, fmaf(a.h, b, -p));
    const float h = p + e;
    return Pair{h, e - (h - p)};
}

// Shared memory of a CTA before its arrays.
struct alignas(16) SelectShared {
    uint32_t hist[kSelectBins];
    uint32_t list[kSelectList];
    uint32_t scan[kSelectThreads / 32];
    uint32_t pick[4];
    uint64_t bar;
    float bound[kSelectCluster * kSelectThreads / 32];   // written by the cluster's warps
    Pair weight[2 * 128];          // -Q-, Q+ for exact scores
};

// The code of a selection runs once per CTA, so its time is that of fetching
// it (128 bytes of instructions in some 45 cycles): loops stay rolled and
// what is used twice is a function.

// Exclusive sum of v over the CTA's threads; *total receives the sum.
template <int NT>
__device__ __noinline__ uint32_t cta_exclusive(uint32_t v, uint32_t *warp_sums, uint32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
        x += lane >= off ? y : 0u;
    }
    __syncthreads();   // the sums of an earlier call are read
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    // a warp's lanes hold the warps' sums
    const uint32_t s = lane < NT / 32 ? warp_sums[lane] : 0u;
    *total = __reduce_add_sync(0xffffffffu, s);
    return __reduce_add_sync(0xffffffffu, lane < warp ? s : 0u) + x - v;
}

// The m-th largest (1 <= m <= their number) of the keys i in [first, last)
// whose bit is set in `mask` (null: all); *left = how many of those equal to it
// are among the m largest.  Each round spreads what is left over 2048 bins
// between its smallest and largest key -- scores of one row share their
// leading bits, and bins of fixed bits would put them all into a few, whose
// atomics then queue -- and keeps the bin of the m-th; once at most 256 keys
// are left, each is ranked against all.
template <int NT>
__device__ __noinline__ uint32_t kth_largest(SelectShared *sh, const uint32_t *key, int first, int last, const uint32_t *mask,
                                             uint32_t m, uint32_t *left)
{
    const int tid = threadIdx.x;
    uint32_t lo = 0xffffffffu, hi = 0;
    // 0: the range; 1: the histogram; 2: the keys of the bin
    auto pass = [&](int what, uint32_t from, uint32_t to, int shift) {
#pragma unroll 2
        for (int i = first + tid; i < last; i += NT) {
            const uint32_t k = key[i];
            if ((mask && !(mask[i / 32] >> (i % 32) & 1u)) || k < from || k > to)
                continue;
            if (what == 0) {
                lo = min(lo, k);
                hi = max(hi, k);
            } else if (what == 1) {
                atomicAdd(&sh->hist[(k - from) >> shift], 1u);
            } else {
                sh->list[atomicAdd(&sh->pick[3], 1u)] = k;   // equal keys are alike: their order does not matter
            }
        }
    };
    uint32_t from = 0, to = 0xffffffffu;
    int what = 0, shift = 0;
    __syncthreads();
    if (tid == 0) {
        sh->pick[0] = 0xffffffffu;
        sh->pick[1] = 0;
    }
#pragma unroll 1
    for (;;) {
        if (what == 1) {
#pragma unroll 1
            for (int k = tid; k < kSelectBins / 4; k += NT)
                *reinterpret_cast<uint4 *>(sh->hist + 4 * k) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
        pass(what, from, to, shift);
        if (what == 0) {
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if ((tid & 31) == 0) {
                atomicMin(&sh->pick[0], lo);
                atomicMax(&sh->pick[1], hi);
            }
            __syncthreads();
            from = sh->pick[0];
            to = sh->pick[1];
            what = 1;
        } else if (what == 1) {
            __syncthreads();
            // thread t adds up bins [at, at + BPT), from the highest down
            constexpr int BPT = kSelectBins / NT;
            const int at = kSelectBins - BPT * (tid + 1);
            uint32_t sum = 0;
#pragma unroll
            for (int k = 0; k < BPT; k += 4) {
                const uint4 a = *reinterpret_cast<const uint4 *>(sh->hist + at + k);
                sum += (a.x + a.y) + (a.z + a.w);
            }
            uint32_t total;
            uint32_t above = cta_exclusive<NT>(sum, sh->scan, &total);
            if (above < m && m <= above + sum) {
                int k = at + BPT - 1;
                while (above + sh->hist[k] < m)
                    above += sh->hist[k--];
                sh->pick[0] = (uint32_t)k;
                sh->pick[1] = m - above;
                sh->pick[2] = sh->hist[k];
                sh->pick[3] = 0;
            }
            __syncthreads();
            m = sh->pick[1];
            const uint32_t base = from + (sh->pick[0] << shift);
            to = base + min(to - base, (1u << shift) - 1u);
            from = base;
            what = shift > 0 && sh->pick[2] <= NT ? 2 : 1;
        } else {
            __syncthreads();
            const uint32_t inside = sh->pick[2];
            if (tid < (int)inside) {
                const uint32_t k = sh->list[tid];
                uint32_t more = 0, same = 0;
#pragma unroll 1
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
        if (from == to) {   // the keys left are equal
            *left = m;
            return from;
        }
        shift = max(0, 32 - __clz(to - from) - 11);   // (to - from) >> shift < 2048
        // the bin's keys are listed with the range as it is
        __syncthreads();   // pick is read
    }
}

__device__ __forceinline__ float select_q(const SelectParams &p, int64_t i)
{
    return p.q_dtype == PKV_F16 ? to_float(static_cast<const __half *>(p.q)[i])
                                : to_float(static_cast<const __nv_bfloat16 *>(p.q)[i]);
}

// -Q- and Q+ of dimension tid < D in pairs, from the group's q, into weight
// [2 D]: for exact scores.  `scale`: a power of two that keeps them below 2^15
// (any that does: only the order of scores counts).
template <int D>
__device__ __forceinline__ void exact_weights(Pair *weight, float (&x)[8], float scale)
{
    Pair lo{0.f, 0.f}, hi{0.f, 0.f};
#pragma unroll 2
    for (int h = 0; h < 8; ++h) {
        const float y = x[0] * scale;
#pragma unroll
        for (int k = 0; k < 7; ++k)
            x[k] = x[k + 1];
        lo = pair_add(lo, Pair{y > 0.f ? 0.f : y, 0.f});
        hi = pair_add(hi, Pair{y < 0.f ? 0.f : y, 0.f});
    }
    weight[threadIdx.x] = lo;
    weight[D + threadIdx.x] = hi;
}

// The power of two that brings the largest of the CTA's `big` (>= 0) to [2^14,
// 2^15); warp_big: a word per warp.  All threads call it.
template <int NW>
__device__ __forceinline__ float weight_scale(float big, uint32_t *warp_big)
{
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
    if ((threadIdx.x & 31) == 0)
        warp_big[threadIdx.x >> 5] = most;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k)
        all = max(all, warp_big[k]);
    const int e = min(max((int)(all >> 23) - 127 - 14, -120), 120);
    return __uint_as_float((uint32_t)(127 - e) << 23);
}

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// A row's number of blocks; a refused length has none (`report`: says so).
__device__ __forceinline__ int row_blocks(const SelectParams &p, int L, bool tell)
{
    if (L < 0 || L > p.max_context_len) {
        if (tell)
            report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
        return 0;
    }
    return (L + p.block_size - 1) / p.block_size;
}

// What a scoring warp gives in place of its S: one of its blocks' ids is
// outside the pool; a copy timed out (and was reported).
constexpr float kBadChunk = -1.f;
constexpr float kLateChunk = -2.f;

// Whether the wait on `bar` ended for all of the CTA's threads (`mine`: for
// this one).  If it did not, thread 0 reports that and sees the copies off,
// whoever gave up.  All threads call it.
__device__ __forceinline__ bool cta_waited(bool mine, uint64_t *bar, uint32_t parity, uint32_t *status,
                                           uint64_t limit_ns = kWaitLimitNs)
{
    if (__syncthreads_and(mine))
        return true;
    if (threadIdx.x == 0) {
        report(status, PKV_DEV_TIMEOUT);
        drain_wait(bar, parity, status, limit_ns);
    }
    return false;
}

// Shared memory of a scoring CTA of NW warps with rings of S tiles: the
// weights [part][2 D] in the summaries' type -- three parts of -Q- (minima) and
// Q+ (maxima), and a bound of their magnitude -- and the rings.
template <int D, int NW, int S>
struct alignas(16) ScoreShared {
    static constexpr int LINE = 4 * D + 16;      // bytes from one summary of a tile to the next
    uint8_t ring[NW][S][16 * LINE];
    uint16_t part[4][2 * D + 8];
    uint64_t bar[NW][S];
    uint32_t big[NW];
};

// Keys of blocks [b0, b0 + p.chunk) of row (seq, kvh) into keys[0 ..], by a CTA
// of NW warps.  Returns each warp's S (in units of the weights' scale), or
// kBadChunk or kLateChunk; nothing is scored in a row that is selected whole.  n receives the row's
// number of blocks, weight (unless null) the weights of exact scores;
// before_stores() runs before the first store.
template <typename T, int D, int NW, int ST, typename Before>
__device__ __forceinline__ float score_blocks(const SelectParams &p, ScoreShared<D, NW, ST> *sw, int seq, int kvh, int b0,
                                              uint32_t *keys, int &n, Pair *weight, bool tell, Before before_stores)
{
    using Sh = ScoreShared<D, NW, ST>;
    constexpr int KS = 2 * D / 16;           // k steps
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    uint64_t *bar = sw->bar[warp];
    // what needs only the arguments leaves at once: the length, the first
    // tiles' ids (as far as the table goes; lane i holds block i of a tile)
    // and q
    const int L = p.context_lens[seq];
    const int32_t *table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq + b0;
    const int there = lane < 16 ? min(p.chunk, p.max_blocks_per_seq - b0) : 0;
    int id[ST];
#pragma unroll
    for (int k = 0; k < ST; ++k) {
        const int i = (warp + k * NW) * 16 + lane;
        id[k] = i < there ? table[i] : 0;
    }
    float x[8];
#pragma unroll
    for (int h = 0; h < 8; ++h)
        x[h] = tid < D && h < p.group ? select_q(p, (((int64_t)seq * p.num_kv_heads + kvh) * p.group + h) * D + tid) : 0.f;
    if (lane == 0) {
        for (int s = 0; s < ST; ++s)
            mbar_init(&bar[s], 1);
        fence_mbar_init();
    }
    __syncwarp();

    n = row_blocks(p, L, tell);
    const int mine = max(0, min(p.chunk, n - b0));
    const int tiles = (mine + 15) / 16, my_n = warp < tiles ? (tiles - 1 - warp) / NW + 1 : 0;
    const bool score = n > p.num_selected && mine > 0;
    bool bad = false;
    const uint8_t *sums = reinterpret_cast<const uint8_t *>(p.summaries) + (int64_t)kvh * (4 * D);
    const int64_t stride = (int64_t)p.num_kv_heads * (4 * D);
    // the warp's k-th tile into stage k % ST
    auto issue = [&](int k, int block) {
        const int i0 = (warp + k * NW) * 16, live = min(16, mine - i0);
        const bool good = block >= 0 && (int64_t)block < p.num_blocks;
        bad |= lane < live && !good;
        if (!score)
            return;
        uint64_t *b = &bar[k % ST];
        if (lane == 0)
            mbar_arrive_expect_tx(b, (uint32_t)(live * 4 * D));
        __syncwarp();
        if (lane < live)
            bulk_load(&sw->ring[warp][k % ST][lane * Sh::LINE], sums + (good ? block : 0) * stride, 4 * D, b);
    };
#pragma unroll
    for (int k = 0; k < ST; ++k)
        if (k < my_n)
            issue(k, id[k]);

    uint32_t bf[KS][2];   // B fragments: column g of k step ks
    if (score) {
        float up[8], down[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            // NaN goes into both sums
            up[h] = x[h] < 0.f ? 0.f : x[h];
            down[h] = x[h] > 0.f ? 0.f : -x[h];
        }
#pragma unroll
        for (int k = 4; k >= 1; k >>= 1) {
#pragma unroll
            for (int h = 0; h < k; ++h) {
                up[h] += up[h + k];
                down[h] += down[h + k];
            }
        }
        // inside both types' range
        const float scale = weight_scale<NW>(fmaxf(up[0], down[0]), sw->big);
        if (weight && tid < D)
            exact_weights<D>(weight, x, scale);
        if (tid < D) {
            auto split = [&](float w, int at) {
                T one;
                float rest = w;
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    one = from_float<T>(rest);
                    sw->part[k][at] = *reinterpret_cast<const uint16_t *>(&one);
                    rest -= to_float(one);
                }
                // an upper bound, and kWeightPad for what the three parts leave out
                one = from_float<T>(fabsf(w) * 1.015625f + kWeightPad<T>);
                sw->part[3][at] = *reinterpret_cast<const uint16_t *>(&one);
            };
            split(-down[0] * scale, tid);
            split(up[0] * scale, D + tid);
        }
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(sw->part[g & 3]) + 8 * ks + c;
            bf[ks][0] = g < 4 ? w[0] : 0u;
            bf[ks][1] = g < 4 ? w[4] : 0u;
        }
    }
    before_stores();

    uint32_t S = 0;   // as its bits: NaN and infinity order above every number
    // this lane's ldmatrix row in a tile
    const uint32_t row = ((lane & 7) + ((lane >> 3) & 1) * 8) * Sh::LINE + (lane >> 4) * 16;
    for (int k = 0; k < my_n; ++k) {
        const int i0 = (warp + k * NW) * 16, st = k % ST;
        const int i_next = i0 + ST * NW * 16 + lane;
        const int next = k + ST < my_n && i_next < there ? table[i_next] : 0;
        if (score) {
            // the warp gives up as one: its products and shuffles need every lane
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bar[st], (uint32_t)((k / ST) & 1)))) {
                // no CTA leaves with copies in flight
                for (int u = k; u < min(my_n, k + ST); ++u)
                    drain_wait(&bar[u % ST], (uint32_t)((u / ST) & 1), p.status);
                if (lane == 0)
                    report(p.status, PKV_DEV_TIMEOUT);
                return __any_sync(0xffffffffu, bad) ? kBadChunk : kLateChunk;
            }
            const uint32_t base = smem_u32(sw->ring[warp][st]) + row;
            float s[8][4], b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                constexpr int PER = KS / 8;   // steps of a chain
                uint32_t a[4];
                ldsm_x4(base + ks * 32, a);
                if (ks % PER == 0)
                    s[ks / PER][0] = s[ks / PER][1] = s[ks / PER][2] = s[ks / PER][3] = 0.f;
                Mma<T>::run(s[ks / PER], a, bf[ks][0], bf[ks][1]);
                // rows past the last block hold anything: theirs alone are wrong
                const uint32_t m[4] = {a[0] & 0x7fff7fffu, a[1] & 0x7fff7fffu, a[2] & 0x7fff7fffu, a[3] & 0x7fff7fffu};
                Mma<T>::run(b, m, bf[ks][0], bf[ks][1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[0][j] = ((s[0][j] + s[1][j]) + (s[2][j] + s[3][j])) + ((s[4][j] + s[5][j]) + (s[6][j] + s[7][j]));
            // columns 0, 1 are in lane c = 0, columns 2, 3 in lane c = 1
            const float p0 = __shfl_down_sync(0xffffffffu, s[0][0], 1), p1 = __shfl_down_sync(0xffffffffu, s[0][2], 1);
            const float m0 = __shfl_down_sync(0xffffffffu, b[1], 1), m1 = __shfl_down_sync(0xffffffffu, b[3], 1);
            if (c == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = i0 + g + 8 * h;
                    if (i < mine) {
                        keys[i] = order_key((s[0][2 * h] + s[0][2 * h + 1]) + (h ? p1 : p0));
                        S = max(S, __float_as_uint(h ? m1 : m0) & 0x7fffffffu);
                    }
                }
            }
        }
        __syncwarp();
        if (k + ST < my_n) {
            if (lane < 16)
                fence_proxy_async_smem();
            issue(k + ST, next);
        }
    }
    if (__any_sync(0xffffffffu, bad))
        return kBadChunk;
    return __uint_as_float(__reduce_max_sync(0xffffffffu, S));
}

// The selection of row (seq, kvh) of n blocks from its keys and its chunks'
// bounds, by one CTA.  in, pend: a bit for each block.
template <typename T, int D, int NT>
__device__ __forceinline__ void select_row(const SelectParams &p, SelectShared *sh, uint32_t *key, uint32_t *in,
                                           uint32_t *pend, const float *bounds, int seq, int kvh, int n)
{
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.num_selected;
    const int32_t *table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
    // the chunks' bounds, a lane each: NaN and infinity order above numbers
    float S;
    bool bad = false, late = false;
    {
        uint32_t most = 0;
        for (int c = lane; c < p.bounds; c += 32) {
            const float x = bounds[c];
            bad |= x == kBadChunk;
            late |= x == kLateChunk;
            most = max(most, __float_as_uint(x) & 0x7fffffffu);
        }
        bad = __any_sync(0xffffffffu, bad);
        late = __any_sync(0xffffffffu, late);
        S = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
        S = !(S <= 3.0e38f) ? INFINITY : S;
    }
    int32_t *out = p.selected + ((int64_t)seq * p.num_kv_heads + kvh) * K;
    if (bad || late || n <= K) {
        // a refused row selects nothing; a short one selects everything
        if (bad && tid == 0)
            report(p.status, PKV_DEV_BAD_BLOCK);
        const int have = bad || late ? 0 : n;
        for (int i = tid; i < K; i += NT)
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
        const float t = key_value(kth_largest<NT>(sh, key, first, last, nullptr, m, &left));
        const bool finite = fabsf(t) < INFINITY && eps < INFINITY;   // else all are in doubt
        hi_edge = finite ? t + 2.f * eps : INFINITY;
        lo_edge = finite ? t - 2.f * eps : -INFINITY;
    }
    uint32_t counts = 0;   // sure ones below, those in doubt above 16 bits, of this thread's
#pragma unroll 2
    for (int i = tid; i < words * 32; i += NT) {   // a warp's 32 blocks are one word
        bool a = i < n, b = false;
        if (i >= first && i < last) {
            const float s = key_value(key[i]);
            a = m > 0 && s > hi_edge;
            b = m > 0 && !a && !(s < lo_edge);
            counts += (uint32_t)a + ((uint32_t)b << 16);
        }
        const uint32_t wa = __ballot_sync(0xffffffffu, a), wb = __ballot_sync(0xffffffffu, b);
        if (lane == 0) {
            in[i / 32] = wa;
            pend[i / 32] = wb;
        }
    }
    uint32_t sure_total, doubt_total;
    {
        const uint32_t a = __reduce_add_sync(0xffffffffu, counts & 0xffffu), b = __reduce_add_sync(0xffffffffu, counts >> 16);
        __syncthreads();
        if (lane == 0) {
            sh->scan[warp] = a;
            sh->list[warp] = b;
        }
        __syncthreads();
        sure_total = __reduce_add_sync(0xffffffffu, lane < NW ? sh->scan[lane] : 0u);
        doubt_total = __reduce_add_sync(0xffffffffu, lane < NW ? sh->list[lane] : 0u);
    }
    ties = m - sure_total;
    bool some_tie = doubt_total > ties;   // of the blocks in doubt, not all are in
    if (some_tie && S > 0.f) {
        // the blocks in doubt by their exact scores; summaries are scaled by
        // 2^-64 where S, for weights up to 2^15, is huge or overflowed
        const float v_scale = S < 0x1p75f ? 1.f : 0x1p-64f;
        auto exact = [&](int i) -> unsigned long long {   // by a warp
            const int64_t at = ((int64_t)table[i] * p.num_kv_heads + kvh) * 2 * D + lane;
            float v[2 * D / 32];
#pragma unroll
            for (int k = 0; k < 2 * D / 32; ++k)
                v[k] = to_float(static_cast<const T *>(p.summaries)[at + k * 32]) * v_scale;
            Pair s{0.f, 0.f};
#pragma unroll 1
            for (int k = 0; k < 2 * D / 32; ++k) {
                s = pair_add(s, pair_mul(sh->weight[k * 32 + lane], v[0]));
#pragma unroll
                for (int j = 0; j + 1 < 2 * D / 32; ++j)
                    v[j] = v[j + 1];
            }
#pragma unroll 1
            for (int off = 16; off > 0; off >>= 1)
                s = pair_add(s, Pair{__shfl_xor_sync(0xffffffffu, s.h, off), __shfl_xor_sync(0xffffffffu, s.l, off)});
            return (unsigned long long)order_key(s.h) << 32 | order_key(fabsf(s.h) < INFINITY ? s.l : 0.f);
        };
        if (doubt_total <= NT) {
            // a few (two, mostly): listed in ascending order, ranked against each other
            const int per = (words + NT - 1) / NT;
            const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
            uint32_t c = 0, total;
            for (int k = w0; k < w1; ++k)
                c += __popc(pend[k]);
            c = cta_exclusive<NT>(c, sh->scan, &total);
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
            for (int k = tid; k < words; k += NT)
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
            some_tie = false;
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
            const uint32_t t = kth_largest<NT>(sh, key, 0, n, pend, ties, &left);
            __syncthreads();
            uint32_t still = 0;
            for (int i = tid; i < words * 32; i += NT) {
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
            (void)cta_exclusive<NT>(still, sh->scan, &total);
            if (total == ties)
                break;
        }
    }
    __syncthreads();

    // ---- emission in ascending order: thread t owns words [w0, w1)
    const int per = (words + NT - 1) / NT;
    const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
    uint32_t total;
    if (some_tie) {
        // the lowest `ties` blocks in doubt are in
        uint32_t c = 0;
#pragma unroll 1
        for (int k = w0; k < w1; ++k)
            c += __popc(pend[k]);
        uint32_t seen = cta_exclusive<NT>(c, sh->scan, &total);
#pragma unroll 1
        for (int k = w0; k < w1; ++k) {
            uint32_t w = pend[k], kept = 0;
            const uint32_t here = (uint32_t)__popc(w);
            for (uint32_t left = seen < ties ? min(ties - seen, here) : 0u; left > 0; --left) {
                kept |= w & (0u - w);
                w &= w - 1;
            }
            seen += here;
            pend[k] = kept;
        }
    }
    uint32_t c = 0;
#pragma unroll 1
    for (int k = w0; k < w1; ++k) {
        in[k] |= pend[k];
        c += __popc(in[k]);
    }
    uint32_t at = cta_exclusive<NT>(c, sh->scan, &total);
#pragma unroll 1
    for (int k = w0; k < w1; ++k) {
        pend[k] = at;   // selected blocks before the word's
        at += __popc(in[k]);
    }
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < n; i += NT) {
        const uint32_t w = in[i / 32];
        if (w >> (i % 32) & 1u)
            out[pend[i / 32] + __popc(w & ((1u << (i % 32)) - 1u))] = i;
    }
}

// One launch: a cluster per row; grid (CTAs of a row, kv head, sequence).
template <typename T, int D, int NT>
__global__ void __launch_bounds__(NT)
select_blocks_kernel(const __grid_constant__ SelectParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int NW = NT / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    SelectShared *sh = reinterpret_cast<SelectShared *>(smem);
    using Score = ScoreShared<D, NW, 1>;
    Score *sw = reinterpret_cast<Score *>(smem + sizeof(SelectShared));
    uint32_t *key = reinterpret_cast<uint32_t *>(smem + sizeof(SelectShared) + sizeof(Score));   // [most], CTA 0's in use
    uint32_t *in = key + p.key_stride;                                            // bit i: block i is selected
    uint32_t *pend = in + (p.most + 31) / 32;                               // bit i: block i is in doubt
    const int me = (int)cluster.block_rank(), kvh = blockIdx.y, seq = blockIdx.z;
    cluster.barrier_arrive();   // CTA 0 has started once this completes: its memory may be written
    wait_for_stream();
    int n;
    const float S = score_blocks<T, D, NW, 1>(p, sw, seq, kvh, me * p.chunk, cluster.map_shared_rank(key, 0) + me * p.chunk, n,
                                           me == 0 ? sh->weight : nullptr, kvh == 0 && me == 0 && threadIdx.x == 0, [&] { cluster.barrier_wait(); });
    if ((threadIdx.x & 31) == 0)
        cluster.map_shared_rank(sh, 0)->bound[me * NW + (threadIdx.x >> 5)] = S;
    cluster.sync();
    if (me == 0)
        select_row<T, D, NT>(p, sh, key, in, pend, sh->bound, seq, kvh, n);
}

// Two launches: scores into the workspace; grid (kv head, chunk, sequence), so
// that the CTAs that read neighbouring parts of a block's summaries run
// together.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreWarps * 32)
score_blocks_kernel(const __grid_constant__ SelectParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    using Score = ScoreShared<D, kScoreWarps, kScoreStages>;
    Score *sw = reinterpret_cast<Score *>(smem);
    wait_for_stream();
    // the second launch's CTAs may come up, and prepare, beside the last of these
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int kvh = blockIdx.x, me = blockIdx.y, seq = blockIdx.z;
    const int64_t row = (int64_t)seq * p.num_kv_heads + kvh;
    int n;
    const float S = score_blocks<T, D, kScoreWarps, kScoreStages>(p, sw, seq, kvh, me * p.chunk, p.ws_keys + row * p.key_stride + me * p.chunk, n,
                                                    nullptr, false, [] {});
    if ((threadIdx.x & 31) == 0)
        p.ws_bound[row * p.bounds + me * kScoreWarps + (threadIdx.x >> 5)] = S;
}

// The second launch, a programmatic dependent of the first: grid (kv head,
// sequence).
template <typename T, int D, int NT>
__global__ void __launch_bounds__(NT)
select_rows_kernel(const __grid_constant__ SelectParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    SelectShared *sh = reinterpret_cast<SelectShared *>(smem);
    uint32_t *key = reinterpret_cast<uint32_t *>(smem + sizeof(SelectShared));   // [most]
    uint32_t *in = key + p.key_stride;
    uint32_t *pend = in + (p.most + 31) / 32;
    const int kvh = blockIdx.x, seq = blockIdx.y;
    const int64_t row = (int64_t)seq * p.num_kv_heads + kvh;
    const int tid = threadIdx.x;
    if (tid == 0) {
        mbar_init(&sh->bar, 1);
        fence_mbar_init();
    }
    // Nothing is read before this wait: the first launch's start says that
    // what precedes it has ended, not that this one sees what it wrote.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int L = p.context_lens[seq];
    float x[8], big = 0.f;
#pragma unroll
    for (int h = 0; h < 8; ++h)
        x[h] = tid < D && h < p.group ? select_q(p, (row * p.group + h) * D + tid) : 0.f;
    int n = row_blocks(p, L, kvh == 0 && tid == 0);
    if (n > p.num_selected && tid == 0) {
        const uint32_t bytes = (uint32_t)(n + 3) / 4 * 16;
        mbar_arrive_expect_tx(&sh->bar, bytes);
        bulk_load(key, p.ws_keys + row * p.key_stride, bytes, &sh->bar);
    }
    // the weights of exact scores, while the keys come
#pragma unroll
    for (int h = 0; h < 8; ++h)
        big = fmaxf(big, fabsf(x[h]) * 8.f);
    const float scale = weight_scale<NT / 32>(big, sh->scan);
    if (tid < D)
        exact_weights<D>(sh->weight, x, scale);
    if (n > p.num_selected && !cta_waited(mbar_wait_bounded(&sh->bar, 0), &sh->bar, 0, p.status))
        n = 0;   // selects nothing
    __syncthreads();
    select_row<T, D, NT>(p, sh, key, in, pend, p.ws_bound + row * p.bounds, seq, kvh, n);
}

// Test hook: what select_rows_kernel and select_row make of waits that gave
// up, on one CTA and a row of 100 blocks.  what 0: the keys' copy never comes,
// and thread 0 alone sees its wait end (on the barrier's other parity); 1: a
// scoring warp gave up; 2: a scoring warp met a bad id.
__global__ void __launch_bounds__(kSelectThreads)
select_timeout_test_kernel(const __grid_constant__ SelectParams p, int what, uint64_t limit_ns)
{
    __shared__ SelectShared sh;
    __shared__ float bounds[2];
    if (threadIdx.x == 0) {
        mbar_init(&sh.bar, 1);
        fence_mbar_init();
        bounds[0] = 1.f;
        bounds[1] = what == 0 ? 1.f : what == 1 ? kLateChunk : kBadChunk;
    }
    __syncthreads();
    int n = 100;
    if (what == 0 && !cta_waited(mbar_wait_bounded(&sh.bar, threadIdx.x == 0 ? 1 : 0, limit_ns), &sh.bar, 0, p.status, limit_ns))
        n = 0;
    __syncthreads();
    // the row is refused or empty: no key, bit or table is looked at
    select_row<__half, 64, kSelectThreads>(p, &sh, nullptr, nullptr, nullptr, bounds, 0, 0, n);
}

}  // namespace pkv
