// q4_attention.cuh -- single-query attention over a 4-bit cache
// (paged_attention_decode_q4):
//   out[s, h] = sum_t softmax_t(scale * q[s, h] . k_t) * v_t,
// a row's numbers s u + m for each group j of 64 dimensions (see q4_cache.cuh):
//   q . k_t   = sum_j s_tj (q_j . u_tj) + m_tj sum(q_j)
//   sum_t w_t v_t = sum_t (w_t s_tj) u_tj + sum_t w_t m_tj
// so that the products take whole numbers, and scales and minima join them in
// fp32.
//
// A CTA owns the G <= 8 query heads of a kv head.  Its four warps take the
// tokens of a row (a sequence's kv head) 32 at a time in turn, each through a
// ring of bulk copies of its own (one per block: codes with their scales), and
// work on two tiles of 16: a tile's tokens are M of S^T = K q^T, its dimensions
// M of O^T += V^T W^T, the query heads N of warp-level MMAs (m16n8k16).
//
// How the work is cut.  Either a CTA per row or per partition of one (merged by
// a cluster or through the workspace, as in list_attention.cuh); or, "streamed",
// as many CTAs as fit on the GPU at once, each of which takes an equal share of
// all rows' tokens put one behind another.  A share's first and last row may be
// parts, which q4_merge_kernel joins.  The rings run on over the rows' ends.
//
// Codes become f16 matrix fragments without a conversion: a word's nibbles
// masked in place are numbers, two at a time.  u in a half's lowest four bits is
// the subnormal u 2^-24, in the next four u 2^-20: a mask is all it takes (five
// instructions for eight codes of K; V's tokens are the products' inner axis, so
// two tokens' words are first paired half by half: six).  The factors go into q
// (a sixteenth for the latter) and the scores, and into the outputs.
//
// A weight w_t s_tj enters the product with V in two f16 parts: off by 2^-22 of
// itself, or 2^-32 of the largest of its head so far.  That needs the largest
// below 2^16 whatever the scales are, so the softmax's reference is not a head's
// largest score alone: weights are 2^(x - m) with m such that the largest
// 2^(x - m) s, not the largest 2^(x - m), is near 2^7.
//
// What bounds it: the latency of dependent instructions, of which no unit is
// full.  Sixteen contexts of 16K to 32K tokens with 8 query heads a kv head (454
// MB) take 109 to 110 us, 4.1 TB/s or 62 % of a copy's rate; one of 128K tokens
// with 4 heads 41 us (151 MB, 55 %); 64 of 128 to 2048 tokens, 32 kv heads, 82 to 88
// us (55 to 58 %).  Of the first: 32 tokens take some 620 warp instructions, a
// third of them the masks and shifts that make codes operands.  168 registers a
// thread leave 12 warps an SM; a scheduler's 2.8 issue in 48 % of the cycles, the
// ALU pipe is busy 47 % of the time, the tensor pipe 32 %.  Of the 5.5 cycles that
// a warp takes per instruction 1.8 are fixed latencies, 1 the issue, 0.65 a pipe
// that is busy, 0.6 another warp's issue, 0.5 reads of shared memory, 0.5 waits
// for other memory, 0.3 dispatch, 0.2 barriers.  1, 2, 4 CTAs per SM: 175, 119,
// 112 us.  Without any loads it took 105 us when it took 112 with them; steps of
// 16 tokens (114) and K's products of one step among V's of the one before (118)
// were compared with 111.
//
// The M axes' order is free: row 2 c + e + 8 f of a tile is its token
// 4 c + 2 f + e (so that a thread's four tokens of V are neighbours), and a
// thread's rows of V^T are the dimensions that its words hold.
#pragma once

#include "list_attention.cuh"
#include "q4_cache.cuh"

namespace pkv {

// Where a streamed CTA's share lies: units [lo, hi) of the stream, of which the
// first is unit `unit` of the `units` of kv head `head` of sequence `seq`.
struct Q4Share {
    int64_t lo, hi;
    int seq, head, unit, units;
};

// The test hook's: copies that are left out, and the limit of the waits.
struct Q4Lost {
    uint64_t limit_ns;
    int cta, warp, unit;   // the warp's unit, counted from its first
};

struct Q4Params {
    ListParams list;             // without selected blocks and scales
    int64_t q_stride;            // elements between two sequences' rows of q
    int shares;                  // streamed: CTAs; else 0
    int part_units;              // tokens / 32 of a partition; 0: a row's, divided by list.np
    Q4Share *ws_share;           // streamed: the shares, for the merge
    Q4Lost lost;                 // the hook's kernel only
};

constexpr int kQ4Unit = 32;      // tokens that a warp takes at a time
// What a row's start and end cost a CTA, in units: shares are of equal cost.
// (us with 0, 4, 8 and 12 units: 64 sequences of 128 to 2048 tokens, 32 kv heads,
// in shares 112, 95.3, 84.0, 84.1; 33 of up to 4095, heads of 64 33.7, 25.5, 23.7,
// 24.2.)
constexpr int kQ4RowCost = 8;
constexpr int kQ4Ring = 40960;   // ring bytes of a CTA at most
constexpr int kQ4Ctas = 3;       // CTAs per SM

template <int D, int BS> struct Q4Cfg {
    using R = Q4Row<D>;
    static constexpr int TILE = 16, TILES = 2;
    static constexpr int REC = R::template record<BS>;
    static constexpr int TOK = kQ4Unit;                        // tokens of a stage
    static constexpr int RECS = TOK / BS;
    // from a tile's codes to the next's
    static constexpr int NEXT_CODE = BS > TILE ? TILE * R::CODES : TILE / BS * REC;
    static constexpr int STAGE_BYTES = 2 * RECS * REC;
    static constexpr int S = kQ4Ring / (kListWarps * STAGE_BYTES);
    static constexpr int CHUNK = 128;                          // units whose blocks are looked up at a time
    static constexpr int AWS = D + 4;                          // row stride of a warp's result, in floats

    static constexpr int OFF_AT = (kListWarps * S * STAGE_BYTES + 127) / 128 * 128;
    // a warp's scales and minima of K in fp32 (and as many of V): all tokens' of
    // the first group, then of the second
    static constexpr int NUMBERS = R::GROUPS * TOK * 16;
    static constexpr int OFF_NUM = OFF_AT + CHUNK * RECS * 8;
    static constexpr int OFF_RESULT = OFF_NUM + kListWarps * 2 * NUMBERS;
    static constexpr int OFF_ML = OFF_RESULT + kListMaxGroup * (D + 2) * 4;
    static constexpr int OFF_BAD = OFF_ML + kListWarps * kListMaxGroup * 8;
    static constexpr int OFF_IDS = OFF_BAD + CHUNK;
    static constexpr int OFF_BAR = OFF_IDS + kListThreads * 4;
    static constexpr int OFF_FLAG = OFF_BAR + kListWarps * S * 8;
    static constexpr int SMEM_BYTES = OFF_FLAG + 128 + 1024;   // slack for the alignment to 1024
    static_assert(REC % 16 == 0 && STAGE_BYTES % 16 == 0 && OFF_RESULT % 16 == 0 && OFF_BAR % 8 == 0 && S >= 2, "alignment");
    static_assert(kListMaxGroup * AWS * 4 <= STAGE_BYTES, "a warp's result fits the stage it took last");
};

// Units of a sequence; one of a refused length has none.
__device__ __forceinline__ int q4_units(const ListParams &p, int seq)
{
    const int L = p.context_lens[seq];
    return L < 0 || L > p.max_context_len ? 0 : (int)(((int64_t)L + kQ4Unit - 1) / kQ4Unit);
}

// Share i's place, by all threads of a CTA.  The stream is cut by cost, a row
// costing its units and kQ4RowCost in front of them, at i / shares of the whole.
// Each thread adds up a run of sequences; the runs that hold the share's two
// ends are walked by their threads.
__device__ __forceinline__ void q4_find_share(const ListParams &p, int shares, int i, Q4Share *share, int64_t *sums)
{
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int run = (p.num_seqs + kListThreads - 1) / kListThreads;
    const int s0 = min(p.num_seqs, t * run), s1 = min(p.num_seqs, s0 + run);
    const int64_t Hk = p.num_kv_heads;
    int64_t mine[2] = {0, 0};   // units of a head, cost of a head
    for (int s = s0; s < s1; ++s) {
        const int n = q4_units(p, s);
        mine[0] += n;
        mine[1] += n ? n + kQ4RowCost : 0;
    }
    int64_t upto[2] = {mine[0], mine[1]}, total = 0;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int64_t other = __shfl_up_sync(0xffffffffu, upto[w], k);
            upto[w] += lane >= k ? other : 0;
        }
    }
    if (lane == 31) {
        sums[2 * warp] = upto[0];
        sums[2 * warp + 1] = upto[1];
    }
    if (t == 0)
        *share = Q4Share{};
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) {
        upto[0] += w < warp ? sums[2 * w] : 0;
        upto[1] += w < warp ? sums[2 * w + 1] : 0;
        total += sums[2 * w + 1];
    }
    total *= Hk;
    int64_t each;
    uint32_t rest;
    if (total >> 32 == 0) {
        each = (uint32_t)total / (uint32_t)shares;
        rest = (uint32_t)total % (uint32_t)shares;
    } else {
        each = total / shares;
        rest = (uint32_t)(total % shares);
    }
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {
        const int64_t at = each * (i + end) + rest * (uint32_t)(i + end) / (uint32_t)shares;
        int64_t cost = (upto[1] - mine[1]) * Hk, units = (upto[0] - mine[0]) * Hk;
        if (cost <= at && at < upto[1] * Hk) {
            int s = s0, n = q4_units(p, s);
            for (int64_t c; at >= cost + (c = n ? (n + kQ4RowCost) * Hk : 0); n = q4_units(p, ++s)) {
                cost += c;
                units += n * Hk;
            }
            int head = 0;
            for (int step = 1 << 15; step; step /= 2)   // (at - cost) / (n + kQ4RowCost), below 2^16
                head += at - cost >= (int64_t)(head + step) * (n + kQ4RowCost) ? step : 0;
            const int unit = max(0, (int)(at - cost - (int64_t)head * (n + kQ4RowCost)) - kQ4RowCost);
            units += (int64_t)head * n + unit;
            if (end == 0) {
                share->seq = s;
                share->head = head;
                share->unit = unit;
                share->units = n;
                share->lo = units;
            } else {
                share->hi = units;
            }
        } else if (at == total && t == kListThreads - 1) {
            share->hi = upto[0] * Hk;
            if (end == 0)   // an empty stream
                share->lo = upto[0] * Hk;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// D = A * B, m16n8k16, f16.
__device__ __forceinline__ void q4_mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// A wait that did not end at once: until the phase completes for every lane, or
// one gives up.  Kept out of the loops that wait.
static __device__ __noinline__ bool q4_wait(uint64_t *bar, uint32_t phase)
{
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase));
}
static __device__ __noinline__ bool q4_wait(uint64_t *bar, uint32_t phase, uint64_t limit_ns)
{
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase, limit_ns));
}

// One warp's state.  Lane (g, c) = (lane / 4, lane % 4).
//
// TWICE (groups of up to four heads): N's columns 4 .. 7 are heads 0 .. 3 once
// more, with the weights' second parts where columns 0 .. 3 have the first, so
// that one product takes both; their sums are added at the end.
template <typename T, int D, int BS, bool TWICE> struct Q4Engine {
    using C = Q4Cfg<D, BS>;
    using R = Q4Row<D>;
    static constexpr int NG = R::GROUPS;
    static constexpr float kMost = 32768.f;      // of a weight times its scale
    static constexpr float kLift = 7.f;          // log2 of the largest one where the reference is set
    static constexpr float kLeast = 0x1p-100f;   // smaller scales count as this: weights stay below 2^115
    // What sums of weights and of values are kept in: 2^25 such weights stay below
    // 2^128, and one beside a scale of 2^123 (2^-116 of it) above 2^-128.
    static constexpr float kSums = 0x1p-12f;

    uint32_t qf[NG][4][2];   // q^T B-fragments of head g: group, step
    // a float2 is of heads 2c, 2c + 1
    float2 fs;               // the softmax's factor, with the powers of two of q and u
    float2 fm[NG];           // sum(q_j), in the same units as q . u
    float o[NG][4][4];       // O^T C-fragments: group, m-tile
    float2 om[NG];           // this lane's tokens' sums of w m
    float2 m, lsum;          // weights' reference and sum, times kSums
    uint32_t nums;           // this warp's numbers in shared memory
    int kcode[2], vcode[4];  // byte offsets of this lane's tokens of K and of V in a stage's records
    int mine;                // of the pairs of the token that this lane makes numbers of
    float second;            // TWICE: -1 where this lane has the weights' second parts
    uint32_t steps;          // taken of the row
    uint32_t flip;           // ~0 in steps that take V's codes from 15
    int g, c;

    // Offset of the record of tile row t in a stage, and the row in it.
    __device__ __forceinline__ static int rec_of(int t) { return BS < C::TILE ? t / BS * C::REC : 0; }

    __device__ __forceinline__ void init(const Q4Params &a, int seq, int kvh, int lane)
    {
        const ListParams &p = a.list;
        g = lane >> 2;
        c = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 4 * (g >> 1) + (g & 1) + 2 * i;
            kcode[i] = rec_of(t) + R::word(t % BS, NG * 2 * c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * c + i;
            vcode[i] = rec_of(t) + R::word(t % BS, NG * g);
        }
        mine = lane / BS * C::REC + R::template pair<BS>(lane % BS, 0);
        // q: dimensions 64 j + 16 c .. + 15 of head g, brought to f16 by a
        // power of two that puts the head's largest magnitude in [2^14, 2^15):
        // what f16 cannot hold is below 2^-35 of it
        const int head = TWICE ? g & 3 : g;
        const bool live = head < p.group;
        const T *qp = static_cast<const T *>(p.q) + (int64_t)seq * a.q_stride + ((int64_t)kvh * p.group + (live ? head : 0)) * D + 16 * c;
        second = TWICE && c >= 2 ? -1.f : 0.f;
        steps = 0;
        using V = typename Pair16<T>::V;
        uint32_t w[NG][8];
        V top = as_pair<T>(0u);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 v = live ? reinterpret_cast<const uint4 *>(qp + 64 * j)[i] : make_uint4(0, 0, 0, 0);
                w[j][4 * i] = v.x;
                w[j][4 * i + 1] = v.y;
                w[j][4 * i + 2] = v.z;
                w[j][4 * i + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = __hmax2(top, __habs2(as_pair<T>(w[j][i])));   // NaN loses
        }
        top = __hmax2(top, as_pair<T>(__shfl_xor_sync(0xffffffffu, as_word(top), 1)));
        top = __hmax2(top, as_pair<T>(__shfl_xor_sync(0xffffffffu, as_word(top), 2)));
        const float2 both = Unpack<T>::pair(as_word(top));
        const float big = fmaxf(both.x, both.y);
        int x = (int)(__float_as_uint(big) >> 23) - 127 - 14;
        x = big < INFINITY ? max(x, -100) : 0;
        const float down = __uint_as_float((uint32_t)(127 - x) << 23);
        const float factor = p.qscale * __uint_as_float((uint32_t)(127 + x) << 23);
        float sum[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            float2 total = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float2 f[4];   // dimensions 2 i, 2 i + 1 of a word's eight
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = fmul2(Unpack<T>::pair(w[j][4 * e + i]), make_float2(down, down));
                    total = fadd2(total, f[i]);
                }
                // a word's pairs (n, n + 4), of which odd n come times 16
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    qf[j][2 * e + i][0] = Mma<__half>::pack(f[i].x, f[i + 2].x);
                    qf[j][2 * e + i][1] = Mma<__half>::pack(f[i].y * 0.0625f, f[i + 2].y * 0.0625f);
                }
            }
            sum[j] = total.x + total.y;
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
        }
        // head h's sits in lanes 4 h ..
        auto heads = [&](float v) { return make_float2(__shfl_sync(0xffffffffu, v, 8 * c), __shfl_sync(0xffffffffu, v, 8 * c + 4)); };
        fs = heads(factor * 16777216.f);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            fm[j] = heads(sum[j] * 0x1p-24f);
            om[j] = make_float2(0.f, 0.f);
        }
        m = make_float2(-INFINITY, -INFINITY);
        lsum = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
                o[j][mt][0] = o[j][mt][1] = o[j][mt][2] = o[j][mt][3] = 0.f;
        }
    }

    // Scales and minima of a step's tokens in fp32, each twice (the factors of
    // two heads), where the warp's lanes find them: a lane makes a token's.
    //  Returns the largest scale of V among all tokens, at least kLeast,
    // with the minima that hold the weights down, too: those of a size that makes
    // the scales' part of the numbers one below fp32's last bit.
    //
    // V's codes are not negative: their sums would grow while the minima's take
    // most of them away again, and tensor cores cut what they add towards zero,
    // which tells in outputs that are means of many numbers.  So half the steps
    // (flip: of four, the second and third) take s u + m as (m + 15 s) + (-s)
    // (15 - u): the sums stay as small as one step's, and of either sign in turn.
    // (Means over 60,000 tokens are then off by 2.6e-5 of their size; where each
    // step only started from zero and was added rounded to nearest, by 2.0e-4.
    // Codes always from one side: 16 long contexts 109.4 us against 109.9, one of
    // 128K tokens 40.2 against 41.0.)
    __device__ __forceinline__ float numbers(uint32_t kbase, uint32_t vbase, int nvalid) const
    {
        float top = kLeast;
        const int lane = 4 * g + c;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                uint32_t w = lds32((v ? vbase : kbase) + mine + 4 * j);
                if (nvalid < C::TOK)
                    w = lane < nvalid ? w : 0u;   // no token: what is there may be anything
                float2 f = Unpack<T>::pair(w);
                if (v)
                    top = fmaxf(top, fmaxf(f.x, fabsf(f.y) * 0x1p-24f));
                if (v) {
                    f.y = fmaf(flip ? 15.f : 0.f, f.x, f.y);
                    f.x = __uint_as_float(__float_as_uint(f.x) ^ (flip & 0x80000000u));
                }
                asm volatile("st.shared.v4.f32 [%0], {%1, %1, %2, %2};" ::"r"(nums + v * C::NUMBERS + (j * C::TOK + lane) * 16), "f"(f.x), "f"(f.y) : "memory");
            }
        }
        return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    }

    // This lane holds tokens t0 = 4 (g / 2) + g % 2 and t0 + 2 of each tile.
    static constexpr int N = 2 * C::TILES;
    __device__ __forceinline__ int token(int n) const { return 4 * (g >> 1) + (g & 1) + 2 * (n & 1) + C::TILE * (n >> 1); }
    // (s, s), (m, m) of token n, group j: K's (v = 0) or V's
    __device__ __forceinline__ void number(int v, int j, int n, float2 &s, float2 &mn) const
    {
        const float4 f = lds128f(nums + v * C::NUMBERS + j * C::TOK * 16 + token(n) * 16);
        s = make_float2(f.x, f.y);
        mn = make_float2(f.z, f.w);
    }

    // Scores of the step whose records start at kbase, up to fs.  Products that
    // add to the same sums stand apart: their latency is four others' time.
    __device__ __forceinline__ void scores(uint32_t kbase, float2 (&x)[N]) const
    {
        uint32_t w[N][2 * NG];   // token, word
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t at = kbase + kcode[n & 1] + (n >> 1) * C::NEXT_CODE;
            if constexpr (NG == 2) {
                const uint4 v = lds128(at);
                w[n][0] = v.x;
                w[n][1] = v.y;
                w[n][2] = v.z;
                w[n][3] = v.w;
            } else {
                const uint2 v = lds64(at);
                w[n][0] = v.x;
                w[n][1] = v.y;
            }
        }
        float acc[C::TILES][NG][4];
#pragma unroll
        for (int step = 0; step < 4; ++step) {
#pragma unroll
            for (int tile = 0; tile < C::TILES; ++tile) {
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const int word = NG * (step >> 1) + j;
                    uint32_t u = w[2 * tile][word], v = w[2 * tile + 1][word];
                    if (step & 1) {
                        u >>= 8;
                        v >>= 8;
                    }
                    const uint32_t a[4] = {u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u};
                    if (step == 0)
                        q4_mma_first(acc[tile][j], a, qf[j][0][0], qf[j][0][1]);
                    else
                        Mma<__half>::run(acc[tile][j], a, qf[j][step][0], qf[j][step][1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float2 s, mn;
                number(0, j, n, s, mn);
                const float2 d = make_float2(acc[n >> 1][j][2 * (n & 1)], acc[n >> 1][j][2 * (n & 1) + 1]);
                x[n] = j ? ffma2(s, d, x[n]) : fmul2(s, d);
                x[n] = ffma2(mn, fm[j], x[n]);
            }
        }
    }

    // Weights of a step from its scores.  Online softmax in the log2 domain:
    // while no weight times a scale can pass kMost, weights are taken against
    // the head's reference m unchanged: no maximum across lanes, no rescaling.
    __device__ __forceinline__ void weights(const float2 (&x)[N], float top, int nvalid, float2 (&p)[N])
    {
        float most = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float2 z = ffma2(x[n], fs, make_float2(-m.x, -m.y));   // infinite before the first token
            p[n] = make_float2(ex2_fast(z.x), ex2_fast(z.y));
        }
        if (nvalid < C::TOK) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (token(n) >= nvalid)
                    p[n] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
            most = fmaxf(most, fmaxf(p[n].x, p[n].y));
        if (!__any_sync(0xffffffffu, most * top > kMost))
            return;
        float2 t = make_float2(-INFINITY, -INFINITY);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float big = kLeast;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                float2 s, mn;
                number(1, j, n, s, mn);
                big = fmaxf(big, fmaxf(fabsf(s.x), fabsf(mn.x) * 0x1p-24f));
            }
            big = __log2f(big) - kLift;
            if (token(n) < nvalid) {
                t.x = fmaxf(t.x, fmaf(x[n].x, fs.x, big));
                t.y = fmaxf(t.y, fmaf(x[n].y, fs.y, big));
            }
        }
#pragma unroll
        for (int k = 4; k < 32; k *= 2) {
            t.x = fmaxf(t.x, __shfl_xor_sync(0xffffffffu, t.x, k));
            t.y = fmaxf(t.y, __shfl_xor_sync(0xffffffffu, t.y, k));
        }
        t = make_float2(fmaxf(m.x, t.x), fmaxf(m.y, t.y));
        const float2 ref = make_float2(reference_of(t.x), reference_of(t.y));
        const Shift<true> sx(m.x, ref.x), sy(m.y, ref.y);
        const float2 alpha = make_float2(sx.factor(), sy.factor());
        m = t;
        lsum = make_float2(sx.of(lsum.x), sy.of(lsum.y));
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            om[j] = fmul2(om[j], alpha);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                o[j][mt][0] *= alpha.x;
                o[j][mt][1] *= alpha.y;
                o[j][mt][2] *= alpha.x;
                o[j][mt][3] *= alpha.y;
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const bool live = token(n) < nvalid;
            p[n].x = live ? ex2_fast(fmaf(x[n].x, fs.x, -ref.x)) : 0.f;
            p[n].y = live ? ex2_fast(fmaf(x[n].y, fs.y, -ref.y)) : 0.f;
        }
    }

    // (w ^ flip) & mask, one instruction
    __device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t mask) const
    {
        uint32_t d;
        asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(d) : "r"(w), "r"(flip), "r"(mask));
        return d;
    }

    // The weights' sums, their products with the minima in fp32, and with the
    // codes of a tile of the step whose records start at vbase.
    __device__ __forceinline__ void value_tile(uint32_t vbase, int tile, const float2 (&p)[N])
    {
        constexpr int PARTS = TWICE ? 1 : 2;
        uint32_t part[PARTS][NG][2];   // weights times scales, as B-fragments
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = 2 * tile + i;
            lsum = ffma2(p[n], make_float2(kSums, kSums), lsum);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                float2 s, mn;
                number(1, j, n, s, mn);
                om[j] = ffma2(p[n], mn, om[j]);
                const float2 w = fmul2(p[n], s);
                const uint32_t h = Mma<__half>::pack(w.x, w.y);
                const float2 f = Unpack<__half>::pair(h);
                if constexpr (TWICE) {
                    const float2 mine = ffma2(f, make_float2(second, second), w);
                    part[0][j][i] = movmatrix_trans(Mma<__half>::pack(mine.x, mine.y));
                } else {
                    const float2 rest = fadd2(w, make_float2(-f.x, -f.y));
                    part[0][j][i] = movmatrix_trans(h);
                    part[PARTS - 1][j][i] = movmatrix_trans(Mma<__half>::pack(rest.x, rest.y));
                }
            }
        }
        uint32_t w[4][NG];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t at = vbase + vcode[i] + tile * C::NEXT_CODE;
            if constexpr (NG == 2) {
                const uint2 v = lds64(at);
                w[i][0] = v.x;
                w[i][1] = v.y;
            } else {
                w[i][0] = lds32(at);
            }
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t u = __byte_perm(w[0][j], w[1][j], e ? 0x7632 : 0x5410);
                const uint32_t v = __byte_perm(w[2][j], w[3][j], e ? 0x7632 : 0x5410);
                uint32_t a[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t uk = u >> (8 * k), vk = v >> (8 * k);
                    a[k][0] = codes(uk, 0x000f000fu);
                    a[k][1] = codes(uk, 0x00f000f0u);
                    a[k][2] = codes(vk, 0x000f000fu);
                    a[k][3] = codes(vk, 0x00f000f0u);
                }
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        Mma<__half>::run(o[j][2 * e + k], a[k], part[i][j][0], part[i][j][1]);
                }
            }
        }
    }

    // The 32 tokens of the stage whose records start at kbase and vbase;
    // nvalid of them count.
    __device__ __forceinline__ void step(uint32_t kbase, uint32_t vbase, int nvalid)
    {
        flip = 0u - ((steps + 1) >> 1 & 1u);
        const float top = numbers(kbase, vbase, nvalid);
        __syncwarp();
        float2 x[N], p[N];
        scores(kbase, x);
        weights(x, top, nvalid, p);
#pragma unroll
        for (int tile = 0; tile < C::TILES; ++tile)
            value_tile(vbase, tile, p);
        ++steps;
    }

    // This warp's reference, sum and sums of values of the heads below `group`,
    // the sums times kSums: ml [kListMaxGroup][2], aw [kListMaxGroup][AWS].
    __device__ __forceinline__ void finish(float2 *ml, float *aw, int group)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = h ? lsum.y : lsum.x, add[NG];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                add[j] = (h ? om[j].y : om[j].x) * kSums;
                add[j] += __shfl_xor_sync(0xffffffffu, add[j], 4);
                add[j] += __shfl_xor_sync(0xffffffffu, add[j], 8);
                add[j] += __shfl_xor_sync(0xffffffffu, add[j], 16);
            }
            const int row = 2 * c + h;
            if ((TWICE ? row & 3 : row) < group) {
                if (TWICE && c >= 2) {
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        add[j] = 0.f;
                }
                if (g == 0 && (!TWICE || c < 2))
                    ml[row] = make_float2(h ? m.y : m.x, l);
                float *dst = aw + row * C::AWS + 8 * g;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
                        *reinterpret_cast<float2 *>(dst + 64 * j + 2 * mt) =
                            make_float2(fmaf(o[j][mt][h], 16777216.f * kSums, add[j]), fmaf(o[j][mt][2 + h], 1048576.f * kSums, add[j]));
                }
            }
        }
    }
};

// Zero rows for the heads of every kv head of a sequence.
template <int D>
__device__ __forceinline__ void q4_zero_rows(const ListParams &p, int seq)
{
    const int64_t heads = (int64_t)p.num_kv_heads * p.group;
    for (int64_t i = (int64_t)threadIdx.x * 4; i < heads * D; i += kListThreads * 4)
        store_out4(p.out, p.out_dtype, seq * heads * D + i, make_float4(0.f, 0.f, 0.f, 0.f));
}

// Grid: streamed (shares); else (partition, kv head, sequence).  HOOK: the test
// hook's kernel, in which a unit's copies are never issued (a.lost).
template <typename T, int D, int BS, bool TWICE, bool HOOK>
__global__ void __launch_bounds__(kListThreads, kQ4Ctas)
q4_attention_kernel(const __grid_constant__ Q4Params a)
{
    using C = Q4Cfg<D, BS>;
    constexpr int S = C::S, NW = kListWarps;
    const ListParams &p = a.list;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    int64_t *record = reinterpret_cast<int64_t *>(smem + C::OFF_AT);   // byte offsets in a cache; -1: none
    ListResult<D> *res = reinterpret_cast<ListResult<D> *>(smem + C::OFF_RESULT);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    uint8_t *bad_row = smem + C::OFF_BAD;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + warp * S;
    uint32_t *flag = reinterpret_cast<uint32_t *>(smem + C::OFF_FLAG);
    Q4Share *share = reinterpret_cast<Q4Share *>(smem + C::OFF_FLAG + 8);
    int64_t *sums = reinterpret_cast<int64_t *>(smem + C::OFF_FLAG + 64);
    if (lane == 0) {
        for (int s = 0; s < S; ++s)
            mbar_init(&bars[s], 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0)
        *flag = 0;
    wait_for_stream();
    // a table that the CTA's threads hold leaves memory together with the length
    int32_t *ids = reinterpret_cast<int32_t *>(smem + C::OFF_IDS);
    const bool early = !a.shares && p.max_context_len <= kListThreads * BS;
    if (early && threadIdx.x * BS < p.max_context_len)
        ids[threadIdx.x] = p.block_tables[(int64_t)blockIdx.z * p.max_blocks_per_seq + threadIdx.x];

    // ---- the share: `left` units from unit `unit` of row (seq, head) on
    int seq, head, unit, L;
    int64_t left;
    if (a.shares) {
        for (int s = blockIdx.x; s < p.num_seqs; s += a.shares) {
            const int len = p.context_lens[s];
            if (len <= 0 || len > p.max_context_len) {
                q4_zero_rows<D>(p, s);
                if (len != 0 && threadIdx.x == 0)
                    report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
            }
        }
        q4_find_share(p, a.shares, blockIdx.x, share, sums);
        if (threadIdx.x == 0)
            a.ws_share[blockIdx.x] = *share;
        left = share->hi - share->lo;
        if (left == 0) {
            if (threadIdx.x < p.group)   // its part of the row that it lies in
                *reinterpret_cast<float2 *>(p.ws_ml + ((int64_t)blockIdx.x * 2 * p.group + threadIdx.x) * 2) = make_float2(-INFINITY, 0.f);
            return;
        }
        seq = share->seq;
        head = share->head;
        unit = share->unit;
        L = p.context_lens[seq];
    } else {
        seq = blockIdx.z;
        head = blockIdx.y;
        L = p.context_lens[seq];
        const int n = q4_units(p, seq);
        const int part = a.part_units ? a.part_units : (n + p.np - 1) / p.np;
        unit = (int)min((int64_t)n, (int64_t)part * blockIdx.x);
        left = min(part, n - unit);
        if (left == 0) {
            const bool refused = L < 0 || L > p.max_context_len;
            if (refused && blockIdx.x == 0 && head == 0 && threadIdx.x == 0)
                report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
            if (threadIdx.x < kListMaxGroup) {
                res->m[threadIdx.x] = -INFINITY;
                res->l[threadIdx.x] = refused ? -1.f : 0.f;
            }
            __syncthreads();
            write_result<D, true>(p, res, seq, head, blockIdx.x);
            return;
        }
    }

    auto units_of = [](int len) { return (int)(((int64_t)len + kQ4Unit - 1) / kQ4Unit); };
    // the row behind (s, h): the next head, or the next sequence that has units
    auto next_row = [&](int &s, int &h, int &len) {
        if (++h < p.num_kv_heads)
            return;
        h = 0;
        do
            len = p.context_lens[++s];
        while (len <= 0 || len > p.max_context_len);
    };

    uint8_t *stages = smem + warp * S * C::STAGE_BYTES;
    int stage = 0;              // the one that this warp takes next
    uint32_t phase = 0;         // its barrier's
    bool dead = false;          // a wait gave up
    bool refused = false;       // the row has a bad block
    bool whole = unit == 0;     // the row starts here
    int rows = 0;               // rows finished
    bool fresh = true;          // the engine has nothing of the row yet
    int issued = 0;             // HOOK: units
    Q4Engine<T, D, BS, TWICE> eng;
    eng.nums = smem_u32(smem + C::OFF_NUM + warp * 2 * C::NUMBERS);

    while (left > 0) {
        // ---- the blocks of the next units; -1 behind a row's last
        int chunk = (int)min(left, (int64_t)C::CHUNK);
        __syncthreads();   // no warp is still in the chunk before, whose last row may go on here
        for (int k = threadIdx.x; k < chunk; k += kListThreads)
            bad_row[k] = 0;
        __syncthreads();
        {
            int s = seq, h = head, u = unit, len = L, row = 0;
            bool bad = false;
            for (int at = 0; at < chunk; ++row) {
                const int n = min(units_of(len) - u, chunk - at);
                const int32_t *table = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
                for (int k = threadIdx.x; k < n * C::RECS; k += kListThreads) {
                    const int64_t b = (int64_t)u * C::RECS + k;
                    int64_t where = -1;
                    if (b * BS < len) {
                        int id = early ? ids[b] : table[b];
                        if (id < 0 || (int64_t)id >= p.num_blocks) {
                            bad = true;
                            bad_row[row] = 1;
                            id = 0;   // a block that there is, for a result that is dropped
                        }
                        where = ((int64_t)id * p.num_kv_heads + h) * C::REC;
                    }
                    record[at * C::RECS + k] = where;
                }
                u += n;
                if (at + n < chunk) {
                    u = 0;
                    next_row(s, h, len);
                } else {
                    // a row that goes on in the next chunk leaves a unit for
                    // every warp there (whose memory takes the warp's result)
                    const int64_t rest = min((int64_t)(units_of(len) - u), left - chunk);
                    if (rest > 0 && rest < NW) {
                        chunk = at > 0 ? at : chunk - NW;
                        break;
                    }
                }
                at += n;
            }
            if (bad)
                report(p.status, PKV_DEV_BAD_BLOCK);
        }
        __syncthreads();

        // ---- this warp's units of the chunk: warp, warp + NW, ...
        // unit k into a stage
        auto issue = [&](int k, int stage) {
            if constexpr (HOOK) {
                const int cta = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
                if (issued++ == a.lost.unit && cta == a.lost.cta && warp == a.lost.warp)
                    return;
            }
            const uint8_t *const kc = p.k_cache, *const vc = p.v_cache;
            uint8_t *kd = stages + stage * C::STAGE_BYTES;
            uint64_t *bar = &bars[stage];
            int64_t at[C::RECS];
            int n = 0;
#pragma unroll
            for (int b = 0; b < C::RECS; ++b) {
                const uint2 v = lds64(smem_u32(record + k * C::RECS + b));
                at[b] = (int64_t)((uint64_t)v.y << 32 | v.x);
                n += at[b] >= 0;
            }
            mbar_arrive_expect_tx(bar, (uint32_t)(n * 2 * C::REC));
#pragma unroll
            for (int b = 0; b < C::RECS; ++b) {
                if (at[b] >= 0) {
                    bulk_load(kd + b * C::REC, kc + at[b], C::REC, bar);
                    bulk_load(kd + (C::RECS + b) * C::REC, vc + at[b], C::REC, bar);
                }
            }
        };
        if (lane == 0 && !dead) {
            fence_proxy_async_smem();
            for (int i = 0; i < S && warp + i * NW < chunk; ++i)
                issue(warp + i * NW, (stage + i) % S);
        }
        int k = warp, row = 0;
        for (int at = 0; at < chunk; ++row) {
            const int n = min(units_of(L) - unit, chunk - at);
            const bool row_ends = unit + n == units_of(L), flush = row_ends || left == n;
            int held = -1, held_stage = 0;   // the unit whose stage takes this warp's result
            if (fresh) {
                eng.init(a, seq, head, lane);
                fresh = false;
            }
            if (k < at + n) {
                const int last = k + (at + n - 1 - k) / NW * NW;
                // units from here on are not followed into their stages by others, or not before the result is out
                const int stop = min(flush ? last : last + 1, chunk - S * NW);
                int valid = (int)min((int64_t)INT32_MAX, L - (int64_t)(unit + k - at) * kQ4Unit);
                for (; k <= last && !dead; k += NW) {
                    // the warp gives up as one: its products and shuffles need every lane
                    bool came = __all_sync(0xffffffffu, mbar_try_wait(&bars[stage], phase));
                    if (!came) {
                        if constexpr (HOOK)
                            came = q4_wait(&bars[stage], phase, a.lost.limit_ns);
                        else
                            came = q4_wait(&bars[stage], phase);
                    }
                    if (!came) {
                        // no CTA leaves with loads in flight
                        for (int i = 0; i < S && k + i * NW < chunk; ++i)
                            drain_wait(&bars[(stage + i) % S], phase ^ (stage + i >= S), lane == 0 ? p.status : nullptr,
                                       HOOK ? a.lost.limit_ns : kWaitLimitNs);
                        if (lane == 0) {
                            report(p.status, PKV_DEV_TIMEOUT);
                            atomicOr(flag, 1u);
                        }
                        dead = true;
                    } else {
                        const uint32_t kbase = smem_u32(stages + stage * C::STAGE_BYTES);
                        eng.step(kbase, kbase + C::RECS * C::REC, valid);
                        valid -= NW * kQ4Unit;
                        __syncwarp();
                        if (lane == 0 && k < stop) {
                            fence_proxy_async_smem();
                            issue(k + S * NW, stage);
                        }
                        held_stage = stage;
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                k = last + NW;
                if (flush && !dead)
                    held = last;
            }
            refused |= bad_row[row] != 0;
            at += n;
            unit += n;
            left -= n;
            if (!flush)
                continue;

            // ---- the warps' parts of the row, through the stages that they took last
            if (held >= 0)
                eng.finish(ml + warp * kListMaxGroup, reinterpret_cast<float *>(stages + held_stage * C::STAGE_BYTES), p.group);
            else if (lane < kListMaxGroup)
                ml[warp * kListMaxGroup + lane] = make_float2(-INFINITY, 0.f);
            int *slot = reinterpret_cast<int *>(sums);
            if (lane == 0)
                slot[warp] = held_stage;
            __syncthreads();
            const bool drop = refused || *reinterpret_cast<volatile uint32_t *>(flag) != 0;
            whole &= row_ends;
            const int64_t head0 = ((int64_t)seq * p.num_kv_heads + head) * p.group;
            const int64_t part0 = ((int64_t)blockIdx.x * 2 + (rows > 0)) * p.group;
            for (int i = threadIdx.x; i < p.group * (D / 4); i += kListThreads) {
                const int r = i / (D / 4), d = i % (D / 4) * 4;
                float Mx = -INFINITY, den = 0.f;
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
                float2 t[NW];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    t[w] = ml[w * kListMaxGroup + r];
                    Mx = fmaxf(Mx, t[w].x);
                }
                const float ref = reference_of(Mx);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    if (t[w].y != 0.f) {   // else the warp had no token; NaN sums stay
                        const Shift<true> by(t[w].x, ref);
                        const float f = by.factor();
                        const float *aw = reinterpret_cast<const float *>(smem + (w * S + slot[w]) * C::STAGE_BYTES) + r * C::AWS + d;
                        float4 x = *reinterpret_cast<const float4 *>(aw);
                        if constexpr (TWICE) {
                            const float4 y = *reinterpret_cast<const float4 *>(aw + 4 * C::AWS);
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        num.x = fmaf(f, x.x, num.x);
                        num.y = fmaf(f, x.y, num.y);
                        num.z = fmaf(f, x.z, num.z);
                        num.w = fmaf(f, x.w, num.w);
                        den = by.add(t[w].y, den);
                    }
                }
                if (!a.shares) {
                    *reinterpret_cast<float4 *>(&res->acc[r][d]) = num;
                    if (d == 0) {
                        res->m[r] = Mx;
                        res->l[r] = drop ? -1.f : den;
                    }
                } else if (whole) {
                    const bool zero = drop || den == 0.f;
                    const float inv = 1.f / den;
                    store_out4(p.out, p.out_dtype, (head0 + r) * D + d,
                               zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv));
                } else {
                    *reinterpret_cast<float4 *>(p.ws_acc + (part0 + r) * D + d) = num;
                    if (d == 0)
                        *reinterpret_cast<float2 *>(p.ws_ml + (part0 + r) * 2) = make_float2(Mx, drop ? -1.f : den);
                }
            }
            __syncthreads();
            if (left == 0)
                break;
            if (lane == 0 && held >= 0 && held + S * NW < chunk && !dead) {
                fence_proxy_async_smem();
                issue(held + S * NW, held_stage);
            }
            ++rows;
            whole = true;
            refused = false;
            unit = 0;
            fresh = true;
            next_row(seq, head, L);
        }
    }
    if (!a.shares) {
        write_result<D, true>(p, res, seq, head, blockIdx.x);
        if (p.np > 1 && !p.cluster)
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    } else {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
}

// Joins the parts of the rows that several shares hold: CTA i looks after the
// row inside which share i is the first to begin, a thread after four
// dimensions of a head in every `ways`th part.  A part of sum -1: the row is
// refused.  CTAs are large where rows have many parts (one context of 128K tokens,
// 57 parts a row: 41.4 us against 43.5) and small where many of them have two (33
// sequences, heads of 64: 25.9 against 29.1).
constexpr int kQ4MergeThreads = 512;   // at most

template <int D>
__global__ void __launch_bounds__(kQ4MergeThreads)
q4_merge_kernel(const __grid_constant__ Q4Params a)
{
    struct Part {
        float m, l;   // l of -1: refused
        float4 sums;
    };
    __shared__ Part parts[kQ4MergeThreads];
    const ListParams &p = a.list;
    const int items = p.group * (D / 4), ways = (int)blockDim.x / items;
    const int way = threadIdx.x / items, item = threadIdx.x - way * items;
    const int i = blockIdx.x, r = item / (D / 4), d = item % (D / 4) * 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Q4Share share = a.ws_share[i];
    const int64_t before = a.ws_share[max(i - 1, 0)].lo;
    // where shares begin: their loads are under way with the share's own (33
    // sequences, heads of 64: 23.6 us; loaded when that had come, 24.8)
    constexpr int B = 4;
    int64_t lo[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int k = b * (int)blockDim.x + threadIdx.x;
        lo[b] = k < a.shares ? a.ws_share[k].lo : INT64_MAX;
    }
    const int64_t row = share.lo - share.unit;
    if (share.unit == 0 || before > row)
        return;
    // the row's last share: the last one that starts before the row's end
    int begun = 0;
#pragma unroll
    for (int b = 0; b < B; ++b)
        begun += lo[b] < row + share.units;
    for (int k = B * (int)blockDim.x + threadIdx.x; k < a.shares; k += (int)blockDim.x)
        begun += a.ws_share[k].lo < row + share.units;
    __shared__ int warp_begun[kQ4MergeThreads / 32];
    begun = __reduce_add_sync(0xffffffffu, begun);
    if (threadIdx.x % 32 == 0)
        warp_begun[threadIdx.x / 32] = begun;
    __syncthreads();
    int last = -1;
    for (int w = 0; w < (int)blockDim.x / 32; ++w)
        last += warp_begun[w];
    float mx = -INFINITY, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    auto join = [&](const float2 &t, const float4 &x, float ref) {
        if (t.y != 0.f) {
            const Shift<true> by(t.x, ref);
            const float f = by.factor();
            den = by.add(t.y, den);
            num.x += f * x.x;
            num.y += f * x.y;
            num.z += f * x.z;
            num.w += f * x.w;
        }
    };
    constexpr int U = 8;
    for (int k0 = i - 1 + way; way < ways && k0 <= last; k0 += U * ways) {
        float2 t[U];
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(k0 + u * ways, last);
            // a share's second place holds the part of a row that is not its first
            const int64_t at = ((int64_t)k * 2 + (k < i && before != row)) * p.group + r;
            t[u] = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml) + at);
            x[u] = __ldcg(reinterpret_cast<const float4 *>(p.ws_acc + at * D + d));
        }
        float mn = mx;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            t[u] = k0 + u * ways <= last ? t[u] : make_float2(-INFINITY, 0.f);
            mn = fmaxf(mn, t[u].x);
            bad |= t[u].y < 0.f;
        }
        const float ref = reference_of(mn);
        const Shift<true> before(mx, ref);
        const float f0 = before.factor();
        den = before.of(den);
        num = make_float4(num.x * f0, num.y * f0, num.z * f0, num.w * f0);
#pragma unroll
        for (int u = 0; u < U; ++u)
            join(t[u], x[u], ref);
        mx = mn;
    }
    parts[threadIdx.x] = Part{mx, bad ? -1.f : den, num};
    __syncthreads();
    if (way > 0)
        return;
    float M = -INFINITY;
    for (int w = 0; w < ways; ++w) {
        M = fmaxf(M, parts[w * items + item].m);
        bad |= parts[w * items + item].l < 0.f;
    }
    const float ref = reference_of(M);
    den = 0.f;
    num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < ways; ++w) {
        const Part &x = parts[w * items + item];
        join(make_float2(x.m, x.l), x.sums, ref);
    }
    const int64_t head = ((int64_t)share.seq * p.num_kv_heads + share.head) * p.group + r;
    const bool zero = bad || den == 0.f;
    const float inv = 1.f / den;
    store_out4(p.out, p.out_dtype, head * D + d,
               zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv));
}

}  // namespace pkv
