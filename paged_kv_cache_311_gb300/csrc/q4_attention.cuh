// q4_attention.cuh -- single-query attention over a 4-bit cache
// (paged_attention_decode_q4):
//   out[s, h] = sum_t softmax_t(scale * q[s, h] . k_t) * v_t,
// a row's numbers s u + m for each group j of 64 dimensions (see q4_cache.cuh):
//   q . k_t   = sum_j s_tj (q_j . u_tj) + m_tj sum(q_j)
//   sum_t w_t v_t = sum_t (w_t s_tj) u_tj + sum_t w_t m_tj
// so that the products take whole numbers, and scales and minima join them in
// fp32.
//
// The frame is that of list_attention.cuh: one CTA per (partition of the
// context, kv head, sequence) with the kv head's G <= 8 query heads, partitions
// merged by a cluster or through the workspace.  Each of four warps streams
// records (bulk copies, one per block, codes with their scales) through a ring
// of its own, 32 tokens at a time, and takes them in two tiles of 16 tokens: a tile's tokens are M of
// S^T = K q^T, its dimensions M of O^T += V^T W^T, the query heads N of
// warp-level MMAs (m16n8k16).
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
// The M axes' order is free: row 2 c + e + 8 f of a tile is its token
// 4 c + 2 f + e (so that a thread's four tokens of V are neighbours), and a
// thread's rows of V^T are the dimensions that its words hold.
#pragma once

#include "list_attention.cuh"
#include "q4_cache.cuh"

namespace pkv {

struct Q4Params {
    ListParams list;             // without selected blocks and scales
    int64_t q_stride;            // elements between two sequences' rows of q
};

constexpr int kQ4Ring = 57344;   // ring bytes of a CTA at most
constexpr int kQ4Ctas = 3;       // CTAs per SM

template <int D, int BS> struct Q4Cfg {
    using R = Q4Row<D>;
    static constexpr int TILE = 16, TILES = 2;
    static constexpr int REC = R::template record<BS>;
    static constexpr int TOK = TILES * TILE;                   // tokens of a stage
    static constexpr int RECS = TOK / BS;
    // from a tile's codes and pairs to the next's
    static constexpr int NEXT_CODE = BS > TILE ? TILE * R::CODES : TILE / BS * REC;
    static constexpr int NEXT_PAIR = BS > TILE ? TILE * R::PAIRS : TILE / BS * REC;
    static constexpr int STAGE_BYTES = 2 * RECS * REC;
    static constexpr int S0 = kQ4Ring / (kListWarps * STAGE_BYTES);
    static constexpr int S = S0 < 2 ? 2 : S0;
    static constexpr int AWS = D + 4;                          // row stride of the merge scratch, in floats

    static constexpr int RING = (kListWarps * S * STAGE_BYTES + 127) / 128 * 128;
    // the warps' results and the CTA's, in the rings' memory once they are done with
    static constexpr int OFF_RESULT = kListWarps * kListMaxGroup * (AWS + 2) * 4;
    static constexpr int RESULT_END = OFF_RESULT + kListMaxGroup * (D + 2) * 4;
    static constexpr int OFF_PHYS = RING > RESULT_END ? RING : RESULT_END;
    static constexpr int OFF_AT = OFF_PHYS + kListCap * 4;
    static constexpr int OFF_BAR = OFF_AT + kListCap * 8;
    static constexpr int OFF_FLAG = OFF_BAR + kListWarps * S * 8;
    static constexpr int SMEM_BYTES = OFF_FLAG + 32 + 1024;    // slack for the alignment to 1024
    static_assert(REC % 16 == 0 && OFF_RESULT % 16 == 0 && OFF_PHYS % 16 == 0, "alignment");
};

// One warp's state.  Lane (g, c) = (lane / 4, lane % 4).
template <typename T, int D, int BS> struct Q4Engine {
    using C = Q4Cfg<D, BS>;
    using R = Q4Row<D>;
    static constexpr int NG = R::GROUPS;
    static constexpr float kMost = 32768.f;      // of a weight times its scale
    static constexpr float kLift = 7.f;          // log2 of the largest one where the reference is set
    static constexpr float kLeast = 0x1p-100f;   // smaller scales count as this: weights stay below 2^115

    uint32_t qf[NG][4][2];   // q^T B-fragments of head g: group, step
    float fs[2];             // heads 2c, 2c + 1: score of s (q . u)
    float fm[NG][2];         //                   score of m
    float o[NG][4][4];       // O^T C-fragments: group, m-tile
    float om[NG][2];         // this lane's tokens' sums of w m
    float m[2], lsum[2];     // heads 2c, 2c + 1: weights' reference and sum
    int kcode[2], kpair[2];  // byte offsets of this lane's tokens of K in a stage's records
    int vcode[4];            // and of V
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
            kpair[i] = rec_of(t) + R::template pair<BS>(t % BS, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * c + i;
            vcode[i] = rec_of(t) + R::word(t % BS, NG * g);
        }
        // q: dimensions 64 j + 16 c .. + 15 of head g, brought to f16 by a
        // power of two that puts the head's largest magnitude in [2^14, 2^15):
        // what f16 cannot hold is below 2^-35 of it
        const bool live = g < p.group;
        const T *qp = static_cast<const T *>(p.q) + (int64_t)seq * a.q_stride + (kvh * p.group + (live ? g : 0)) * D + 16 * c;
        uint32_t w[NG][8];
        float big = 0.f;
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
            for (int i = 0; i < 8; ++i) {
                const float2 f = Unpack<T>::pair(w[j][i] & 0x7fff7fffu);
                big = fmaxf(big, fmaxf(f.x, f.y));
            }
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        int x = (int)(__float_as_uint(big) >> 23) - 127 - 14;
        x = big < INFINITY ? max(x, -100) : 0;
        const float down = __uint_as_float((uint32_t)(127 - x) << 23);
        const float factor = p.qscale * __uint_as_float((uint32_t)(127 + x) << 23);
        float sum[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            sum[j] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = Unpack<T>::pair(w[j][4 * e + i]);
                    f[2 * i] = v.x * down;
                    f[2 * i + 1] = v.y * down;
                }
                // a word's pairs (n, n + 4), of which odd n come times 16
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float up = n & 1 ? 0.0625f : 1.f;
                    const uint32_t h = Mma<__half>::pack(f[n] * up, f[n + 4] * up);
                    qf[j][2 * e + (n >> 1)][n & 1] = h;
                    const float2 back = Unpack<__half>::pair(h);
                    sum[j] += (back.x + back.y) / up;
                }
            }
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
        }
        // head h's sits in lanes 4 h ..
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float f = __shfl_sync(0xffffffffu, factor, 8 * c + 4 * i);
            fs[i] = f * 16777216.f;
            m[i] = -INFINITY;
            lsum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                fm[j][i] = f * __shfl_sync(0xffffffffu, sum[j], 8 * c + 4 * i);
                om[j][i] = 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
                o[j][mt][0] = o[j][mt][1] = o[j][mt][2] = o[j][mt][3] = 0.f;
        }
    }

    // (scale, minimum) of each group of a row, from shared memory.
    __device__ __forceinline__ static void pairs(uint32_t at, float (&s)[NG], float (&mn)[NG])
    {
        if constexpr (NG == 2) {
            const uint2 v = lds64(at);
            const float2 a = Unpack<T>::pair(v.x), b = Unpack<T>::pair(v.y);
            s[0] = a.x;
            mn[0] = a.y;
            s[1] = b.x;
            mn[1] = b.y;
        } else {
            const float2 a = Unpack<T>::pair(lds32(at));
            s[0] = a.x;
            mn[0] = a.y;
        }
    }

    // S^T of a tile.
    __device__ __forceinline__ void scores(uint32_t kbase, int tile, float (&acc)[NG][4]) const
    {
        uint32_t w[2][2 * NG];   // token, word
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at = kbase + kcode[i] + tile * C::NEXT_CODE;
            if constexpr (NG == 2) {
                const uint4 v = lds128(at);
                w[i][0] = v.x;
                w[i][1] = v.y;
                w[i][2] = v.z;
                w[i][3] = v.w;
            } else {
                const uint2 v = lds64(at);
                w[i][0] = v.x;
                w[i][1] = v.y;
            }
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t u = w[0][NG * e + j], v = w[1][NG * e + j];
                const uint32_t a0[4] = {u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u};
                Mma<__half>::run(acc[j], a0, qf[j][2 * e][0], qf[j][2 * e][1]);
                const uint32_t a1[4] = {(u >> 8) & 0x000f000fu, (v >> 8) & 0x000f000fu, (u >> 8) & 0x00f000f0u, (v >> 8) & 0x00f000f0u};
                Mma<__half>::run(acc[j], a1, qf[j][2 * e + 1][0], qf[j][2 * e + 1][1]);
            }
        }
    }

    // The 32 tokens of the stage whose records start at kbase and vbase;
    // nvalid of them count.
    __device__ __forceinline__ void step(uint32_t kbase, uint32_t vbase, int nvalid)
    {
        // Online softmax in the log2 domain; this lane holds tokens t0 = 4 (g /
        // 2) + g % 2 and t0 + 2 of each tile, heads 2c, 2c + 1.  While no weight
        // times its scale passes kMost, weights are taken against the head's
        // reference m unchanged: no maximum across lanes, no rescaling.
        constexpr int N = 2 * C::TILES;          // this lane's tokens
        const int t0 = 4 * (g >> 1) + (g & 1);
        float x[N][2], p[N][2], s[N][NG], mn[N][NG], top[N];
        bool over = false;
#pragma unroll
        for (int tile = 0; tile < C::TILES; ++tile) {
            float acc[NG][4];
            scores(kbase, tile, acc);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = 2 * tile + i;
                pairs(kbase + kpair[i] + tile * C::NEXT_PAIR, s[n], mn[n]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float dot = s[n][0] * acc[0][2 * i + h], low = mn[n][0] * fm[0][h];
                    if constexpr (NG == 2) {
                        dot = fmaf(s[n][1], acc[1][2 * i + h], dot);
                        low = fmaf(mn[n][1], fm[1][h], low);
                    }
                    x[n][h] = fmaf(fs[h], dot, low);
                }
                pairs(vbase + kpair[i] + tile * C::NEXT_PAIR, s[n], mn[n]);
            }
        }
        if (nvalid < C::TOK) {
            // no token: what is there may be anything
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (t0 + 2 * (n & 1) + C::TILE * (n >> 1) >= nvalid) {
                    x[n][0] = x[n][1] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        s[n][j] = mn[n][j] = 0.f;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            // minima of a size that makes the scales' part of the numbers one
            // below fp32's last bit hold the weights down, too
            top[n] = NG == 2 ? fmaxf(fmaxf(s[n][0], s[n][NG - 1]), 0x1p-24f * fmaxf(fabsf(mn[n][0]), fabsf(mn[n][NG - 1])))
                             : fmaxf(s[n][0], 0x1p-24f * fabsf(mn[n][0]));
            top[n] = fmaxf(top[n], kLeast);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                p[n][h] = ex2_fast(x[n][h] - m[h]);   // infinite before the first token
                over |= p[n][h] * top[n] > kMost;
            }
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float t = -INFINITY;
#pragma unroll
                for (int n = 0; n < N; ++n)
                    t = fmaxf(t, x[n][h] + __log2f(top[n]) - kLift);
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                t = fmaxf(m[h], t);
                const float ref = reference_of(t), alpha = ex2_fast(m[h] - ref);
                m[h] = t;
                lsum[h] *= alpha;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    om[j][h] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        o[j][mt][h] *= alpha;
                        o[j][mt][2 + h] *= alpha;
                    }
                }
#pragma unroll
                for (int n = 0; n < N; ++n)
                    p[n][h] = ex2_fast(x[n][h] - ref);
            }
        }

        // The weights' sums, their products with the minima in fp32, and with
        // the scales in two f16 parts each, as B-fragments.
#pragma unroll
        for (int tile = 0; tile < C::TILES; ++tile) {
            uint32_t hi[NG][2], lo[NG][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = 2 * tile + i;
                lsum[0] += p[n][0];
                lsum[1] += p[n][1];
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    om[j][0] = fmaf(p[n][0], mn[n][j], om[j][0]);
                    om[j][1] = fmaf(p[n][1], mn[n][j], om[j][1]);
                    const float a = p[n][0] * s[n][j], b = p[n][1] * s[n][j];
                    const uint32_t h = Mma<__half>::pack(a, b);
                    const float2 f = Unpack<__half>::pair(h);
                    hi[j][i] = movmatrix_trans(h);
                    lo[j][i] = movmatrix_trans(Mma<__half>::pack(a - f.x, b - f.y));
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
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t a[4] = {(u >> (8 * k)) & 0x000f000fu, (u >> (8 * k)) & 0x00f000f0u,
                                               (v >> (8 * k)) & 0x000f000fu, (v >> (8 * k)) & 0x00f000f0u};
                        Mma<__half>::run(o[j][2 * e + k], a, hi[j][0], hi[j][1]);
                        Mma<__half>::run(o[j][2 * e + k], a, lo[j][0], lo[j][1]);
                    }
                }
            }
        }
    }

    // This warp's (max, sum, sums of values) of the heads below `group` into
    // the merge scratch.
    __device__ __forceinline__ void finish(float *mw, float *lw, float *aw, int warp, int group)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = lsum[h], add[NG];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                add[j] = om[j][h];
                add[j] += __shfl_xor_sync(0xffffffffu, add[j], 4);
                add[j] += __shfl_xor_sync(0xffffffffu, add[j], 8);
                add[j] += __shfl_xor_sync(0xffffffffu, add[j], 16);
            }
            const int row = 2 * c + h;
            if (row < group) {
                if (g == 0) {
                    mw[warp * kListMaxGroup + row] = m[h];
                    lw[warp * kListMaxGroup + row] = l;
                }
                float *dst = aw + (warp * kListMaxGroup + row) * C::AWS + 8 * g;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
                        *reinterpret_cast<float2 *>(dst + 64 * j + 2 * mt) = make_float2(fmaf(o[j][mt][h], 16777216.f, add[j]), fmaf(o[j][mt][2 + h], 1048576.f, add[j]));
                }
            }
        }
    }
};

// Grid (partition, kv head, sequence).
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kListThreads, kQ4Ctas)
q4_attention_kernel(const __grid_constant__ Q4Params a)
{
    using C = Q4Cfg<D, BS>;
    constexpr int S = C::S, NW = kListWarps;
    const ListParams &p = a.list;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    int32_t *phys = reinterpret_cast<int32_t *>(smem + C::OFF_PHYS);
    int64_t *record = reinterpret_cast<int64_t *>(smem + C::OFF_AT);   // byte offsets of the partition's records
    const int part = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + warp * S;
    uint32_t *flag = reinterpret_cast<uint32_t *>(smem + C::OFF_FLAG);
    int *warp_tokens = reinterpret_cast<int *>(smem + C::OFF_FLAG + 16);
    if (lane == 0) {
        for (int s = 0; s < S; ++s)
            mbar_init(&bars[s], 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0)
        *flag = 0;
    wait_for_stream();
    const int L = p.context_lens[seq];
    const int e0 = part * p.part_blocks;
    ListEntries<BS> entries;
    entries.load(p, seq, kvh, e0);
    ListResult<D> *res = reinterpret_cast<ListResult<D> *>(smem + C::OFF_RESULT);
    int tokens = 0;
    if (L < 0 || L > p.max_context_len) {
        if (part == 0 && kvh == 0 && threadIdx.x == 0)
            report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
        tokens = -1;
    } else if ((int64_t)e0 * BS < L) {
        tokens = entries.resolve(p, phys, e0, L);
        const int most = __reduce_max_sync(0xffffffffu, tokens);
        if (lane == 0)
            warp_tokens[warp] = most;
        if (__syncthreads_or(tokens < 0)) {
            if (threadIdx.x == 0)
                report(p.status, PKV_DEV_BAD_BLOCK);
            tokens = -1;
        } else {
#pragma unroll
            for (int w = 0; w < NW; ++w)
                tokens = max(tokens, warp_tokens[w]);
        }
    }
    if (tokens <= 0) {
        if (threadIdx.x < kListMaxGroup) {
            res->m[threadIdx.x] = -INFINITY;
            res->l[threadIdx.x] = tokens < 0 ? -1.f : 0.f;
        }
        __syncthreads();
        write_result<D>(p, res, seq, kvh, part);
        return;
    }

#pragma unroll 1
    for (int k = threadIdx.x; k * BS < tokens; k += kListThreads)
        record[k] = ((int64_t)phys[k] * p.num_kv_heads + kvh) * C::REC;
    __syncthreads();

    // ---- this warp's stages: warp, warp + NW, ...
    const int nstages = (tokens + C::TOK - 1) / C::TOK;
    const int my_n = warp < nstages ? (nstages - 1 - warp) / NW + 1 : 0;
    uint8_t *stages = smem + warp * S * C::STAGE_BYTES;
    auto issue = [&](int i, int st) {
        const int t0 = (warp + i * NW) * C::TOK;
        uint8_t *kd = stages + st * C::STAGE_BYTES, *vd = kd + C::RECS * C::REC;
        const int n = min(C::RECS, (tokens - t0 + BS - 1) / BS);
        mbar_arrive_expect_tx(&bars[st], (uint32_t)(n * 2 * C::REC));
        for (int b = 0; b < n; ++b) {
            const int64_t at = record[t0 / BS + b];
            bulk_load(kd + b * C::REC, p.k_cache + at, C::REC, &bars[st]);
            bulk_load(vd + b * C::REC, p.v_cache + at, C::REC, &bars[st]);
        }
    };
    if (lane == 0) {
        for (int i = 0; i < min(my_n, S); ++i)
            issue(i, i);
    }
    Q4Engine<T, D, BS> eng;
    eng.init(a, seq, kvh, lane);

    int failed_at = -1;
    for (int i = 0; i < my_n; ++i) {
        const int st = i % S;
        // the warp gives up as one: its products and shuffles need every lane
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[st], (uint32_t)((i / S) & 1)))) {
            failed_at = i;
            break;
        }
        const int t0 = (warp + i * NW) * C::TOK;
        const uint32_t kbase = smem_u32(stages + st * C::STAGE_BYTES);
        eng.step(kbase, kbase + C::RECS * C::REC, tokens - t0);
        __syncwarp();
        if (lane == 0 && i + S < my_n) {
            fence_proxy_async_smem();
            issue(i + S, st);
        }
    }
    if (failed_at >= 0) {
        // no CTA leaves with loads in flight
        for (int i = failed_at; i < min(my_n, failed_at + S); ++i)
            drain_wait(&bars[i % S], (uint32_t)((i / S) & 1), p.status);
        if (lane == 0) {
            report(p.status, PKV_DEV_TIMEOUT);
            atomicOr(flag, 1u);
        }
    }

    // ---- the warps' parts, through the rings' memory
    __syncthreads();
    const bool failed = *reinterpret_cast<volatile uint32_t *>(flag) != 0;
    float *mw = reinterpret_cast<float *>(smem);
    float *lw = mw + NW * kListMaxGroup;
    float *aw = lw + NW * kListMaxGroup;
    eng.finish(mw, lw, aw, warp, p.group);
    __syncthreads();
    for (int i = threadIdx.x; i < p.group * D; i += kListThreads) {
        const int r = i / D, d = i % D;
        float Mx = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            Mx = fmaxf(Mx, mw[w * kListMaxGroup + r]);
        const float ref = reference_of(Mx);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2f(mw[w * kListMaxGroup + r] - ref);   // 0 for a warp without tokens; NaN sums stay
            num += f * aw[(w * kListMaxGroup + r) * C::AWS + d];
            den += f * lw[w * kListMaxGroup + r];
        }
        res->acc[r][d] = num;
        if (d == 0) {
            res->m[r] = Mx;
            res->l[r] = failed ? -1.f : den;
        }
    }
    __syncthreads();
    write_result<D>(p, res, seq, kvh, part);
    if (p.np > 1 && !p.cluster)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace pkv
