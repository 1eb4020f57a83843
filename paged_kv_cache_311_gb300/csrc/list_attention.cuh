// list_attention.cuh -- single-query attention over a list of a sequence's
// blocks: all of them in an e4m3 cache (paged_attention_decode_q8), or the
// selected ones of a 16-bit or an e4m3 cache (paged_attention_decode_selected).
//
//   out[s, h] = sum_i softmax_i(scale * ks_b(i) * q[s, h] . k_i) * vs_b(i) * v_i
// over the tokens i of the listed blocks, ks and vs the block's scales (1 in a
// 16-bit cache).
//
// One CTA per (partition of the list, kv head, sequence); it owns the kv
// head's G <= 8 query heads, so each K/V byte is read from HBM once.  With more
// than one partition each CTA has (max, sum, unnormalised sum of values) to
// give.  Up to eight partitions are a cluster: they exchange them through
// their shared memory, and each writes a part of the output.  More of them
// write them to the workspace for list_merge_kernel.
//
// Each of the CTA's four warps streams tiles of 16 tokens through a ring of
// TMA loads of its own (128-byte swizzled boxes, one per block) and runs the
// online softmax over them with warp-level MMAs (m16n8k16): the tile's tokens
// are M of S^T = K q^T, its dimensions M of O^T += V^T P^T, the query heads N.
//
// An e4m3 tile is multiplied in f16, which holds every e4m3 value exactly; the
// conversion is one instruction per two values, on fragments as ldmatrix
// leaves them:
//   K: a thread gets four neighbouring dimensions of a row where a 16-bit
//      tile gives two.  A dot product may take its dimensions in any order, so
//      the low pair plays dimensions 2c, 2c + 1 of the MMA's k axis and the
//      high pair 2c + 8, 2c + 9; q is laid out to match.
//   V: transposed ldmatrix moves byte pairs (dimensions 2g, 2g + 1) of tokens
//      2c, 2c + 1; one byte permute pairs them by dimension.  Row g of the
//      MMA's M axis is then dimension 2g and row g + 8 dimension 2g + 1.
// The K scale multiplies the scores (exactly: a power of two); the V scale
// multiplies the tile's product as it joins the accumulators, so no weight
// has to fit a 16-bit range together with it.
//
// What bounds it: HBM.  Sixteen q8 contexts of 16K to 32K tokens (808 MB) take
// 134 to 139 us, 6.0 TB/s or 90 to 87 % of a copy's rate (93 % while the SMs have
// work); 64 of 128 to 2048 tokens with 32 kv heads 91 to 102 us (94 to 84 %);
// 128 blocks of 16 tokens of a 16-bit cache for 32 x 8 rows 43.5 us (93 %).  Over
// the 8-bit cache those rows take 29 us (70 %): too few warps for the chain of
// dependent instructions that each runs per tile.  One
// request of 700 tokens takes 5.6 us, a launch and the latencies of length and
// table, tile, products and merge.
#pragma once

#include <cooperative_groups.h>

#include "pa_decode.cuh"
#include "q8_cache.cuh"

namespace pkv {

// The reference that weights are taken against: the largest score, or 0 where
// there is none yet, so that 2^(-inf - reference) is 0 and not NaN.
__device__ __forceinline__ float reference_of(float m) { return m == -INFINITY ? 0.f : m; }

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
    int cluster;                 // nonzero: the np CTAs of a row are a cluster
    int out_dtype, q_dtype;
    float qscale;                // softmax scale * log2(e)
};

constexpr int kListWarps = 4;
constexpr int kListThreads = kListWarps * 32;
constexpr int kListMaxGroup = 8;
constexpr int kListCap = 512;    // list entries one CTA stages

// The element an MMA works on, and the cache's bytes per element.
template <typename T> struct ListElem {
    using M = T;
    static constexpr int bytes = 2;
    static constexpr CUtensorMapDataType tma = Elem<T>::tma;
};
template <> struct ListElem<uint8_t> {
    using M = __half;
    static constexpr int bytes = 1;
    static constexpr CUtensorMapDataType tma = CU_TENSOR_MAP_DATA_TYPE_UINT8;
};

// Ring bytes of a CTA (at least two stages a warp), and CTAs per SM: four with
// 48 KB against three with 64 took q8 contexts of 16K to 32K tokens from 142
// to 138 us, a batch of 64 from 95.6 to 93.6; five with 32 KB: 146 and 96.
constexpr int kListRing = 49152;
constexpr int kListCtas = 4;

template <typename T, int D, int BS>
struct ListCfg {
    static constexpr bool Q8 = ListElem<T>::bytes == 1;
    static constexpr int TILE = 16;
    static constexpr int ROW = D * ListElem<T>::bytes;         // bytes of a token's row
    // a box's lines are 128 bytes: a row's chunk, or two rows of 64 bytes
    static constexpr int TPL = ROW < 128 ? 128 / ROW : 1;      // tokens per line
    static constexpr int CHUNKS = ROW < 128 ? 1 : ROW / 128;
    static constexpr int PPT = (ROW < 128 ? ROW : 128) / 16;   // 16-byte pieces of a token in a line
    static constexpr int BOX_TOK = BS < TILE ? BS : TILE;
    static constexpr int BOXES = TILE / BOX_TOK;
    static constexpr int BOX_LINES = BOX_TOK / TPL;
    static constexpr int BOX_BYTES = BOX_TOK * ROW;
    static constexpr int BOX_STRIDE = BOX_BYTES < 1024 ? 1024 : BOX_BYTES;   // swizzle atoms are 1024 bytes
    static constexpr int TILE_BYTES = BOXES * BOX_STRIDE;      // K (or V) of a tile
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int S0 = kListRing / (kListWarps * STAGE_BYTES);
    static constexpr int S = S0 < 2 ? 2 : S0;
    static constexpr int KS = D / 16;                          // k-steps of QK, m-tiles of PV
    static constexpr int AWS = D + 4;                          // row stride of the merge scratch, in floats

    static constexpr int OFF_PHYS = kListWarps * S * STAGE_BYTES;
    static constexpr int OFF_KS = OFF_PHYS + kListCap * 4;
    static constexpr int OFF_VS = OFF_KS + (Q8 ? kListCap * 4 : 0);
    static constexpr int OFF_BAR = OFF_VS + (Q8 ? kListCap * 4 : 0);
    static constexpr int OFF_FLAG = OFF_BAR + kListWarps * S * 8;
    static constexpr int SMEM_BYTES = OFF_FLAG + 32 + 1024;    // slack for the alignment to 1024

    static_assert(BOX_BYTES % 512 == 0 && BOX_STRIDE % 1024 == 0 && S >= 2, "ring");
    // the CTA's result, behind the warps' in the rings' memory
    static constexpr int OFF_RESULT = kListWarps * kListMaxGroup * (AWS + 2) * 4;
    static_assert(OFF_RESULT % 16 == 0 && OFF_RESULT + kListMaxGroup * (D + 2) * 4 <= OFF_PHYS, "merge scratch fits in the ring");

    // Shared-memory offset of 16-byte piece q of token t of a tile.
    __device__ __forceinline__ static uint32_t addr(int t, int q)
    {
        const int bx = t / BOX_TOK, r = t % BOX_TOK;
        const int line = r / TPL, pc = (r % TPL) * PPT + q % PPT;
        return bx * BOX_STRIDE + ((q / PPT) * BOX_LINES + line) * 128 + ((pc ^ (line & 7)) << 4);
    }
};

// The list entries of a CTA's partition: thread t looks at entries t, t + 128,
// ... of it.  Two steps, so that every load that can leave at once does: load()
// needs nothing but the arguments, resolve() the row's length.  The loops stay
// rolled: code that runs once costs its fetching, about 128 bytes in 45 cycles.
//
// A selected list is refused unless it is strictly ascending and inside the
// sequence's blocks, with -1 only behind its last entry: so no block counts
// twice and only the last entry can be partial.
template <int BS>
struct ListEntries {
    const int32_t *src, *table;
    int id, before;   // entry t, and the list's entry in front (selected lists)

    __device__ __forceinline__ void get(const ListParams &p, int e0, int k)
    {
        id = src[k];
        before = p.selected && e0 + k > 0 ? src[k - 1] : -1;
    }

    __device__ __forceinline__ void load(const ListParams &p, int seq, int kvh, int e0)
    {
        table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
        src = p.selected ? p.selected + ((int64_t)seq * p.num_kv_heads + kvh) * p.num_selected + e0 : table + e0;
        const int k = (int)threadIdx.x;
        if (k < min(p.part_blocks, (p.selected ? p.num_selected : p.max_blocks_per_seq) - e0))
            get(p, e0, k);
    }

    // Physical block ids into phys; returns the tokens of this thread's
    // entries counted from the partition's start, or -1 for a refused entry.
    __device__ __forceinline__ int resolve(const ListParams &p, int32_t *phys, int e0, int L)
    {
        const int nblk = (L + BS - 1) / BS;
        const int have = min(p.part_blocks, (p.selected ? p.num_selected : nblk) - e0);
        int tokens = 0;
        bool bad = false;
#pragma unroll 1
        for (int k = (int)threadIdx.x; k < have; k += kListThreads) {
            if (k >= kListThreads)
                get(p, e0, k);
            int b = id, here = L - e0 * BS - k * BS;   // tokens from the entry on
            if (p.selected) {
                if (id < 0 || id >= nblk || (e0 + k > 0 && (before < 0 || before >= id))) {
                    bad |= id != -1;
                    continue;
                }
                b = table[id];
                here = L - id * BS;
            }
            bad |= b < 0 || (int64_t)b >= p.num_blocks;
            phys[k] = b;
            tokens = max(tokens, k * BS + min(BS, here));
        }
        return bad ? -1 : tokens;
    }
};

// What a CTA has of its row's heads: (max, sum) and, for a positive sum, the
// sums of values; a sum of -1: refused.  In the rings' memory once they are
// done with.
template <int D>
struct ListResult {
    float m[kListMaxGroup], l[kListMaxGroup];
    float acc[kListMaxGroup][D];
};

// Writes the CTA's result where it goes: the output (one partition, or a
// cluster, which all CTAs of it have to reach) or the workspace.  All threads
// call it after a barrier behind the result's last store.
template <int D>
__device__ __forceinline__ void write_result(const ListParams &p, ListResult<D> *res, int seq, int kvh, int part)
{
    const int64_t head0 = ((int64_t)seq * p.num_kv_heads + kvh) * p.group;
    const int total = p.group * D;
    if (p.cluster) {
        namespace cg = cooperative_groups;
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        for (int i = (part * kListThreads + (int)threadIdx.x) * 4; i < total; i += p.np * kListThreads * 4) {
            const int r = i / D, d = i % D;
            float m[8], l[8], M = -INFINITY;
            float4 a[8];
            bool bad = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                m[k] = -INFINITY;
                l[k] = 0.f;
                a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < p.np) {
                    const ListResult<D> *other = cluster.map_shared_rank(res, k);
                    m[k] = other->m[r];
                    l[k] = other->l[r];
                    a[k] = *reinterpret_cast<const float4 *>(&other->acc[r][d]);
                }
                M = fmaxf(M, m[k]);
                bad |= l[k] < 0.f;
            }
            const float ref = reference_of(M);
            float den = 0.f;
            float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (l[k] != 0.f) {   // else its sums of values were not stored
                    const float f = exp2f(m[k] - ref);
                    den += f * l[k];
                    num.x += f * a[k].x;
                    num.y += f * a[k].y;
                    num.z += f * a[k].z;
                    num.w += f * a[k].w;
                }
            }
            const bool zero = bad || den == 0.f;
            const float inv = 1.f / den;
            store_out4(p.out, p.out_dtype, (head0 + r) * D + d,
                       zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv));
        }
        cluster.sync();   // no CTA leaves while another reads its shared memory
        return;
    }
    for (int i = (int)threadIdx.x * 4; i < total; i += kListThreads * 4) {
        const int r = i / D, d = i % D;
        const float l = res->l[r];
        const float4 a = *reinterpret_cast<const float4 *>(&res->acc[r][d]);
        if (p.np == 1) {
            const float inv = 1.f / l;
            const bool zero = l == 0.f || l < 0.f;
            store_out4(p.out, p.out_dtype, (head0 + r) * D + d,
                       zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
        } else {
            const int64_t slot = (head0 + r) * p.np + part;
            if (l != 0.f)
                *reinterpret_cast<float4 *>(p.ws_acc + slot * D + d) = a;
            if (d == 0)
                *reinterpret_cast<float2 *>(p.ws_ml + slot * 2) = make_float2(res->m[r], l);
        }
    }
}

// One warp's state: its rows of q, running maxima, sums and accumulators.
// Lane (g, c) = (lane / 4, lane % 4).
template <typename T, int D, int BS>
struct ListEngine {
    using C = ListCfg<T, D, BS>;
    using M = typename ListElem<T>::M;
    static constexpr int KS = C::KS;
    // What a weight (at most 2^kSlack) is multiplied by on its way to its parts
    // of M's type: f16's numbers end at 2^-24, and weights of that size count
    // where a context has many of them beside one large weight of value 0.
    // Taken back from a tile's product with the V scale, or at the end.
    static constexpr float kLift = std::is_same<M, __half>::value ? 128.f : 1.f;

    uint32_t qf[KS][2];      // q^T B-fragments of head g
    float o[KS][4];          // O^T C-fragments
    float m[2], lsum[2];     // heads 2c, 2c + 1
    float qs[2];             // score factors of heads 2c, 2c + 1
    uint32_t koff[4], voff[4];   // this lane's ldmatrix offsets in a tile, 64 bytes of a row
    int g, c;

    // Issues the loads of q.
    __device__ __forceinline__ void load(const ListParams &p, int seq, int kvh, int lane)
    {
        g = lane >> 2;
        c = lane & 3;
        const bool live = g < p.group;
        const int64_t row = ((int64_t)seq * p.num_kv_heads + kvh) * p.group + (live ? g : 0);
        const uint32_t *qp = reinterpret_cast<const uint32_t *>(p.q) + row * (D / 2);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if constexpr (C::Q8) {
                const uint2 w = live ? *reinterpret_cast<const uint2 *>(qp + 8 * ks + 2 * c) : make_uint2(0u, 0u);
                qf[ks][0] = w.x;
                qf[ks][1] = w.y;
            } else {
                qf[ks][0] = live ? qp[8 * ks + c] : 0u;
                qf[ks][1] = live ? qp[8 * ks + c + 4] : 0u;
            }
        }
    }

    __device__ __forceinline__ void init(const ListParams &p)
    {
        const int lane = threadIdx.x & 31;
        const int tk = (lane & 7) + ((lane >> 3) & 1) * 8, dk = lane >> 4;
        const int tv = C::Q8 ? tk : (lane & 7) + (lane >> 4) * 8, dv = C::Q8 ? dk : (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            koff[k] = C::addr(tk, (2 * k + dk) % (C::CHUNKS * C::PPT));
            voff[k] = C::addr(tv, (2 * k + dv) % (C::CHUNKS * C::PPT));
        }
        float factor = p.qscale;
        if constexpr (C::Q8) {
            if (p.q_dtype == PKV_BF16) {
                // bfloat16 to f16: the row's largest magnitude is brought to
                // [2^14, 2^15) by a power of two, so that what f16 cannot
                // hold is below 2^-38 of it
                __nv_bfloat162 mx = as_pair<__nv_bfloat16>(0u);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    mx = __hmax2(mx, as_pair<__nv_bfloat16>(qf[ks][0] & 0x7fff7fffu));
                    mx = __hmax2(mx, as_pair<__nv_bfloat16>(qf[ks][1] & 0x7fff7fffu));
                }
                const float2 f = Unpack<__nv_bfloat16>::pair(as_word(mx));
                float a = fmaxf(f.x, f.y);
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                int x = (int)(__float_as_uint(a) >> 23) - 127 - 14;
                x = a < INFINITY ? max(x, -100) : 0;
                const float down = __uint_as_float((uint32_t)(127 - x) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = Unpack<__nv_bfloat16>::pair(qf[ks][i]);
                        qf[ks][i] = Mma<__half>::pack(v.x * down, v.y * down);
                    }
                }
                factor *= __uint_as_float((uint32_t)(127 + x) << 23);
            }
        }
        // head h's factor sits in lanes 4 h ..
        qs[0] = __shfl_sync(0xffffffffu, factor, 8 * c);
        qs[1] = __shfl_sync(0xffffffffu, factor, 8 * c + 4);
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
            o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        lsum[0] = lsum[1] = 0.f;
    }

    // Byte offset of the chunk that holds 32 bytes group k of a row.
    __device__ __forceinline__ static uint32_t chunk_off(int k) { return (uint32_t)((k >> 2) * C::BOX_LINES * 128); }

    // A tile's tokens: rows 0..7 with scales ks0, vs0, rows 8..15 with ks1,
    // vs1 (the same unless a block holds 8 tokens; vs0 and vs1 divided by
    // kLift); nvalid of them count.
    __device__ __forceinline__ void tile(uint32_t kbase, uint32_t vbase, int nvalid, int lane, float ks0, float ks1,
                                         float vs0, float vs1)
    {
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (C::Q8) {
#pragma unroll
            for (int j = 0; j < KS / 2; ++j) {
                uint32_t w[4];
                ldsm_x4(kbase + chunk_off(j) + koff[j & 3], w);
                const uint32_t a0[4] = {f16x2_of_e4m3(w[0] & 0xffffu), f16x2_of_e4m3(w[1] & 0xffffu),
                                        f16x2_of_e4m3(w[0] >> 16), f16x2_of_e4m3(w[1] >> 16)};
                const uint32_t a1[4] = {f16x2_of_e4m3(w[2] & 0xffffu), f16x2_of_e4m3(w[3] & 0xffffu),
                                        f16x2_of_e4m3(w[2] >> 16), f16x2_of_e4m3(w[3] >> 16)};
                Mma<M>::run(s, a0, qf[2 * j][0], qf[2 * j][1]);
                Mma<M>::run(s2, a1, qf[2 * j + 1][0], qf[2 * j + 1][1]);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a[4];
                ldsm_x4(kbase + chunk_off(ks) + koff[ks & 3], a);
                Mma<M>::run(ks & 1 ? s2 : s, a, qf[ks][0], qf[ks][1]);
            }
        }

        // Online softmax in the log2 domain; this lane holds tokens g, g + 8
        // of heads 2c, 2c + 1.  While every score stays within kSlack of its
        // head's reference m, the weights 2^(x - m) <= 2^kSlack are taken
        // against it unchanged: no maximum across lanes, no rescaling.
        constexpr float kSlack = 8.f;
        const bool ok0 = g < nvalid, ok1 = g + 8 < nvalid;
        float x0[2], x1[2], p0[2], p1[2];
        bool over = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x0[j] = ok0 ? (s[j] + s2[j]) * (qs[j] * ks0) : -INFINITY;
            x1[j] = ok1 ? (s[2 + j] + s2[2 + j]) * (qs[j] * ks1) : -INFINITY;
            over |= fmaxf(x0[j], x1[j]) > m[j] + kSlack;
        }
        if (__any_sync(0xffffffffu, over)) {
            float alpha[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float tm = fmaxf(x0[j], x1[j]);
                tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 4));
                tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 8));
                tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
                const float mn = fmaxf(m[j], tm);
                // no number yet: the sums are zero (or NaN), whatever alpha is
                alpha[j] = ex2_fast(m[j] - reference_of(mn));
                lsum[j] *= alpha[j];
                m[j] = mn;
            }
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                o[mt][0] *= alpha[0];
                o[mt][1] *= alpha[1];
                o[mt][2] *= alpha[0];
                o[mt][3] *= alpha[1];
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float mr = reference_of(m[j]);   // a NaN score stays NaN
            p0[j] = ex2_fast(x0[j] - mr);
            p1[j] = ex2_fast(x1[j] - mr);
            lsum[j] += p0[j] + p1[j];
        }

        // Rows of V past the valid tokens may hold anything; zero them so that
        // a weight of 0 leaves 0.
        if (nvalid < C::TILE) {
            constexpr int NPC = C::CHUNKS * C::PPT;
            for (int i = lane; i < (C::TILE - nvalid) * NPC; i += 32)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vbase + C::addr(nvalid + i / NPC, i % NPC)),
                             "r"(0u)
                             : "memory");
            // a later load into the stage must not overtake these stores: each
            // lane orders its own before it
            fence_proxy_async_smem();
            __syncwarp();
        }

        // The weights enter the product in two 16-bit parts (whatever the
        // output's type: what one part drops is not small beside values that
        // cancel): off by (half a step)^2 of themselves, 2^-22 in f16, 2^-16 in
        // bfloat16; f16 parts of tiny ones by half their last bit, 2^-25 / kLift
        // of the largest weight.
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            p0[j] *= kLift;
            p1[j] *= kLift;
        }
        const uint32_t h0 = Mma<M>::pack(p0[0], p0[1]), h1 = Mma<M>::pack(p1[0], p1[1]);
        const uint32_t bh0 = movmatrix_trans(h0), bh1 = movmatrix_trans(h1);
        const float2 f0 = Mma<M>::unpack(h0), f1 = Mma<M>::unpack(h1);
        const uint32_t bl0 = movmatrix_trans(Mma<M>::pack(p0[0] - f0.x, p0[1] - f0.y));
        const uint32_t bl1 = movmatrix_trans(Mma<M>::pack(p1[0] - f1.x, p1[1] - f1.y));
        if constexpr (C::Q8) {
#pragma unroll
            for (int j = 0; j < KS / 2; ++j) {
                uint32_t w[4];
                ldsm_x4_trans(vbase + chunk_off(j) + voff[j & 3], w);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t u = __byte_perm(w[2 * i], 0, 0x3120), v = __byte_perm(w[2 * i + 1], 0, 0x3120);
                    const uint32_t a[4] = {f16x2_of_e4m3(u & 0xffffu), f16x2_of_e4m3(u >> 16),
                                           f16x2_of_e4m3(v & 0xffffu), f16x2_of_e4m3(v >> 16)};
                    float t[4] = {0.f, 0.f, 0.f, 0.f};
                    float *acc = o[2 * j + i];
                    if constexpr (BS == 8) {
                        mma_k8(t, a[0], a[1], bh0);
                        mma_k8(t, a[0], a[1], bl0);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            acc[k] = fmaf(vs0, t[k], acc[k]);
                            t[k] = 0.f;
                        }
                        mma_k8(t, a[2], a[3], bh1);
                        mma_k8(t, a[2], a[3], bl1);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[k] = fmaf(vs1, t[k], acc[k]);
                    } else {
                        Mma<M>::run(t, a, bh0, bh1);
                        Mma<M>::run(t, a, bl0, bl1);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[k] = fmaf(vs0, t[k], acc[k]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                uint32_t a[4];
                ldsm_x4_trans(vbase + chunk_off(mt) + voff[mt & 3], a);
                Mma<M>::run(o[mt], a, bh0, bh1);
                Mma<M>::run(o[mt], a, bl0, bl1);
            }
        }
    }

    // D = A * B + D, m16n8k8, f16.
    __device__ __forceinline__ static void mma_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b)
    {
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(b));
    }

    // This warp's (max, sum, sums of values) of the heads below `group` into
    // the merge scratch.
    __device__ __forceinline__ void finish(float *mw, float *lw, float *aw, int warp, int group)
    {
        if constexpr (!C::Q8 && kLift != 1.f) {
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[mt][k] *= 1.f / kLift;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l = lsum[j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int row = 2 * c + j;
            if (row < group) {
                if (g == 0) {
                    mw[warp * kListMaxGroup + row] = m[j];
                    lw[warp * kListMaxGroup + row] = l;
                }
                float *dst = aw + (warp * kListMaxGroup + row) * C::AWS;
#pragma unroll
                for (int mt = 0; mt < KS; ++mt) {
                    if constexpr (C::Q8) {
                        *reinterpret_cast<float2 *>(dst + 16 * mt + 2 * g) = make_float2(o[mt][j], o[mt][2 + j]);
                    } else {
                        dst[16 * mt + g] = o[mt][j];
                        dst[16 * mt + g + 8] = o[mt][2 + j];
                    }
                }
            }
        }
    }
};

// T: __half, __nv_bfloat16, or uint8_t for an e4m3 cache.  Grid (partition,
// kv head, sequence).
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kListThreads, kListCtas)
list_attention_kernel(const __grid_constant__ ListParams p, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv)
{
    using C = ListCfg<T, D, BS>;
    constexpr int S = C::S, TILE = C::TILE, NW = kListWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    int32_t *phys = reinterpret_cast<int32_t *>(smem + C::OFF_PHYS);
    float *ks_s = reinterpret_cast<float *>(smem + C::OFF_KS);
    float *vs_s = reinterpret_cast<float *>(smem + C::OFF_VS);
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
    if (threadIdx.x == 0) {
        *flag = 0;
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    wait_for_stream();
    // what needs nothing but the arguments leaves first: the length, the
    // list's entries and q
    const int L = p.context_lens[seq];
    const int e0 = part * p.part_blocks;
    ListEntries<BS> entries;
    entries.load(p, seq, kvh, e0);
    ListEngine<T, D, BS> eng;
    eng.load(p, seq, kvh, lane);
    ListResult<D> *res = reinterpret_cast<ListResult<D> *>(smem + C::OFF_RESULT);
    int tokens = 0;
    if (L < 0 || L > p.max_context_len) {
        if (part == 0 && kvh == 0 && threadIdx.x == 0)
            report(p.status, PKV_DEV_BAD_CONTEXT_LEN);
        tokens = -1;
    } else if (p.selected || e0 * BS < L) {
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

    // ---- this warp's tiles: warp, warp + NW, ...
    const int ntiles = (tokens + TILE - 1) / TILE;
    const int my_n = warp < ntiles ? (ntiles - 1 - warp) / NW + 1 : 0;
    uint8_t *stages = smem + warp * S * C::STAGE_BYTES;
    auto issue = [&](int i, int st) {
        const int t0 = (warp + i * NW) * TILE;
        uint8_t *kd = stages + st * C::STAGE_BYTES, *vd = kd + C::TILE_BYTES;
        const int nbox = min(C::BOXES, (tokens - t0 + C::BOX_TOK - 1) / C::BOX_TOK);
        mbar_arrive_expect_tx(&bars[st], (uint32_t)(nbox * 2 * C::BOX_BYTES));
        for (int b = 0; b < nbox; ++b) {
            const int tok = t0 + b * C::BOX_TOK;
            const int blk = phys[tok / BS], line = (tok % BS) / C::TPL;
            tma_load_5d(kd + b * C::BOX_STRIDE, &tmk, &bars[st], 0, line, 0, kvh, blk);
            tma_load_5d(vd + b * C::BOX_STRIDE, &tmv, &bars[st], 0, line, 0, kvh, blk);
        }
    };
    if (lane == 0) {
        for (int i = 0; i < min(my_n, S); ++i)
            issue(i, i);
    }
    if constexpr (C::Q8) {
#pragma unroll 1
        for (int k = (int)threadIdx.x; k * BS < tokens; k += kListThreads) {
            const int64_t at = (int64_t)phys[k] * p.scale_stride + kvh;
            ks_s[k] = p.k_scales[at];
            vs_s[k] = p.v_scales[at] * (1.f / ListEngine<T, D, BS>::kLift);   // exact: a power of two
        }
    }
    eng.init(p);
    if constexpr (C::Q8)
        __syncthreads();   // every thread's scales

    int failed_at = -1;
    for (int i = 0; i < my_n; ++i) {
        const int st = i % S;
        // the warp gives up as one: its products and shuffles need every lane
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[st], (uint32_t)((i / S) & 1)))) {
            failed_at = i;
            break;
        }
        const int t0 = (warp + i * NW) * TILE;
        const int nvalid = min(TILE, tokens - t0);
        const uint32_t kbase = smem_u32(stages + st * C::STAGE_BYTES);
        float ks0 = 1.f, ks1 = 1.f, vs0 = 1.f, vs1 = 1.f;
        if constexpr (C::Q8) {
            const int e = t0 / BS;
            ks0 = ks1 = ks_s[e];
            vs0 = vs1 = vs_s[e];
            if constexpr (BS == 8) {
                // a second block that is not there weighs nothing
                ks1 = nvalid > 8 ? ks_s[e + 1] : 0.f;
                vs1 = nvalid > 8 ? vs_s[e + 1] : 0.f;
            }
        }
        eng.tile(kbase, kbase + C::TILE_BYTES, nvalid, lane, ks0, ks1, vs0, vs1);
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

// The log-sum-exp merge of the np partials of every (sequence, head),
// launched as a programmatic dependent of the partitions' kernel.  A head's
// partials are dealt to `per_head` warps (a power of two up to 8) of one CTA;
// a lane holds D / 32 dimensions.  A sum of -1 marks a refused partition: the
// row is zero.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
list_merge_kernel(const __grid_constant__ ListParams p, int per_head)
{
    constexpr int N = D / 32, U = 8;
    using V = typename std::conditional<N == 4, float4, float2>::type;
    __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
    __shared__ int s_bad[kMergeWarps];
    __shared__ V s_acc[kMergeWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t heads = (int64_t)p.num_seqs * p.num_kv_heads * p.group;
    const int64_t sh = ((int64_t)blockIdx.x * kMergeWarps + warp) / per_head;
    const int first = warp % per_head;
    const bool live = sh < heads;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml) + (live ? sh : 0) * p.np;
    const V *acc = reinterpret_cast<const V *>(p.ws_acc + (live ? sh : 0) * p.np * D) + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float mx = -INFINITY, den = 0.f, num[N];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
        num[i] = 0.f;
    for (int k0 = first; live && k0 < p.np; k0 += per_head * U) {
        float2 t[U];
        V a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // every load leaves before one is used: an empty partial's sums
            // of values are read too, and dropped
            const int k = k0 + u * per_head;
            t[u] = make_float2(-INFINITY, 0.f);
            a[u] = V{};
            if (k < p.np) {
                t[u] = __ldcg(ml + k);
                a[u] = __ldcg(acc + (int64_t)k * 32);
            }
        }
        float mn = mx;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mn = fmaxf(mn, t[u].x);
            bad |= t[u].y < 0.f;
        }
        const float ref = reference_of(mn);
        const float f0 = exp2f(mx - ref);
        den *= f0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            num[i] *= f0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t[u].y != 0.f) {
                const float f = exp2f(t[u].x - ref);
                den += f * t[u].y;
                num[0] += f * a[u].x;
                num[1] += f * a[u].y;
                if constexpr (N == 4) {
                    num[2] += f * a[u].z;
                    num[3] += f * a[u].w;
                }
            }
        }
        mx = mn;
    }
    if (per_head > 1) {
        V v;
        v.x = num[0];
        v.y = num[1];
        if constexpr (N == 4) {
            v.z = num[2];
            v.w = num[3];
        }
        s_acc[warp][lane] = v;
        if (lane == 0) {
            s_m[warp] = mx;
            s_l[warp] = den;
            s_bad[warp] = bad;
        }
        __syncthreads();
        if (first != 0)
            return;
        float M = -INFINITY;
        for (int w = warp; w < warp + per_head; ++w) {
            M = fmaxf(M, s_m[w]);
            bad |= s_bad[w] != 0;
        }
        const float ref = reference_of(M);
        den = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            num[i] = 0.f;
        for (int w = warp; w < warp + per_head; ++w) {
            const float f = exp2f(s_m[w] - ref);
            const V x = s_acc[w][lane];
            den += f * s_l[w];
            num[0] += f * x.x;
            num[1] += f * x.y;
            if constexpr (N == 4) {
                num[2] += f * x.z;
                num[3] += f * x.w;
            }
        }
    }
    if (!live)
        return;
    const bool zero = bad || den == 0.f;
    const float inv = 1.f / den;
    const int64_t at = sh * D + lane * N;
    if constexpr (N == 4)
        store_out4(p.out, p.out_dtype, at, zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                : make_float4(num[0] * inv, num[1] * inv, num[2] * inv, num[3] * inv));
    else {
        store_out(p.out, p.out_dtype, at, zero ? 0.f : num[0] * inv);
        store_out(p.out, p.out_dtype, at + 1, zero ? 0.f : num[1] * inv);
    }
}

}  // namespace pkv
