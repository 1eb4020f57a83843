// q4_cache.cuh -- the 4-bit cache: its format, reshape_and_cache_q4_kernel (new
// tokens' K and V into it) and gather_cache_q4_kernel (rows back as numbers).
//
// The cache.  A group is 64 neighbouring dimensions of one token's row of one
// kv head.  It has a scale s and a minimum m of the model's 16-bit type and 64
// codes u of 4 bits; a number is s u + m.  With m the group's smallest value,
// which the type holds exactly, and s a fifteenth of its range, a number is off
// by at most about s / 2.  A scale per row and group needs nothing of the rows
// around it: a row is written once and never again, whatever comes into its
// block later (one scale for a whole block would have to grow with its rows,
// and 4 bits have no room for coding a row twice).
//
// A block's rows of one kv head are a record of block_size * (D / 2 + D / 16)
// bytes: the rows' codes, then their (s, m) pairs.  One bulk copy fetches it.
// The codes' order inside is that in which attention's matrix fragments want
// them: see Q4Row.
//
// What bounds them, at large sizes: HBM.  130K tokens of 8 heads of 128 are read
// back in 105 us (6.5 TB/s, 97 % of a copy's rate), prompts of 12.0K tokens of 40
// heads written in 58.8 (5.35 TB/s, 80 %: some 180 instructions for a warp's four
// rows keep issue at 70 %) and read in 50.6 (93 %).  What it took: rows of several
// tokens in flight in a thread (one row a thread, a CTA for every 16 rows: 207 us
// and 180 for both), addresses by additions, no 64-bit division.  A decode step's
// call is a launch and a chain of loads: 2.6 us each.
#pragma once

#include "q8_cache.cuh"

namespace pkv {

constexpr int kQ4Group = 64;      // dimensions that share a scale and a minimum

// A row of codes: D / 8 words of eight, word G i + j (G = D / 64 groups) holds
// dimensions 64 j + 8 i .. + 7, the lowest in the lowest bits.  So any 8 or 16
// bytes of a row hold equal parts of its groups, and a thread that reads them
// can feed products that keep to one group.  Rows fill lines of 128 bytes, and
// a line's 16-byte pieces are exchanged (piece p of line n is stored at
// p ^ x(n)) such that reads of one row by four threads and reads of 16 rows at
// the same place meet no bank of shared memory twice.
template <int D> struct Q4Row {
    static constexpr int GROUPS = D / kQ4Group;
    static constexpr int CODES = D / 2;            // bytes of codes
    static constexpr int PAIRS = GROUPS * 4;       // bytes of (scale, minimum) pairs

    // Byte offset of word w of row r in a record.
    __host__ __device__ __forceinline__ static int word(int r, int w)
    {
        const int at = r * CODES + w * 4, line = at >> 7;
        const int x = D == 128 ? line & 7 : (line & 1) << 2 | (line & 2);
        return at ^ (x << 4);
    }
    // Byte offset of group j's pair of row r.
    template <int BS> __host__ __device__ __forceinline__ static int pair(int r, int j)
    {
        return BS * CODES + r * PAIRS + j * 4;
    }
    template <int BS> static constexpr int record = BS * (CODES + PAIRS);
};

struct Q4RowsParams {
    const void *key;              // write: read from; gather: written to
    const void *value;
    uint8_t *k_cache;
    uint8_t *v_cache;
    const int64_t *slot_mapping;
    uint32_t *status;
    int64_t key_stride, value_stride;   // elements between two tokens
    int64_t num_blocks;
    int num_tokens, num_kv_heads;
    int tokens_per_cta;
    int step;                     // tokens whose rows a CTA takes at a time
};

constexpr int kQ4Threads = 256;

// Which rows a thread of a CTA works on, LANES threads to a row: always the same
// row (K's heads, then V's) of `left` tokens first, first + step, ...  Where a
// token has fewer rows than a CTA takes at a time, the CTA takes several tokens
// (`step`); where it has more, blockIdx.y tells the rows.
template <int LANES> struct Q4Rows {
    static constexpr int AT_ONCE = kQ4Threads / LANES;
    int head, step, left;
    int64_t first;
    bool is_v;
    __device__ __forceinline__ explicit Q4Rows(const Q4RowsParams &p) : step(p.step)
    {
        const int rows = 2 * p.num_kv_heads, mine = threadIdx.x / LANES;
        const int token = step > 1 ? mine / rows : 0;
        const int row = step > 1 ? mine - token * rows : mine + (int)blockIdx.y * AT_ONCE;
        is_v = row >= p.num_kv_heads;
        head = is_v ? row - p.num_kv_heads : row;
        const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
        first = t0 + token;
        const int here = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - t0) - token;
        left = row < rows && token < step && here > 0 ? (step > 1 ? (here + step - 1) / step : here) : 0;
    }
};

// A slot's record: `base` is the first block's record of the head, blocks are
// `apart` bytes apart.  Null for padding and for a slot out of range (reported).
template <int D, int BS>
__device__ __forceinline__ uint8_t *q4_record(const Q4RowsParams &p, uint8_t *base, uint32_t apart, int64_t slot, int &row)
{
    row = (int)slot & (BS - 1);
    if ((uint64_t)slot < (uint64_t)(p.num_blocks * BS))
        return base + (uint64_t)(uint32_t)(slot / BS) * apart;
    if (slot >= 0)
        report(p.status, PKV_DEV_BAD_SLOT);
    return nullptr;
}

// Eight values of 32-bit words (pairs of T) -> eight codes; mh = m / 2, c = 2 / s.
//
// u = min(15, rint(q)), q = (x - m) / s taken as (x / 2 - m / 2) * c, which
// overflows nowhere.  q is first rounded to 16 binary places by an addition of
// 192, then to a whole number by one of 1.5 * 2^23: c is rounded, and a
// quotient halfway between two codes, common among 16-bit numbers, has to come
// out as one (it goes to the even code).  The codes stand in the sums' lowest
// bits; the sums' other bits add up to kCodesOffset.  CAP: quotients may pass
// 15.5, which takes a scale that was rounded by more than a thirtieth of itself:
// one of f16's subnormal numbers.
constexpr uint32_t kCodesOffset = 0x4b400000u * 0x11111111u;
template <typename T, bool CAP>
__device__ __forceinline__ uint32_t q4_codes(const uint32_t *in, float mh, float c)
{
    uint32_t w = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        float2 f = Unpack<T>::pair(in[i]);
        f = ffma2(f, make_float2(0.5f, 0.5f), make_float2(-mh, -mh));
        f = ffma2(f, make_float2(c, c), make_float2(192.f, 192.f));
        f = __fadd2_rn(f, make_float2(12582720.f, 12582720.f));
        if (CAP) {
            f.x = fminf(f.x, 12582927.f);
            f.y = fminf(f.y, 12582927.f);
        }
        w = (w << 4) + __float_as_uint(f.y);
        w = (w << 4) + __float_as_uint(f.x);
    }
    return w - kCodesOffset;
}

__device__ __forceinline__ uint16_t half_bits(__half x) { return __half_as_ushort(x); }
__device__ __forceinline__ uint16_t half_bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
template <typename T> __device__ __forceinline__ T round16(float x);
template <> __device__ __forceinline__ __half round16<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 round16<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// R / 7.5, rounded to nearest: the product with the rounded reciprocal, corrected
// by its remainder's (P. Markstein, IBM J. Res. Dev. 34, 1990: with a correctly
// rounded reciprocal that is the correctly rounded quotient).  Remainders of
// smaller numbers would not be exact.
__device__ __forceinline__ float q4_scale(float range)
{
    const float c = 1.f / 7.5f;
    const float q = range * c;
    return range > 0x1p-90f ? fmaf(fmaf(-7.5f, q, range), c, q) : range / 7.5f;
}

// New tokens' rows into the cache.  A thread holds 16 dimensions of a row, the
// four threads of a group find its range by two exchanges; two threads of the
// two groups of a row swap a word, so that each stores eight bytes.  Rows leave
// memory before their slots are known, kQ4WriteAhead at a time.
constexpr int kQ4WriteAhead = 2;

template <typename T, int D, int BS> struct Q4Writer {
    using R = Q4Row<D>;
    using V = typename Pair16<T>::V;
    static constexpr int LPR = D / 16;
    const Q4RowsParams &p;
    uint8_t *base;
    uint32_t apart;
    int c, j, first;   // place in the group, group, first of the words that this thread stores

    // Every thread of a warp calls it.
    __device__ __forceinline__ void write(uint4 x0, uint4 x1, int64_t slot) const
    {
        // the smallest value and the smallest of the negated ones, in one word
        const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        V lo = as_pair<T>(w[0]), hi = lo;
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = __hmin2_nan(lo, as_pair<T>(w[i]));
            hi = __hmax2_nan(hi, as_pair<T>(w[i]));
        }
        const uint32_t a = as_word(lo), b = as_word(__hneg2(hi));
        V both = __hmin2_nan(as_pair<T>(__byte_perm(a, b, 0x5410)), as_pair<T>(__byte_perm(a, b, 0x7632)));
        both = __hmin2_nan(both, as_pair<T>(__shfl_xor_sync(0xffffffffu, as_word(both), 1)));
        both = __hmin2_nan(both, as_pair<T>(__shfl_xor_sync(0xffffffffu, as_word(both), 2)));
        const float2 ends = Unpack<T>::pair(as_word(both));
        const float mh = 0.5f * ends.x;
        T s = round16<T>(q4_scale(fmaf(-0.5f, ends.y, -mh)));
        uint32_t m = as_word(both) & 0xffffu;
        if (to_float(s) < 1.17549435e-38f)        // 2 / s would not be a number
            s = round16<T>(0.f);
        if (!(fmaxf(fabsf(ends.x), fabsf(ends.y)) < INFINITY) || ends.x != ends.x || ends.y != ends.y) {
            // a NaN or an infinity among the values: the group's numbers are NaN
            s = round16<T>(NAN);
            m = half_bits(s);
        }
        const float s32 = to_float(s);
        const float inv = s32 > 0.f ? 2.f * __frcp_rn(s32) : 0.f;   // 2 / s, rounded once
        uint2 codes = make_uint2(q4_codes<T, false>(w, mh, inv), q4_codes<T, false>(w + 4, mh, inv));
        if constexpr (std::is_same<T, __half>::value) {
            if (__any_sync(0xffffffffu, s32 > 0.f && s32 < 6.103515625e-05f))
                codes = make_uint2(q4_codes<T, true>(w, mh, inv), q4_codes<T, true>(w + 4, mh, inv));
        }
        if constexpr (R::GROUPS == 2) {
            // words 4 c + j and 4 c + 2 + j -> 4 c + 2 j and the next
            const uint32_t other = __shfl_xor_sync(0xffffffffu, j ? codes.x : codes.y, 4);
            codes = j ? make_uint2(other, codes.y) : make_uint2(codes.x, other);
        }
        int row;
        uint8_t *rec = q4_record<D, BS>(p, base, apart, slot, row);
        if (rec) {
            *reinterpret_cast<uint2 *>(rec + R::word(row, first)) = codes;
            if (c == 0)
                *reinterpret_cast<uint32_t *>(rec + R::template pair<BS>(row, j)) = half_bits(s) | m << 16;
        }
    }
};

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kQ4Threads)
reshape_and_cache_q4_kernel(const __grid_constant__ Q4RowsParams p)
{
    using R = Q4Row<D>;
    using W = Q4Writer<T, D, BS>;
    constexpr int U = kQ4WriteAhead;
    const Q4Rows<W::LPR> mine(p);
    const int l = threadIdx.x % W::LPR, c = l & 3, j = l >> 2;
    const W writer{p, (mine.is_v ? p.v_cache : p.k_cache) + mine.head * R::template record<BS>,
                   (uint32_t)p.num_kv_heads * R::template record<BS>, c, j, R::GROUPS == 2 ? 4 * c + 2 * j : 2 * c};
    const int64_t stride = mine.is_v ? p.value_stride : p.key_stride, step = stride * mine.step;
    const T *src = static_cast<const T *>(mine.is_v ? p.value : p.key) + mine.first * stride + mine.head * D + 16 * l;
    const int64_t *at = p.slot_mapping + mine.first;
    int left = mine.left;
    wait_for_stream();
    for (; __all_sync(0xffffffffu, left >= U); left -= U) {
        uint4 x[U][2];
        int64_t slot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u][0] = __ldcs(reinterpret_cast<const uint4 *>(src));
            x[u][1] = __ldcs(reinterpret_cast<const uint4 *>(src) + 1);
            slot[u] = *at;
            src += step;
            at += mine.step;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            writer.write(x[u][0], x[u][1], slot[u]);
    }
    // threads without a row of their own take part in the exchanges
    for (; __any_sync(0xffffffffu, left > 0); --left) {
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        int64_t slot = -1;
        if (left > 0) {
            x[0] = __ldcs(reinterpret_cast<const uint4 *>(src));
            x[1] = __ldcs(reinterpret_cast<const uint4 *>(src) + 1);
            slot = *at;
        }
        writer.write(x[0], x[1], slot);
        src += step;
        at += mine.step;
    }
}

// Two codes as numbers of type T: the word's bits 0..3 and 16..19.  The codes
// become the last bits of a power of two's mantissa, which is taken off again.
template <typename T> __device__ __forceinline__ typename Pair16<T>::V q4_pair(uint32_t w);
template <> __device__ __forceinline__ __half2 q4_pair<__half>(uint32_t w)
{
    return __hsub2(as_pair<__half>((w & 0x000f000fu) | 0x64006400u), __float2half2_rn(1024.f));
}
template <> __device__ __forceinline__ __nv_bfloat162 q4_pair<__nv_bfloat16>(uint32_t w)
{
    return __hsub2(as_pair<__nv_bfloat16>((w & 0x000f000fu) | 0x43004300u), __float2bfloat162_rn(128.f));
}

// Rows back as numbers, O: T or float.  A thread has a word of codes (eight
// neighbouring dimensions) of each group, of kQ4ReadAhead rows at a time.  In
// T's own arithmetic s u + m is rounded once.
constexpr int kQ4ReadAhead = 4;

template <typename T, typename O, int D, int BS> struct Q4Reader {
    using R = Q4Row<D>;
    using V = typename Pair16<T>::V;
    static constexpr int LPR = 8, NG = R::GROUPS;
    using Words = typename std::conditional<NG == 2, uint2, uint32_t>::type;
    struct Row {
        Words codes, pairs;
        bool there;
    };
    const Q4RowsParams &p;
    const uint8_t *base;
    uint32_t apart;
    int i;

    __device__ __forceinline__ Row read(int64_t slot) const
    {
        Row r{};
        int row;
        const uint8_t *rec = q4_record<D, BS>(p, const_cast<uint8_t *>(base), apart, slot, row);
        r.there = rec != nullptr;
        if (r.there) {
            r.codes = *reinterpret_cast<const Words *>(rec + R::word(row, NG * i));
            r.pairs = *reinterpret_cast<const Words *>(rec + R::template pair<BS>(row, 0));
        }
        return r;
    }

    __device__ __forceinline__ static void group(uint32_t w, uint32_t sm, O *to)
    {
        if constexpr (std::is_same<O, float>::value) {
            const float2 f = Unpack<T>::pair(sm);
            float o[8];
#pragma unroll
            for (int n = 0; n < 8; ++n)
                o[n] = fmaf((float)((w >> (4 * n)) & 15u), f.x, f.y);
            __stcs(reinterpret_cast<float4 *>(to), make_float4(o[0], o[1], o[2], o[3]));
            __stcs(reinterpret_cast<float4 *>(to) + 1, make_float4(o[4], o[5], o[6], o[7]));
        } else {
            const V s = as_pair<T>(__byte_perm(sm, 0, 0x1010)), m = as_pair<T>(__byte_perm(sm, 0, 0x3232));
            uint32_t v[4];   // dimensions n, n + 4
#pragma unroll
            for (int n = 0; n < 4; ++n)
                v[n] = as_word(__hfma2(q4_pair<T>(w >> (4 * n)), s, m));
            __stcs(reinterpret_cast<uint4 *>(to), make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                                                             __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)));
        }
    }

    __device__ __forceinline__ static void write(const Row &r, O *to)
    {
        if (!r.there)
            return;
        if constexpr (NG == 2) {
            group(r.codes.x, r.pairs.x, to);
            group(r.codes.y, r.pairs.y, to + kQ4Group);
        } else {
            group(r.codes, r.pairs, to);
        }
    }
};

template <typename T, typename O, int D, int BS>
__global__ void __launch_bounds__(kQ4Threads)
gather_cache_q4_kernel(const __grid_constant__ Q4RowsParams p)
{
    using R = Q4Row<D>;
    using G = Q4Reader<T, O, D, BS>;
    constexpr int U = kQ4ReadAhead;
    const Q4Rows<G::LPR> mine(p);
    const G reader{p, (mine.is_v ? p.v_cache : p.k_cache) + mine.head * R::template record<BS>,
                   (uint32_t)p.num_kv_heads * R::template record<BS>, (int)threadIdx.x % G::LPR};
    const int64_t stride = mine.is_v ? p.value_stride : p.key_stride, step = stride * mine.step;
    O *dst = static_cast<O *>(const_cast<void *>(mine.is_v ? p.value : p.key)) + mine.first * stride + mine.head * D + 8 * reader.i;
    const int64_t *at = p.slot_mapping + mine.first;
    int left = mine.left;
    wait_for_stream();
    auto batch = [&](auto all) {
        int64_t slot[U];
        typename G::Row r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            slot[u] = decltype(all)::value || u < left ? at[(int64_t)u * mine.step] : -1;
#pragma unroll
        for (int u = 0; u < U; ++u)
            r[u] = reader.read(slot[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            G::write(r[u], dst + u * step);
        at += U * (int64_t)mine.step;
        dst += U * step;
    };
    for (; left >= U; left -= U)
        batch(std::true_type{});
    if (left > 1)
        batch(std::false_type{});
    else if (left == 1)
        G::write(reader.read(*at), dst);
}

}  // namespace pkv
