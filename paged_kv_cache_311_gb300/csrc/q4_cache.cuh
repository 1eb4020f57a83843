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
    static constexpr int WORDS = D / 8;

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
};

constexpr int kQ4Threads = 256;

// The record of kv head h in the block of a slot and the slot's row there;
// null for padding and for a slot out of range (reported).
template <int D, int BS>
__device__ __forceinline__ uint8_t *q4_record(const Q4RowsParams &p, int64_t slot, int h, bool is_v, int &row)
{
    if (slot < 0)
        return nullptr;
    if (slot >= p.num_blocks * BS) {
        report(p.status, PKV_DEV_BAD_SLOT);
        return nullptr;
    }
    row = (int)(slot % BS);
    return (is_v ? p.v_cache : p.k_cache) + (slot / BS * p.num_kv_heads + h) * Q4Row<D>::template record<BS>;
}

// Eight values of 32-bit words (pairs of T) -> eight codes; mh = m / 2, c = 2 / s.
//
// u = min(15, rint(q)), q = (x - m) / s taken as (x / 2 - m / 2) * c, which
// overflows nowhere.  q is first rounded to 16 binary places by an addition of
// 192, then to a whole number by one of 1.5 * 2^23: c is rounded, and a
// quotient halfway between two codes, common among 16-bit numbers, has to come
// out as one (it goes to the even code).  The codes stand in the sums' lowest
// bits; the sums' other bits add up to kCodesOffset.
constexpr uint32_t kCodesOffset = 0x4b400000u * 0x11111111u;
template <typename T>
__device__ __forceinline__ uint32_t q4_codes(uint4 x, float mh, float c)
{
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t w = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float2 f = Unpack<T>::pair(in[i]);
        const float a = fmaf(fmaf(f.x, 0.5f, -mh), c, 192.f) + 12582720.f;
        const float b = fmaf(fmaf(f.y, 0.5f, -mh), c, 192.f) + 12582720.f;
        w = (w << 4) + __float_as_uint(fminf(b, 12582927.f));
        w = (w << 4) + __float_as_uint(fminf(a, 12582927.f));
    }
    return w - kCodesOffset;
}

__device__ __forceinline__ uint16_t half_bits(__half x) { return __half_as_ushort(x); }
__device__ __forceinline__ uint16_t half_bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
template <typename T> __device__ __forceinline__ T round16(float x);
template <> __device__ __forceinline__ __half round16<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 round16<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// New tokens' rows into the cache.  A thread holds 16 dimensions of a row, the
// four threads of a group find its range by two exchanges; two threads of the
// two groups of a row swap a word, so that each stores eight bytes.  A CTA
// takes the rows of K and of V of all heads of tokens_per_cta tokens.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kQ4Threads)
reshape_and_cache_q4_kernel(const __grid_constant__ Q4RowsParams p)
{
    using R = Q4Row<D>;
    using V = typename Pair16<T>::V;
    constexpr int LPR = D / 16;                   // threads of a row
    constexpr int RPC = kQ4Threads / LPR;         // rows a CTA has at a time
    const int l = threadIdx.x % LPR, c = l & 3, j = l >> 2;
    const int Hk = p.num_kv_heads;
    wait_for_stream();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
    const int rows = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - t0) * 2 * Hk;
    // every thread of a warp takes part in the exchanges
    for (int r0 = blockIdx.y * RPC; r0 < rows; r0 += gridDim.y * RPC) {
        const int r = r0 + threadIdx.x / LPR;
        const int64_t t = t0 + r / (2 * Hk);
        const int h = r % (2 * Hk) >> 1;
        const bool is_v = r & 1;
        int row = 0;
        uint8_t *rec = r < rows ? q4_record<D, BS>(p, p.slot_mapping[t], h, is_v, row) : nullptr;
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (rec) {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(is_v ? p.value : p.key) +
                                                               t * (is_v ? p.value_stride : p.key_stride) + h * D) + 2 * l;
            x[0] = src[0];
            x[1] = src[1];
        }
        // the smallest value and the smallest of the negated ones, in one word
        const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
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
        T s = round16<T>(fmaf(-0.5f, ends.y, -mh) / 7.5f);
        uint32_t m = as_word(both) & 0xffffu;
        if (to_float(s) < 1.17549435e-38f)        // 2 / s would not be a number
            s = round16<T>(0.f);
        if (!(fabsf(ends.x) < INFINITY && fabsf(ends.y) < INFINITY)) {
            // a NaN or an infinity among the values: the group's numbers are NaN
            s = round16<T>(NAN);
            m = half_bits(s);
        }
        const float s32 = to_float(s);
        const float inv = s32 > 0.f ? 2.f / s32 : 0.f;
        uint2 codes = make_uint2(q4_codes<T>(x[0], mh, inv), q4_codes<T>(x[1], mh, inv));
        if constexpr (R::GROUPS == 2) {
            // words 4 c + j and 4 c + 2 + j -> 4 c + 2 j and the next
            const uint32_t other = __shfl_xor_sync(0xffffffffu, j ? codes.x : codes.y, 4);
            codes = j ? make_uint2(other, codes.y) : make_uint2(codes.x, other);
        }
        if (rec) {
            const int first = R::GROUPS == 2 ? 4 * c + 2 * j : 2 * c;
            *reinterpret_cast<uint2 *>(rec + R::word(row, first)) = codes;
            if (c == 0)
                *reinterpret_cast<uint32_t *>(rec + R::template pair<BS>(row, j)) = half_bits(s) | m << 16;
        }
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

// Rows back as numbers, O: T or float.  A thread has a word of codes, eight
// neighbouring dimensions.  In T's own arithmetic s u + m is rounded once.
template <typename T, typename O, int D, int BS>
__global__ void __launch_bounds__(kQ4Threads)
gather_cache_q4_kernel(const __grid_constant__ Q4RowsParams p)
{
    using R = Q4Row<D>;
    using V = typename Pair16<T>::V;
    constexpr int RPC = kQ4Threads / R::WORDS;
    const int l = threadIdx.x % R::WORDS, j = l >> 3, i = l & 7;
    const int Hk = p.num_kv_heads;
    wait_for_stream();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
    const int rows = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - t0) * 2 * Hk;
    for (int r = blockIdx.y * RPC + threadIdx.x / R::WORDS; r < rows; r += gridDim.y * RPC) {
        const int64_t t = t0 + r / (2 * Hk);
        const int h = r % (2 * Hk) >> 1;
        const bool is_v = r & 1;
        int row = 0;
        const uint8_t *rec = q4_record<D, BS>(p, p.slot_mapping[t], h, is_v, row);
        if (!rec)
            continue;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + R::word(row, R::GROUPS * i + j));
        const uint32_t sm = *reinterpret_cast<const uint32_t *>(rec + R::template pair<BS>(row, j));
        O *dst = static_cast<O *>(const_cast<void *>(is_v ? p.value : p.key)) + t * (is_v ? p.value_stride : p.key_stride) + h * D + 8 * l;
        if constexpr (std::is_same<O, float>::value) {
            const float2 f = Unpack<T>::pair(sm);
            float o[8];
#pragma unroll
            for (int n = 0; n < 8; ++n)
                o[n] = fmaf((float)((w >> (4 * n)) & 15u), f.x, f.y);
            *reinterpret_cast<float4 *>(dst) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4 *>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
        } else {
            const V s = as_pair<T>(__byte_perm(sm, 0, 0x1010)), m = as_pair<T>(__byte_perm(sm, 0, 0x3232));
            uint32_t v[4];   // dimensions n, n + 4
#pragma unroll
            for (int n = 0; n < 4; ++n)
                v[n] = as_word(__hfma2(q4_pair<T>(w >> (4 * n)), s, m));
            *reinterpret_cast<uint4 *>(dst) = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                                                         __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
        }
    }
}

}  // namespace pkv
