// q4_cache.cu -- host side of reshape_and_cache_q4 and gather_cache_q4: checks
// of arguments and the compile-time dispatch over type, head_dim and block size.
#include <cuda_runtime.h>

#include "pkv_host.cuh"
#include "q4_cache.cuh"

namespace pkv {
namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What both calls ask of their arguments; PKV_OK or an error.
int check_rows(const Q4RowsParams &p, int head_dim, int block_size, int elem_bytes)
{
    if (p.num_tokens < 0 || p.num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || p.num_blocks <= 0 ||
        p.num_blocks > INT32_MAX)
        return PKV_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 8 && block_size != 16 && block_size != 32) ||
        p.num_kv_heads > 65535)
        return PKV_EUNSUPPORTED;
    const int64_t row = (int64_t)p.num_kv_heads * head_dim;
    // tokens may lie apart, as in a slice of a fused projection's output
    if (p.num_tokens > 1 && (p.key_stride < row || p.value_stride < row || p.key_stride > INT64_MAX / 4 / INT32_MAX ||
                             p.value_stride > INT64_MAX / 4 / INT32_MAX || p.key_stride * elem_bytes % 16 ||
                             p.value_stride * elem_bytes % 16))
        return PKV_EINVAL;
    if (p.num_tokens == 0)
        return PKV_OK;
    if (!p.key || !p.value || !p.k_cache || !p.v_cache || !p.slot_mapping || !aligned(p.key, 16) || !aligned(p.value, 16) ||
        !aligned(p.k_cache, 16) || !aligned(p.v_cache, 16) || !aligned(p.slot_mapping, 8))
        return PKV_EINVAL;
    return PKV_OK;
}

// Tokens per CTA: what it takes at a time (its rows over the token's, at least
// one token), then times two while that leaves two CTAs per SM, until a thread
// has the `ahead` rows that it holds in flight; further while it leaves 16.  (us,
// write and read: 8000 tokens of 8 heads of 128 10.2 and 6.9, with 16 CTAs per SM
// from the start 13.0 and 9.4; prompts of 12.0K tokens of 40 heads 58.7 and 50.4
// either way, 63.8 and 55.0 where four CTAs per SM are enough throughout.)
template <typename K>
int launch(K kern, Q4RowsParams p, int rows_per_cta, int ahead, cudaStream_t stream)
{
    const int rows = 2 * p.num_kv_heads;
    const int64_t y = ((int64_t)rows + rows_per_cta - 1) / rows_per_cta;
    const int64_t sms = device_sm_count();
    p.step = rows < rows_per_cta ? rows_per_cta / rows : 1;
    int64_t tokens = p.step;
    while (tokens < p.num_tokens && (p.num_tokens / (2 * tokens) + 1) * y > (2 * tokens <= (int64_t)ahead * p.step ? 2 : 16) * sms)
        tokens *= 2;
    p.tokens_per_cta = (int)(tokens < p.num_tokens ? tokens : p.num_tokens);
    const unsigned x = (unsigned)((p.num_tokens + (int64_t)p.tokens_per_cta - 1) / p.tokens_per_cta);
    return launch_pdl(kern, dim3(x, (unsigned)y), dim3(kQ4Threads), 0, stream, p);
}

template <typename T, int D>
int write_block(const Q4RowsParams &p, int bs, cudaStream_t s)
{
    constexpr int rows = kQ4Threads / Q4Writer<T, D, 8>::LPR;
    switch (bs) {
    case 8: return launch(reshape_and_cache_q4_kernel<T, D, 8>, p, rows, kQ4WriteAhead, s);
    case 16: return launch(reshape_and_cache_q4_kernel<T, D, 16>, p, rows, kQ4WriteAhead, s);
    default: return launch(reshape_and_cache_q4_kernel<T, D, 32>, p, rows, kQ4WriteAhead, s);
    }
}

template <typename T, typename O, int D>
int gather_block(const Q4RowsParams &p, int bs, cudaStream_t s)
{
    constexpr int rows = kQ4Threads / Q4Reader<T, O, D, 8>::LPR;
    switch (bs) {
    case 8: return launch(gather_cache_q4_kernel<T, O, D, 8>, p, rows, kQ4ReadAhead, s);
    case 16: return launch(gather_cache_q4_kernel<T, O, D, 16>, p, rows, kQ4ReadAhead, s);
    default: return launch(gather_cache_q4_kernel<T, O, D, 32>, p, rows, kQ4ReadAhead, s);
    }
}

template <typename T, typename O>
int gather_dim(const Q4RowsParams &p, int head_dim, int bs, cudaStream_t s)
{
    return head_dim == 64 ? gather_block<T, O, 64>(p, bs, s) : gather_block<T, O, 128>(p, bs, s);
}

Q4RowsParams rows_params(const void *key, int64_t key_stride, const void *value, int64_t value_stride, void *k_cache,
                         void *v_cache, const int64_t *slot_mapping, int num_tokens, int num_kv_heads, int64_t num_blocks,
                         uint32_t *device_status)
{
    Q4RowsParams p;
    p.key = key;
    p.value = value;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.slot_mapping = slot_mapping;
    p.status = device_status;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.num_blocks = num_blocks;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.tokens_per_cta = p.step = 1;
    return p;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_reshape_and_cache_q4(const void *key, int64_t key_stride, const void *value, int64_t value_stride, int dtype,
                             void *k_cache, void *v_cache, const int64_t *slot_mapping, int num_tokens, int num_kv_heads,
                             int head_dim, int block_size, int64_t num_blocks, uint32_t *device_status, void *stream)
{
    if (dtype < PKV_F32 || dtype > PKV_BF16)
        return PKV_EINVAL;
    const Q4RowsParams p = rows_params(key, key_stride, value, value_stride, k_cache, v_cache, slot_mapping, num_tokens,
                                       num_kv_heads, num_blocks, device_status);
    const int rc = check_rows(p, head_dim, block_size, 2);
    if (rc)
        return rc;
    if (dtype == PKV_F32)
        return PKV_EUNSUPPORTED;
    if (num_tokens == 0)
        return PKV_OK;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_F16)
        return head_dim == 64 ? write_block<__half, 64>(p, block_size, s) : write_block<__half, 128>(p, block_size, s);
    return head_dim == 64 ? write_block<__nv_bfloat16, 64>(p, block_size, s)
                          : write_block<__nv_bfloat16, 128>(p, block_size, s);
}

int pkv_gather_cache_q4(void *key, int64_t key_stride, void *value, int64_t value_stride, int out_dtype,
                        const void *k_cache, const void *v_cache, int dtype, const int64_t *slot_mapping, int num_tokens,
                        int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, uint32_t *device_status,
                        void *stream)
{
    if (dtype < PKV_F32 || dtype > PKV_BF16 || out_dtype < PKV_F32 || out_dtype > PKV_BF16)
        return PKV_EINVAL;
    const Q4RowsParams p = rows_params(key, key_stride, value, value_stride, const_cast<void *>(k_cache),
                                       const_cast<void *>(v_cache), slot_mapping, num_tokens, num_kv_heads, num_blocks,
                                       device_status);
    const int rc = check_rows(p, head_dim, block_size, out_dtype == PKV_F32 ? 4 : 2);
    if (rc)
        return rc;
    if (dtype == PKV_F32 || (out_dtype != dtype && out_dtype != PKV_F32))
        return PKV_EUNSUPPORTED;
    if (num_tokens == 0)
        return PKV_OK;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_F16)
        return out_dtype == PKV_F32 ? gather_dim<__half, float>(p, head_dim, block_size, s)
                                    : gather_dim<__half, __half>(p, head_dim, block_size, s);
    return out_dtype == PKV_F32 ? gather_dim<__nv_bfloat16, float>(p, head_dim, block_size, s)
                                : gather_dim<__nv_bfloat16, __nv_bfloat16>(p, head_dim, block_size, s);
}

}  // extern "C"
