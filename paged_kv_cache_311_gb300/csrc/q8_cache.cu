// q8_cache.cu -- host side of append_cache_q8 and summarize_blocks: checks of
// arguments and the compile-time dispatch over type, head_dim and block size.
#include <cuda_runtime.h>

#include "pkv_host.cuh"
#include "q8_cache.cuh"

namespace pkv {
namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What both calls ask of the sizes; PKV_OK or an error.
int check_sizes(int num_seqs, int num_tokens, int num_kv_heads, int head_dim, int block_size,
                int64_t num_blocks, int max_blocks_per_seq, const void *query_start)
{
    if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0)
        return PKV_EINVAL;
    if (!query_start && num_tokens != num_seqs)
        return PKV_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 8 && block_size != 16 && block_size != 32) ||
        num_kv_heads > 65535 || (int64_t)max_blocks_per_seq * block_size > INT32_MAX)
        return PKV_EUNSUPPORTED;
    return PKV_OK;
}

// Tokens per CTA: one while the grid has fewer than four CTAs per SM (a decode
// step's tokens all lead a block: their heads then spread over blockIdx.y, a
// warp each), else as many as leave it four, up to kUnitTokens, a leader's
// heads dealt four to a warp.  (Prompts of 12.8K tokens of 40 heads: 65 us; with
// eight CTAs per SM and all heads in one CTA 70, with one head to a warp 72.)
//
// The carveout between L1 and shared memory is left to the driver.  The
// largest shared memory, which the library's other kernels ask for, leaves
// these too little L1 for the loads that they have in flight (append of those
// prompts 65.8 -> 81.5 us, summaries of prompts of 4K to 16K tokens 39.5 ->
// 44.4) and saves nothing where they run between the others: a step of append,
// summaries, selection and attention takes 17.05 us for one request, 21.1 for
// 8, 62.9 for 32, either way.
template <typename K, typename P>
int launch(K kern, P p, int units, cudaStream_t stream)
{
    const int most = p.num_tokens / (4 * device_sm_count());
    p.tokens_per_cta = 1;
    while (p.tokens_per_cta * 2 <= most && p.tokens_per_cta < kUnitTokens)
        p.tokens_per_cta *= 2;
    const int per_cta = kUnitWarps * (p.tokens_per_cta == 1 ? 1 : 4);
    const unsigned x = (unsigned)(((int64_t)p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta);
    return launch_pdl(kern, dim3(x, (unsigned)((units + per_cta - 1) / per_cta)), dim3(kUnitThreads), 0, stream, p);
}

template <typename T, int D>
int append_block(const AppendParams &p, int bs, cudaStream_t s)
{
    const int units = 2 * p.num_kv_heads;
    switch (bs) {
    case 8: return launch(append_cache_q8_kernel<T, D, 8>, p, units, s);
    case 16: return launch(append_cache_q8_kernel<T, D, 16>, p, units, s);
    default: return launch(append_cache_q8_kernel<T, D, 32>, p, units, s);
    }
}

template <typename T, int D, bool Q8>
int summarize_block(const SummarizeParams &p, int bs, cudaStream_t s)
{
    switch (bs) {
    case 8: return launch(summarize_blocks_kernel<T, D, 8, Q8>, p, p.num_kv_heads, s);
    case 16: return launch(summarize_blocks_kernel<T, D, 16, Q8>, p, p.num_kv_heads, s);
    default: return launch(summarize_blocks_kernel<T, D, 32, Q8>, p, p.num_kv_heads, s);
    }
}

template <typename T>
int summarize_type(const SummarizeParams &p, int head_dim, int bs, cudaStream_t s)
{
    if (p.k_scales)
        return head_dim == 64 ? summarize_block<T, 64, true>(p, bs, s) : summarize_block<T, 128, true>(p, bs, s);
    return head_dim == 64 ? summarize_block<T, 64, false>(p, bs, s) : summarize_block<T, 128, false>(p, bs, s);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_append_cache_q8(const void *key, const void *value, int dtype, void *k_cache, void *v_cache,
                        float *k_scales, float *v_scales, const int32_t *block_tables,
                        int max_blocks_per_seq, const int32_t *context_lens,
                        const int32_t *query_start, int num_seqs, int num_tokens, int num_kv_heads,
                        int head_dim, int block_size, int64_t num_blocks, uint32_t *device_status,
                        void *stream)
{
    if (dtype != PKV_F32 && dtype != PKV_F16 && dtype != PKV_BF16)
        return PKV_EINVAL;
    const int rc = check_sizes(num_seqs, num_tokens, num_kv_heads, head_dim, block_size, num_blocks,
                               max_blocks_per_seq, query_start);
    if (rc)
        return rc;
    if (dtype == PKV_F32)
        return PKV_EUNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0)
        return PKV_OK;
    if (!key || !value || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !context_lens)
        return PKV_EINVAL;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(query_start, 4))
        return PKV_EINVAL;
    AppendParams p;
    p.key = key;
    p.value = value;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.status = device_status;
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.scale_stride = q8_scale_stride(num_kv_heads);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_F16)
        return head_dim == 64 ? append_block<__half, 64>(p, block_size, s) : append_block<__half, 128>(p, block_size, s);
    return head_dim == 64 ? append_block<__nv_bfloat16, 64>(p, block_size, s)
                          : append_block<__nv_bfloat16, 128>(p, block_size, s);
}

int pkv_summarize_blocks(const void *k_cache, int cache_dtype, const float *k_scales, void *summaries,
                         int summary_dtype, const int32_t *block_tables, int max_blocks_per_seq,
                         const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                         int num_tokens, int num_kv_heads, int head_dim, int block_size,
                         int64_t num_blocks, uint32_t *device_status, void *stream)
{
    if (cache_dtype < PKV_F32 || cache_dtype > PKV_E4M3 || summary_dtype < PKV_F32 || summary_dtype > PKV_BF16)
        return PKV_EINVAL;
    const int rc = check_sizes(num_seqs, num_tokens, num_kv_heads, head_dim, block_size, num_blocks,
                               max_blocks_per_seq, query_start);
    if (rc)
        return rc;
    // an e4m3 value times a power of two is a bfloat16; a 16-bit key is its own type
    if (cache_dtype == PKV_F32 || summary_dtype != (cache_dtype == PKV_E4M3 ? PKV_BF16 : cache_dtype))
        return PKV_EUNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0)
        return PKV_OK;
    if (!k_cache || !summaries || !block_tables || !context_lens || (cache_dtype == PKV_E4M3) != (k_scales != nullptr))
        return PKV_EINVAL;
    if (!aligned(k_cache, 16) || !aligned(summaries, 16) || !aligned(k_scales, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(query_start, 4))
        return PKV_EINVAL;
    SummarizeParams p;
    p.k_cache = k_cache;
    p.k_scales = k_scales;
    p.summaries = summaries;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.status = device_status;
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.scale_stride = q8_scale_stride(num_kv_heads);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return summary_dtype == PKV_F16 ? summarize_type<__half>(p, head_dim, block_size, s)
                                    : summarize_type<__nv_bfloat16>(p, head_dim, block_size, s);
}

}  // extern "C"
