// q4_attention.cu -- host side of paged_attention_decode_q4: checks of
// arguments, launches.
#include <cuda_runtime.h>

#include <cmath>

#include "pkv_host.cuh"
#include "q4_attention.cuh"

namespace pkv {
namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename T, int D, int BS>
int run_q4(const Q4Params &p, int num_seqs, cudaStream_t stream)
{
    return launch_pdl(q4_attention_kernel<T, D, BS>, dim3(p.num_kv_heads, num_seqs), dim3(kQ4Warps * 32), 0, stream, p);
}

template <typename T, int D>
int run_q4_block(const Q4Params &p, int num_seqs, int bs, cudaStream_t s)
{
    switch (bs) {
    case 8: return run_q4<T, D, 8>(p, num_seqs, s);
    case 16: return run_q4<T, D, 16>(p, num_seqs, s);
    default: return run_q4<T, D, 32>(p, num_seqs, s);
    }
}

template <typename T>
int run_q4_type(const Q4Params &p, int num_seqs, int head_dim, int bs, cudaStream_t s)
{
    return head_dim == 64 ? run_q4_block<T, 64>(p, num_seqs, bs, s) : run_q4_block<T, 128>(p, num_seqs, bs, s);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_paged_attention_q4_workspace_bytes(int, int, int, int, int, int, int) { return 0; }

int pkv_paged_attention_decode_q4(void *out, int out_dtype, const void *q, int64_t q_stride, int q_dtype,
                                  const void *k_cache, const void *v_cache, const int32_t *block_tables,
                                  int max_blocks_per_seq, const int32_t *context_lens, int num_seqs, int num_heads,
                                  int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                  int max_context_len, float scale, int partition_size, void *workspace,
                                  size_t workspace_bytes, uint32_t *device_status, void *stream)
{
    (void)workspace;
    (void)workspace_bytes;
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0 || block_size <= 0 ||
        max_context_len < 0 || partition_size < 0 || !std::isfinite(scale) ||
        (int64_t)max_context_len > (int64_t)max_blocks_per_seq * block_size)
        return PKV_EINVAL;
    if (out_dtype < PKV_F32 || out_dtype > PKV_BF16 || q_dtype < PKV_F32 || q_dtype > PKV_BF16)
        return PKV_EINVAL;
    if (q_dtype == PKV_F32 || (head_dim != 64 && head_dim != 128) ||
        (block_size != 8 && block_size != 16 && block_size != 32) || num_heads / num_kv_heads > kListMaxGroup ||
        num_kv_heads > 65535 || num_seqs > 65535 || (int64_t)num_seqs * num_heads > INT32_MAX / 8 ||
        max_context_len > INT32_MAX - 64)
        return PKV_EUNSUPPORTED;
    if (partition_size % 32 || partition_size % block_size)
        return PKV_EINVAL;
    if (num_seqs > 1 && (q_stride < (int64_t)num_heads * head_dim || q_stride % 8 || q_stride > INT64_MAX / 4 / 65536))
        return PKV_EINVAL;
    if (num_seqs == 0)
        return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
        return PKV_EINVAL;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_EINVAL;
    Q4Params p;
    p.out = out;
    p.q = q;
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.status = device_status;
    p.num_blocks = num_blocks;
    p.q_stride = q_stride;
    p.num_kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.out_dtype = out_dtype;
    p.qscale = scale * 1.4426950408889634f;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return q_dtype == PKV_F16 ? run_q4_type<__half>(p, num_seqs, head_dim, block_size, s)
                              : run_q4_type<__nv_bfloat16>(p, num_seqs, head_dim, block_size, s);
}

}  // extern "C"
