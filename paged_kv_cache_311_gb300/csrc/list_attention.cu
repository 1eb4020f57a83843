// list_attention.cu -- host side of paged_attention_decode_q8 and
// paged_attention_decode_selected: checks of arguments, launches.
#include <cuda_runtime.h>

#include <cmath>

#include "list_host.cuh"

namespace pkv {
namespace {

template <typename T, int D, int BS>
int run_list(const ListParams &p, cudaStream_t stream)
{
    using C = ListCfg<T, D, BS>;
    constexpr int E = ListElem<T>::bytes;
    alignas(64) CUtensorMap tmk;
    alignas(64) CUtensorMap tmv;
    // rows of 64 bytes are read in pairs: lines of 128 bytes, half as many
    for (int i = 0; i < 2; ++i) {
        const int rc = encode_kv_map(i ? &tmv : &tmk, i ? p.v_cache : p.k_cache, ListElem<T>::tma, E, D * C::TPL, BS / C::TPL,
                                     p.num_kv_heads, p.num_blocks, C::BOX_LINES);
        if (rc)
            return rc;
    }
    static unsigned long long done = 0;
    auto kern = list_attention_kernel<T, D, BS>;
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM_BYTES, &done);
    if (rc)
        return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.np, (unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
    cfg.blockDim = dim3(kListThreads);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.np;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, p, tmk, tmv) != cudaSuccess)
        return PKV_ECUDA;
    if (p.np > 1 && !p.cluster) {
        rc = launch_list_merge<D>(p, stream);
        if (rc)
            return rc;
    }
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

template <typename T, int D>
int run_list_block(const ListParams &p, int bs, cudaStream_t s)
{
    switch (bs) {
    case 8: return run_list<T, D, 8>(p, s);
    case 16: return run_list<T, D, 16>(p, s);
    default: return run_list<T, D, 32>(p, s);
    }
}

template <typename T>
int run_list_type(const ListParams &p, int head_dim, int bs, cudaStream_t s)
{
    return head_dim == 64 ? run_list_block<T, 64>(p, bs, s) : run_list_block<T, 128>(p, bs, s);
}

int decode_list(void *out, int out_dtype, const void *q, int q_dtype, const void *k_cache, const void *v_cache,
                int kv_dtype, const float *k_scales, const float *v_scales, const int32_t *block_tables,
                int max_blocks_per_seq, const int32_t *context_lens, const int32_t *selected, int num_selected,
                int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                int max_context_len, float scale, int partition_size, void *workspace, size_t workspace_bytes,
                uint32_t *device_status, void *stream, bool select)
{
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0 || block_size <= 0 ||
        max_context_len < 0 || partition_size < 0 || !std::isfinite(scale) ||
        (int64_t)max_context_len > (int64_t)max_blocks_per_seq * block_size || (select && num_selected <= 0))
        return PKV_EINVAL;
    if (out_dtype < PKV_F32 || out_dtype > PKV_BF16 || q_dtype < PKV_F32 || q_dtype > PKV_BF16 ||
        kv_dtype < PKV_F32 || kv_dtype > PKV_E4M3 || (kv_dtype != PKV_E4M3 && kv_dtype != q_dtype))
        return PKV_EINVAL;
    if (q_dtype == PKV_F32 || (head_dim != 64 && head_dim != 128) ||
        (block_size != 8 && block_size != 16 && block_size != 32) || num_heads / num_kv_heads > kListMaxGroup ||
        num_kv_heads > 65535 || num_seqs > 65535 || (int64_t)num_seqs * num_heads > INT32_MAX / 8 ||
        max_context_len > INT32_MAX - 64)
        return PKV_EUNSUPPORTED;
    if (partition_size % 32 || partition_size % block_size)
        return PKV_EINVAL;
    if (num_seqs == 0)
        return PKV_OK;
    const bool q8 = kv_dtype == PKV_E4M3;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || (select && !selected) ||
        q8 != (k_scales != nullptr) || q8 != (v_scales != nullptr))
        return PKV_EINVAL;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(selected, 4))
        return PKV_EINVAL;

    const int table_blocks = (int)((max_context_len + (int64_t)block_size - 1) / block_size);
    const int blocks = select ? num_selected : (table_blocks > 0 ? table_blocks : 1);
    const long long rows = (long long)num_seqs * num_kv_heads;
    ListCut cut = list_cut(rows, blocks, block_size, partition_size);
    // a list longer than the contexts ends in -1: it stays whole where the
    // blocks that it can name would (1664 rows of up to 17 blocks of 32 tokens in
    // lists of 129: 37 us, cut in three 88)
    if (select && partition_size == 0 && table_blocks < blocks && blocks <= kListCap &&
        list_cut(rows, table_blocks, block_size, 0).np == 1)
        cut = ListCut{blocks, 1, false};
    const int part = cut.part, np = cut.np;
    if (part > kListCap && blocks > kListCap)
        return PKV_EUNSUPPORTED;
    ListParams p;
    p.ws_ml = nullptr;
    p.ws_acc = nullptr;
    if (np > 1 && !cut.cluster) {
        ListLayout lay;
        if (!list_layout(num_seqs, num_heads, np, head_dim, &lay))
            return PKV_EUNSUPPORTED;
        if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 16))
            return PKV_EWORKSPACE;
        p.ws_ml = static_cast<float *>(workspace);
        p.ws_acc = reinterpret_cast<float *>(static_cast<char *>(workspace) + lay.acc_off);
    }
    p.out = out;
    p.q = q;
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.selected = select ? selected : nullptr;
    p.status = device_status;
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.num_selected = num_selected;
    p.scale_stride = q8_scale_stride(num_kv_heads);
    p.part_blocks = part;
    p.np = np;
    p.cluster = cut.cluster;
    p.out_dtype = out_dtype;
    p.q_dtype = q_dtype;
    p.qscale = scale * 1.4426950408889634f;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (kv_dtype) {
    case PKV_F16: return run_list_type<__half>(p, head_dim, block_size, s);
    case PKV_BF16: return run_list_type<__nv_bfloat16>(p, head_dim, block_size, s);
    default: return run_list_type<uint8_t>(p, head_dim, block_size, s);
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_paged_attention_list_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                int block_size, int max_list_blocks, int partition_size)
{
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        block_size > 32 || max_list_blocks <= 0 || partition_size < 0 || partition_size % block_size ||
        (partition_size > 0 && partition_size < block_size))
        return 0;
    const ListCut cut = list_cut((long long)num_seqs * num_kv_heads, max_list_blocks, block_size, partition_size);
    if (cut.np <= 1 || cut.cluster)
        return 0;
    ListLayout lay;
    return list_layout(num_seqs, num_heads, cut.np, head_dim, &lay) ? lay.total : 0;
}

int pkv_paged_attention_decode_q8(void *out, int out_dtype, const void *q, int q_dtype, const void *k_cache,
                                  const void *v_cache, const float *k_scales, const float *v_scales,
                                  const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                                  int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                  int64_t num_blocks, int max_context_len, float scale, int partition_size,
                                  void *workspace, size_t workspace_bytes, uint32_t *device_status, void *stream)
{
    return decode_list(out, out_dtype, q, q_dtype, k_cache, v_cache, PKV_E4M3, k_scales, v_scales, block_tables,
                       max_blocks_per_seq, context_lens, nullptr, 0, num_seqs, num_heads, num_kv_heads, head_dim,
                       block_size, num_blocks, max_context_len, scale, partition_size, workspace, workspace_bytes,
                       device_status, stream, false);
}

int pkv_paged_attention_decode_selected(void *out, int out_dtype, const void *q, int q_dtype, const void *k_cache,
                                        const void *v_cache, int kv_dtype, const float *k_scales,
                                        const float *v_scales, const int32_t *block_tables, int max_blocks_per_seq,
                                        const int32_t *context_lens, const int32_t *selected, int num_selected,
                                        int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                        int64_t num_blocks, int max_context_len, float scale, int partition_size,
                                        void *workspace, size_t workspace_bytes, uint32_t *device_status, void *stream)
{
    return decode_list(out, out_dtype, q, q_dtype, k_cache, v_cache, kv_dtype, k_scales, v_scales, block_tables,
                       max_blocks_per_seq, context_lens, selected, num_selected, num_seqs, num_heads, num_kv_heads,
                       head_dim, block_size, num_blocks, max_context_len, scale, partition_size, workspace,
                       workspace_bytes, device_status, stream, true);
}

}  // extern "C"
