// block_select.cu -- host side of select_blocks.
#include <cuda_runtime.h>

#include "block_select.cuh"
#include "pkv_host.cuh"

namespace pkv {
namespace {

constexpr int kSelectMaxBlocks = 40960;   // their scores fit CTA 0's shared memory

size_t select_smem(int chunk, int most, int head_dim)
{
    return sizeof(SelectShared) + (size_t)head_dim * 8 + (size_t)chunk * 4 + (size_t)most * 4 + (size_t)(most + 31) / 32 * 8;
}

template <typename T, int D>
int launch_select(const SelectParams &p, int ctas, cudaStream_t stream)
{
    static unsigned long long done = 0;
    auto kern = select_blocks_kernel<T, D>;
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(kern), (int)select_smem(kSelectMaxBlocks / kSelectCluster, kSelectMaxBlocks, D), &done);
    if (rc)
        return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = select_smem(p.chunk, p.most, D);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_select_blocks(int32_t *selected, const void *q, int q_dtype, const void *summaries,
                                 int summary_dtype, const int32_t *block_tables, int max_blocks_per_seq,
                                 const int32_t *context_lens, int num_seqs, int num_heads, int num_kv_heads,
                                 int head_dim, int block_size, int64_t num_blocks, int max_context_len,
                                 int num_selected, int keep_first, int keep_last, uint32_t *device_status,
                                 void *stream)
{
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0 ||
        max_context_len < 0 || num_selected <= 0 || keep_first < 0 || keep_last < 0 ||
        (int64_t)keep_first + keep_last > num_selected ||
        (int64_t)max_context_len > (int64_t)max_blocks_per_seq * block_size)
        return PKV_EINVAL;
    if (q_dtype < PKV_F32 || q_dtype > PKV_BF16 || summary_dtype < PKV_F32 || summary_dtype > PKV_BF16)
        return PKV_EINVAL;
    if (q_dtype == PKV_F32 || summary_dtype == PKV_F32 || (head_dim != 64 && head_dim != 128) ||
        (block_size != 8 && block_size != 16 && block_size != 32) || num_heads / num_kv_heads > 8 ||
        num_kv_heads > 65535 || num_seqs > 65535)
        return PKV_EUNSUPPORTED;
    const int most = (max_context_len + block_size - 1) / block_size;
    if (most > kSelectMaxBlocks)
        return PKV_EUNSUPPORTED;
    if (num_seqs == 0)
        return PKV_OK;
    if (!selected || !q || !summaries || !block_tables || !context_lens)
        return PKV_EINVAL;
    if (!aligned(selected, 4) || !aligned(q, 16) || !aligned(summaries, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PKV_EINVAL;

    // CTAs per row: as many as leave each 64 blocks (a load of eight per warp)
    // and as are resident together, four to an SM
    const long long rows = (long long)num_seqs * num_kv_heads;
    int ctas = 1;
    while (ctas < kSelectCluster && most > ctas * 64 && rows * ctas * 2 <= 4LL * device_sm_count())
        ctas *= 2;
    SelectParams p;
    p.selected = selected;
    p.q = q;
    p.summaries = summaries;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.status = device_status;
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.block_size = block_size;
    p.num_selected = num_selected;
    p.keep_first = keep_first;
    p.keep_last = keep_last;
    p.most = most;
    p.chunk = most > 0 ? (most + ctas - 1) / ctas : 1;
    p.q_dtype = q_dtype;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (summary_dtype == PKV_F16)
        return head_dim == 64 ? launch_select<__half, 64>(p, ctas, s) : launch_select<__half, 128>(p, ctas, s);
    return head_dim == 64 ? launch_select<__nv_bfloat16, 64>(p, ctas, s)
                          : launch_select<__nv_bfloat16, 128>(p, ctas, s);
}
