// block_select.cu -- host side of select_blocks.
#include <cuda_runtime.h>

#include "block_select.cuh"
#include "pkv_host.cuh"

namespace pkv {
namespace {

constexpr int kSelectMaxBlocks = 40960;   // a row's scores fit one CTA's shared memory
// One launch: blocks of a row, and rows x blocks of the call, at most; half of
// those where rows exceed the 608 CTAs of 128 threads that are resident.  (One
// launch against two, us: 512 rows of up to 256 blocks 18 against 22, 64 of
// 2048 19 against 21, 128 of 512 13 against 18; but 800 of 163 26 against 22,
// 3200 of 128 44 against 38, 128 of 2048 56 against 36.)
constexpr int kSelectOneBlocks = 2048;
constexpr int64_t kSelectOne = 131072;

int key_stride(int n) { return (n + 3) / 4 * 4; }

// How a call runs: `ctas` CTAs score `chunk` blocks of a row each, in one
// launch as a cluster or in two through the workspace.
struct SelectCut {
    int chunk, ctas, bounds, threads;
    bool cluster;
    size_t bound_off, total;   // workspace: keys, then bounds
};

// One launch while its summaries are few: it saves a launch, but clusters are
// not spread evenly over the SMs.
SelectCut select_cut(int64_t rows, int most)
{
    SelectCut c{};
    const int n = most > 0 ? most : 1;
    constexpr int kOne = 128;   // blocks of a cluster's CTA, a tile per warp
    const int64_t sms = device_sm_count();
    c.cluster = n <= kSelectOneBlocks && rows * n <= (rows <= 4 * sms ? kSelectOne : kSelectOne / 2);
    if (c.cluster) {
        // CTAs per row: as many as have a tile per warp while two an
        // SM are resident together
        c.ctas = 1;
        while (c.ctas < kSelectCluster && n > c.ctas * kOne && rows * c.ctas <= sms)
            c.ctas *= 2;
        c.chunk = (n + c.ctas - 1) / c.ctas;
        c.threads = rows * c.ctas > 2 * sms ? 128 : 256;
        c.bounds = c.ctas * (c.threads / 32);
    } else {
        c.threads = rows > 4 * sms ? 128 : 256;
        c.chunk = kScoreWarps * kScoreTiles * 16;
        c.ctas = (n + c.chunk - 1) / c.chunk;
        c.bounds = c.ctas * kScoreWarps;
        c.bound_off = ((size_t)rows * key_stride(n) * 4 + 255) & ~size_t(255);
        c.total = c.bound_off + (size_t)rows * c.bounds * 4;
    }
    return c;
}

size_t row_smem(int most) { return sizeof(SelectShared) + (size_t)key_stride(most) * 4 + (size_t)(most + 31) / 32 * 8; }

template <typename T, int D, int NT>
int launch_select(const SelectParams &p, int ctas, bool one, cudaStream_t stream)
{
    static unsigned long long done_one = 0, done_score = 0, done_rows = 0;
    if (one) {
        auto kern = select_blocks_kernel<T, D, NT>;
        constexpr size_t score = sizeof(ScoreShared<D, NT / 32, 1>);
        const int rc = ensure_smem_attr(reinterpret_cast<const void *>(kern), (int)(score + row_smem(kSelectOneBlocks)), &done_one);
        if (rc)
            return rc;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas, (unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
        cfg.blockDim = dim3(NT);
        cfg.dynamicSmemBytes = score + row_smem(p.most);
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)ctas;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PKV_OK : PKV_ECUDA;
    }
    constexpr int score = (int)sizeof(ScoreShared<D, kScoreWarps, kScoreStages>);
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(score_blocks_kernel<T, D>), score, &done_score);
    if (!rc)
        rc = ensure_smem_attr(reinterpret_cast<const void *>(select_rows_kernel<T, D, NT>), (int)row_smem(kSelectMaxBlocks), &done_rows);
    if (rc)
        return rc;
    rc = launch_pdl(score_blocks_kernel<T, D>, dim3((unsigned)p.num_kv_heads, (unsigned)ctas, (unsigned)p.num_seqs),
                    dim3(kScoreWarps * 32), score, stream, p);
    if (rc)
        return rc;
    rc = launch_pdl(select_rows_kernel<T, D, NT>, dim3((unsigned)p.num_kv_heads, (unsigned)p.num_seqs), dim3(NT),
                    row_smem(p.most), stream, p);
    if (rc)
        return rc;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

template <typename T, int D>
int launch_select(const SelectParams &p, const SelectCut &cut, cudaStream_t stream)
{
    return cut.threads == 128 ? launch_select<T, D, 128>(p, cut.ctas, cut.cluster, stream)
                              : launch_select<T, D, 256>(p, cut.ctas, cut.cluster, stream);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_select_blocks_workspace_bytes(int num_seqs, int num_kv_heads, int max_context_len, int block_size)
{
    if (num_seqs <= 0 || num_seqs > 65535 || num_kv_heads <= 0 || num_kv_heads > 65535 || max_context_len < 0 ||
        block_size <= 0 || (max_context_len + (int64_t)block_size - 1) / block_size > kSelectMaxBlocks)
        return 0;
    return select_cut((int64_t)num_seqs * num_kv_heads, (int)((max_context_len + (int64_t)block_size - 1) / block_size)).total;
}

extern "C" int pkv_select_blocks(int32_t *selected, const void *q, int q_dtype, const void *summaries,
                                 int summary_dtype, const int32_t *block_tables, int max_blocks_per_seq,
                                 const int32_t *context_lens, int num_seqs, int num_heads, int num_kv_heads,
                                 int head_dim, int block_size, int64_t num_blocks, int max_context_len,
                                 int num_selected, int keep_first, int keep_last, void *workspace,
                                 size_t workspace_bytes, uint32_t *device_status, void *stream)
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
    const int most = (int)((max_context_len + (int64_t)block_size - 1) / block_size);
    if (most > kSelectMaxBlocks)
        return PKV_EUNSUPPORTED;
    if (num_seqs == 0)
        return PKV_OK;
    if (!selected || !q || !summaries || !block_tables || !context_lens)
        return PKV_EINVAL;
    if (!aligned(selected, 4) || !aligned(q, 16) || !aligned(summaries, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PKV_EINVAL;

    const SelectCut cut = select_cut((int64_t)num_seqs * num_kv_heads, most);
    if (cut.total && (!workspace || workspace_bytes < cut.total || !aligned(workspace, 16)))
        return PKV_EWORKSPACE;
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
    p.key_stride = key_stride(most > 0 ? most : 1);
    p.chunk = cut.chunk;
    p.bounds = cut.bounds;
    p.ws_keys = static_cast<uint32_t *>(workspace);
    p.ws_bound = reinterpret_cast<float *>(static_cast<char *>(workspace) + cut.bound_off);
    p.q_dtype = q_dtype;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (summary_dtype == PKV_F16)
        return head_dim == 64 ? launch_select<__half, 64>(p, cut, s)
                              : launch_select<__half, 128>(p, cut, s);
    return head_dim == 64 ? launch_select<__nv_bfloat16, 64>(p, cut, s)
                          : launch_select<__nv_bfloat16, 128>(p, cut, s);
}

extern "C" int pkv_test_select_timeout(int what, uint64_t limit_ns, int32_t *selected, int num_selected,
                                       uint32_t *device_status, void *stream)
{
    if (what < 0 || what > 2 || limit_ns == 0 || limit_ns > kWaitLimitNs || !selected || num_selected <= 0 ||
        num_selected >= 100 || !device_status || !aligned(selected, 4) || !aligned(device_status, 4))
        return PKV_EINVAL;
    SelectParams p = {};
    p.selected = selected;
    p.status = device_status;
    p.num_selected = num_selected;
    p.num_seqs = p.num_kv_heads = 1;
    p.bounds = 2;
    select_timeout_test_kernel<<<1, kSelectThreads, 0, static_cast<cudaStream_t>(stream)>>>(p, what, limit_ns);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}
