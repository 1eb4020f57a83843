// q4_attention.cu -- host side of paged_attention_decode_q4: checks of
// arguments, the cut of the work, the workspace's layout.
#include <cuda_runtime.h>

#include <cmath>

#include "q4_attention_host.cuh"

namespace pkv {
namespace {

// How a call is cut: streamed into `shares`, or rows into `list.np` partitions.
struct Q4Cut {
    ListCut list;
    int shares, part_units;
};

// Rows that leave CTAs idle are divided among clusters, by each row's own length,
// as long as all CTAs are resident at once; other short rows stay whole; the rest
// is streamed, in shares of equal cost.  us, in that order (whole: one CTA a row),
// 8 kv heads of 128 where nothing else is said:
//   1 sequence of 4000 tokens (8 per row)          9.6   34.2   13.5
//   8 of 2000 (6 per row)                         11.0   19.2   14.0
//   16 of 2000 (3 per row)                        15.3   19.8   18.1
//   16 of 8K to 16K (3 per row)                   73.9  135.0   62.1
//   30 of 2000                                      -    25.1   26.7
//   57 of 2048: a row for each place               -    31.7   34.6
//   64 of 2048                                      -    46.5   43.8
//   75 of 2048                                      -    46.9   49.2
//   64 of 128 to 2048, 32 kv heads                  -    82.4   83.9
//   128 of 512 to 2048                              -    58.5   56.0
//   256 of 512                                      -    50.0   53.2
//   256 of 1 to 64                                  -    22.3   23.8
//   256 of 1 to 64, 40 kv heads                     -   100.8   84.6
//   33 of up to 4095, heads of 64                   -    34.2   23.9
//   64 of 512 to 4000                               -    57.7   48.5
// The rule goes by the longest length that the call names.  What it gives away is
// in the lines where short rows come in a wave and a little, and in those of ten
// thousand rows of one step, where either form is far from the bytes' time (9 us).
// (Clusters of 8 whatever the rows, which come in waves: 16.8, 22.1, 82.3 for 8 of
// 2000, 16 of 2000, 16 of 8K to 16K.)
Q4Cut q4_cut(long long rows, long long max_context_len, int block_size, int partition_size)
{
    Q4Cut c{};
    if (partition_size > 0) {
        const long long blocks = max_context_len > 0 ? (max_context_len + block_size - 1) / block_size : 1;
        c.list = list_cut(rows, blocks, block_size, partition_size);
        c.part_units = partition_size / kQ4Unit;
        return c;
    }
    const long long slots = (long long)kQ4Ctas * device_sm_count();
    const long long units = (max_context_len + kQ4Unit - 1) / kQ4Unit;
    // (clusters of CTAs on nearby SMs do not fill every slot: at 448 of 456, 64 rows
    // of 700 tokens take 12.8 us, at 384 8.0)
    long long np = slots * 7 / 8 / rows;
    np = np > 8 ? 8 : np;
    np = np > units ? units : np;
    np = np < 1 ? 1 : np;
    if (units > np * (np > 1 ? 32 : 64))
        c.shares = (int)slots;
    else
        c.list = ListCut{0, (int)np, np > 1};
    return c;
}

// The workspace of a cut; false if it passes 64 bits.
struct Q4Layout {
    ListLayout list;
    size_t share_off, total;
};
bool q4_layout(const Q4Cut &c, uint64_t seqs, uint64_t heads, uint64_t kv_heads, uint64_t head_dim, Q4Layout *lay)
{
    *lay = Q4Layout{};
    if (c.shares) {
        // two parts of each share, of a group's heads, and where the share lies
        if (!list_layout(2 * (uint64_t)c.shares, heads / kv_heads, 1, head_dim, &lay->list))
            return false;
        lay->share_off = (lay->list.total + 15) / 16 * 16;
        lay->total = lay->share_off + c.shares * sizeof(Q4Share);
        return true;
    }
    if (c.list.np > 1 && !c.list.cluster && !list_layout(seqs, heads, c.list.np, head_dim, &lay->list))
        return false;
    lay->total = lay->list.total;
    return true;
}

// pkv_paged_attention_decode_q4; `lost`: the test hook's.
int decode_q4(void *out, int out_dtype, const void *q, int64_t q_stride, int q_dtype,
              const void *k_cache, const void *v_cache, const int32_t *block_tables,
              int max_blocks_per_seq, const int32_t *context_lens, int num_seqs, int num_heads,
              int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
              int max_context_len, float scale, int partition_size, void *workspace,
              size_t workspace_bytes, uint32_t *device_status, void *stream, const Q4Lost *lost)
{
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

    const Q4Cut cut = q4_cut((long long)num_seqs * num_kv_heads, max_context_len, block_size, partition_size);
    Q4Params p = {};
    ListParams &l = p.list;
    Q4Layout lay;
    if (!q4_layout(cut, num_seqs, num_heads, num_kv_heads, head_dim, &lay))
        return PKV_EUNSUPPORTED;
    if (lay.total) {
        if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 16))
            return PKV_EWORKSPACE;
        l.ws_ml = static_cast<float *>(workspace);
        l.ws_acc = reinterpret_cast<float *>(static_cast<char *>(workspace) + lay.list.acc_off);
        p.ws_share = reinterpret_cast<Q4Share *>(static_cast<char *>(workspace) + lay.share_off);
    }
    p.shares = cut.shares;
    p.part_units = cut.part_units;
    l.out = out;
    l.q = q;
    l.k_cache = static_cast<const uint8_t *>(k_cache);
    l.v_cache = static_cast<const uint8_t *>(v_cache);
    l.block_tables = block_tables;
    l.context_lens = context_lens;
    l.status = device_status;
    l.num_blocks = num_blocks;
    l.num_seqs = num_seqs;
    l.num_kv_heads = num_kv_heads;
    l.group = num_heads / num_kv_heads;
    l.max_blocks_per_seq = max_blocks_per_seq;
    l.max_context_len = max_context_len;
    l.np = cut.shares ? 1 : cut.list.np;
    l.cluster = !cut.shares && cut.list.cluster;
    l.out_dtype = out_dtype;
    l.q_dtype = q_dtype;
    l.qscale = scale * 1.4426950408889634f;
    p.q_stride = q_stride;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (lost) {
        p.lost = *lost;
        return launch_q4_lost(p, s);
    }
    return q_dtype == PKV_F16 ? launch_q4_f16(p, head_dim, block_size, s) : launch_q4_bf16(p, head_dim, block_size, s);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_paged_attention_q4_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                              int max_context_len, int partition_size)
{
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
        block_size <= 0 || block_size > 32 || max_context_len < 0 || partition_size < 0 || partition_size % kQ4Unit)
        return 0;
    Q4Layout lay;
    const Q4Cut cut = q4_cut((long long)num_seqs * num_kv_heads, max_context_len, block_size, partition_size);
    return q4_layout(cut, num_seqs, num_heads, num_kv_heads, head_dim, &lay) ? lay.total : 0;
}

int pkv_paged_attention_decode_q4(void *out, int out_dtype, const void *q, int64_t q_stride, int q_dtype,
                                  const void *k_cache, const void *v_cache, const int32_t *block_tables,
                                  int max_blocks_per_seq, const int32_t *context_lens, int num_seqs, int num_heads,
                                  int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                  int max_context_len, float scale, int partition_size, void *workspace,
                                  size_t workspace_bytes, uint32_t *device_status, void *stream)
{
    return decode_q4(out, out_dtype, q, q_stride, q_dtype, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                     num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale,
                     partition_size, workspace, workspace_bytes, device_status, stream, nullptr);
}

int pkv_test_q4_timeout(uint64_t limit_ns, int cta, int warp, int unit, float *out, const void *q, const void *k_cache,
                        const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                        int num_seqs, int num_heads, int num_kv_heads, int64_t num_blocks, int max_context_len, float scale,
                        int partition_size, void *workspace, size_t workspace_bytes, uint32_t *device_status, void *stream)
{
    if (limit_ns == 0 || limit_ns > kWaitLimitNs || cta < 0 || warp < 0 || warp >= kListWarps || unit < 0 || num_kv_heads <= 0 ||
        num_heads / num_kv_heads > 4 || !device_status || !aligned(device_status, 4))
        return PKV_EINVAL;
    const Q4Lost lost{limit_ns, cta, warp, unit};
    return decode_q4(out, PKV_F32, q, (int64_t)num_heads * 64, PKV_BF16, k_cache, v_cache, block_tables, max_blocks_per_seq,
                     context_lens, num_seqs, num_heads, num_kv_heads, 64, 16, num_blocks, max_context_len, scale, partition_size,
                     workspace, workspace_bytes, device_status, stream, &lost);
}

}  // extern "C"
