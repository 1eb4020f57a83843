// list_host.cuh -- host-side parts of attention over lists of blocks, shared by
// its translation units: the cut of a row's list into partitions, the layout of
// the workspace, the launch of the merge.
#pragma once

#include <cuda_runtime.h>

#include "list_attention.cuh"
#include "pkv_host.cuh"

namespace pkv {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The cut of a row's list of at most `blocks` entries: entries per partition,
// partitions, and whether a row's partitions are a cluster.
struct ListCut {
    int part, np;
    bool cluster;
};

inline ListCut list_cut(long long rows, long long blocks, int block_size, int partition_size)
{
    if (blocks < 1)
        blocks = 1;
    ListCut c{0, 1, false};
    const int least = 64 / block_size;
    const int sms = device_sm_count();
    long long part = blocks;
    if (partition_size > 0) {
        part = partition_size / block_size;
    } else if (rows >= sms) {
        // rows that fill the SMs stay whole up to 4096 tokens, else 2048 each
        if (blocks > 4096 / block_size)
            part = 2048 / block_size;
    } else {
        // four CTAs per SM; as a cluster where that leaves a CTA 512 tokens
        const long long np = (4LL * sms + rows - 1) / rows;
        part = (blocks + np - 1) / np;
        const long long eighth = (blocks + 7) / 8;
        if (part < eighth && eighth <= 512 / block_size)
            part = eighth;
        part = part > 2048 / block_size ? 2048 / block_size : part;
        part = (part + least - 1) / least * least;
    }
    if (partition_size == 0 && part > kListCap)
        part = kListCap;
    c.part = (int)part;
    c.np = (int)((blocks + part - 1) / part);
    c.cluster = partition_size == 0 && c.np > 1 && c.np <= 8;
    return c;
}

struct ListLayout {
    size_t acc_off, total;
};
inline bool list_layout(uint64_t seqs, uint64_t heads, uint64_t np, uint64_t head_dim, ListLayout *s)
{
    uint64_t rows, ml, acc;
    if (__builtin_mul_overflow(seqs, heads, &rows) || __builtin_mul_overflow(rows, np, &rows) ||
        __builtin_mul_overflow(rows, (uint64_t)8, &ml) || __builtin_mul_overflow(rows, head_dim * 4, &acc) ||
        ml > UINT64_MAX - 256 || ((ml + 255) & ~uint64_t(255)) > UINT64_MAX - acc)
        return false;
    s->acc_off = (size_t)((ml + 255) & ~uint64_t(255));
    s->total = s->acc_off + (size_t)acc;
    return true;
}

template <int D, bool WIDE = false>
int launch_list_merge(const ListParams &p, cudaStream_t stream)
{
    static unsigned long long merge_done = 0;
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(list_merge_kernel<D, WIDE>), 0, &merge_done);
    if (rc)
        return rc;
    // a warp for each head where the heads fill the GPU, else several
    const int64_t heads = (int64_t)p.num_seqs * p.num_kv_heads * p.group;
    int per_head = 1;
    while (per_head < kMergeWarps && per_head * 8 < p.np && heads * per_head * 2 <= 32LL * device_sm_count())
        per_head *= 2;
    return launch_pdl(list_merge_kernel<D, WIDE>, dim3((unsigned)((heads * per_head + kMergeWarps - 1) / kMergeWarps)),
                      dim3(kMergeWarps * 32), 0, stream, p, per_head);
}

}  // namespace pkv
