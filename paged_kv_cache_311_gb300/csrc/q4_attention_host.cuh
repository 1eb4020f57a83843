// q4_attention_host.cuh -- launches of paged_attention_decode_q4, compiled by type
// in q4_attention_f16.cu and q4_attention_bf16.cu.
#pragma once

#include "list_host.cuh"
#include "q4_attention.cuh"

namespace pkv {

int launch_q4_f16(const Q4Params &p, int head_dim, int block_size, cudaStream_t stream);
int launch_q4_bf16(const Q4Params &p, int head_dim, int block_size, cudaStream_t stream);
int launch_q4_lost(const Q4Params &p, cudaStream_t stream);   // the test hook's: bfloat16, heads of 64, blocks of 16, groups up to 4

template <typename T, int D, int BS, bool TWICE, bool HOOK = false>
int run_q4(const Q4Params &p, cudaStream_t stream)
{
    using C = Q4Cfg<D, BS>;
    static unsigned long long done = 0;
    auto kern = q4_attention_kernel<T, D, BS, TWICE, HOOK>;
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM_BYTES, &done);
    if (rc)
        return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = p.shares ? dim3((unsigned)p.shares)
                           : dim3((unsigned)p.list.np, (unsigned)p.list.num_kv_heads, (unsigned)p.list.num_seqs);
    cfg.blockDim = dim3(kListThreads);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.list.np;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.list.cluster ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess)
        return PKV_ECUDA;
    if (p.shares) {
        static unsigned long long merge_done = 0;
        const int rm = ensure_smem_attr(reinterpret_cast<const void *>(q4_merge_kernel<D>), 0, &merge_done);
        if (rm)
            return rm;
        // at least a thread for each four dimensions of a group's heads
        const bool many = p.shares >= 8LL * p.list.num_seqs * p.list.num_kv_heads;
        const int threads = many ? kQ4MergeThreads : p.list.group * (D / 4) <= 128 ? 128 : 256;
        return launch_pdl(q4_merge_kernel<D>, dim3((unsigned)p.shares), dim3(threads), 0, stream, p);
    }
    return p.list.np > 1 && !p.list.cluster ? launch_list_merge<D, true>(p.list, stream) : PKV_OK;
}

template <typename T, int D, int BS>
int run_q4_group(const Q4Params &p, cudaStream_t s)
{
    return p.list.group <= 4 ? run_q4<T, D, BS, true>(p, s) : run_q4<T, D, BS, false>(p, s);
}

template <typename T, int D>
int run_q4_block(const Q4Params &p, int bs, cudaStream_t s)
{
    switch (bs) {
    case 8: return run_q4_group<T, D, 8>(p, s);
    case 16: return run_q4_group<T, D, 16>(p, s);
    default: return run_q4_group<T, D, 32>(p, s);
    }
}

template <typename T>
int run_q4_type(const Q4Params &p, int head_dim, int bs, cudaStream_t s)
{
    return head_dim == 64 ? run_q4_block<T, 64>(p, bs, s) : run_q4_block<T, 128>(p, bs, s);
}

}  // namespace pkv
