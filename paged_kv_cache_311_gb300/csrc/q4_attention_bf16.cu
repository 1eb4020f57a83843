// Attention over 4-bit caches of bfloat16.
#include "q4_attention_host.cuh"

namespace pkv {
int launch_q4_bf16(const Q4Params &p, int head_dim, int block_size, cudaStream_t stream)
{
    return run_q4_type<__nv_bfloat16>(p, head_dim, block_size, stream);
}
}  // namespace pkv
