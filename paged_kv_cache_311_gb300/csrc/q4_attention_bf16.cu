// Attention over 4-bit caches of bfloat16, and the test hook's kernel.
#include "q4_attention_host.cuh"

namespace pkv {
int launch_q4_bf16(const Q4Params &p, int head_dim, int block_size, cudaStream_t stream)
{
    return run_q4_type<__nv_bfloat16>(p, head_dim, block_size, stream);
}
int launch_q4_lost(const Q4Params &p, cudaStream_t stream)
{
    return run_q4<__nv_bfloat16, 64, 16, true, true>(p, stream);
}
}  // namespace pkv
