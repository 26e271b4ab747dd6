// Tensor-core decode stage 1 with score modifiers: its instantiations,
// compiled apart from the others (the kernel is in tq_decode_mma_scored.cuh).
#include "tq_decode_mma_scored.cuh"

namespace tq {

cudaError_t launch_mma_scored(const MmaArgs& a, int q_dtype, int B, size_t smem, cudaStream_t st)
{
    return q_dtype == TQ_F16 ? launch_scored_q<__half, kScored>(a, B, smem, st)
                             : launch_scored_q<__nv_bfloat16, kScored>(a, B, smem, st);
}

}  // namespace tq
