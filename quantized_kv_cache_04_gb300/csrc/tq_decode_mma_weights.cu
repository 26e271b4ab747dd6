// Tensor-core decode stage 1 that keeps the scores for the attention weights: its instantiations,
// compiled apart from the others (the kernel is in tq_decode_mma_scored.cuh).
#include "tq_decode_mma_scored.cuh"

namespace tq {

cudaError_t launch_mma_weights(const MmaArgs& a, int q_dtype, int B, size_t smem, cudaStream_t st)
{
    return q_dtype == TQ_F16 ? launch_scored_q<__half, kWeights>(a, B, smem, st)
                             : launch_scored_q<__nv_bfloat16, kWeights>(a, B, smem, st);
}

}  // namespace tq
