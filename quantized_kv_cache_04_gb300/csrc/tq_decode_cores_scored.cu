// CUDA-core decode stage 1 with score modifiers: its instantiations, compiled
// apart from the plain ones (the kernel is in tq_decode_cores.cuh).
#include "tq_decode_cores.cuh"

namespace tq {

cudaError_t launch_cores_scored(int preset, int q_dtype, const DecodeArgs& a, cudaStream_t st)
{
    return q_dtype == TQ_F16 ? launch_stage1<__half, true>(preset, a, st)
                             : launch_stage1<__nv_bfloat16, true>(preset, a, st);
}

}  // namespace tq
