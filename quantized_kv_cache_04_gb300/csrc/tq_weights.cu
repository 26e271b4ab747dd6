// Accumulated attention weight per cached token: the third kernel of
// tq_decode_attention_weights.
//
// Stage 1 keeps the (capped, biased) scores x of every listed token; after
// stage 2 has merged the splits' log-sum-exps,
//   acc[b][h][t] += sum_g exp(x[g][t] - lse[g])
// over the query heads g of kv head h.  Each running sum has one writer and a
// fixed order of additions.
#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kThreads = 256;

// One thread per listed token.
__global__ void __launch_bounds__(kThreads) weights_kernel(ScoreArgs m, const int32_t* seq_lens, const float* lse,
                                                           float* acc, long long stride_b, long long stride_h,
                                                           int Hk, int G)
{
    __shared__ float s_lse[kMaxGroup];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.z, h = blockIdx.y;
    const int L = seq_lens[b];
    if (L > m.max_len) return;               // its scores were not kept
    const VisibleSet vis(m, L, b);
    const int v = blockIdx.x * kThreads + threadIdx.x;
    if (blockIdx.x * kThreads >= 32 * vis.tiles()) return;
    if (threadIdx.x < G)
        s_lse[threadIdx.x] = lse[((long long)b * Hk + h) * G + threadIdx.x] * 1.4426950408889634f;
    __syncthreads();
    if (v >= 32 * vis.tiles()) return;
    const int t = vis.base(v >> 5) + (v & 31);
    if (!vis.sees(t)) return;
    const float* x = m.scores + (((long long)b * Hk + h) * m.vtok + v) * m.gp;
    float w = 0.f;
    for (int g = 0; g < G; ++g) w += exp2f(x[g] - s_lse[g]);
    acc[b * stride_b + h * stride_h + t] += w;
}

}  // namespace

cudaError_t launch_weights(const ScoreArgs& m, const int32_t* seq_lens, const float* lse, float* acc,
                           long long stride_b, long long stride_h, int B, int Hk, int G, cudaStream_t st)
{
    if (m.vtok == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((m.vtok + kThreads - 1) / kThreads, Hk, B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_kernel, m, seq_lens, lse, acc, stride_b, stride_h, Hk, G);
}

}  // namespace tq
