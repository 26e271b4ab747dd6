// Accumulated attention weight per cached token: the third kernel of
// tq_decode_attention_weights.
//
// Stage 1 keeps the (capped, biased) scores x of every listed token, in log2
// units, [sequence][kv head][listed token][query head]; after stage 2 has merged
// the splits' log-sum-exps,
//   acc[b][h][t] += sum_g 2^(x[g][t] - lse[g] log2 e)
// over the G query heads of kv head h.  Each running sum has one writer and a
// fixed order of additions.  Bound by bytes: 4 G per token of scores, which come
// from L2 where they fit it, and 8 of sums.
#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                  // tokens per thread, kThreads apart

// GP: columns per listed token (0: m.gp).
template <int GP>
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
    const int v0 = blockIdx.x * kThreads * kPer, end = min(32 * vis.tiles(), v0 + kThreads * kPer);
    if (v0 >= end) return;
    if (threadIdx.x < G)
        s_lse[threadIdx.x] = lse[((long long)b * Hk + h) * G + threadIdx.x] * 1.4426950408889634f;
    const float* x = m.scores + ((long long)b * Hk + h) * m.vtok * m.gp;
    float* sums = acc + b * stride_b + h * stride_h;
    float s[kPer][GP ? GP : 1], was[kPer];
    int t[kPer];
    // every load of the thread's tokens before the arithmetic
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int v = v0 + u * kThreads + threadIdx.x;
        t[u] = v < end ? vis.base(v >> 5) + (v & 31) : -1;
        if (t[u] >= 0 && !vis.sees(t[u])) t[u] = -1;
        if (t[u] >= 0) was[u] = sums[t[u]];
        if constexpr (GP > 0) {
            if (t[u] >= 0) {
                if constexpr (GP % 4 == 0) {
#pragma unroll
                    for (int g = 0; g < GP; g += 4) {
                        const float4 q = *reinterpret_cast<const float4*>(x + (long long)v * GP + g);
                        s[u][g] = q.x; s[u][g + 1] = q.y; s[u][g + 2] = q.z; s[u][g + 3] = q.w;
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < GP; ++g) s[u][g] = x[(long long)v * GP + g];
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        if (t[u] < 0) continue;
        float w = 0.f;
        if constexpr (GP > 0) {
#pragma unroll
            for (int g = 0; g < GP; ++g)
                if (g < G) w += exp2f(s[u][g] - s_lse[g]);
        } else {
            const long long v = v0 + u * kThreads + threadIdx.x;
            for (int g = 0; g < G; ++g) w += exp2f(x[v * m.gp + g] - s_lse[g]);
        }
        sums[t[u]] = was[u] + w;
    }
}

}  // namespace

cudaError_t launch_weights(const ScoreArgs& m, const int32_t* seq_lens, const float* lse, float* acc,
                           long long stride_b, long long stride_h, int Hk, int G, cudaStream_t st)
{
    if (m.vtok == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((m.vtok + kThreads * kPer - 1) / (kThreads * kPer), Hk, m.B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // groups of up to 8 keep their tokens' scores in registers
    auto k = m.gp == 8 ? weights_kernel<8> : m.gp == 6 ? weights_kernel<6> : m.gp == 4 ? weights_kernel<4>
             : m.gp == 3 ? weights_kernel<3> : m.gp == 2 ? weights_kernel<2> : m.gp == 1 ? weights_kernel<1>
                                                                                         : weights_kernel<0>;
    return cudaLaunchKernelEx(&cfg, k, m, seq_lens, lse, acc, stride_b, stride_h, Hk, G);
}

}  // namespace tq
