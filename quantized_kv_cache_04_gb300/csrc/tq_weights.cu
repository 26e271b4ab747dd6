// Accumulated attention weight per cached token: the third kernel of
// tq_decode_attention_weights.
//
// Stage 1 keeps the (capped, biased) scores x of every listed token, in log2
// units, [sequence][kv head][listed token][query head]; after stage 2 has merged
// the splits' log-sum-exps,
//   acc[b][h][t] += sum_g 2^(x[g][t] - lse[g] log2 e)
// over the G query heads of kv head h.  Each running sum has one writer and a
// fixed order of additions.  Bound by bytes: 4 G per token of scores, which come
// from L2 where they fit it, and 8 of sums.  Measured: 524K tokens, 8 kv heads,
// groups of 8 (134 MB of scores): 27 us, 5.7 TB/s at the DRAM; with one token per
// thread at a time 36 us.
#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kThreads = 256;

// tokens per thread, kThreads apart: as many as keep their scores in registers
template <int GP> constexpr int kPerThread = GP > 8 ? 2 : 4;

// GP: columns per listed token (m.gp).
template <int GP>
__global__ void __launch_bounds__(kThreads) weights_kernel(ScoreArgs m, const int32_t* seq_lens, const float* lse,
                                                           float* acc, long long stride_b, long long stride_h,
                                                           int Hk, int G)
{
    constexpr int kPer = kPerThread<GP>;
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
    const float* x = m.scores + ((long long)b * Hk + h) * m.vtok * GP;
    float* sums = acc + b * stride_b + h * stride_h;
    float s[kPer][GP], was[kPer];
    int t[kPer];
    // every load of the thread's tokens before the arithmetic
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int v = v0 + u * kThreads + threadIdx.x;
        t[u] = v < end ? vis.base(v >> 5) + (v & 31) : -1;
        if (t[u] >= 0 && !vis.sees(t[u])) t[u] = -1;
        if (t[u] < 0) continue;
        was[u] = sums[t[u]];
        const float* xv = x + (unsigned long long)unsigned(v) * unsigned(GP);
        if constexpr (GP % 4 == 0) {
#pragma unroll
            for (int g = 0; g < GP; g += 4) {
                const float4 q = __ldcs(reinterpret_cast<const float4*>(xv + g));
                s[u][g] = q.x; s[u][g + 1] = q.y; s[u][g + 2] = q.z; s[u][g + 3] = q.w;
            }
        } else if constexpr (GP % 2 == 0) {
#pragma unroll
            for (int g = 0; g < GP; g += 2) {
                const float2 q = __ldcs(reinterpret_cast<const float2*>(xv + g));
                s[u][g] = q.x; s[u][g + 1] = q.y;
            }
        } else {
#pragma unroll
            for (int g = 0; g < GP; ++g) s[u][g] = __ldcs(xv + g);
        }
    }
    __syncthreads();
    float l[GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) l[g] = s_lse[g];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        float w = 0.f;
#pragma unroll
        for (int g = 0; g < GP; ++g)
            if (g < G) w += fast_exp2(s[u][g] - l[g]);           // a padding column may hold anything
        if (t[u] >= 0) sums[t[u]] = was[u] + w;
    }
}

template <int GP>
cudaError_t launch_gp(const ScoreArgs& m, const int32_t* seq_lens, const float* lse, float* acc, long long stride_b,
                      long long stride_h, int Hk, int G, cudaStream_t st)
{
    constexpr int kTokens = kThreads * kPerThread<GP>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((m.vtok + kTokens - 1) / kTokens, Hk, m.B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_kernel<GP>, m, seq_lens, lse, acc, stride_b, stride_h, Hk, G);
}

}  // namespace

cudaError_t launch_weights(const ScoreArgs& m, const int32_t* seq_lens, const float* lse, float* acc,
                           long long stride_b, long long stride_h, int Hk, int G, cudaStream_t st)
{
    if (m.vtok == 0) return cudaSuccess;
    switch (m.gp) {                          // score_heads(G), G <= 16
#define TQ_GP(n) case n: return launch_gp<n>(m, seq_lens, lse, acc, stride_b, stride_h, Hk, G, st);
    TQ_GP(1) TQ_GP(2) TQ_GP(3) TQ_GP(4) TQ_GP(6) TQ_GP(8) TQ_GP(10) TQ_GP(12) TQ_GP(14) TQ_GP(16)
#undef TQ_GP
    }
    return cudaErrorInvalidValue;
}

}  // namespace tq
