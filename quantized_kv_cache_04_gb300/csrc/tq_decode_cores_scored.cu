// CUDA-core decode stage 1 with score modifiers, for the shapes the tensor-core
// scored kernel (tq_decode_mma_scored.cuh) does not serve.  As the plain one
// (tq_decode.cu): one CTA per (split, kv head), four warps striding over the
// split's tokens, 4 coordinates per lane; the splits are those of the batch's
// plan, hidden tokens are skipped with their pages.  A kernel of its own for the
// plain one's registers.
#include "tq_decode_cores.cuh"

namespace tq {
namespace {

template <typename TQ, bool KEY_FP8, int KBITS, int VBITS, int GM>
__global__ void __launch_bounds__(kWarps * 32) scored_kernel(DecodeArgs a)
{
    const int h = blockIdx.y;
    // which sequence's split this is goes by the plan of the batch
    __shared__ int s_plan[kPlanMax + 4];
    const int id = blockIdx.z * a.num_splits + blockIdx.x;
    const SplitPlan plan(a.mods, a.seq_lens, a.num_splits, id, blockIdx.x + blockIdx.y + blockIdx.z == 0, s_plan);
    if (plan.b < 0) return;
    const int b = plan.b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.G;
    const int L = a.seq_lens[b];
    const VisibleSet vis(a.mods, min(L, a.mods.max_len), b);
    // this split's partial of query head hq, and its positions in the list of
    // tiles that hold visible tokens
    auto partial = [&](int hq) { return a.mid + ((long long)id * a.Hq + hq) * (kHeadDim + 1); };
    const int t0 = (id - plan.base) * 32 * plan.chunk;
    const int t1 = min(32 * vis.tiles(), t0 + 32 * plan.chunk);

    __shared__ float s_cent[16];
    __shared__ float s_m[kWarps][GM], s_l[kWarps][GM];
    __shared__ float s_acc[kWarps][GM][kHeadDim];

    if (L > a.mods.max_len) {                // past what can be listed: a NaN lse, nothing read
        if (threadIdx.x < G) partial(h * G + threadIdx.x)[kHeadDim] = __int_as_float(0x7fc00000);
        return;
    }
    __shared__ int s_bad;        // a block-table entry outside [0, num_blocks) was met
    if (threadIdx.x == 0) s_bad = 0;
    if constexpr (!KEY_FP8) {
        if (threadIdx.x < (1 << KBITS)) s_cent[threadIdx.x] = a.centroids[threadIdx.x];
    }

    // q (rotated once for MSE keys), pre-multiplied by the softmax scale
    float qv[GM][4];
    const TQ* Q = static_cast<const TQ*>(a.query);
    float sgn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sgn[i] = KEY_FP8 ? 1.f : float(a.signs[4 * lane + i]);
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        if (g < G) {
            const TQ* qp = Q + ((long long)b * a.Hq + h * G + g) * kHeadDim + 4 * lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[g][i] = sgn[i] * to_f32(qp[i]);
            if constexpr (!KEY_FP8) {
                fwht128_warp(qv[g], lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) qv[g][i] *= 0.08838834764831845f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[g][i] *= a.scale;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[g][i] = 0.f;
        }
    }
    __syncthreads();

    float m[GM], l[GM], acc[GM][4];
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][i] = 0.f;
    }

    const int32_t* bt = a.block_table + (long long)b * a.bt_stride;
    const int lgbs = 31 - __clz(a.bs);       // block sizes are powers of two
    bool bad = false;
    for (int v = t0 + warp; v < t1; v += kWarps) {
        const int t = vis.base(v >> 5) + (v & 31);
        if (!vis.sees(t)) continue;
        const long long page = bt[t >> lgbs];
        if (page < 0 || page >= a.num_blocks) { bad = true; continue; }   // not read; the rows become NaN
        const uint8_t *sp, *mp;              // data and metadata of the record
        slot_ptrs(a.g, a.cache, page, t & (a.bs - 1), h, a.bs, a.Hk, sp, mp);

        float kv[4];
        float knorm = 1.f;
        if constexpr (KEY_FP8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __half_raw hr = __nv_cvt_fp8_to_halfraw(sp[4 * lane + i], __NV_E4M3);
                kv[i] = __half2float(__half(hr));
            }
        } else {
            int c[4];
            load_codes<KBITS>(sp, lane, c);
#pragma unroll
            for (int i = 0; i < 4; ++i) kv[i] = s_cent[c[i]];
            knorm = __half2float(__ushort_as_half(ld_u16(mp + a.g.m_norm)));
        }
        float s[GM];
#pragma unroll
        for (int g = 0; g < GM; ++g)
            s[g] = warp_sum(qv[g][0] * kv[0] + qv[g][1] * kv[1] + qv[g][2] * kv[2] + qv[g][3] * kv[3]) * knorm;

        float mine = 0.f;                // the score this lane writes (query head `lane`)
        if (a.mods.cap > 0.f) softcap_warp(s, a.mods.cap, a.mods.inv_cap);
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            if (a.mods.slopes && g < G) s[g] = fmaf(-a.mods.slopes[h * G + g], float(L - 1 - t), s[g]);
            if (lane == g) mine = s[g];
        }
        if (a.mods.scores && lane < G)
            a.mods.scores[(((long long)b * a.Hk + h) * a.mods.vtok + v) * a.mods.gp + lane] =
                mine * 1.4426950408889634f;

        // online softmax
        float al[GM], pv[GM];
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            const float mn = fmaxf(m[g], s[g]);
            const float p = expf(s[g] - mn);
            al[g] = expf(m[g] - mn);
            l[g] = l[g] * al[g] + p;
            m[g] = mn;
            pv[g] = p;
        }
        float vv[4];
        int vc[4];
        load_codes<VBITS>(sp + a.g.v_off, lane, vc);
        const float vs = __half2float(__ushort_as_half(ld_u16(mp + a.g.m_scale)));
        const float vz = __half2float(__ushort_as_half(ld_u16(mp + a.g.m_zero)));
#pragma unroll
        for (int i = 0; i < 4; ++i) vv[i] = float(vc[i]) * vs + vz;
#pragma unroll
        for (int g = 0; g < GM; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[g][i] = acc[g][i] * al[g] + pv[g] * vv[i];
    }

    // merge the four warps' partials
    if (bad && lane == 0) s_bad = 1;
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        if (lane == 0) { s_m[warp][g] = m[g]; s_l[warp][g] = l[g]; }
#pragma unroll
        for (int i = 0; i < 4; ++i) s_acc[warp][g][4 * lane + i] = acc[g][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * kHeadDim; i += blockDim.x) {
        const int g = i / kHeadDim, d = i % kHeadDim;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][g]);
        float lsum = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = s_m[w][g] == -INFINITY ? 0.f : expf(s_m[w][g] - M);
            lsum += s_l[w][g] * f;
            o += s_acc[w][g][d] * f;
        }
        float* mp = partial(h * G + g);
        mp[d] = lsum == 0.f ? 0.f : o / lsum;    // every page of the split lay outside the cache
        if (d == 0) mp[kHeadDim] = s_bad ? __int_as_float(0x7fc00000) : M + logf(lsum);
    }
}

template <typename TQ, bool FP8, int KB, int VB>
cudaError_t launch_scored_g(const DecodeArgs& a, cudaStream_t st)
{
    dim3 grid(a.num_splits, a.Hk, a.B);
    if (a.G <= 1) scored_kernel<TQ, FP8, KB, VB, 1><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.G <= 2) scored_kernel<TQ, FP8, KB, VB, 2><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.G <= 4) scored_kernel<TQ, FP8, KB, VB, 4><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.G <= 8) scored_kernel<TQ, FP8, KB, VB, 8><<<grid, kWarps * 32, 0, st>>>(a);
    else scored_kernel<TQ, FP8, KB, VB, 16><<<grid, kWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename TQ>
cudaError_t launch_scored(int preset, const DecodeArgs& a, cudaStream_t st)
{
    switch (preset & 0xFF) {
    case TQ_K8V4:    return launch_scored_g<TQ, true, 4, 4>(a, st);
    case TQ_4BIT_NC: return launch_scored_g<TQ, false, 4, 4>(a, st);
    case TQ_K3V4_NC: return launch_scored_g<TQ, false, 3, 4>(a, st);
    case TQ_3BIT_NC: return launch_scored_g<TQ, false, 3, 3>(a, st);
    case TQ_2BIT_NC: return launch_scored_g<TQ, false, 2, 2>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cores_scored(int preset, int q_dtype, const DecodeArgs& a, cudaStream_t st)
{
    return q_dtype == TQ_F16 ? launch_scored<__half>(preset, a, st) : launch_scored<__nv_bfloat16>(preset, a, st);
}

}  // namespace tq
