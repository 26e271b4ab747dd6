// CUDA-core decode stage 1, for the shapes the tensor-core stage 1
// (tq_decode_mma.cuh) does not serve: one CTA per (split, kv head, sequence),
// four warps striding over the split's tokens, 4 coordinates per lane, fp32
// scores and online softmax, partials merged across warps in shared memory.
// Method sources: as tq_decode.cu.
#pragma once

#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

struct DecodeArgs {
    const void* query;
    const uint8_t* cache;
    long long num_blocks;
    const int32_t* block_table;
    int bt_stride;
    const int32_t* seq_lens;
    float scale;
    int num_splits;
    const int8_t* signs;
    const float* centroids;
    float* mid;          // (B, Hq, S, D+1)
    void* out;
    float* lse;
    int B, Hq, Hk, G, bs;
    float vthr;          // sparse V: rows with p <= vthr skip the value sum (0: off)
    SlotGeom g;
    ScoreArgs mods;      // SCORED instantiations only
};

// CUDA-core stage 1 with score modifiers (its own translation unit)
cudaError_t launch_cores_scored(int preset, int q_dtype, const DecodeArgs& a, cudaStream_t st);

namespace {

constexpr int kWarps = 4;

// Codes 4*lane .. 4*lane+3 of a packed code stream starting at p (2-byte
// aligned).  Every width is an LSB-first bitstream: 4 bits low nibble first,
// 2 bits four per byte, 3 bits 8 codes per 3 bytes (the lane's 12 bits start
// at bit 12*lane, i.e. byte 3*lane/2 plus 0 or 4 bits).
template <int BITS>
__device__ __forceinline__ void load_codes(const uint8_t* p, int lane, int (&c)[4])
{
    if constexpr (BITS == 2) {
        const uint32_t w = p[lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = (w >> (2 * i)) & 3u;
    } else if constexpr (BITS == 4) {
        const uint32_t w = ld_u16(p + 2 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = (w >> (4 * i)) & 15u;
    } else {
        static_assert(BITS == 3, "2, 3 or 4 bits");
        const uint8_t* q = p + ((3 * lane) >> 1);
        const uint32_t w = (uint32_t(q[0]) | uint32_t(q[1]) << 8) >> (4 * (lane & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = (w >> (3 * i)) & 7u;
    }
}

// SCORED: softcap, distance bias and the visible tokens of ScoreArgs, with the
// scores kept when asked; the splits then share the list of visible tiles.
template <typename TQ, bool KEY_FP8, int KBITS, int VBITS, int GM, bool SCORED>
__global__ void __launch_bounds__(kWarps * 32) stage1_kernel(DecodeArgs a)
{
    const int h = blockIdx.y;
    int split = blockIdx.x, b = blockIdx.z, chunk = 0;
    // scored: the launch's splits go by the plan of the batch (SplitPlan)
    [[maybe_unused]] int id = 0;
    if constexpr (SCORED) {
        __shared__ int s_plan[kPlanMax + 4];
        id = blockIdx.z * a.num_splits + blockIdx.x;
        const SplitPlan plan(a.mods, a.seq_lens, a.num_splits, id, blockIdx.x + blockIdx.y + blockIdx.z == 0, s_plan);
        if (plan.b < 0) return;
        b = plan.b;
        split = id - plan.base;
        chunk = 32 * plan.chunk;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.G, S = a.num_splits;
    const int L = a.seq_lens[b];
    [[maybe_unused]] VisibleSet vis(SCORED ? a.mods : ScoreArgs{}, SCORED ? min(L, a.mods.max_len) : 0, b);
    const int n = SCORED ? 32 * vis.tiles() : L;     // positions the splits share
    if constexpr (!SCORED) chunk = (n + S - 1) / S;
    // this split's partial of query head hq
    auto partial = [&](int hq) {
        return a.mid + (SCORED ? (long long)id * a.Hq + hq : ((long long)b * a.Hq + hq) * S + split) * (kHeadDim + 1);
    };
    const int t0 = split * chunk;
    const int t1 = min(n, t0 + chunk);
    const bool too_long = SCORED && L > a.mods.max_len;   // past what can be listed

    __shared__ float s_cent[16];
    __shared__ float s_m[kWarps][GM], s_l[kWarps][GM];
    __shared__ float s_acc[kWarps][GM][kHeadDim];

    if (t0 >= t1 || too_long) {   // empty split: lse = -inf (too long: NaN), zero partial output
        for (int i = threadIdx.x; i < G * (kHeadDim + 1); i += blockDim.x) {
            const int g = i / (kHeadDim + 1), d = i % (kHeadDim + 1);
            partial(h * G + g)[d] = d == kHeadDim ? (too_long ? __int_as_float(0x7fc00000) : -INFINITY) : 0.f;
        }
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
        const int t = SCORED ? vis.base(v >> 5) + (v & 31) : v;
        if (SCORED && !vis.sees(t)) continue;
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

        if constexpr (SCORED) {
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
        }

        // online softmax; sparse V: a row whose p is at most vthr keeps its
        // weight in l but adds nothing to the value sum, and the value codes
        // are not read when no head keeps the row (s is warp-uniform)
        float al[GM], pv[GM];
        bool anyv = false;
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            const float mn = fmaxf(m[g], s[g]);
            const float p = expf(s[g] - mn);
            al[g] = expf(m[g] - mn);
            l[g] = l[g] * al[g] + p;
            m[g] = mn;
            pv[g] = p > a.vthr ? p : 0.f;
            anyv |= g < G && pv[g] > 0.f;
        }
        float vv[4] = {0.f, 0.f, 0.f, 0.f};
        if (anyv) {
            int vc[4];
            load_codes<VBITS>(sp + a.g.v_off, lane, vc);
            const float vs = __half2float(__ushort_as_half(ld_u16(mp + a.g.m_scale)));
            const float vz = __half2float(__ushort_as_half(ld_u16(mp + a.g.m_zero)));
#pragma unroll
            for (int i = 0; i < 4; ++i) vv[i] = float(vc[i]) * vs + vz;
        }
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
        mp[d] = SCORED && lsum == 0.f ? 0.f : o / lsum;      // a split may list no visible token
        if (d == 0) mp[kHeadDim] = s_bad ? __int_as_float(0x7fc00000) : M + logf(lsum);
    }
}

template <typename TQ, bool FP8, int KB, int VB, bool SCORED>
cudaError_t launch_stage1_g(const DecodeArgs& a, cudaStream_t st)
{
    dim3 grid(a.num_splits, a.Hk, a.B);
    if (a.G <= 1) stage1_kernel<TQ, FP8, KB, VB, 1, SCORED><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.G <= 2) stage1_kernel<TQ, FP8, KB, VB, 2, SCORED><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.G <= 4) stage1_kernel<TQ, FP8, KB, VB, 4, SCORED><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.G <= 8) stage1_kernel<TQ, FP8, KB, VB, 8, SCORED><<<grid, kWarps * 32, 0, st>>>(a);
    else stage1_kernel<TQ, FP8, KB, VB, 16, SCORED><<<grid, kWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename TQ, bool SCORED>
cudaError_t launch_stage1(int preset, const DecodeArgs& a, cudaStream_t st)
{
    switch (preset & 0xFF) {
    case TQ_K8V4:    return launch_stage1_g<TQ, true, 4, 4, SCORED>(a, st);
    case TQ_4BIT_NC: return launch_stage1_g<TQ, false, 4, 4, SCORED>(a, st);
    case TQ_K3V4_NC: return launch_stage1_g<TQ, false, 3, 4, SCORED>(a, st);
    case TQ_3BIT_NC: return launch_stage1_g<TQ, false, 3, 3, SCORED>(a, st);
    case TQ_2BIT_NC: return launch_stage1_g<TQ, false, 2, 2, SCORED>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace tq
