// What the CUDA-core decode stages 1 share (tq_decode.cu: plain,
// tq_decode_cores_scored.cu: with score modifiers): their arguments and the
// reading of packed codes.
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
    ScoreArgs mods;      // scored kernel only (tq_decode_cores_scored.cu)
};

// CUDA-core stage 1 with score modifiers (tq_decode_cores_scored.cu)
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

}  // namespace
}  // namespace tq
