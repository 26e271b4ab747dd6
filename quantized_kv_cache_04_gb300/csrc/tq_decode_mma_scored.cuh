// Decode stage 1 on tensor cores with score modifiers: distance bias and visible
// tokens (kScored), softcap too (kCapped), and the scores kept for the attention
// weights as well (kWeights, where a cap of 0 is none).
//
// The tile pipeline is the plain kernel's (tq_decode_mma.cuh: layout of the
// ring, score and value MMAs, precision, launch chain) with the same helpers.
// It is a kernel of its own, not a mode of that one: modes of one text moved
// the plain decode's register allocation (up to 3% of its time).  What differs:
//   - splits are given out by the batch's visible lengths (SplitPlan);
//   - the list of tiles that hold visible tokens in place of all tiles, newest
//     first; pages without a visible token are not looked up;
//   - between scores and softmax: cap, bias, and the kept scores;
//   - the value sum about the middle code.
// Bound, like the plain kernel, by instruction issue and shared-memory lookups for
// 2- to 4-bit keys, by the copies for FP8 keys: 4 to 9% above the plain decode of
// the same tokens, up to 15% for groups of 8 (4 sequences of 65536 tokens, 8 kv
// heads, capped; plain in brackets: 32 query heads k8v4 74 us (75) = 0.82 of the
// copy bandwidth, k3v4 92 (85) = 0.40, 4bit 101 (94), 3bit 99 (93); 64 query
// heads 96 (84), 122 (106), 130 (117), 131 (120)).
// Modes are instantiations, not branches: a branch between the scores and the
// softmax ends the block in which the compiler overlaps a tile's loads, lookups
// and MMAs.  The bias is always added (a slope of 0).
#pragma once

#include "tq_decode_mma.cuh"

namespace tq {
namespace {

constexpr int kScored = 0, kCapped = 1, kWeights = 2;
constexpr int kWordRows = 0, kSoa = 1, kHalfRows = 2;

// The same with the bytes first to leave the L2: cache rows of a call that
// keeps its scores, so that the scores stay there for the weights kernel
// (524K tokens, 64 query heads: 239 -> 234 us).
__device__ __forceinline__ void bulk_g2s_once(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// Stores of kept scores where `put`, without a branch and, as nothing in the
// kernel reads them, without a memory clobber that would keep the compiler from
// moving a tile's loads across.
__device__ __forceinline__ void store_if(float* p, float x, int put)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %2, 0;\n\t@q st.global.f32 [%0], %1;\n\t}"
                 ::"l"(p), "f"(x), "r"(put));
}
__device__ __forceinline__ void store_if(float* p, float x, float y, int put)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %3, 0;\n\t@q st.global.v2.f32 [%0], {%1, %2};\n\t}"
                 ::"l"(p), "f"(x), "f"(y), "r"(put));
}

// LAY: kWordRows (AoS, token rows of whole 32-bit words), kSoa, or kHalfRows (AoS
// rows of 2 mod 4 bytes, e.g. 3 kv heads of 118-byte slots: every load finds its
// own misalignment).
template <typename TQ, int KMODE, int VBITS, int G, int LAY, int MODE>
__global__ void __launch_bounds__(512) scored_mma_kernel(const __grid_constant__ MmaArgs a)
{
    constexpr bool CAPPED = MODE != kScored, KEEP = MODE == kWeights, SOA = LAY == kSoa;
    extern __shared__ __align__(128) uint8_t smem[];
    // 3-bit keys: the code-pair centroid table (8 KB; one element elsewhere)
    __shared__ __align__(16) uint2 key_lut[KMODE == 3 ? kLut3Entries : KMODE == 4 ? kLut4Entries : 1];
    // launched as a programmatic dependent of the previous kernel in the
    // stream (typically the store of the step's new tokens): wait for it to
    // complete before the first read of global memory
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // blockIdx.x = (split * nqg + qg) * (Hk / hpc) + kv-head group: the
    // CTAs that read the parts of the same token rows (kv-head groups) and
    // the same pages (query-head groups) are neighbours in launch order, so
    // they run together (DRAM pages and L2 lines are used once)
    const int ngroups = a.Hk / a.hpc;
    const int kvg = blockIdx.x % ngroups;     // which hpc kv heads
    const int qg = (blockIdx.x / ngroups) % a.nqg;   // which 8 query heads of each kv head (G > 8)
    // which sequence's split this is goes by the plan of the batch
    const int id = blockIdx.y * a.num_splits + blockIdx.x / ngroups / a.nqg;
    const SplitPlan plan(a.mods, a.seq_lens, a.num_splits, id, blockIdx.x == 0 && blockIdx.y == 0,
                         reinterpret_cast<int*>(smem));
    if (plan.b < 0) return;
    const int b = plan.b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3;
    const int h0 = kvg * a.hpc;               // first kv head of this CTA
    const int h = h0 + warp;                   // this warp's kv head
    // query heads of this CTA per kv head: Greal of them from qh0 (all G
    // when G <= 8); query head of (kv head hh, column g) = hh * Gall + qh0 + g
    const int Hq = a.Hq, Gall = a.G;
    const int qh0 = 8 * qg;
    const int Greal = a.nqg > 1 ? min(8, Gall - qh0) : Gall;
    const int Hc = a.hpc;
    const int nwarps = blockDim.x >> 5;

    const int L = a.seq_lens[b];
    // this split's partial of query head hq
    auto partial = [&](int hq) { return a.mid + ((long long)id * Hq + hq) * (kHeadDim + 1); };
    const int t_begin = (id - plan.base) * plan.chunk * kTile;
    int t_end = 0;
    // t_begin and t_end are positions in the list of tiles that hold
    // visible tokens (32 per tile).  What the tile loop needs of the visible set
    // lies in shared memory (registers are what G = 8 runs out of), as do the
    // heads' slopes
    __shared__ int s_vis[sizeof(VisibleSet) / 4];
    __shared__ float s_slope[16 * 8];
    __shared__ float* s_keep[KEEP ? 16 : 1];      // where each warp's kv head keeps its scores
    __shared__ __align__(16) int s_tiles[4];      // na, token of tile 0, of tile na less 32 na, last tile
    const VisibleSet& vis = *reinterpret_cast<const VisibleSet*>(s_vis);
    {
        const VisibleSet v(a.mods, min(L, a.mods.max_len), b);
        t_end = min(v.tiles() * kTile, t_begin + plan.chunk * kTile);
        if (threadIdx.x == 0) {
            *reinterpret_cast<VisibleSet*>(s_vis) = v;
            *reinterpret_cast<int4*>(s_tiles) = make_int4(v.na, v.base(0), (v.b0 - v.na) << 5, v.tiles() - 1);
        }
        if (KEEP && lane == 0)
            s_keep[warp] = a.mods.scores + ((long long)b * a.Hk + h) * a.mods.vtok * a.mods.gp + qh0;
        for (int i = threadIdx.x; i < Hc * 8; i += blockDim.x)
            s_slope[i] = a.mods.slopes && i % 8 < Greal
                             ? a.mods.slopes[(h0 + i / 8) * Gall + qh0 + i % 8] * 1.4426950408889634f : 0.f;
    }
    // listed tile v: its first token, and whether it surely holds nothing hidden
    auto vis_base = [&](int v) { return (v << 5) + (v < s_tiles[0] ? s_tiles[1] : s_tiles[2]); };
    auto vis_whole = [&](int v) { return v != 0 && v + 1 != s_tiles[0] && v != s_tiles[0] && v != s_tiles[3]; };

    if (L > a.mods.max_len || a.num_blocks <= 0) {
        // a sequence past what can be listed, or no cache block to read from: a
        // NaN lse, nothing read
        for (int i = threadIdx.x; i < Hc * Greal; i += blockDim.x)
            partial((h0 + i / Greal) * Gall + qh0 + i % Greal)[kHeadDim] = __int_as_float(0x7fc00000);
        return;
    }

    // ---------------- shared-memory ring of 32 token rows (the CTA's kv
    // heads), filled by bulk (TMA) copies.  Rows of one page are contiguous in
    // global memory: one copy per page segment when the CTA takes whole rows
    // and the shared row stride equals the global one, else one copy per row
    // (issued by the 32 lanes of one warp).
    const int row_bytes = a.row_bytes;        // global token row (Hk slots)
    const int cb = a.copy_bytes;              // bytes of it this CTA copies (SoA: data part)
    const int rs = a.smem_row;                // shared row stride: 16 mod 32 bytes
    const int mb = SOA ? a.meta_bytes : 0;    // SoA: metadata part per token, rows after the data rows
    const int stage_bytes = kTile * (rs + mb);
    const int NST = a.nstages;
    const int ntiles = (t_end - t_begin + kTile - 1) / kTile;
    // the newest tokens first, whose biased scores are the largest, so
    // that the running maximum seldom moves
    auto vis_tile = [&](int tile) { return (t_begin >> 5) + ntiles - 1 - tile; };
    const int32_t* bt = a.block_table + (long long)b * a.bt_stride;
    const int lg = a.bs_log2;
    const int seg_rows = kTile < (1 << lg) ? kTile : (1 << lg);   // rows per page segment
    const int seg_lg = lg < 5 ? lg : 5;                                  // log2(seg_rows)
    // Per stage: `full` completes when the stage's bytes have landed; `done`
    // counts the warps finished with it.  The warp that finishes a stage last
    // refills it, so warps never wait on each other, only on data.
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + NST * stage_bytes);
    int* done = reinterpret_cast<int*>(full + NST);
    int* bad_pages = done + NST;               // a block-table entry outside the cache was met
    int* finished = bad_pages + 1;             // warps past their epilogue
    // MSE keys with G = 8 keep their q fragments (hi and lo, 32 words per
    // thread) in tensor memory: 32 columns per group of 4 warps, the address
    // written by the allocation to the word after the stage counters
    constexpr bool kQt = KMODE != 8 && G == 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + NST * stage_bytes + 16 * NST);
    const uint32_t q_cols = nwarps <= 4 ? 32u : nwarps <= 8 ? 64u : 128u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) { mbar_init(&full[i], 1); done[i] = 0; }
        *bad_pages = 0;
        *finished = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if constexpr (kQt) {
        if (warp == 0) tmem_alloc(tmem_slot, q_cols);
        tmem_fence_before_sync();
    }
    __syncthreads();
    uint32_t tq = 0;                           // this thread's q columns (k-step 0)
    if constexpr (kQt) {
        tmem_fence_after_sync();
        tq = *reinterpret_cast<volatile uint32_t*>(tmem_slot) + ((32u * uint32_t(warp & 3)) << 16) +
             32u * uint32_t(warp >> 2);
    }
    // Only rows of tokens < L are copied: block-table entries past the
    // sequence's last page are never read.  Skipped rows keep stale bytes and
    // are masked out of the softmax.
    // SoA blocks: the token rows' data parts and metadata parts lie in two
    // regions of the block; each row (or page segment) takes one copy per
    // region, the metadata landing in rows of mb bytes after the data rows.
    constexpr bool soa = SOA;                  // the block convention (a.g.soa), fixed per instantiation
    const long long hs_g = soa ? a.g.data_bytes : a.g.slot;    // head stride in a global data row
    const long long drow = soa ? (long long)a.Hk * a.g.data_bytes : row_bytes;
    bool bad_seen = false;                     // this lane replaced a page outside the cache
    // tensor copies land on 128-byte aligned stage and segment offsets
    // (stage_bytes and the segment size are multiples of 128 for these
    // rows); a ring base that is not would take the per-row copies
    // (FP8 keys only: the other instantiations carry no tensor-copy code)
    const bool use_tm = KMODE == 8 && !soa && a.use_tmap && (smem_u32(smem) & 127u) == 0;
    auto issue = [&](int tile, int stage) {   // called by all lanes of one warp
        if (tile >= ntiles) return;
        uint8_t* dst = smem + stage * stage_bytes;
        uint64_t* bar = &full[stage];
        const int tbase = vis_base(vis_tile(tile));
        // data rows: one copy per page segment when the CTA takes whole rows
        // and the shared stride equals the global one, or through the tensor
        // map (a box of the CTA's part of a segment's rows), else one per
        // row; SoA metadata rows (unpadded in shared memory): one copy per
        // page segment when the CTA takes every kv head
        const bool seg_d = (rs == drow && cb == drow) || use_tm;
        const bool seg_m = soa && mb == a.Hk * a.g.meta_bytes;
        const int len_d = seg_d ? seg_rows : 1, len_m = seg_m ? seg_rows : 1;   // rows per copy
        const int lg_d = seg_d ? seg_lg : 0, lg_m = seg_m ? seg_lg : 0;      // (powers of two)
        const int nd = kTile >> lg_d;
        const int nm = soa ? kTile >> lg_m : 0;
        // only copies that bring a visible token (the pages of others
        // may have been freed)
        bool want_d = true, want_m = true;
        int cnt_d = nd, cnt_m = nm;
        if (!vis_whole(vis_tile(tile))) {     // warp-uniform
            want_d = vis.any(tbase + lane * len_d, len_d);
            want_m = vis.any(tbase + lane * len_m, len_m);
            cnt_d = __popc(__ballot_sync(0xffffffffu, lane < nd && want_d));
            if constexpr (soa) cnt_m = __popc(__ballot_sync(0xffffffffu, lane < nm && want_m));
        }
        if (lane == 0) {
            fence_async_shared();             // prior generic reads of this stage before the async writes
            mbar_expect_tx(bar, uint32_t(cnt_d * len_d * cb + cnt_m * len_m * mb));
        }
        __syncwarp();
        const bool same = !soa || len_d == len_m;     // one address computation for both copies
        // a block-table entry outside [0, num_blocks) is replaced by page 0,
        // so nothing outside the cache is read, and noted: the CTA's rows
        // come out NaN (see the end of the kernel)
        if (lane < nd && want_d) {
            const int t = tbase + lane * len_d;
            long long page = bt[t >> lg];
            if ((unsigned long long)page >= (unsigned long long)a.num_blocks) { page = 0; bad_seen = true; }
            const int off = t & ((1 << lg) - 1);
            const uint8_t* blk = a.cache + (page << lg) * (long long)row_bytes;
            if (KMODE == 8 && !soa && use_tm) {
                tma_load_2d(dst + lane * len_d * rs, &a.tmap, int(h0 * hs_g) >> 2, int((page << lg) + off), bar);
            } else {
                const uint8_t* src =
                    soa ? blk + off * drow + h0 * hs_g : blk + off * (long long)row_bytes + h0 * hs_g;
                if constexpr (KEEP) bulk_g2s_once(dst + lane * len_d * rs, src, uint32_t(len_d * cb), bar);
                else                bulk_g2s(dst + lane * len_d * rs, src, uint32_t(len_d * cb), bar);
            }
            if (soa && same) {
                const uint8_t* meta = blk + (1LL << lg) * drow + ((long long)off * a.Hk + h0) * a.g.meta_bytes;
                bulk_g2s(dst + kTile * rs + lane * len_m * mb, meta, uint32_t(len_m * mb), bar);
            }
        }
        if (!same && lane < nm && want_m) {
            const int t = tbase + lane * len_m;
            long long page = bt[t >> lg];
            if ((unsigned long long)page >= (unsigned long long)a.num_blocks) { page = 0; bad_seen = true; }
            const int off = t & ((1 << lg) - 1);
            const uint8_t* blk = a.cache + (page << lg) * (long long)row_bytes;
            const uint8_t* meta = blk + (1LL << lg) * drow + ((long long)off * a.Hk + h0) * a.g.meta_bytes;
            bulk_g2s(dst + kTile * rs + lane * len_m * mb, meta, uint32_t(len_m * mb), bar);
        }
    };
    // The q staging area (hpc x (4 or 8) heads x 512 B) sits at the end of the
    // ring: the tiles whose stages lie wholly before it are requested first,
    // so their latency overlaps the preparation of q.
    const int q_base = NST * stage_bytes - Hc * G * kHeadDim * 4;
    const int s_q = q_base / stage_bytes;
    if (warp == 0)
        for (int i = 0; i < s_q; ++i) issue(i, i);

    // ---------------- q columns: B operand of the score MMA.  Each warp
    // rotates (MSE keys) and scales its G query heads with lane l holding dims
    // 4l..4l+3, parks them in the staging area, and every thread reads back
    // the 32 values of its column.  The k index of k-step kk and thread tig
    // maps to dims
    //   FP8 keys:   16 kk + 4 tig + j   one key word per k-step, bank-conflict
    //               free across the warp
    //   3-bit keys: 32 tig + 4 kk + j   12 bytes (32 codes) per thread and row
    //   4-bit keys: the same, 16 bytes per thread
    //   2-bit keys: 32 tig + 16 (kk >> 2) + 8 (kk & 1) + ((kk >> 1) & 1) + 2 j
    //               (8 bytes per thread; see qk_tile)
    // 2-bit keys: the host passes a scale alpha that makes every alpha * c_k
    // of the library's codebook an fp16 value to 5e-7 relative.  If that holds
    // for the centroids given (the same test in every thread), the keys use
    // fp16(alpha c_k) alone and q carries 1 / alpha: no lo lookups or MMAs.
    float key_alpha = 1.f;
    bool key_lo = KMODE != 8;
    if constexpr (KMODE == 2) {
        const float al = a.key_alpha;
        float err = (al >= 1.f && al < 2.f) ? 0.f : INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = al * a.centroids[k];
            const float d = fabsf(x - __half2float(__float2half_rn(x)));
            err = fmaxf(err, x != 0.f ? d / fabsf(x) : d);
        }
        if (err <= 5e-7f) { key_alpha = al; key_lo = false; }
    }

    // 3- and 4-bit keys: entry e (codes e mod 2^bits and e >> bits) of the
    // pair table holds fp16x2 (hi) and fp16x2 (lo) of the two centroids, once
    // per half-warp lane; the barrier after the q staging below orders it
    // before any use
    if constexpr (KMODE == 3 || KMODE == 4) {
        // one (entry, two copies) per step: a 16-byte store of the entry twice
        constexpr int NE = KMODE == 3 ? kLut3Entries : kLut4Entries;
        for (int i = threadIdx.x; i < NE / 2; i += blockDim.x) {
            const int e = i >> 3;
            float h0, l0, h1, l1;
            split_f16(a.centroids[e & ((1 << KMODE) - 1)], h0, l0);
            split_f16(a.centroids[e >> KMODE], h1, l1);
            const uint32_t x = pack_half2(h0, h1), y = pack_half2(l0, l1);
            reinterpret_cast<uint4*>(key_lut)[i] = make_uint4(x, y, x, y);
        }
    }

    // MSE keys with G = 8 keep their q fragments in tensor memory (read once
    // per k-step) instead of 32 registers (the register file is the limit of
    // that instantiation) or 4 KB of shared memory per warp (which a third
    // ring stage needs).
    uint32_t bq[8][2], bql[8][2];
    {
        float* sq = reinterpret_cast<float*>(smem + q_base) + warp * G * kHeadDim;
        float sgn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sgn[i] = KMODE == 8 ? 1.f : float(a.signs[4 * lane + i]);
        const TQ* Q = static_cast<const TQ*>(a.query);
        for (int g = 0; g < G; ++g) {
            float qv[4] = {0.f, 0.f, 0.f, 0.f};
            if (g < Greal) {        // warp-uniform
                const TQ* qp = Q + ((long long)b * Hq + h * Gall + qh0 + g) * kHeadDim + 4 * lane;
#pragma unroll
                for (int i = 0; i < 4; ++i) qv[i] = sgn[i] * to_f32(qp[i]);
                if constexpr (KMODE != 8) {
                    fwht128_warp(qv, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) qv[i] *= 0.08838834764831845f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) qv[i] *= a.qscale / key_alpha;
            }
            reinterpret_cast<float4*>(sq + g * kHeadDim)[lane] = make_float4(qv[0], qv[1], qv[2], qv[3]);
        }
        __syncwarp();
        const int col_head = G == 4 ? (gid >> 1) : gid;
        const bool col_lo = G == 4 && (gid & 1);
        const float* qc = sq + col_head * kHeadDim;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            float4 x;
            if constexpr (KMODE == 2) {
                // dims 32 tig + 16 (kk >> 2) + 8 (kk & 1) + ((kk >> 1) & 1) + 2 j
                const float* qd = qc + 32 * tig + 16 * (kk >> 2) + 8 * (kk & 1) + ((kk >> 1) & 1);
                x = make_float4(qd[0], qd[2], qd[4], qd[6]);
            } else {
                x = reinterpret_cast<const float4*>(qc + (KMODE == 8 ? 16 * kk + 4 * tig : 32 * tig + 4 * kk))[0];
            }
            float hi[4], lo[4];
            split_f16(x.x, hi[0], lo[0]);
            split_f16(x.y, hi[1], lo[1]);
            split_f16(x.z, hi[2], lo[2]);
            split_f16(x.w, hi[3], lo[3]);
            if (G == 4) {
                bq[kk][0] = col_lo ? pack_half2(lo[0], lo[1]) : pack_half2(hi[0], hi[1]);
                bq[kk][1] = col_lo ? pack_half2(lo[2], lo[3]) : pack_half2(hi[2], hi[3]);
                bql[kk][0] = bql[kk][1] = 0u;
            } else {
                bq[kk][0] = pack_half2(hi[0], hi[1]);
                bq[kk][1] = pack_half2(hi[2], hi[3]);
                bql[kk][0] = pack_half2(lo[0], lo[1]);
                bql[kk][1] = pack_half2(lo[2], lo[3]);
                if constexpr (kQt) {
                    tmem_st4(tq + 4 * kk, make_uint4(bq[kk][0], bq[kk][1], bql[kk][0], bql[kk][1]));
                    bq[kk][0] = bq[kk][1] = bql[kk][0] = bql[kk][1] = 0u;
                }
            }
        }
        if constexpr (kQt) tmem_wait_st();
        __syncthreads();            // every warp is done with the staging area
    }
    if (warp == 0)
        for (int i = s_q; i < NST; ++i) issue(i, i);

    // ---------------- centroid byte planes for the PRMT lookup (2-bit keys):
    // plane 0/1 = low/high byte of fp16(c), plane 2/3 = low/high byte of the
    // fp16 residual c - fp16(c), with c = key_alpha * c_k; T[p][0] holds the
    // four codes' bytes of plane p
    uint32_t T[4][2] = {};
    if constexpr (KMODE == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float c = key_alpha * a.centroids[k];
            const __half chi = __float2half_rn(c);
            const __half clo = __float2half_rn(c - __half2float(chi));
            const uint32_t hb = __half_as_ushort(chi), lb = __half_as_ushort(clo);
            const int sh = 8 * k;
            T[0][0] |= (hb & 0xFFu) << sh;
            T[1][0] |= (hb >> 8) << sh;
            T[2][0] |= (lb & 0xFFu) << sh;
            T[3][0] |= (lb >> 8) << sh;
        }
    }

    constexpr int NH = G == 8 ? 2 : 1;        // query heads per thread (softmax state)
    float m_run[NH], l_run[NH], z_run[NH];
#pragma unroll
    for (int j = 0; j < NH; ++j) { m_run[j] = -INFINITY; l_run[j] = 0.f; z_run[j] = 0.f; }
    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    constexpr float kMidCode = 0.5f * float((1 << VBITS) - 1);
    const int tau0 = gid, tau1 = gid + 8;      // this thread's QK rows
    const uint32_t l8 = uint32_t(lane & 15) * 8;   // this lane's copy in a pair-table entry
    const int hoff = warp * int(hs_g);         // this warp's slot (SoA: data record) in a shared row
    const int kmis = hoff & 2;
    const int vmis = (hoff + a.g.v_off) & 2;
    // metadata rows: AoS = the data rows (fields inside the slot); SoA = the
    // rows after the data rows, mb bytes each
    const int mrs = soa ? mb : rs;
    const int moff = soa ? kTile * rs + warp * a.g.meta_bytes : hoff;

    // One 32-token tile in stage memory st (this warp's slot at offset 0).
    // PARTIAL: some of its tokens lie at or past t_end and are masked.
    // KGEN: the general key path; false: 2-bit keys without the lo part
    // (key_alpha)
    // KM / VM: the key / value misalignment of this warp's slot (0 or 2)
    // vt: the tile's first position in the list of visible tiles
    auto tile = [&](const uint8_t* st, const uint8_t* sm, int t0, [[maybe_unused]] int vt, auto partial_tag,
                    auto lo_tag, auto km_tag, auto vm_tag) {
        constexpr bool PARTIAL = decltype(partial_tag)::value;
        [[maybe_unused]] constexpr bool KGEN = decltype(lo_tag)::value;
        constexpr int KM = decltype(km_tag)::value, VM = decltype(vm_tag)::value;
        // ---- scores of both 16-row tiles
        float s[NH][2][2], vs[2][2], vz[2][2];
        bool ok[2][2];
        [[maybe_unused]] float sc2[2][4], scl2[2][4];
        if constexpr (KMODE == 3 || KMODE == 4) {
            const uint8_t* const rr[4] = {st + tau0 * rs, st + tau1 * rs, st + (16 + tau0) * rs,
                                          st + (16 + tau1) * rs};
            qk_pairs<KMODE, G, KM>(rr, tig, kmis, bq, tq, key_lut, l8, sc2, scl2);
        }
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            [[maybe_unused]] const uint8_t* r0 = st + (16 * rt + tau0) * rs;
            [[maybe_unused]] const uint8_t* r1 = st + (16 * rt + tau1) * rs;
            const uint8_t* m0 = sm + (16 * rt + tau0) * mrs;
            const uint8_t* m1 = sm + (16 * rt + tau1) * mrs;
            float sc[4], scl[4];
            if constexpr (KMODE == 3 || KMODE == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) { sc[i] = sc2[rt][i]; scl[i] = scl2[rt][i]; }
            } else {
                qk_tile<KMODE, G, KGEN, KM>(r0, r1, tig, kmis, bq, bql, tq, T, key_lut, l8, sc, scl);
            }
            float n0 = 1.f, n1 = 1.f;
            if constexpr (KMODE != 8) { n0 = lds_f16(m0 + a.g.m_norm); n1 = lds_f16(m1 + a.g.m_norm); }
            vs[rt][0] = lds_f16(m0 + a.g.m_scale);
            vz[rt][0] = lds_f16(m0 + a.g.m_zero);
            vs[rt][1] = lds_f16(m1 + a.g.m_scale);
            vz[rt][1] = lds_f16(m1 + a.g.m_zero);
            vz[rt][0] = fmaf(kMidCode, vs[rt][0], vz[rt][0]);      // see the value sums below
            vz[rt][1] = fmaf(kMidCode, vs[rt][1], vz[rt][1]);
            ok[rt][0] = !PARTIAL || vis.sees(t0 + 16 * rt + tau0);
            ok[rt][1] = !PARTIAL || vis.sees(t0 + 16 * rt + tau1);
            if constexpr (G == 4) {
                s[0][rt][0] = (sc[0] + sc[1]) * n0;
                s[0][rt][1] = (sc[2] + sc[3]) * n1;
            } else {
                s[0][rt][0] = (sc[0] + scl[0]) * n0;
                s[1][rt][0] = (sc[1] + scl[1]) * n0;
                s[0][rt][1] = (sc[2] + scl[2]) * n1;
                s[1][rt][1] = (sc[3] + scl[3]) * n1;
            }
        }

        // softcap, then the distance bias (distance: to the newest token),
        // in log2 units like the scores
        if (CAPPED && (!KEEP || a.mods.cap > 0.f)) {
#pragma unroll
            for (int j = 0; j < NH; ++j) {
                float x[4] = {s[j][0][0], s[j][0][1], s[j][1][0], s[j][1][1]};
                softcap_warp(x, a.mods.cap, a.mods.inv_cap);
                s[j][0][0] = x[0];
                s[j][0][1] = x[1];
                s[j][1][0] = x[2];
                s[j][1][1] = x[3];
            }
        }
        const float dist0 = float(vis.L - 1 - t0 - tau0);
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            const float slope = s_slope[8 * warp + (G == 4 ? tig : 2 * tig + j)];
#pragma unroll
            for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                for (int r = 0; r < 2; ++r) s[j][rt][r] = fmaf(-slope, dist0 - float(16 * rt + 8 * r), s[j][rt][r]);
        }

        // ---- one online-softmax update for the 32 tokens (log2 units).  The
        // running max only moves when a head's tile max exceeds it by more
        // than 8 (so p <= 2^8 otherwise), or when a value scale above 128
        // could take p * v_scale out of the fp16 range of P'.  Moving it
        // rescales the accumulators; keeping it changes no result, since
        // o and l share the same reference.
        float mt[NH];
        bool need = false;
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            float m = -INFINITY;
#pragma unroll
            for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (!ok[rt][r]) s[j][rt][r] = -INFINITY;
                    m = fmaxf(m, s[j][rt][r]);
                }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            mt[j] = m;               // finite: the tile holds a valid token
            need |= m > m_run[j] + 8.f;
        }
        if constexpr (KEEP) {
            // the scores for the attention weights, masked tokens as -inf
            float* p = s_keep[warp] + (unsigned long long)unsigned(vt + tau0) * unsigned(a.mods.gp) +
                       (G == 4 ? tig : 2 * tig);
            const int put = (G == 4 ? tig : 2 * tig) < Greal;
#pragma unroll
            for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if constexpr (G == 4) store_if(p, s[0][rt][r], put);
                    else                  store_if(p, s[0][rt][r], s[1][rt][r], put);
                    p += 8 * a.mods.gp;
                }
        }
        need |= fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1])) > 128.f;
        if (__any_sync(0xffffffffu, need)) {
            float alpha[NH];
#pragma unroll
            for (int j = 0; j < NH; ++j) {
                const float mn = fmaxf(m_run[j], mt[j]);
                alpha[j] = fast_exp2(m_run[j] - mn);
                m_run[j] = mn;
                l_run[j] *= alpha[j];
                z_run[j] *= alpha[j];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (G == 4) {
                    acc[i][0] *= alpha[0]; acc[i][1] *= alpha[0]; acc[i][2] *= alpha[0]; acc[i][3] *= alpha[0];
                } else {
                    acc[i][0] *= alpha[0]; acc[i][2] *= alpha[0]; acc[i][1] *= alpha[1]; acc[i][3] *= alpha[1];
                }
            }
        }
        float pp[2][NH][2];   // [row tile][head][row]: P' = p * v_scale
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            float lsum = 0.f, zsum = 0.f;
#pragma unroll
            for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p = fast_exp2(s[j][rt][r] - m_run[j]);   // 0 for masked rows
                    lsum += p;
                    zsum += ok[rt][r] ? p * vz[rt][r] : 0.f;
                    pp[rt][j][r] = ok[rt][r] ? p * vs[rt][r] : 0.f;
                }
            l_run[j] += lsum;
            z_run[j] += zsum;
            // The value sum is kept about the middle code, sum p scale (code - mid) +
            // sum p (zero + mid scale): over long contexts its two parts, sum p scale
            // code and sum p zero, nearly cancel, and the MMAs' accumulation rounds
            // towards zero.  So the accumulators give up mid times the tile's sum of P'
            // (without it the output is 3.5e-4 off, relatively, at 131072 tokens and
            // groups of 8; with it 5e-6).
            float d = (pp[0][j][0] + pp[0][j][1]) + (pp[1][j][0] + pp[1][j][1]);
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
            d *= kMidCode / 512.f;             // the accumulators hold 2^-9 of the sums
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i][j] -= d;                // G = 4: column 2 tig, the head's hi part
                acc[i][j + 2] -= d;
            }
        }

        // ---- values
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            uint32_t pb[2][2];
            p_to_b<G>(pp[rt], gid, tig, pb);
            pv_tile<VBITS, G, VM>(st + 16 * rt * rs + a.g.v_off, rs, gid, tig, vmis, pb, acc);
        }
    };

    // The tile loop; returns the tile whose wait gave up, or -1.  2-bit keys
    // instantiate it with and without the lo part and pick once per CTA.
    auto run = [&](auto lo_tag, auto km_tag, auto vm_tag) {
        int stage = 0;               // it mod NST
        uint32_t parity = 0;         // (it / NST) mod 2
        for (int it = 0; it < ntiles; ++it) {
            // tile `it` has landed; a copy that never completes ends this warp's
            // heads with a NaN lse instead of hanging (bounded wait)
            const bool ok_wait = mbar_wait(&full[stage], parity, a.wait_polls);
            if (!__all_sync(0xffffffffu, ok_wait)) return it;
            const uint8_t* st = smem + stage * stage_bytes + hoff;
            const uint8_t* sm = smem + stage * stage_bytes + moff;
            const int v = vis_tile(it), t0 = vis_base(v);
            if (vis_whole(v)) tile(st, sm, t0, v << 5, std::false_type{}, lo_tag, km_tag, vm_tag);
            else              tile(st, sm, t0, v << 5, std::true_type{}, lo_tag, km_tag, vm_tag);

            // ---- this warp is done with the stage; the last warp refills it
            __syncwarp();
            int last = 0;
            if (lane == 0) {
                // release: this warp's reads of the stage come before the
                // count; acquire: the last warp's refill comes after all
                uint32_t prev;
                asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;"
                             : "=r"(prev) : "r"(smem_u32(&done[stage])) : "memory");
                last = prev == uint32_t(nwarps - 1);
                if (last) done[stage] = 0;
            }
            if (__shfl_sync(0xffffffffu, last, 0)) issue(it + NST, stage);
            if (++stage == NST) { stage = 0; parity ^= 1u; }
        }
        return -1;
    };
    // Misalignment of the warp's key and value loads: FP8 keys are read as
    // aligned words and their values start aligned; the others test it in the
    // loop (instances per misalignment, which the plain kernel has for 3-bit keys
    // with 3-bit values, spill here: groups of 8 151 -> 131 us without them, 4 sequences
    // of 65536 tokens).
    using M0 = std::integral_constant<int, 0>;
    using MR = std::integral_constant<int, -1>;
    using ML = std::integral_constant<int, -2>;
    auto run_mis = [&](auto lo_tag) {
        if constexpr (LAY == kHalfRows) return run(lo_tag, ML{}, ML{});
        else if constexpr (KMODE == 8)  return run(lo_tag, M0{}, M0{});
        else                            return run(lo_tag, MR{}, MR{});
    };
    int failed_at;
    if constexpr (KMODE == 2) failed_at = key_lo ? run_mis(std::true_type{}) : run_mis(std::false_type{});
    else                      failed_at = run_mis(std::true_type{});
    // stage 2 (a programmatic dependent launch) may start its launch now; it
    // waits for this grid's completion before it reads the partials
    asm volatile("griddepcontrol.launch_dependents;");
    // Run by every warp once its partials are written.  If any warp's copies
    // replaced a page outside the cache, the last warp to get here (when
    // every epilogue of the CTA is done) gives all the CTA's heads a NaN lse.
    auto finish = [&]() {
        __syncwarp();                          // the warp's partial writes before lane 0's count
        const bool wbad = __any_sync(0xffffffffu, bad_seen);
        int last = 0;
        if (lane == 0) {
            if (wbad) atomicOr(bad_pages, 1);
            __threadfence_block();
            last = atomicAdd(finished, 1) == nwarps - 1;
            __threadfence_block();
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        __syncwarp();
        if (last && *reinterpret_cast<volatile int*>(bad_pages))
            for (int i = lane; i < Hc * Greal; i += 32)
                partial((h0 + i / Greal) * Gall + qh0 + i % Greal)[kHeadDim] = __int_as_float(0x7fc00000);
    };
    if (failed_at >= 0) {
        // let the copies that may still be in flight (tiles failed_at ..
        // failed_at + NST - 1) land, with the same bounded wait, then mark
        // this warp's heads as failed
        for (int it = failed_at; it < min(ntiles, failed_at + NST); ++it)
            mbar_wait(&full[it % NST], uint32_t((it / NST) & 1), a.wait_polls);
        if (lane < Greal)
            partial(h * Gall + qh0 + lane)[kHeadDim] = __int_as_float(0x7fc00000);
        finish();
    } else {
        // ---------------- epilogue: finish the row sums, write o_s and lse_s.
        // The value accumulators hold 2^-9 of sum_t p_t v_scale_t code_t.
#pragma unroll
        for (int j = 0; j < NH; ++j) {
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) {
                l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], m);
                z_run[j] += __shfl_xor_sync(0xffffffffu, z_run[j], m);
            }
        }
#pragma unroll
        for (int j = 0; j < NH; ++j) {
            const int g = G == 4 ? tig : 2 * tig + j;
            if (g >= Greal) continue;
            const int hq = h * Gall + qh0 + g;
            float* mp = partial(hq);
            const float inv = 1.f / l_run[j];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int d = 16 * gid + 2 * i;
                float e, o;
                if constexpr (G == 4) { e = acc[i][0] + acc[i][1]; o = acc[i][2] + acc[i][3]; }
                else { e = j == 0 ? acc[i][0] : acc[i][1]; o = j == 0 ? acc[i][2] : acc[i][3]; }
                mp[d] = (e * 512.f + z_run[j]) * inv;
                mp[d + 1] = (o * 512.f + z_run[j]) * inv;
            }
            if (gid == 0) mp[kHeadDim] = (m_run[j] + log2f(l_run[j])) * 0.6931471805599453f;
        }
        finish();
    }
    // every warp of the CTA is done with its q columns: free them (the
    // allocating warp; all warps reach this point, the waits being bounded)
    if constexpr (kQt) {
        tmem_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
            tmem_fence_after_sync();
            tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(tmem_slot), q_cols);
        }
    }
}

template <typename TQ, int KMODE, int VBITS, int G, int MODE>
cudaError_t launch_scored_t(const MmaArgs& a, int B, size_t smem, cudaStream_t st)
{
    auto k = a.g.soa ? scored_mma_kernel<TQ, KMODE, VBITS, G, kSoa, MODE>
                     : scored_mma_kernel<TQ, KMODE, VBITS, G, kWordRows, MODE>;
    if constexpr (KMODE != 8)                // FP8-key slots are whole words
        if (!a.g.soa && a.row_bytes % 4) k = scored_mma_kernel<TQ, KMODE, VBITS, G, kHalfRows, MODE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_splits * a.nqg * (a.Hk / a.hpc), B, 1);   // see the kernel's blockIdx.x
    cfg.blockDim = dim3(32 * a.hpc);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename TQ, int KMODE, int VBITS, int MODE>
cudaError_t launch_scored_g(const MmaArgs& a, int B, size_t smem, cudaStream_t st)
{
    return a.G <= 4 ? launch_scored_t<TQ, KMODE, VBITS, 4, MODE>(a, B, smem, st)
                    : launch_scored_t<TQ, KMODE, VBITS, 8, MODE>(a, B, smem, st);
}

template <typename TQ, int MODE>
cudaError_t launch_scored_q(const MmaArgs& a, int B, size_t smem, cudaStream_t st)
{
    if (a.g.key_fp8) return launch_scored_g<TQ, 8, 4, MODE>(a, B, smem, st);
    if (a.g.key_bits == 4) return launch_scored_g<TQ, 4, 4, MODE>(a, B, smem, st);
    if (a.g.key_bits == 2) return launch_scored_g<TQ, 2, 2, MODE>(a, B, smem, st);
    if (a.g.value_bits == 4) return launch_scored_g<TQ, 3, 4, MODE>(a, B, smem, st);
    return launch_scored_g<TQ, 3, 3, MODE>(a, B, smem, st);
}

}  // namespace
}  // namespace tq
