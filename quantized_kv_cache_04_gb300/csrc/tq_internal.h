// Internal declarations shared by the host and CUDA translation units of the
// TurboQuant library.  Not part of the public ABI (include/tq.h is).
#pragma once

#include "tq.h"

#include <cstdint>
#include <cuda_runtime.h>

namespace tq {

constexpr int kHeadDim = 128;     // the served head dimension
constexpr int kMaxGroup = 16;     // query heads per kv head served by decode
constexpr int kNumSMs = 152;      // GB300

int fill_layout(int preset, int head_dim, tq_layout* L);
// Split count for num_splits = 0 (tq_decode.cu): the one that minimises the
// stage-1 critical path over the resident CTA slots of the kernel that runs.
int pick_splits(const tq_layout& L, bool soa, int batch, int num_q_heads, int num_kv_heads, int max_seq_len,
                int min_split = 128, bool scored = false);

inline bool block_size_ok(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }
inline bool in_dtype_ok(int dt) { return dt == TQ_F16 || dt == TQ_BF16; }
inline bool out_dtype_ok(int dt) { return dt == TQ_F16 || dt == TQ_BF16 || dt == TQ_F32; }

// Plain-old-data copy of the slot layout handed to kernels by value, with
// the block byte convention.  Field addresses of record (token t of a block,
// kv head h) come from two pointers, `data` (key data at 0, value data at
// v_off) and `meta` (k_norm / v_scale / v_zero at m_norm / m_scale /
// m_zero): AoS: both are the slot, offsets as in tq_layout; SoA: data record
// and metadata record (TQ_LAYOUT_SOA in tq.h).
struct SlotGeom {
    int key_fp8, key_bits, value_bits, norm_correction;
    int key_data_bytes, off_k_norm, off_v_data, off_v_scale, off_v_zero;
    int slot;        // slot_size_aligned
    int soa;         // 1: TQ_LAYOUT_SOA
    int data_bytes;  // SoA data record: key_data_bytes + value_data_bytes
    int meta_bytes;  // SoA metadata record: 2 * fields
    int v_off;       // value data offset from `data`
    int m_norm, m_scale, m_zero;   // field offsets from `meta`
};

inline SlotGeom geom_of(const tq_layout& L, bool soa = false)
{
    SlotGeom g;
    g.key_fp8 = L.key_fp8;
    g.key_bits = L.key_bits;
    g.value_bits = L.value_bits;
    g.norm_correction = L.norm_correction;
    g.key_data_bytes = L.key_data_bytes;
    g.off_k_norm = L.off_k_norm;
    g.off_v_data = L.off_v_data;
    g.off_v_scale = L.off_v_scale;
    g.off_v_zero = L.off_v_zero;
    g.slot = L.slot_size_aligned;
    g.soa = soa ? 1 : 0;
    g.data_bytes = L.key_data_bytes + L.value_data_bytes;
    g.meta_bytes = L.key_fp8 ? 4 : 6;
    if (soa) {
        g.v_off = L.key_data_bytes;
        g.m_norm = L.key_fp8 ? -1 : 0;
        g.m_scale = L.key_fp8 ? 0 : 2;
        g.m_zero = L.key_fp8 ? 2 : 4;
    } else {
        g.v_off = L.off_v_data;
        g.m_norm = L.off_k_norm;
        g.m_scale = L.off_v_scale;
        g.m_zero = L.off_v_zero;
    }
    return g;
}

// Preset argument: low byte = preset, TQ_LAYOUT_SOA bit = block convention.
inline bool layout_flags_ok(int preset) { return (preset & ~(0xFF | TQ_LAYOUT_SOA)) == 0; }
inline bool is_soa(int preset) { return (preset & TQ_LAYOUT_SOA) != 0; }

#ifdef __CUDACC__
// Data and metadata pointers of record (block `page`, token `off`, head h).
__device__ __forceinline__ void slot_ptrs(const SlotGeom& g, const uint8_t* cache, long long page, int off,
                                          int h, int bs, int Hk, const uint8_t*& data, const uint8_t*& meta)
{
    if (g.soa) {
        const uint8_t* blk = cache + page * bs * (long long)Hk * g.slot;
        const long long rec = (long long)off * Hk + h;
        data = blk + rec * g.data_bytes;
        meta = blk + (long long)bs * Hk * g.data_bytes + rec * g.meta_bytes;
    } else {
        data = cache + ((page * bs + off) * (long long)Hk + h) * g.slot;
        meta = data;
    }
}
#endif

// Longest sequence the scored decode and the eviction take: positions of
// 32-token tiles then stay clear of 2^31.
constexpr int kMaxListedLen = 1 << 30;

// Score modifiers as the stage-1 kernels take them (tq_score_mods in tq.h),
// and where the scores of a call that accumulates attention weights go.
struct ScoreArgs {
    float cap, inv_cap;        // softcap and its reciprocal (cap 0: none)
    const float* slopes;       // distance biases per query head (null: none)
    int window, prefix;        // window 0: every token of the document
    const int32_t* doc_start;  // first token of the current document (null: 0)
    float* scores;             // [B][Hk][vtok][gp] scores in log2 units (null: not kept)
    int vtok;                  // listed tokens per (sequence, kv head): a multiple of 32
    int gp;                    // query heads per kv head, padded (score_heads)
    int max_len;               // sequences longer than this cannot be listed: a NaN lse
    int B;
    int* plan;                 // [B][2]: a sequence's first split and its number of splits
};

// columns per listed token in ScoreArgs::scores: even above 4 heads, where
// the tensor-core stage 1 writes pairs
inline int score_heads(int G) { return G <= 4 ? G : (G + 1) & ~1; }

// 32-token tiles that hold the visible tokens of a sequence of at most
// max_len tokens (VisibleSet): a window or prefix of n tokens meets at most
// n / 32 + 2 of them
inline int visible_tiles(int max_len, int window, int prefix)
{
    const long long all = ((long long)max_len + 31) / 32;
    if (window <= 0) return int(all);
    const long long some = (long long)window / 32 + 2 + (prefix > 0 ? (long long)prefix / 32 + 2 : 0);
    return int(all < some ? all : some);
}

// Workspace of a scored decode: the split partials, then for each sequence
// where its splits begin and how many there are (SplitPlan); of one that
// accumulates attention weights also an lse per query head (when the caller
// takes none) and the scores.  Byte offsets on 256-byte
// boundaries.
struct ScoredLayout {
    size_t off_plan, off_lse, off_scores, bytes;
    int vtok;
};
inline ScoredLayout scored_layout(int batch, int Hq, int Hk, int S, int max_len, int window, int prefix, bool scores)
{
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    ScoredLayout w;
    w.vtok = 32 * visible_tiles(max_len, window, prefix);
    w.off_plan = up(tq_decode_workspace_bytes(batch, Hq, S, kHeadDim));
    w.off_lse = w.off_plan + up(size_t(batch) * 2 * sizeof(int));
    w.off_scores = w.off_lse + (scores ? up(size_t(batch) * Hq * sizeof(float)) : 0);
    w.bytes = w.off_scores + (scores ? size_t(batch) * Hk * w.vtok * score_heads(Hq / Hk) * sizeof(float) : 0);
    return w;
}

// acc[b][h][t] += sum of the softmax weights of token t over the G query
// heads of kv head h, from the kept scores and the lse (tq_weights.cu).
cudaError_t launch_weights(const ScoreArgs& m, const int32_t* seq_lens, const float* lse, float* acc,
                           long long stride_b, long long stride_h, int Hk, int G, cudaStream_t st);

// Whether rows acc + b * sb + h * sh of max_len elements do not overlap:
// sequences of heads or heads of sequences (one writer per running sum).
inline bool acc_strides_ok(int B, int Hk, long long sb, long long sh, int max_len)
{
    if (sb < 0 || sh < 0) return false;
    if (Hk > 1 && sh < max_len) return false;
    if (B > 1 && sb < max_len) return false;
    if (B <= 1 || Hk <= 1) return true;
    return sb >= (Hk - 1) * sh + max_len || sh >= (B - 1) * sb + max_len;
}

#ifdef __CUDACC__
// The visible tokens of a sequence: [lo, pend) and [first, L), with
// lo <= pend <= first, listed by the 32-token tiles (of the sequence) that
// hold any of them: tiles a0 .. a0 + na - 1 for the prefix, then b0 ..
// b0 + nb - 1.  Every listed tile holds a visible token; tiles between the
// prefix and the window are not listed, so their pages are never looked at.
struct VisibleSet {
    int L, lo, pend, first;
    int a0, na, b0, nb;
    __device__ __forceinline__ VisibleSet(const ScoreArgs& m, int len, int b)
    {
        L = max(len, 0);
        lo = m.doc_start ? max(m.doc_start[b], 0) : 0;
        lo = min(lo, L);
        first = m.window > 0 ? max(lo, L - m.window) : lo;
        pend = lo + (m.window > 0 ? min(m.prefix, first - lo) : 0);
        a0 = lo >> 5;
        na = pend > lo ? ((pend + 31) >> 5) - a0 : 0;
        b0 = max(first >> 5, na ? a0 + na : 0);
        nb = first < L ? max(((L + 31) >> 5) - b0, 0) : 0;
    }
    __device__ __forceinline__ int tiles() const { return na + nb; }
    // first token of listed tile v
    __device__ __forceinline__ int base(int v) const { return (v < na ? a0 + v : b0 + v - na) << 5; }
    __device__ __forceinline__ bool sees(int t) const
    {
        return (t >= lo && t < pend) || (t >= first && t < L);
    }
    // whether [t, t + n) holds a visible token / nothing else
    __device__ __forceinline__ bool any(int t, int n) const
    {
        return max(t, lo) < min(t + n, pend) || max(t, first) < min(t + n, L);
    }
    __device__ __forceinline__ bool all(int t, int n) const
    {
        return (t >= lo && t + n <= pend) || (t >= first && t + n <= L);
    }
};
// Which splits a batch of scored sequences has: all of `chunk` tiles (a
// sequence's last one may be shorter), with the smallest chunk that gives at
// most B * S of them, so that every CTA has the same work however the lengths,
// windows and documents differ.  Split `id` of the launch belongs to sequence
// b, as its split number id - base.  All threads of the block call this;
// `area` is B + 4 ints of shared memory, free again afterwards.  The launch's
// first block (`writer`) stores the plan for stage 2.  Batches above kPlanMax
// sequences keep S splits for each.  (Four sequences of packed documents, 3-bit
// keys, 282K visible tokens in all: 209 us with S splits for each, 143 us so.)
constexpr int kPlanMax = 512;
struct SplitPlan {
    int b, base, n, chunk;     // b < 0: no split of this number
    __device__ SplitPlan(const ScoreArgs& m, const int32_t* seq_lens, int S, int id, bool writer, int* area)
    {
        auto tiles = [&](int i) {
            const int len = seq_lens[i];
            return len > m.max_len ? 1 : VisibleSet(m, len, i).tiles();      // too long: one split, which says so
        };
        if (m.B == 1 || m.B > kPlanMax) {
            b = id / S;
            const int t = tiles(b);
            base = b * S;
            chunk = max((t + S - 1) / S, 1);
            n = (t + chunk - 1) / chunk;
            if ((m.B == 1 ? writer : id == base) && threadIdx.x == 0) { m.plan[2 * b] = base; m.plan[2 * b + 1] = n; }
            if (id - base >= n) b = -1;
            return;
        }
        const int lane = threadIdx.x & 31;
        if (m.B <= 32) {               // every warp for itself, a sequence per lane
            const int t = lane < m.B ? tiles(lane) : 0;
            chunk = chunk_of(t, t, S * m.B, m.B, [&](int c) { return (t + c - 1) / c; });
            const int k = (t + chunk - 1) / chunk;
            int incl = k;
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            if (writer && threadIdx.x < m.B) { m.plan[2 * lane] = incl - k; m.plan[2 * lane + 1] = k; }
            const unsigned here = __ballot_sync(0xffffffffu, id >= incl - k && id < incl);
            b = here ? __ffs(here) - 1 : -1;
            base = __shfl_sync(0xffffffffu, incl - k, max(b, 0));
            n = __shfl_sync(0xffffffffu, k, max(b, 0));
            return;
        }
        for (int i = threadIdx.x; i < m.B; i += blockDim.x) area[i] = tiles(i);
        __syncthreads();
        if (threadIdx.x < 32) {
            const int B = m.B;
            long long total = 0;
            int most = 0;
            for (int i = lane; i < B; i += 32) { total += area[i]; most = max(most, area[i]); }
            const int c = chunk_of(total, most, S * B, B, [&](int c) {
                int k = 0;
                for (int i = lane; i < B; i += 32) k += (area[i] + c - 1) / c;
                return k;
            });
            int run = 0;
            if (lane == 0) area[B] = -1;
            __syncwarp();
            for (int i0 = 0; i0 < B; i0 += 32) {
                const int i = i0 + lane, k = i < B ? (area[i] + c - 1) / c : 0;
                int incl = k;
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += o;
                }
                const int first = run + incl - k;
                if (id >= first && id < first + k) { area[B] = i; area[B + 1] = first; area[B + 2] = k; }
                if (writer && i < B) { m.plan[2 * i] = first; m.plan[2 * i + 1] = k; }
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) area[B + 3] = c;
        }
        __syncthreads();
        b = area[m.B];
        base = area[m.B + 1];
        n = area[m.B + 2];
        chunk = area[m.B + 3];
        __syncthreads();
    }

    // The smallest chunk with at most `slots` splits: a warp's search between
    // the average share and what surely suffices.  total, most: each lane's
    // share of the sequences' tiles and its longest; splits(c): its splits.
    template <typename F>
    static __device__ int chunk_of(long long total, int most, int slots, int B, F splits)
    {
        for (int k = 16; k; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
        most = __reduce_max_sync(0xffffffffu, most);
        int lo = int(max((total + slots - 1) / slots, 1LL));
        int hi = max(slots > B ? int(min((total + slots - B - 1) / (slots - B), (long long)most)) : most, lo);
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (__reduce_add_sync(0xffffffffu, splits(mid)) <= slots) hi = mid;
            else                                                      lo = mid + 1;
        }
        return lo;
    }
};
#endif

// Tensor-core stage 1 (tq_decode_mma.cu): which shapes it serves, and its launcher.
bool mma_stage1_supported(const tq_layout& L, bool soa, int num_kv_heads, int group);
bool mma_scored_supported(const tq_layout& L, bool soa, int num_kv_heads, int group);   // its scored kernel
// CTAs one split of one sequence launches, and resident CTA slots on num_sms
// SMs (0 when the occupancy query fails, e.g. without a device).
void mma_stage1_shape(const tq_layout& L, bool soa, int num_kv_heads, int group, int num_sms,
                      int* ctas_per_split, int* slots);
// Polls of a stage's mbarrier before stage 1 gives up on it (the split's
// lse becomes NaN); each poll sleeps at most 20 us waiting for the phase,
// so a stage that never completes is given up after about 1.3 s.  A test
// may pass a small count and a stuck tile.
constexpr uint32_t kWaitPolls = 1u << 16;
int launch_mma_stage1(const tq_layout& L, bool soa, int q_dtype, const void* query, const uint8_t* kv_cache,
                      long long num_blocks, const int32_t* block_table, int bt_stride, const int32_t* seq_lens,
                      float softmax_scale, int num_splits, const int8_t* signs,
                      const float* centroids, float* mid, int B, int Hq, int Hk, int bs,
                      float v_threshold, cudaStream_t st, int stuck_tile = -1,
                      uint32_t wait_polls = kWaitPolls, const ScoreArgs* mods = nullptr);

}  // namespace tq
