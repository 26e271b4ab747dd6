// Eviction by accumulated attention weight: which tokens each kv head keeps
// (tq_evict_select), and the move of the kept slots to the front of their
// sequence, in place (tq_evict_compact).
#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

#include <cooperative_groups.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace tq {
namespace {

// ------------------------------------------------------------------ select
//
// One thread-block cluster per (sequence, kv head) row.  Every CTA of the
// cluster holds its part of the row in shared memory as order-preserving
// 32-bit keys, so the row is read from memory once (rows beyond the shared
// memory of 8 CTAs read the rest again in each pass).  The budget-th largest
// key T is found by histograms of its top 12, middle 10 and low 10 bits;
// then the keys above T and the first keys equal to T (in token order) are
// written out in order, from counts per warp segment.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHist1 = 4096, kHist2 = 1024;
constexpr int kSelMaxKeys = 49152;      // keys of a row a CTA holds: 192 KB

struct SelectArgs {
    const float* acc;
    long long stride_b, stride_h;
    const int32_t* seq_lens;
    int max_len, Hk, budget, prefix, recent, cap;
    int32_t* keep;
    int32_t* new_lens;
};

struct SelectShared {
    unsigned h1[kHist1], h2[kHist2], h3[kHist2];
    int bin, above;                      // the picked bin and the keys above it
    int warp_gt[kSelWarps], warp_eq[kSelWarps];
    int cta_gt[8], cta_eq[8];
    int scan[kSelWarps];
};

// Larger floats have larger keys; -0 counts as 0, and a NaN is above every
// number (a sum that cannot be judged is kept).  Always-kept tokens are above all.
__device__ __forceinline__ unsigned order_key(float x)
{
    if (x != x) return 0xFFFFFFFEu;
    const unsigned u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The bin in which the need-th largest key lies, and how many keys lie above
// it.  All threads of the block; n is a multiple of kSelThreads.
__device__ void pick_bin(const unsigned* hist, int n, int need, SelectShared& sh)
{
    const int per = n / kSelThreads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int top = n - 1 - threadIdx.x * per;      // this thread's bins: top, top - 1, ...
    int mine = 0;
    for (int i = 0; i < per; ++i) mine += hist[top - i];
    int incl = mine;
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += o;
    }
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    int before = incl - mine;
    for (int w = 0; w < warp; ++w) before += sh.scan[w];
    if (before < need && need <= before + mine) {   // one thread
        int i = 0;
        while (before + int(hist[top - i]) < need) before += hist[top - i++];
        sh.bin = top - i;
        sh.above = before;
    }
    __syncthreads();
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a, int csize)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SelectShared& sh = *reinterpret_cast<SelectShared*>(smem_raw);
    unsigned* keys = reinterpret_cast<unsigned*>(smem_raw + sizeof(SelectShared));
    cg::cluster_group cl = cg::this_cluster();
    const int rank = CLUSTER ? int(blockIdx.x % csize) : 0;
    const int row = CLUSTER ? blockIdx.x / csize : blockIdx.x;
    const int b = row / a.Hk, h = row % a.Hk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int L = max(a.seq_lens[b], 0);
    int32_t* keep = a.keep + (long long)row * a.budget;
    const bool too_long = L > a.max_len;             // caller error: nothing read, nothing evicted
    if (h == 0 && rank == 0 && tid == 0) a.new_lens[b] = too_long ? L : min(L, a.budget);
    if (L <= a.budget || too_long) {                 // uniform in the cluster
        for (int i = rank * kSelThreads + tid; i < a.budget; i += csize * kSelThreads)
            keep[i] = i < L && !too_long ? i : -1;
        return;
    }
    auto sync = [&]() { if constexpr (CLUSTER) cl.sync(); else __syncthreads(); };

    for (int i = tid; i < kHist1 + 2 * kHist2; i += kSelThreads) sh.h1[i] = 0;   // h1, h2, h3 are adjacent
    sync();

    // ---- this CTA's part of the row
    const int seg = (L + csize - 1) / csize;
    const int c0 = min(L, rank * seg), n = min(L, c0 + seg) - c0;
    const float* x = a.acc + b * a.stride_b + h * a.stride_h + c0;
    const int kept_hi = L - a.recent;
    auto fresh_key = [&](int i) {
        const int t = c0 + i;
        return t < a.prefix || t >= kept_hi ? 0xFFFFFFFFu : order_key(x[i]);
    };
    auto key = [&](int i) { return i < a.cap ? keys[i] : fresh_key(i); };
#pragma unroll 4
    for (int i = tid; i < n; i += kSelThreads) {
        const unsigned k = fresh_key(i);
        if (i < a.cap) keys[i] = k;
        atomicAdd(&sh.h1[k >> 20], 1u);
    }
    // every CTA's counts go to the first CTA, which picks the bin for all
    auto pick = [&](unsigned* hist, int bins, int need) {
        __syncthreads();
        if constexpr (CLUSTER) {
            if (rank != 0) {
                unsigned* to = cl.map_shared_rank(hist, 0);
                for (int i = tid; i < bins; i += kSelThreads)
                    if (hist[i]) atomicAdd(&to[i], hist[i]);
            }
            cl.sync();
            if (rank == 0) {
                pick_bin(hist, bins, need, sh);
                if (tid > 0 && tid < csize) {
                    SelectShared* to = cl.map_shared_rank(&sh, tid);
                    to->bin = sh.bin;
                    to->above = sh.above;
                }
            }
            cl.sync();
        } else {
            pick_bin(hist, bins, need, sh);
        }
    };
    int need = a.budget;
    pick(sh.h1, kHist1, need);
    const unsigned p1 = sh.bin;
    need -= sh.above;
    for (int i = tid; i < n; i += kSelThreads) {
        const unsigned k = key(i);
        if (k >> 20 == p1) atomicAdd(&sh.h2[(k >> 10) & 1023u], 1u);
    }
    pick(sh.h2, kHist2, need);
    const unsigned p2 = p1 << 10 | unsigned(sh.bin);
    need -= sh.above;
    for (int i = tid; i < n; i += kSelThreads) {
        const unsigned k = key(i);
        if (k >> 10 == p2) atomicAdd(&sh.h3[k & 1023u], 1u);
    }
    pick(sh.h3, kHist2, need);
    const unsigned T = p2 << 10 | unsigned(sh.bin);
    need -= sh.above;                                // keys equal to T that are kept

    // ---- counts above and equal per warp segment, then the ordered output
    const int wseg = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int w0 = min(n, warp * wseg), w1 = min(n, w0 + wseg);
    int gt = 0, eq = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const unsigned k = key(i);
        gt += k > T;
        eq += k == T;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) { sh.warp_gt[warp] = gt; sh.warp_eq[warp] = eq; }
    __syncthreads();
    int pos_gt = 0, pos_eq = 0;
    for (int w = 0; w < warp; ++w) { pos_gt += sh.warp_gt[w]; pos_eq += sh.warp_eq[w]; }
    if constexpr (CLUSTER) {
        if (tid < csize) {
            int g = 0, e = 0;
            for (int w = 0; w < kSelWarps; ++w) { g += sh.warp_gt[w]; e += sh.warp_eq[w]; }
            SelectShared* to = cl.map_shared_rank(&sh, tid);
            to->cta_gt[rank] = g;
            to->cta_eq[rank] = e;
        }
        cl.sync();
        for (int r = 0; r < rank; ++r) { pos_gt += sh.cta_gt[r]; pos_eq += sh.cta_eq[r]; }
    }
    const unsigned below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const unsigned k = i < w1 ? key(i) : 0u;
        const bool isg = i < w1 && k > T, ise = i < w1 && k == T;
        const unsigned mg = __ballot_sync(0xffffffffu, isg), me = __ballot_sync(0xffffffffu, ise);
        const int eq_before = pos_eq + __popc(me & below);
        const int at = pos_gt + __popc(mg & below) + min(eq_before, need);
        if (isg || (ise && eq_before < need)) keep[at] = c0 + i;
        pos_gt += __popc(mg);
        pos_eq += __popc(me);
    }
}

// ------------------------------------------------------------------ compact
//
// One cluster per (sequence, kv head).  The kept tokens ascend, so slot i
// comes from slot keep[i] >= i: a chunk of destinations may be written once
// the chunk's sources (all at or past its start) have been read by every
// warp of the cluster, and the next chunk's sources are never among the
// slots written.  One barrier per chunk, between its reads and its writes.
constexpr int kCmpThreads = 256;
constexpr int kCmpWarps = kCmpThreads / 32;

struct CompactArgs {
    uint8_t* cache;
    long long num_blocks;
    const int32_t* block_table;
    int bt_stride;
    const int32_t* keep;
    const int32_t* seq_lens;
    int max_len, budget, Hk, bs_log2;
    float* acc;                          // null: no running sums
    long long stride_b, stride_h;
    SlotGeom g;
};

__device__ __forceinline__ uint32_t ldg_u16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// K slots per warp and chunk; IT 128-byte steps cover the record.
template <int K, int IT, bool SOA>
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(CompactArgs a, int csize)
{
    const int rank = blockIdx.x % csize, row = blockIdx.x / csize;
    const int b = row / a.Hk, h = row % a.Hk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int L = a.seq_lens[b];
    if (L <= a.budget || L > a.max_len) return;      // uniform in the cluster
    const int32_t* keep = a.keep + (long long)row * a.budget;
    const int32_t* bt = a.block_table + (long long)b * a.bt_stride;
    float* acc = a.acc ? a.acc + b * a.stride_b + h * a.stride_h : nullptr;
    const int bs = 1 << a.bs_log2;
    const int nbytes = SOA ? a.g.data_bytes : a.g.slot;      // even
    const int per_chunk = csize * kCmpWarps * K;
    const int nchunks = (a.budget + per_chunk - 1) / per_chunk;
    for (int c = 0; c < nchunks; ++c) {
        const int i0 = c * per_chunk + (rank * kCmpWarps + warp) * K;
        // lane k: slot i0 + k
        long long src = -1, dst = -1, msrc = 0, mdst = 0;
        float w = 0.f;
        const int i = i0 + lane;
        if (lane < K && i < a.budget) {
            const int t = keep[i];
            if (t != i && t >= 0 && t < L) {
                const long long sp = bt[t >> a.bs_log2], dp = bt[i >> a.bs_log2];
                if ((unsigned long long)sp < (unsigned long long)a.num_blocks &&
                    (unsigned long long)dp < (unsigned long long)a.num_blocks) {
                    const uint8_t *d, *m;
                    slot_ptrs(a.g, a.cache, sp, t & (bs - 1), h, bs, a.Hk, d, m);
                    src = d - a.cache;
                    msrc = m - a.cache;
                    slot_ptrs(a.g, a.cache, dp, i & (bs - 1), h, bs, a.Hk, d, m);
                    dst = d - a.cache;
                    mdst = m - a.cache;
                    if (acc) w = acc[t];
                }
            }
        }
        uint32_t v[K][IT], mv[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long s = __shfl_sync(0xffffffffu, src, k), d = __shfl_sync(0xffffffffu, dst, k);
            const int lead = int(d & 2);             // the first destination word may begin 2 bytes early
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int o = 4 * (lane + 32 * it) - lead;
                uint32_t lo = 0, hi = 0;
                if (s >= 0 && o >= 0 && o < nbytes) lo = ldg_u16(a.cache + s + o);
                if (s >= 0 && o + 2 < nbytes) hi = ldg_u16(a.cache + s + o + 2);
                v[k][it] = lo | hi << 16;
            }
            if constexpr (SOA) {
                const long long ms = __shfl_sync(0xffffffffu, msrc, k);
                mv[k] = s >= 0 && 2 * lane < a.g.meta_bytes ? ldg_u16(a.cache + ms + 2 * lane) : 0u;
            }
        }
        if (csize > 1) cg::this_cluster().sync();
        else           __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long d = __shfl_sync(0xffffffffu, dst, k);
            if (d < 0) continue;
            const int lead = int(d & 2);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int o = 4 * (lane + 32 * it) - lead;
                uint8_t* p = a.cache + d + o;
                if (o >= 0 && o + 2 < nbytes) *reinterpret_cast<uint32_t*>(p) = v[k][it];
                else if (o >= 0 && o < nbytes) *reinterpret_cast<uint16_t*>(p) = uint16_t(v[k][it]);
                else if (o < 0) *reinterpret_cast<uint16_t*>(p + 2) = uint16_t(v[k][it] >> 16);
            }
            if constexpr (SOA) {
                const long long md = __shfl_sync(0xffffffffu, mdst, k);
                if (2 * lane < a.g.meta_bytes)
                    *reinterpret_cast<uint16_t*>(a.cache + md + 2 * lane) = uint16_t(mv[k]);
            }
        }
        if (acc && dst >= 0) acc[i] = w;
    }
    // past the last barrier every source has been read: the evicted tail's sums start again at 0
    if (acc)
        for (int t = a.budget + rank * kCmpThreads + threadIdx.x; t < L; t += csize * kCmpThreads) acc[t] = 0.f;
}

template <typename K, typename A>
cudaError_t launch_cluster(K kernel, const A& a, long long rows, int csize, int threads, size_t smem, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows * csize));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(csize);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, csize);
}

}  // namespace
}  // namespace tq

extern "C" int tq_evict_select(int batch, int num_kv_heads, const float* acc, long long acc_stride_seq,
                               long long acc_stride_head, const int32_t* seq_lens, int max_seq_len, int budget,
                               int prefix, int recent, int32_t* keep, int32_t* new_lens, void* stream)
{
    using namespace tq;
    if (batch < 0 || num_kv_heads < 1 || max_seq_len < 0 || max_seq_len > kMaxListedLen || budget < 1 || prefix < 0 || recent < 0 ||
        (long long)prefix + recent > budget || !acc_strides_ok(batch, num_kv_heads, acc_stride_seq, acc_stride_head, max_seq_len) ||
        (long long)batch * num_kv_heads > (1LL << 27))
        return TQ_ERR_INVALID_ARG;
    if (batch == 0) return TQ_OK;
    if (!acc || !seq_lens || !keep || !new_lens) return TQ_ERR_INVALID_ARG;
    SelectArgs a;
    a.acc = acc;
    a.stride_b = acc_stride_seq;
    a.stride_h = acc_stride_head;
    a.seq_lens = seq_lens;
    a.max_len = max_seq_len;
    a.Hk = num_kv_heads;
    a.budget = budget;
    a.prefix = prefix;
    a.recent = recent;
    a.keep = keep;
    a.new_lens = new_lens;
    const long long rows = (long long)batch * num_kv_heads;
    auto seg = [&](int c) { return (max_seq_len + c - 1) / c; };
    int csize = 1;
    while (csize < 8 && (seg(csize) > kSelMaxKeys || (rows * csize < 2 * kNumSMs && seg(csize) >= 4096))) csize *= 2;
    a.cap = std::min(seg(csize), kSelMaxKeys);
    const size_t smem = sizeof(SelectShared) + 4 * size_t(a.cap);
    auto k = csize > 1 ? select_kernel<true> : select_kernel<false>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
        return TQ_ERR_CUDA;
    return launch_cluster(k, a, rows, csize, kSelThreads, smem, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? TQ_OK : TQ_ERR_CUDA;
}

extern "C" int tq_evict_compact(int preset, int head_dim, int batch, int num_kv_heads, int block_size,
                                uint8_t* kv_cache, long long num_blocks, const int32_t* block_table,
                                int block_table_stride, const int32_t* keep, int budget,
                                const int32_t* seq_lens, int max_seq_len, float* acc,
                                long long acc_stride_seq, long long acc_stride_head, void* stream)
{
    using namespace tq;
    tq_layout L;
    const int rc = fill_layout(preset, head_dim, &L);
    if (rc) return rc;
    if (head_dim != kHeadDim || !block_size_ok(block_size)) return TQ_ERR_UNSUPPORTED;
    if (batch < 0 || num_kv_heads < 1 || num_blocks < 0 || block_table_stride < 0 || budget < 1 || max_seq_len < 0 || max_seq_len > kMaxListedLen ||
        (long long)batch * num_kv_heads > (1LL << 27))
        return TQ_ERR_INVALID_ARG;
    if (acc && !acc_strides_ok(batch, num_kv_heads, acc_stride_seq, acc_stride_head, max_seq_len))
        return TQ_ERR_INVALID_ARG;
    if (batch == 0) return TQ_OK;
    if (!kv_cache || !block_table || !keep || !seq_lens || (reinterpret_cast<uintptr_t>(kv_cache) & 15))
        return TQ_ERR_INVALID_ARG;
    CompactArgs a;
    a.cache = kv_cache;
    a.num_blocks = num_blocks;
    a.block_table = block_table;
    a.bt_stride = block_table_stride;
    a.keep = keep;
    a.seq_lens = seq_lens;
    a.max_len = max_seq_len;
    a.budget = budget;
    a.Hk = num_kv_heads;
    a.bs_log2 = block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
    a.acc = acc;
    a.stride_b = acc_stride_seq;
    a.stride_h = acc_stride_head;
    const bool soa = is_soa(preset);
    a.g = geom_of(L, soa);
    const long long rows = (long long)batch * num_kv_heads;
    const int nbytes = soa ? a.g.data_bytes : a.g.slot;
    const bool wide = nbytes + 2 > 128;
    const int K = wide ? 4 : 8;
    int csize = 1;
    while (csize < 8 && rows * csize < 8 * kNumSMs && csize * kCmpWarps * K < budget) csize *= 2;
    auto k = wide ? (soa ? compact_kernel<4, 2, true> : compact_kernel<4, 2, false>)
                  : (soa ? compact_kernel<8, 1, true> : compact_kernel<8, 1, false>);
    return launch_cluster(k, a, rows, csize, kCmpThreads, 0, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? TQ_OK : TQ_ERR_CUDA;
}
