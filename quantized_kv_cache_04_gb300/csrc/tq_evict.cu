// Eviction by accumulated attention weight: which tokens each kv head keeps
// (tq_evict_select), and the move of the kept slots to the front of their
// sequence, in place (tq_evict_compact).
#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

namespace cg = cooperative_groups;

namespace tq {
namespace {

// ------------------------------------------------------------------ select
//
// One thread-block cluster per (sequence, kv head) row.  Every CTA of the
// cluster holds its part of the row in shared memory as order-preserving
// 32-bit keys; of a part above kSelMaxKeys the rest is read a second time in
// step 2, from L2.
//   1. A histogram of the keys' top 12 bits, merged in the first CTA, gives the
//      bin that holds the budget-th largest key.
//   2. Every 32 keys leave a word of bits "above the bin" and one of "in it";
//      the keys in the bin, usually a few per cent, are listed in the first CTA.
//   3. The first CTA finds the budget-th key T from the list by histograms of
//      the middle and low 10 bits (a list that overflows, e.g. of many equal
//      sums, is not used: both histograms are then taken over the bit words).
//   4. The bits become "above T" and "equal to T"; the tokens are written in
//      order from the words' counts, of the equal ones the first.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHist1 = 4096, kHist2 = 1024;
constexpr int kList = 4096;             // listed keys of the bin
constexpr int kSelMaxKeys = 16384;      // keys a CTA holds: 64 KB, two CTAs to an SM
constexpr int kSelMaxWords = 4096;      // words whose bits a CTA holds (rows of up to 2^20 tokens)

struct SelectArgs {
    const float* acc;
    long long stride_b, stride_h;
    const int32_t* seq_lens;
    int max_len, Hk, budget, prefix, recent;
    int cap, wcap;                       // keys (a multiple of 32) and words of bits a CTA holds
    int32_t* keep;
    int32_t* new_lens;
};

struct SelectShared {
    unsigned h1[kHist1];                 // later the list
    unsigned h2[kHist2], h3[kHist2];
    int bin, above;                      // the picked bin and the keys above it
    int listed;                          // keys offered to the list
    unsigned T;
    int need;                            // keys equal to T that are kept
    int warp_gt[kSelWarps], warp_eq[kSelWarps];
    int cta_gt[8], cta_eq[8];
    int scan[kSelWarps];
};
static_assert(kList <= kHist1, "the list takes the first histogram's place");

// Larger floats have larger keys; -0 counts as 0, and a NaN is above every
// number (a sum that cannot be judged is kept).  Always-kept tokens are above all.
__device__ __forceinline__ unsigned order_key(float x)
{
    if (x != x) return 0xFFFFFFFEu;
    const unsigned u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The bin in which the need-th largest key lies, and how many keys lie above
// it, to sh.bin and sh.above.  All threads of the block; n is a multiple of
// kSelThreads.
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
    unsigned* keys = reinterpret_cast<unsigned*>(smem_raw + (sizeof(SelectShared) + 15) / 16 * 16);
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
    auto first = [&](auto* p) { if constexpr (CLUSTER) return cl.map_shared_rank(p, 0); else return p; };

    for (int i = tid; i < kHist1 + 2 * kHist2; i += kSelThreads) sh.h1[i] = 0;   // h1, h2, h3 are adjacent
    if (tid == 0) sh.listed = 0;

    // ---- this CTA's part of the row: words of 32 keys
    const int seg = ((L + csize - 1) / csize + 31) & ~31;
    const int c0 = min(L, rank * seg), n = min(L, c0 + seg) - c0;
    const int nwords = (n + 31) >> 5;
    unsigned* bits_gt = keys + a.cap;
    unsigned* bits_eq = bits_gt + a.wcap;
    const float* x = a.acc + b * a.stride_b + h * a.stride_h + c0;
    const int kept_hi = L - a.recent;
    auto key_of = [&](float v, int i) {
        const int t = c0 + i;
        return t < a.prefix || t >= kept_hi ? 0xFFFFFFFFu : order_key(v);
    };
    auto key = [&](int i) { return i < a.cap ? keys[i] : key_of(x[i], i); };
    __syncthreads();
    // four keys a thread and step, as one 16-byte load where the row allows it
    const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0;
    auto take = [&](auto vec_tag) {
        constexpr bool V = decltype(vec_tag)::value;
        constexpr int U = 4;
        for (int i0 = 4 * tid; i0 < n; i0 += 4 * kSelThreads * U) {
            float4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * 4 * kSelThreads;
                if (V && i + 4 <= n) v[u] = *reinterpret_cast<const float4*>(x + i);
                else {
                    v[u].x = i < n ? x[i] : 0.f;
                    v[u].y = i + 1 < n ? x[i + 1] : 0.f;
                    v[u].z = i + 2 < n ? x[i + 2] : 0.f;
                    v[u].w = i + 3 < n ? x[i + 3] : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * 4 * kSelThreads;
                if (i >= n) break;
                uint4 k;
                if (c0 + i >= a.prefix && c0 + i + 4 <= kept_hi)
                    k = make_uint4(order_key(v[u].x), order_key(v[u].y), order_key(v[u].z), order_key(v[u].w));
                else
                    k = make_uint4(key_of(v[u].x, i), key_of(v[u].y, i + 1), key_of(v[u].z, i + 2), key_of(v[u].w, i + 3));
                if (i < a.cap) *reinterpret_cast<uint4*>(keys + i) = k;      // cap and i are multiples of 4
                atomicAdd(&sh.h1[k.x >> 20], 1u);
                if (i + 1 < n) atomicAdd(&sh.h1[k.y >> 20], 1u);
                if (i + 2 < n) atomicAdd(&sh.h1[k.z >> 20], 1u);
                if (i + 3 < n) atomicAdd(&sh.h1[k.w >> 20], 1u);
            }
        }
    };
    if (vec) take(std::true_type{}); else take(std::false_type{});

    // every CTA's counts go to the first CTA, which picks the bin for all
    // (the first CTA's histogram is zeroed before its part of the row is
    // taken; the others add theirs after the first barrier)
    auto pick = [&](unsigned* hist, int bins, int need) {
        sync();
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
    pick(sh.h1, kHist1, a.budget);
    const unsigned p1 = sh.bin;
    int need = a.budget - sh.above;

    // ---- bits of the words, and the list of the bin's keys (in the first
    // CTA's h1: every CTA is past its use of it)
    unsigned* list = first(sh.h1);
    int* listed = first(&sh.listed);
    auto word_key = [&](int w) { return (w << 5) + lane < n ? key((w << 5) + lane) : 0u; };
    for (int w = warp; w < nwords; w += kSelWarps) {
        const int i = (w << 5) + lane;
        const unsigned k = word_key(w);
        const bool in = i < n && k >> 20 == p1;
        const unsigned g = __ballot_sync(0xffffffffu, i < n && k >> 20 > p1), e = __ballot_sync(0xffffffffu, in);
        if (w < a.wcap && lane == 0) { bits_gt[w] = g; bits_eq[w] = e; }
        if (e) {
            int at = 0;
            if (lane == 0) at = atomicAdd(listed, __popc(e));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(e & ((1u << lane) - 1u));
            if (in && at < kList) list[at] = k;
        }
    }
    sync();
    const int total = *listed;
    if (total <= kList) {
        if (rank == 0) {
            for (int i = tid; i < total; i += kSelThreads) atomicAdd(&sh.h2[(sh.h1[i] >> 10) & 1023u], 1u);
            __syncthreads();
            pick_bin(sh.h2, kHist2, need, sh);
            const unsigned p2 = p1 << 10 | unsigned(sh.bin);
            need -= sh.above;
            for (int i = tid; i < total; i += kSelThreads)
                if (sh.h1[i] >> 10 == p2) atomicAdd(&sh.h3[sh.h1[i] & 1023u], 1u);
            __syncthreads();
            pick_bin(sh.h3, kHist2, need, sh);
            if (tid < csize) {
                SelectShared* to = &sh;
                if constexpr (CLUSTER) to = cl.map_shared_rank(&sh, tid);
                to->T = p2 << 10 | unsigned(sh.bin);
                to->need = need - sh.above;
            }
        }
        sync();
    } else {
        for (int w = warp; w < nwords; w += kSelWarps) {
            if (w < a.wcap && !bits_eq[w]) continue;
            const unsigned k = word_key(w);
            if ((w << 5) + lane < n && k >> 20 == p1) atomicAdd(&sh.h2[(k >> 10) & 1023u], 1u);
        }
        pick(sh.h2, kHist2, need);
        const unsigned p2 = p1 << 10 | unsigned(sh.bin);
        need -= sh.above;
        for (int w = warp; w < nwords; w += kSelWarps) {
            if (w < a.wcap && !bits_eq[w]) continue;
            const unsigned k = word_key(w);
            if ((w << 5) + lane < n && k >> 10 == p2) atomicAdd(&sh.h3[k & 1023u], 1u);
        }
        pick(sh.h3, kHist2, need);
        if (tid == 0) { sh.T = p2 << 10 | unsigned(sh.bin); sh.need = need - sh.above; }
        __syncthreads();
    }
    const unsigned T = sh.T;
    need = sh.need;

    // ---- the words' final bits, their counts per warp (consecutive words),
    // then the output in order
    const int wper = (nwords + kSelWarps - 1) / kSelWarps;
    const int w0 = min(nwords, warp * wper), w1 = min(nwords, w0 + wper);
    auto word_bits = [&](int w, unsigned& g, unsigned& e) {
        const int i = (w << 5) + lane;
        const unsigned k = word_key(w);
        g = __ballot_sync(0xffffffffu, i < n && k > T);
        e = __ballot_sync(0xffffffffu, i < n && k == T);
    };
    int gt = 0, eq = 0;
    for (int w = w0; w < w1; ++w) {
        unsigned g, e;
        if (w < a.wcap) {
            g = bits_gt[w];
            e = bits_eq[w];
            if (e) {
                word_bits(w, g, e);
                __syncwarp();
                if (lane == 0) { bits_gt[w] = g; bits_eq[w] = e; }
            }
        } else {
            word_bits(w, g, e);
        }
        gt += __popc(g);
        eq += __popc(e);
    }
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
    for (int w = w0; w < w1; ++w) {
        unsigned g, e;
        if (w < a.wcap) { g = bits_gt[w]; e = bits_eq[w]; }
        else            word_bits(w, g, e);
        const int eq_before = pos_eq + __popc(e & below);
        const int at = pos_gt + __popc(g & below) + min(eq_before, need);
        if ((g >> lane & 1u) || ((e >> lane & 1u) && eq_before < need)) keep[at] = c0 + (w << 5) + lane;
        pos_gt += __popc(g);
        pos_eq += __popc(e);
    }
}

// ------------------------------------------------------------------ compact
//
// One cluster per (sequence, kv head).  The kept tokens ascend, so slot i
// comes from slot keep[i] >= i: a chunk of destinations may be written once
// the chunk's sources (all at or past its start) have been read by every
// warp of the cluster, and the next chunk's sources are never among the
// slots written.  One barrier per chunk, between its reads and its writes;
// the next chunk's addresses are looked up before it.
//
// A record of this kv head begins at the same place of every token row.  Where
// token rows are whole 32-bit words (WORDS), source and destination agree
// modulo 4, and records move as aligned words: a load may take the two bytes
// around the record's ends along (they lie in the cache, whose size is a
// multiple of 32), a store leaves them out.  Other rows move as 16-bit halves.
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

__device__ __forceinline__ uint32_t ld_half(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// K slots per warp and chunk; IT 128-byte steps cover the record.
template <int K, int IT, bool SOA, bool WORDS>
__global__ void __launch_bounds__(1024) compact_kernel(CompactArgs a, int csize)
{
    const int rank = blockIdx.x % csize, row = blockIdx.x / csize;
    const int b = row / a.Hk, h = row % a.Hk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int L = a.seq_lens[b];
    if (L <= a.budget || L > a.max_len) return;      // uniform in the cluster
    const int32_t* keep = a.keep + (long long)row * a.budget;
    const int32_t* bt = a.block_table + (long long)b * a.bt_stride;
    float* acc = a.acc ? a.acc + b * a.stride_b + h * a.stride_h : nullptr;
    const int bs = 1 << a.bs_log2;
    const int nbytes = SOA ? a.g.data_bytes : a.g.slot;      // even
    const int per_chunk = csize * nwarps * K;
    const int nchunks = (a.budget + per_chunk - 1) / per_chunk;
    int i = (rank * nwarps + warp) * K + lane;       // lane k < K: slot i of the chunk

    // slot i's source token and the places of both records; src < 0: nothing to move
    struct Place { int t; long long src, dst, msrc, mdst; };
    auto place = [&](int i) {
        Place p = {0, -1, -1, 0, 0};
        if (lane < K && i < a.budget) {
            p.t = keep[i];
            if (p.t != i && p.t >= 0 && p.t < L) {
                const long long sp = bt[p.t >> a.bs_log2], dp = bt[i >> a.bs_log2];
                if ((unsigned long long)sp < (unsigned long long)a.num_blocks &&
                    (unsigned long long)dp < (unsigned long long)a.num_blocks) {
                    const uint8_t *d, *m;
                    slot_ptrs(a.g, a.cache, sp, p.t & (bs - 1), h, bs, a.Hk, d, m);
                    p.src = d - a.cache;
                    p.msrc = m - a.cache;
                    slot_ptrs(a.g, a.cache, dp, i & (bs - 1), h, bs, a.Hk, d, m);
                    p.dst = d - a.cache;
                    p.mdst = m - a.cache;
                }
            }
        }
        return p;
    };
    Place p = place(i);
    for (int c = 0; c < nchunks; ++c, i += per_chunk) {
        const float w = acc && p.src >= 0 ? acc[p.t] : 0.f;
        uint32_t v[K][IT], mv[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long s = __shfl_sync(0xffffffffu, p.src, k);
            const int lead = int(__shfl_sync(0xffffffffu, uint32_t(p.dst), k) & 2);   // the first word may begin 2 bytes early
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int o = 4 * (lane + 32 * it) - lead;
                const uint8_t* q = a.cache + s + o;
                if constexpr (WORDS) {
                    v[k][it] = s >= 0 && o < nbytes ? *reinterpret_cast<const uint32_t*>(q) : 0u;
                } else {
                    uint32_t lo = 0, hi = 0;
                    if (s >= 0 && o >= 0 && o < nbytes) lo = ld_half(q);
                    if (s >= 0 && o + 2 < nbytes) hi = ld_half(q + 2);
                    v[k][it] = lo | hi << 16;
                }
            }
            if constexpr (SOA) {
                const long long ms = __shfl_sync(0xffffffffu, p.msrc, k);
                mv[k] = s >= 0 && 2 * lane < a.g.meta_bytes ? ld_half(a.cache + ms + 2 * lane) : 0u;
            }
        }
        const Place next = place(c + 1 < nchunks ? i + per_chunk : a.budget);
        if (csize > 1) cg::this_cluster().sync();
        else           __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long d = __shfl_sync(0xffffffffu, p.dst, k);
            if (d < 0) continue;
            const int lead = int(d & 2);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int o = 4 * (lane + 32 * it) - lead;
                uint8_t* q = a.cache + d + o;
                if (o >= 0 && o + 2 < nbytes) *reinterpret_cast<uint32_t*>(q) = v[k][it];
                else if (o >= 0 && o < nbytes) *reinterpret_cast<uint16_t*>(q) = uint16_t(v[k][it]);
                else if (o < 0) *reinterpret_cast<uint16_t*>(q + 2) = uint16_t(v[k][it] >> 16);
            }
            if constexpr (SOA) {
                const long long md = __shfl_sync(0xffffffffu, p.mdst, k);
                if (2 * lane < a.g.meta_bytes)
                    *reinterpret_cast<uint16_t*>(a.cache + md + 2 * lane) = uint16_t(mv[k]);
            }
        }
        if (acc && p.src >= 0) acc[i] = w;
        p = next;
    }
    // past the last barrier every source has been read: the evicted tail's sums start again at 0
    if (acc)
        for (int t = a.budget + rank * blockDim.x + threadIdx.x; t < L; t += csize * blockDim.x) acc[t] = 0.f;
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
    // A CTA's part of the longest row is at most 8192 keys where 8 CTAs suffice
    // for that (four CTAs then share an SM, and one's loads overlap another's
    // passes), and shorter when the rows are too few to fill the GPU.
    auto seg = [&](int c) { return ((max_seq_len + c - 1) / c + 31) & ~31; };
    int csize = 1;
    while (csize < 8 && (seg(csize) > 8192 || (rows * csize < 2 * kNumSMs && seg(csize) > 2048))) csize *= 2;
    a.cap = std::min(seg(csize), kSelMaxKeys);
    a.wcap = std::min(seg(csize) / 32, kSelMaxWords);
    const size_t smem = (sizeof(SelectShared) + 15) / 16 * 16 + 4 * size_t(a.cap) + 8 * size_t(a.wcap);
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
    const bool words = soa ? nbytes % 4 == 0 : num_kv_heads * nbytes % 4 == 0;
    const int K = wide ? 4 : 8;
    // CTAs of 8 warps, eight to an SM, in clusters of up to 8; of 32 warps
    // where even clusters of 8 leave SMs idle (the chunks are then fewer)
    int csize = 1, threads = 256;
    while (csize < 8 && rows * csize < 8 * kNumSMs && csize * threads / 32 * K < budget) csize *= 2;
    while (threads < 1024 && rows * csize * threads < 1024LL * kNumSMs && csize * threads / 32 * K < budget) threads *= 2;
    auto k = compact_kernel<8, 1, false, false>;
    if (wide) k = soa ? (words ? compact_kernel<4, 2, true, true> : compact_kernel<4, 2, true, false>)
                      : (words ? compact_kernel<4, 2, false, true> : compact_kernel<4, 2, false, false>);
    else      k = soa ? (words ? compact_kernel<8, 1, true, true> : compact_kernel<8, 1, true, false>)
                      : (words ? compact_kernel<8, 1, false, true> : compact_kernel<8, 1, false, false>);
    return launch_cluster(k, a, rows, csize, threads, 0, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? TQ_OK : TQ_ERR_CUDA;
}
