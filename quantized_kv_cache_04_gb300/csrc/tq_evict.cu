// Eviction by accumulated attention weight: which tokens each kv head keeps
// (tq_evict_select), and the move of the kept slots to the front of their
// sequence, in place (tq_evict_compact).
#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

namespace cg = cooperative_groups;

namespace tq {
namespace {

// ------------------------------------------------------------------ select
//
// One CTA, or a thread-block cluster, per (sequence, kv head) row.  A CTA holds
// its part of the row in shared memory as order-preserving 32-bit keys; of a
// part above kSelMaxKeys the rest is read again, from L2.
//   1. A histogram of the keys' top 11 bits, merged in the first CTA, gives the
//      bin that holds the budget-th largest key.
//   2. A second look at the keys counts those above the bin and lists those in
//      it, usually a few per cent.
//   3. Histograms of the middle 11 and the low 10 bits of the listed keys give
//      the budget-th key T.  A list that overflows (many equal sums) is not
//      used: the CTA looks at its keys again instead.
//   4. The tokens with keys above T, and the first of those equal to T, are
//      written in order, each warp's from the counts of those before it.
// Bound by instructions (28.6 M warp instructions for 12.4 M keys, issued 60% of
// the time), not by the one read of the sums.  Measured: 512 rows of up to 32768
// tokens, budget 8192: 49 us with one CTA a row, 56 / 84 / 147 us with clusters of
// 2 / 4 / 8 (each barrier of a cluster costs about 1 us); 32 rows of 65536: 39 us
// with one CTA, 25 / 14 / 14 us; 32 rows of 262144: 258 us, 136 / 45 / 39 us.
// Holding 4096 to 40960 keys changes those by 5%, but for one CTA of 164 KB per SM
// in the last case (61 us).
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHist1 = 2048, kHist2 = 2048, kHist3 = 1024;
constexpr int kList = 2048;             // listed keys of the bin
constexpr int kSelMaxKeys = 20480;      // keys a CTA holds: 80 KB, two CTAs to an SM

struct SelectArgs {
    const float* acc;
    long long stride_b, stride_h;
    const int32_t* seq_lens;
    int max_len, Hk, budget, prefix, recent;
    int cap;                             // keys a CTA holds: a multiple of 128
    int32_t* keep;
    int32_t* new_lens;
};

struct SelectShared {
    unsigned h1[kHist1];                 // later the listed keys
    unsigned h2[kHist2], h3[kHist3];
    int list_at[kList];                  // where in the CTA's part
    int bin, above;                      // the picked bin and the keys above it
    int listed;                          // keys offered to the list
    int warp_gt[kSelWarps], warp_eq[kSelWarps];
    int cta_gt[8], cta_eq[8];
    int scan[kSelWarps];
};
static_assert(kList <= kHist1, "the list takes the first histogram's place");

// Larger floats have larger keys; -0 counts as 0, and a NaN is above every
// number (a sum that cannot be judged is kept).  Always-kept tokens are above all.
__device__ __forceinline__ unsigned order_key(float x)
{
    const unsigned u = __float_as_uint(x + 0.f);     // a NaN's sum is the canonical, positive NaN
    return min(u ^ (unsigned(int(u) >> 31) | 0x80000000u), 0xFFFFFFFEu);
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
    auto first = [&](unsigned* p) { if constexpr (CLUSTER) return cl.map_shared_rank(p, 0); else return p; };

    for (int i = tid; i < (kHist1 + kHist2 + kHist3) / 4; i += kSelThreads)      // h1, h2, h3 are adjacent
        reinterpret_cast<uint4*>(sh.h1)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sh.listed = 0;
    if (tid < kSelWarps) sh.warp_eq[tid] = 0;
    __syncthreads();

    // ---- this CTA's part of the row, in steps of 128 keys: four per lane
    const int seg = ((L + csize - 1) / csize + 127) & ~127;
    const int c0 = min(L, rank * seg), n = min(L, c0 + seg) - c0;
    const float* x = a.acc + b * a.stride_b + h * a.stride_h + c0;
    const int kept_hi = L - a.recent;
    const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0;
    auto load4 = [&](int i) {                        // i a multiple of 4, below n
        if (vec && i + 4 <= n) return *reinterpret_cast<const float4*>(x + i);
        return make_float4(x[i], i + 1 < n ? x[i + 1] : 0.f, i + 2 < n ? x[i + 2] : 0.f, i + 3 < n ? x[i + 3] : 0.f);
    };
    // keys of the sums of tokens i .. i + 3; past the part 0, below every key
    // that is ever above or equal (T >= order_key(-inf) > 0)
    // (plain4: none of the four is kept always; then none is past the part either)
    const unsigned plain = kept_hi - 4 >= a.prefix ? unsigned(kept_hi - 4 - a.prefix) : 0u;
    const int plain_from = kept_hi - 4 >= a.prefix ? a.prefix - c0 : INT_MAX;
    auto plain4 = [&](int i) { return unsigned(i - plain_from) <= plain; };
    auto keys4 = [&](const float4& v, int i) {
        uint4 k = make_uint4(order_key(v.x), order_key(v.y), order_key(v.z), order_key(v.w));
        const int t = c0 + i;
        if (!plain4(i)) {
            auto one = [&](unsigned kk, int j) {
                return i + j >= n ? 0u : t + j < a.prefix || t + j >= kept_hi ? 0xFFFFFFFFu : kk;
            };
            k = make_uint4(one(k.x, 0), one(k.y, 1), one(k.z, 2), one(k.w, 3));
        }
        return k;
    };
    auto count = [&](const float4& v, int i) {
        const uint4 k = keys4(v, i);
        if (i < a.cap) *reinterpret_cast<uint4*>(keys + i) = k;
        // keys past the part are 0: they count in the lowest bin, below every pick
        atomicAdd(&sh.h1[k.x >> 21], 1u);
        atomicAdd(&sh.h1[k.y >> 21], 1u);
        atomicAdd(&sh.h1[k.z >> 21], 1u);
        atomicAdd(&sh.h1[k.w >> 21], 1u);
    };
    {
        // four 16-byte loads a thread on their way at a time
        constexpr int U = 4, kStep = 4 * kSelThreads;
        int i = 4 * tid;
        if (vec)
            for (; i + (U - 1) * kStep + 4 <= n; i += U * kStep) {
                float4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const float4*>(x + i + u * kStep);
#pragma unroll
                for (int u = 0; u < U; ++u) count(v[u], i + u * kStep);
            }
        for (; i < n; i += kStep) count(load4(i), i);
    }
    auto look = [&](int i) {                         // keys i .. i + 3 again
        if (i >= n) return make_uint4(0, 0, 0, 0);
        return i < a.cap ? *reinterpret_cast<const uint4*>(keys + i) : keys4(load4(i), i);
    };

    // The bin of the need-th key, from the histograms of all CTAs: the others'
    // counts are added to the first CTA's (merge: they are still in their own).
    auto pick = [&](unsigned* hist, int bins, int need, bool merge) {
        sync();
        if constexpr (CLUSTER) {
            if (merge) {
                if (rank != 0) {
                    unsigned* to = first(hist);
                    for (int i = tid; i < bins; i += kSelThreads)
                        if (hist[i]) atomicAdd(&to[i], hist[i]);
                }
                cl.sync();
            }
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
    pick(sh.h1, kHist1, a.budget, true);
    const unsigned p1 = sh.bin;
    int need = a.budget - sh.above;

    // ---- each warp's consecutive keys: how many lie above the bin; the list
    // of those in it (keys in h1, which no CTA needs any more)
    const int wseg = ((n + kSelWarps - 1) / kSelWarps + 127) & ~127;
    const int w0 = min(n, warp * wseg), w1 = min(n, w0 + wseg);
    unsigned* list = sh.h1;
    // f(i, k): this warp's steps in order, four keys k of i .. i + 3 per lane; the
    // whole steps held in shared memory apart, where a look is one load
    const int w_held = min(w1 & ~127, a.cap);
    auto steps = [&](auto f) {
        int i = w0 + 4 * lane;
        for (; i < w_held; i += 128) {
            const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
            f(i, k);
        }
        for (; i < w1 + 4 * lane; i += 128) f(i, look(i));
    };
    // bounds of the bin as keys: in it p1_lo <= k <= p1_hi; no real key is 0
    const unsigned p1_lo = max(p1 << 21, 1u), p1_hi = p1 << 21 | 0x1FFFFFu;
    int gt = 0;
    steps([&](int i, const uint4& k4) {
        const unsigned k[4] = {k4.x, k4.y, k4.z, k4.w};
        bool in[4];
        int cnt = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gt += k[j] > p1_hi;
            in[j] = k[j] - p1_lo <= p1_hi - p1_lo;
            cnt += in[j];
        }
        if (cnt) {                                   // few lanes: their order in the list does not matter
            int at = atomicAdd(&sh.listed, cnt);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in[j] && at < kList) { list[at] = k[j]; sh.list_at[at++] = i + j; }
        }
    });
    gt = __reduce_add_sync(0xffffffffu, gt);
    if (lane == 0) sh.warp_gt[warp] = gt;
    __syncthreads();
    const int listed = sh.listed;
    const bool use_list = listed <= kList;
    // one level: the listed keys with these leading bits, by the next ones
    auto level = [&](unsigned* hist, int bins, int lead, unsigned prefix, int shift) {
        if (use_list) {
            unsigned* to = first(hist);
            for (int i = tid; i < listed; i += kSelThreads)
                if (list[i] >> lead == prefix) atomicAdd(&to[(list[i] >> shift) & (bins - 1)], 1u);
        } else {
            for (int i = 4 * tid; i < n; i += 4 * kSelThreads) {
                const uint4 k4 = look(i);
                const unsigned k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k[j] >> lead == prefix && i + j < n) atomicAdd(&hist[(k[j] >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
            if (rank != 0) {
                unsigned* to = first(hist);
                for (int i = tid; i < bins; i += kSelThreads)
                    if (hist[i]) atomicAdd(&to[i], hist[i]);
            }
        }
        pick(hist, bins, need, false);
    };
    level(sh.h2, kHist2, 21, p1, 10);
    const unsigned p2 = p1 << 11 | unsigned(sh.bin);
    need -= sh.above;
    level(sh.h3, kHist3, 10, p2, 0);
    const unsigned T = p2 << 10 | unsigned(sh.bin);
    need -= sh.above;                                // keys equal to T that are kept

    // ---- counts above T and equal to T per warp
    if (use_list) {
        for (int i = tid; i < listed; i += kSelThreads) {
            const unsigned k = list[i];
            if (k >= T) atomicAdd(k > T ? &sh.warp_gt[sh.list_at[i] / wseg] : &sh.warp_eq[sh.list_at[i] / wseg], 1);
        }
    } else {
        int g = 0, e = 0;
        steps([&](int, const uint4& k) {
            g += (k.x > T) + (k.y > T) + (k.z > T) + (k.w > T);
            e += (k.x == T) + (k.y == T) + (k.z == T) + (k.w == T);
        });
        g = __reduce_add_sync(0xffffffffu, g);
        e = __reduce_add_sync(0xffffffffu, e);
        if (lane == 0) { sh.warp_gt[warp] = g; sh.warp_eq[warp] = e; }
    }
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
    // each warp writes its kept tokens in order: a lane's four follow those of the lanes below it
    int32_t* to = keep + pos_gt + min(pos_eq, need);
    steps([&](int i, const uint4& k4) {
        const unsigned k[4] = {k4.x, k4.y, k4.z, k4.w};
        bool take[4];
        int cnt = 0, eq = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            take[j] = k[j] > T;
            eq += k[j] == T;
        }
        if (__any_sync(0xffffffffu, eq)) {           // warp-uniform: ties, the first `need` of the row are kept
            int incl = eq;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, m);
                if (lane >= m) incl += o;
            }
            int at = pos_eq + incl - eq;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k[j] == T) take[j] = at++ < need;
            pos_eq += __shfl_sync(0xffffffffu, incl, 31);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) cnt += take[j];
        int incl = cnt;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, m);
            if (lane >= m) incl += o;
        }
        int32_t* at = to + (incl - cnt);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (take[j]) *at++ = c0 + i + j;
        to += __shfl_sync(0xffffffffu, incl, 31);
    });
}

// ------------------------------------------------------------------ compact
//
// One cluster per (sequence, kv head).  The kept tokens ascend, so slot i
// comes from slot keep[i] >= i: a chunk of destinations may be written once
// the chunk's sources (all at or past its start) have been read by every
// warp of the cluster, and the sources of later chunks are never among the
// slots written.  One barrier per chunk, between its reads and its writes.
//
// A half-warp moves a record.  It is read by asynchronous copies of the aligned
// 16-byte units that hold it (they lie in the cache, whose size is a multiple
// of 32) into a ring of kStages chunks in shared memory, so two more chunks are
// on their way while one is written: records lie scattered in memory, and bytes
// in flight are what the kernel lives on.  It is written in units of UNIT bytes,
// the largest power of two, up to 16, that divides a token row: a kv head's
// record begins at the same place of every row, so source and destination
// agree modulo UNIT (SoA data records are whole 16-byte units).  The bytes before
// the first and after the last whole unit, and SoA metadata, go as 16-bit halves.
//
// Bound by memory: a kept record lies alone, so its bytes are read in 64-byte
// pieces (118-byte slots: 214 MB from DRAM for 129 MB).  Measured, 256 rows of
// 16384 tokens (ragged) cut to 4096: 118-byte slots 68 us (3.8 TB/s of records read
// and written, 4.5 TB/s at the DRAM), 196-byte slots 95 us (4.4 TB/s), SoA 118 99
// us, 3 kv heads (2-byte units) 31 us; 8 rows of 262144 cut to 32768: 37 us.
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

template <int UNIT> struct UnitOf;
template <> struct UnitOf<2> { using type = uint16_t; };
template <> struct UnitOf<4> { using type = uint32_t; };
template <> struct UnitOf<8> { using type = uint2; };
template <> struct UnitOf<16> { using type = uint4; };

constexpr int kSlots = 8;                // slots per warp and chunk: four per half-warp
constexpr int kStages = 3;
constexpr int kCmpMaxThreads = 1024;

// What the writes of a chunk need to know of a slot.
struct __align__(16) Move {
    long long dst;                       // byte offset of the destination record; < 0: nothing moves
    int lead;                            // bytes of the first 16-byte unit before the source record
    int meta;                            // SoA: the same for its metadata record (dst: the block convention)
};

// 16-byte units that hold a record of nbytes at any even place, and with SoA
// its aligned record and the metadata record's two.
__host__ __device__ constexpr int record_units(int nbytes, bool soa)
{
    return soa ? nbytes / 16 + 2 : (nbytes + 14 + 15) / 16;
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy_async4(void* dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src)
                 : "memory");
}

// STEPS steps of 16 units of UNIT bytes cover a record.
template <int UNIT, int STEPS, bool SOA>
__global__ void __maxnreg__(40) compact_kernel(CompactArgs a, int csize)
{
    using unit_t = typename UnitOf<UNIT>::type;
    extern __shared__ __align__(16) uint8_t ring[];
    const int rank = blockIdx.x % csize, row = blockIdx.x / csize;
    const int b = row / a.Hk, h = row % a.Hk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int half = lane >> 4, l = lane & 15;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int L = a.seq_lens[b];
    if (L <= a.budget || L > a.max_len) return;      // uniform in the cluster
    const int32_t* keep = a.keep + (long long)row * a.budget;
    const int32_t* bt = a.block_table + (long long)b * a.bt_stride;
    float* acc = a.acc ? a.acc + b * a.stride_b + h * a.stride_h : nullptr;
    const int nbytes = SOA ? a.g.data_bytes : a.g.slot;      // even
    const int per_chunk = csize * nwarps * kSlots;
    const int nchunks = (a.budget + per_chunk - 1) / per_chunk;
    const int i_warp = (rank * nwarps + warp) * kSlots;      // lane k < kSlots: slot i_warp + k of a chunk

    // this warp's part of the ring: per stage the records, their moves, their sums
    const int units = record_units(nbytes, SOA);
    const int slot_bytes = 16 * units, stage_bytes = kSlots * (slot_bytes + 16 + 4);   // a multiple of 16
    uint8_t* mine = ring + warp * kStages * stage_bytes;

    // byte offsets of the record (SoA: data, metadata) of token t in block `page`
    // (a block's size fits 32 bits: at most 4096 kv heads)
    const unsigned row_bytes = a.Hk * nbytes, block_lg = a.bs_log2, off_mask = (1u << block_lg) - 1u;
    const unsigned block_bytes = unsigned(a.Hk * a.g.slot) << block_lg;
    auto record = [&](int page, int t) -> long long {
        return (unsigned long long)unsigned(page) * block_bytes + ((t & off_mask) * row_bytes + h * nbytes);
    };
    auto meta = [&](int page, int t) -> long long {
        return (unsigned long long)unsigned(page) * block_bytes +
               ((row_bytes << block_lg) + ((t & off_mask) * a.Hk + h) * a.g.meta_bytes);
    };
    auto inside = [&](int page) { return page >= 0 && page < a.num_blocks; };

    // The lookups run ahead of the requests: a chunk's tokens are read two
    // requests early, their pages one request early.
    auto token = [&](int c) {                        // lane k: slot k's source token; < 0: nothing moves
        const int i = c * per_chunk + i_warp + lane;
        if (lane >= kSlots || c >= nchunks || i >= a.budget) return -1;
        const int t = keep[i];
        return t != i && t < L ? t : -1;
    };
    struct Pages { int t, src, dst; };
    auto pages = [&](int c, int t) {
        Pages p = {t, -1, -1};
        if (t >= 0) {
            p.src = bt[t >> block_lg];
            p.dst = bt[(c * per_chunk + i_warp + lane) >> block_lg];
        }
        return p;
    };
    Pages ahead = pages(0, token(0));
    int ahead_token = token(1);
    // request chunk c's sources; called for c = 0, 1, 2, ...; every call is one copy group
    auto request = [&](int c) {
        const Pages p = ahead;
        ahead = pages(c + 1, ahead_token);
        ahead_token = token(c + 2);
        if (c < nchunks) {
            uint8_t* st = mine + (c % kStages) * stage_bytes;
            const int i = c * per_chunk + i_warp + lane;
            long long src = -1, msrc = 0;
            if (lane < kSlots) {
                Move m = {-1, 0, 0};
                if (p.t >= 0 && inside(p.src) && inside(p.dst)) {
                    src = record(p.src, p.t);
                    m.dst = record(p.dst, i);
                    m.lead = int(src) & 15;
                    if (SOA) { msrc = meta(p.src, p.t); m.meta = int(msrc) & 15; }
                    if (acc) copy_async4(st + kSlots * (slot_bytes + 16) + 4 * lane, acc + p.t);
                }
                reinterpret_cast<Move*>(st + kSlots * slot_bytes)[lane] = m;
            }
#pragma unroll
            for (int k = 0; k < kSlots / 2; ++k) {
                const int from = 2 * k + half;       // the lane that looked the slot up
                const long long s = __shfl_sync(0xffffffffu, src, from);
                uint8_t* to = st + from * slot_bytes + 16 * l;
                if constexpr (SOA) {
                    const long long ms = __shfl_sync(0xffffffffu, msrc, from);
                    const int data = units - 2, j = l - data;
                    if (s >= 0 && l < data) copy_async16(to, a.cache + s + 16 * l);
                    else if (s >= 0 && j >= 0 && 16 * j < (int(ms) & 15) + a.g.meta_bytes)
                        copy_async16(to, a.cache + (ms & ~15LL) + 16 * j);
                } else {
                    if (s >= 0 && 16 * l < (int(s) & 15) + nbytes) copy_async16(to, a.cache + (s & ~15LL) + 16 * l);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // write chunk c from the ring
    auto write = [&](int c) {
        const uint8_t* st = mine + (c % kStages) * stage_bytes;
        const Move* moves = reinterpret_cast<const Move*>(st + kSlots * slot_bytes);
#pragma unroll
        for (int k = 0; k < kSlots / 2; ++k) {
            const int from = 2 * k + half;
            const Move m = moves[from];
            if (m.dst < 0) continue;
            const uint8_t* q = st + from * slot_bytes + m.lead;
            uint8_t* d = a.cache + m.dst;
            const int head = -m.lead & (UNIT - 1), whole = (nbytes - head) / UNIT;
#pragma unroll
            for (int step = 0; step < STEPS; ++step) {
                const int o = head + (l + 16 * step) * UNIT;
                if (l + 16 * step < whole) *reinterpret_cast<unit_t*>(d + o) = *reinterpret_cast<const unit_t*>(q + o);
            }
            if constexpr (SOA) {
                // the metadata record of destination slot i: the block's metadata region
                const int i = c * per_chunk + i_warp + from;
                if (2 * l < a.g.meta_bytes)
                    *reinterpret_cast<uint16_t*>(a.cache + meta(bt[i >> block_lg], i) + 2 * l) =
                        *reinterpret_cast<const uint16_t*>(st + from * slot_bytes + 16 * (units - 2) + m.meta + 2 * l);
            } else if constexpr (UNIT > 2) {
                // lanes 0 .. 7: the halves before the first whole unit, 8 .. 15: after the last
                const int o = l < 8 ? 2 * l : head + whole * UNIT + 2 * (l - 8);
                if (l < 8 ? o < head : o < nbytes)
                    *reinterpret_cast<uint16_t*>(d + o) = *reinterpret_cast<const uint16_t*>(q + o);
            }
        }
        if (acc && lane < kSlots && moves[lane].dst >= 0)
            acc[c * per_chunk + i_warp + lane] = reinterpret_cast<const float*>(st + kSlots * (slot_bytes + 16))[lane];
    };

    // A chunk's barrier opens once every warp has read its sources; what a warp
    // does between its arrival and its wait is the request two chunks on.  The
    // arrival is relaxed: what it orders are reads, and those have returned
    // (wait_group); a releasing one would also wait for the last chunk's writes,
    // which no CTA of the cluster reads (4 of 10 stalled cycles).
    for (int c = 0; c < kStages - 1; ++c) request(c);
    for (int c = 0; c < nchunks; ++c) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");       // chunk c is here
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
        __syncwarp();                            // chunk c - 1's reads of the ring, before its stage is refilled
        request(c + kStages - 1);
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        write(c);
    }
    // past the last barrier every source has been read: the evicted tail's sums start again at 0
    if (acc)
        for (int t = a.budget + rank * blockDim.x + threadIdx.x; t < L; t += csize * blockDim.x) acc[t] = 0.f;
}

// The kernel for AoS records of nbytes.
template <int UNIT>
auto compact_of(int nbytes)
{
    constexpr int kMost = (196 / UNIT + 15) / 16, kSome = (134 / UNIT + 15) / 16;
    return nbytes > 134 ? compact_kernel<UNIT, kMost, false> : compact_kernel<UNIT, kSome, false>;
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
    // every row reads the old lengths while the new ones are written
    if (new_lens < seq_lens + batch && seq_lens < new_lens + batch) return TQ_ERR_INVALID_ARG;
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
    // One CTA per row of up to 32768 tokens when the rows fill the GPU (two to an
    // SM); clusters of up to 8 for longer rows, and for fewer rows as long as
    // a CTA's part is above 2048 keys (figures at the kernel).
    auto seg = [&](int c) { return ((max_seq_len + c - 1) / c + 127) & ~127; };
    int csize = 1;
    while (csize < 8 && (seg(csize) > 32768 || (rows * csize < 2 * kNumSMs && seg(csize) > 2048))) csize *= 2;
    a.cap = std::min(seg(csize), kSelMaxKeys);
    const size_t smem = (sizeof(SelectShared) + 15) / 16 * 16 + 4 * size_t(a.cap);
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
    if (batch < 0 || num_kv_heads < 1 || num_kv_heads > 4096 || num_blocks < 0 || block_table_stride < 0 || budget < 1 || max_seq_len < 0 || max_seq_len > kMaxListedLen ||
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
    // a power of two that divides every token row (the cache starts at a
    // multiple of 16)
    const int row_bytes = num_kv_heads * nbytes;
    // CTAs of 8 warps, several to an SM, in clusters of up to 8; of 32
    // warps where even clusters of 8 leave SMs idle (the chunks are then fewer)
    int csize = 1, threads = 256;
    while (csize < 8 && rows * csize < 8 * kNumSMs && csize * threads / 32 * kSlots < budget) csize *= 2;
    if (rows * csize < 4 * kNumSMs && csize * threads / 32 * kSlots < budget) threads = kCmpMaxThreads;
    const size_t smem = size_t(threads / 32) * kStages * kSlots * (16 * record_units(nbytes, soa) + 20);
    auto k = soa                   ? compact_kernel<16, 1, true>
             : row_bytes % 16 == 0 ? compact_of<16>(nbytes)
             : row_bytes % 8 == 0  ? compact_of<8>(nbytes)
             : row_bytes % 4 == 0  ? compact_of<4>(nbytes)
                                   : compact_of<2>(nbytes);
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
        return TQ_ERR_CUDA;
    return launch_cluster(k, a, rows, csize, threads, smem, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? TQ_OK : TQ_ERR_CUDA;
}
