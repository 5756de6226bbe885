// Attention of new tokens over a paged bf16 cache on the tensor cores (heads of
// up to 128 columns).  Contract and masks: include/usm.h; how the work is
// divided: usm_paged.cuh.
//
// One CTA an SM walks over its share of tiles of 128 keys.  A block has up to
// 256 rows (tokens x the heads that share keys) in two halves of 128, one row a
// lane of tensor memory:
//   S = Q·K^T    both from shared memory, 128 x 128 fp32 in tensor memory;
//   P = 2^(S·c - m·c), a row a thread, over S's own columns: two bf16 parts, the
//     rounded weight and what that leaves, which hold a weight to 2^-16 (the rounding
//     alone, 2^-8, is as large as the output's own);
//   O += P·V     P from tensor memory, V from shared memory, fp32 in tensor memory,
//     one part of P after the other.
// While one half's softmax runs the tensor cores work for the other.  Where a
// block has no more than 128 rows (single tokens, drafts) the halves take the
// same rows over alternate tiles (on from one segment to the next), and the half
// that is done first leaves its sums to the other and goes on.
//
// Bounds and figures (measured at the sizes given): single tokens by HBM and the
// softmax's latency (64 over 8192 keys, 1.55 GB: 263 us, 5.9 TB/s); chunks by the
// products beside the softmax's latency (two of 2048 over 16384 keys: 1000 us, 1010
// TFLOP/s, half as many again with the second part's); prompts of a few thousand
// tokens by start and joining as well (8x4096 of 64 columns: 56 us).  With the
// rounded weight alone these are 242, 735 and 48 us: tokens pay for the forming of the
// second part (without its products they take the same time), chunks mostly for its
// products (without them 800 us); its storing costs nothing.
//
// The reference m of a row is its maximum, but it is raised only when a tile's
// maximum passes it by more than 2^8 in the weights: fp32 sums and weights keep
// their relative precision, and O is rescaled (a pass over tensor memory) once or
// twice a row instead of in most tiles.
//
// Roles: warps 0-3 and 4-7 softmax and output of the halves, 8-11 copies of
// queries, keys and values (through the page table, rows outside
// the sequence zeros), 12 issues the matrix products, 13 hands out the segments,
// 14 and 15 help with the copies.
#include <cuda_bf16.h>

#include <algorithm>

#include "usm_internal.h"
#include "usm_paged.cuh"
#include "usm_tmem.cuh"

namespace usm {
namespace {

constexpr int kRows = 256, kKeys = 128, kThreads = 512;
// What an item costs a CTA beyond its tiles (its queries, the first products and the
// output), in tiles: 8000 to 14000 cycles where a tile takes 2400 to 4200.  (3 to 8
// measured: a prompt of 8x4096 takes 56.5 us with 4, 56.4 with 3, 59.4 with 8; 64
// tokens 262, 263, 266; local attention 141.5, 139.8, 137.8.)
constexpr int kSegmentCost = 4;
constexpr int kRing = 4;       // segments handed out ahead
constexpr int kConsumers = 13; // warps that read a segment (and two more where they copy queries)
constexpr float kRaise = 8.f;  // log2 of the largest weight before a row's reference is raised
// Largest |m·c| for which S·c - m·c is formed by one FMA: the rounding of m·c changes
// the weights that share the reference by one factor, which differs where the
// reference was raised, in the other half and in other parts; up to here it stays
// within 2^-17, below a weight's own 2^-16.
constexpr float kNear = 256.f;

using Shares = PagedShares<kRows, kKeys, kThreads, kSegmentCost>;

template <int DP>  // columns of shared memory: 64 or 128
struct Sizes {
    static constexpr int kTile = DP * 256;              // bytes of 128 rows
    static constexpr int kStages = DP == 128 ? 5 : 10;  // tiles of keys or values in flight
    static constexpr int kStage0 = 2 * kTile;           // behind the two halves' queries
    static constexpr int kControl = kStage0 + kStages * kTile;
};

struct Control {
    unsigned long long full[10], empty[10], started[10], cleaned[10];  // stages
    unsigned long long q_full, q_empty;
    unsigned long long s_full[2], p_full[2], o_full[2];
    unsigned long long seg_full[kRing], seg_empty[kRing];
    unsigned long long box_full, box_free;  // the halves' exchange
    unsigned long long drained;
    long long scratch[kThreads / 32 + 2];
    PagedSegment seg[kRing];
    float2 stats[128];  // (reference, sum) of the rows that one half leaves to the other
    uint32_t tmem;
    int abort;
    int progress;  // changes with every tile that a stage was free for and every step of the search for segments
    int joined;  // warps that have joined a segment's halves, over all segments
};
static_assert(Sizes<128>::kControl + sizeof(Control) <= 227 * 1024, "shared memory");

// Waits are bounded: a wait that gives up says so to all others of the CTA.  Those for a
// whole segment (kLong; it may have millions of tiles) count from the last progress.
template <bool kLong>
__device__ bool wait_slow(uint32_t bar, uint32_t parity, Control* ct, int* status) {
    unsigned long long t0 = global_timer_ns();
    volatile int* abort = &ct->abort;
    volatile int* progress = &ct->progress;
    int seen = kLong ? *progress : 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            if (kLong && *progress != seen) {
                seen = *progress;
                t0 = global_timer_ns();
                continue;
            }
            *abort = 1;
            record_status(status, USM_ERR_TIMEOUT);
            return false;
        }
    }
}
// By a whole warp, with one answer.
template <bool kLong = false>
__device__ __forceinline__ bool wait(const unsigned long long& b, uint32_t parity, Control* ct, int* status) {
    const uint32_t bar = smem_addr(&b);
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) ok = wait_slow<kLong>(bar, parity, ct, status);
    return __all_sync(kFullMask, ok);
}
__device__ __forceinline__ void arrive_warp(const unsigned long long& b) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&b));
}

// Loads of a segment of n tiles come in the order K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ uint32_t k_load(uint32_t base, int t) { return base + (t == 0 ? 0 : 2 * t - 1); }
__device__ __forceinline__ uint32_t v_load(uint32_t base, int t, int n) { return base + (t == n - 1 ? 2 * n - 1 : 2 * t + 2); }

// The keys that every row of the segment's block sees.
__device__ __forceinline__ void set_edges(const PagedArgs& a, PagedSegment& g) {
    const int2 first = paged_seen(a, g, 0), last = paged_seen(a, g, g.rows - 1);
    const bool none = first.y <= first.x || last.y <= last.x;
    g.hi_least = none ? 0 : first.y;
    g.lo_most = none ? 0x7fffffff : last.x;
}
// Whether some row does not see all of the tile's keys that lie in [lo, hi).
__device__ __forceinline__ bool partly_seen(const PagedSegment& g, int key0) {
    return min(key0 + kKeys, g.hi) > g.hi_least || max(key0, g.lo) < g.lo_most;
}
// Whether a tile's values need cleaning: that, or keys of it lie outside [lo, hi).
__device__ __forceinline__ bool needs_cleaning(const PagedSegment& g, int key0) {
    return partly_seen(g, key0) || key0 < g.lo || key0 + kKeys > g.hi;
}

__device__ __forceinline__ bool odd_bf16(uint32_t w) {  // an infinity or NaN in either half
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t nan_if_odd(uint32_t sum, uint32_t w) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0), "r"(sum));
    return r;
}
__device__ __forceinline__ uint32_t without_odd(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// ---------------------------------------------------------------------------
// Copies.  Pages that divide a tile, or that tiles divide, come by TMA, a box of a
// page's slots and 64 columns at a time: a warp for keys and one for values wait for
// room and start the boxes, two put right what boxes bring beyond the sequence,
// and two copy the queries.  Other page sizes (and those under 8) come in 16-byte
// copies by the first four; these complete on the tile's barrier by themselves too,
// and the thread that multiplies makes them visible to the tensor cores.
// (16-byte copies for all: 64 tokens over 8192 keys take 502 us, 263 with boxes; two
// chunks over 16384 keys 1365, 1000 with boxes.)
// ---------------------------------------------------------------------------
template <int DP>
struct Copies {
    using Z = Sizes<DP>;
    static constexpr int kChunks = DP / 8;      // 16-byte chunks of a row
    static constexpr int kSide = 32 / kChunks;  // rows of a warp's copy
    static constexpr int kPanels = DP / 64;

    const PagedArgs& a;
    Control* ct;
    uint32_t smem;
    int warp, lane, chunk, side;

    __device__ Copies(const PagedArgs& a, Control* ct, uint32_t smem) : a(a), ct(ct), smem(smem) {
        warp = (threadIdx.x >> 5) & 3;
        lane = threadIdx.x & 31;
        chunk = lane % kChunks;
        side = lane / kChunks;
    }
    __device__ __forceinline__ static uint32_t place(uint32_t tile, int row, int chunk) {
        return tile + (chunk >> 3) * 16384 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
    }

    // Rows row0.. (32 of them) of a tile; row: where the lane's one begins, null for zeros.
    __device__ __forceinline__ void rows(uint32_t tile, int row0, const char* row) {
        const bool used = chunk * 8 < (a.head_dim + 15) / 16 * 16;  // a column of the products
#pragma unroll 4
        for (int i = side; i < 32; i += kSide) {
            const unsigned long long from = __shfl_sync(kFullMask, (unsigned long long)row, i);
            const bool there = from != 0 && chunk * 8 < a.head_dim;
            if (used)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place(tile, row0 + i, chunk)),
                             "l"(there ? (const char*)from + chunk * 16 : (const char*)a.q), "r"(there ? 16 : 0)
                             : "memory");
        }
    }
    __device__ __forceinline__ void complete_on(const unsigned long long& b) {
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&b)) : "memory");
    }

    // Segment `it`'s queries may come: those before are no longer read, and, where
    // there is a second tile of them, no halves are being joined through it: all
    // `joins` segments before whose halves are have been.
    __device__ __forceinline__ bool room_for_queries(const PagedSegment& g, uint32_t it, int& joins) {
        const int before = joins;
        if (g.rows <= 128 && g.tiles > 1) ++joins;
        if (it == 0) return true;
        if (!wait<true>(ct->q_empty, (it - 1) & 1, ct, a.status)) return false;
        if (g.rows <= 128) return true;
        const unsigned long long t0 = global_timer_ns();
        bool ok = true;
        while (ok && *(volatile int*)&ct->joined < 4 * before) {
            if (*(volatile int*)&ct->abort) ok = false;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *(volatile int*)&ct->abort = 1;
                record_status(a.status, USM_ERR_TIMEOUT);
                ok = false;
            }
        }
        __threadfence_block();
        return __all_sync(kFullMask, ok);
    }

    // The segment's queries, by warps first, first + step, ...; rows past the last
    // group of 32 are left as they are (a row's results depend on nothing else).
    __device__ void queries(const PagedSegment& g, int first, int step) {
#pragma unroll 1
        for (int row0 = 32 * first; row0 < g.rows; row0 += 32 * step) {
            const int r = row0 + lane;
            const char* row = nullptr;
            if (r < g.rows) {
                const int flat = g.row0 + r, token = by_group(a, flat);
                row = (const char*)a.q + 2 * ((g.start + token) * a.q_token + (g.head * a.group + flat - token * a.group) * a.q_head);
            }
            rows(smem + (row0 >> 7) * Z::kTile, row0 & 127, row);
        }
        complete_on(ct->q_full);
    }

    // Values that must not reach the products: rows outside [lo, hi), which may hold
    // anything (a weight of 0 does not silence NaN), and infinities and NaN in keys
    // that not every row sees, which are added at the end where they are seen.
    // Rows begin..end-1 of a tile, by `threads` threads.
    __device__ __forceinline__ static void zero(uint32_t tile, int begin, int end, int thread, int threads) {
        const int chunk = thread % kChunks;
        for (int row = begin + thread / kChunks; row < end; row += threads / kChunks)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(place(tile, row, chunk)), "r"(0) : "memory");
    }
    __device__ __forceinline__ static void silence(uint32_t tile, int begin, int end, int thread, int threads, int* found) {
        const int chunk = thread % kChunks, step = threads / kChunks;
#pragma unroll 1
        for (int row = begin + thread / kChunks; row < end; row += 4 * step) {
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = row + u * step < end ? lds128(place(tile, row + u * step, chunk)) : make_uint4(0, 0, 0, 0);
            uint32_t sum = 0;  // x·0 + sum: NaN once some x is one or infinite
#pragma unroll
            for (int u = 0; u < 4; ++u) sum = nan_if_odd(nan_if_odd(nan_if_odd(nan_if_odd(sum, w[u].x), w[u].y), w[u].z), w[u].w);
            if ((sum & 0x7fff7fffu) == 0) continue;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (!(odd_bf16(w[u].x) || odd_bf16(w[u].y) || odd_bf16(w[u].z) || odd_bf16(w[u].w))) continue;
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(place(tile, row + u * step, chunk)), "r"(without_odd(w[u].x)),
                             "r"(without_odd(w[u].y)), "r"(without_odd(w[u].z)), "r"(without_odd(w[u].w))
                             : "memory");
                *(volatile int*)found = 1;
            }
        }
    }
    // Of the tile's rows first..first+count-1; lo, most, least, hi: the edges, from its first key.
    __device__ __noinline__ static void clean(uint32_t tile, int lo, int most, int least, int hi, int first, int count, int chunks,
                                              int thread, int threads, int* found) {
        if (thread % kChunks >= chunks) return;  // columns that no copy wrote
        const int end = first + count;
        lo = min(max(lo, first), end);
        hi = min(max(hi, lo), end);
        most = min(max(most, lo), hi);
        least = max(min(least, hi), most);
        zero(tile, first, lo, thread, threads);
        zero(tile, hi, end, thread, threads);
#pragma unroll 1
        for (int i = 0; i < 2; ++i) silence(tile, i ? least : lo, i ? hi : most, thread, threads, found);
    }
    __device__ __forceinline__ void clean(const PagedSegment& g, uint32_t stage, int key0, int first, int count, int thread, int threads) {
        clean(smem + Z::kStage0 + stage * Z::kTile, g.lo - key0, (int)min((long long)g.lo_most - key0, 1LL << 30), g.hi_least - key0, g.hi - key0,
              first, count, (a.head_dim + 7) / 8, thread, threads, const_cast<int*>(&g.odd_values));
        fence_proxy_async_smem();
    }

    // Load i of a segment's 2n: K0 K1 V0 K2 V1 ... V(n-1).
    __device__ __forceinline__ static int tile_of(int i, int n, bool& values) {
        values = i == 2 * n - 1 || (i > 0 && i % 2 == 0);
        return i == 2 * n - 1 ? n - 1 : values ? i / 2 - 1 : (i + 1) / 2;
    }

    // One warp for keys, one for values: boxes, all issued by one thread (threads of
    // a warp side by side take 100 cycles for each).  The pages of 32 entries of the
    // table are kept a lane each, and the next 32 behind them: a look-up takes
    // longer than a tile.
    // False where a wait gave up.
    __device__ bool boxes(const CUtensorMap* map, bool values) {
        const int slots = min(a.page_size, kKeys), per_tile = kKeys / slots;  // of a box; pages of a tile
        const int tiles_of_page = a.page_size / slots;
        const bool lead = elect_one();
        uint32_t base = 0;
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!wait<true>(ct->seg_full[slot], it / kRing & 1, ct, a.status)) return false;
            const PagedSegment& g = ct->seg[slot];
            if (!g.live) break;
            const int n = g.tiles, tile0 = g.tile0, lo = g.lo, hi = g.hi, head = g.head;
            const int* table = a.table + (long long)g.seq * a.table_stride;
            int group = -1, now = 0, next = 0;
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                const int tile = tile0 + t, first = tile * kKeys;
                const int entry = tiles_of_page == 1 ? tile * per_tile : tile / tiles_of_page;
                if (entry >> 5 != group) {
                    const int i = (entry & ~31) + lane;
                    now = entry >> 5 == group + 1 && group >= 0 ? next : i < a.table_pages ? table[i] : 0;
                    next = i + 32 < a.table_pages ? table[i + 32] : 0;
                    group = entry >> 5;
                    now = min(max(now, 0), a.num_pages - 1);
                }
                // Pages of the tile with keys in [lo, hi): begin..end-1.
                const int begin = first < lo ? (lo - first) / slots : 0;
                const int end = first + kKeys > hi ? (hi - first + slots - 1) / slots : per_tile;
                const int in_page = tiles_of_page == 1 ? 0 : first - entry * a.page_size;
                const uint32_t load = values ? v_load(base, t, n) : k_load(base, t);
                const uint32_t stage = load % Z::kStages;
                if (!wait(ct->empty[stage], (load / Z::kStages & 1) ^ 1, ct, a.status)) return false;
                const uint32_t bar = smem_addr(&ct->full[stage]), to = smem + Z::kStage0 + stage * Z::kTile;
                if (lead) *(volatile int*)&ct->progress = (int)load;
                if (lead) mbar_arrive_expect_tx(bar, max(end - begin, 0) * kPanels * slots * 128);
                loaded |= 1u << stage;
                phases = (phases & ~(1u << stage)) | ((load / Z::kStages & 1) << stage);
                for (int j = begin; j < end; j += 8) {
                    int page[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) page[u] = __shfl_sync(kFullMask, now, (entry + j + u) & 31);
                    if (lead)
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            if (j + u < end)
#pragma unroll
                                for (int panel = 0; panel < kPanels; ++panel)
                                    tma_load_4d(to + panel * 16384 + (j + u) * slots * 128, map, panel * 64, in_page, head, page[u], bar);
                }
                if (lead && values && needs_cleaning(g, first)) mbar_arrive(smem_addr(&ct->started[stage]));
                __syncwarp();
            }
            base += 2 * n;
            arrive_warp(ct->seg_empty[slot]);
        }
        return true;
    }
    uint32_t loaded = 0, phases = 0;  // a bit a stage: by this warp, and in which phase last
    // After a wait that gave up: the boxes have landed before the CTA ends, or had
    // long enough to.
    __device__ void landed() {
        for (int i = 0; i < Z::kStages; ++i)
            if (loaded >> i & 1) mbar_wait_bounded(smem_addr(&ct->full[i]), phases >> i & 1, kWaitLimitNs);
    }

    // Two further warps: the queries.
    __device__ void all_queries() {
        int joins = 0;
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!wait<true>(ct->seg_full[slot], it / kRing & 1, ct, a.status)) return;
            const PagedSegment& g = ct->seg[slot];
            if (!g.live || !room_for_queries(g, it, joins)) return;
            queries(g, warp & 1, 2);
            arrive_warp(ct->seg_empty[slot]);
        }
    }

    // And two: the cleaning.
    __device__ void all_cleaning() {
        uint32_t load = 0, startings = 0;  // startings: parity of each stage's
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!wait<true>(ct->seg_full[slot], it / kRing & 1, ct, a.status)) return;
            const PagedSegment& g = ct->seg[slot];
            if (!g.live) return;
            const int n = g.tiles;
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                const int key0 = (g.tile0 + t) * kKeys;
                if (!needs_cleaning(g, key0)) continue;
                const uint32_t i = v_load(load, t, n), stage = i % Z::kStages;
                // Its phase of `full` can be told from others only once it has begun.
                if (!wait<true>(ct->started[stage], startings >> stage & 1, ct, a.status)) return;
                startings ^= 1u << stage;
                if (!wait(ct->full[stage], i / Z::kStages & 1, ct, a.status)) return;
                clean(g, stage, key0, 0, kKeys, threadIdx.x & 63, 64);
                arrive_warp(ct->cleaned[stage]);
            }
            load += 2 * n;
            arrive_warp(ct->seg_empty[slot]);
        }
    }

    // Where this lane's row of load i begins; null outside [lo, hi).
    __device__ __forceinline__ const char* key_row(const PagedSegment& g, int i) const {
        bool values;
        const int key = (g.tile0 + tile_of(i, g.tiles, values)) * kKeys + 32 * warp + lane;
        if (key < g.lo || key >= g.hi) return nullptr;
        const int2 w = paged_slot(a, g.seq, key);
        return values ? (const char*)a.v + 2 * (w.x * a.v_page + w.y * a.v_slot + g.head * a.v_head)
                      : (const char*)a.k + 2 * (w.x * a.k_page + w.y * a.k_slot + g.head * a.k_head);
    }

    // All four warps: 16-byte copies.
    __device__ void chunks() {
        uint32_t stage = 0, parity = 1;
        int joins = 0;
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!wait<true>(ct->seg_full[slot], it / kRing & 1, ct, a.status)) return;
            const PagedSegment& g = ct->seg[slot];
            if (!g.live) break;
            const int n = g.tiles, key0 = g.tile0 * kKeys;
            if (!room_for_queries(g, it, joins)) return;
            queries(g, warp, 4);
            const char* next = key_row(g, 0);
#pragma unroll 1
            for (int i = 0; i < 2 * n; ++i) {
                bool values;
                const int at = key0 + tile_of(i, n, values) * kKeys;
                const char* row = next;
                next = i + 1 < 2 * n ? key_row(g, i + 1) : nullptr;  // its look-up runs behind this tile's copies
                if (!wait(ct->empty[stage], parity, ct, a.status)) return;
                if (lane == 0) *(volatile int*)&ct->progress = i;
                rows(smem + Z::kStage0 + stage * Z::kTile, 32 * warp, row);
                if (values && partly_seen(g, at)) {
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    __syncwarp();  // this warp's rows alone
                    clean(g, stage, at, 32 * warp, 32, lane, 32);
                    mbar_arrive(smem_addr(&ct->full[stage]));
                } else {
                    complete_on(ct->full[stage]);
                }
                if (++stage == Z::kStages) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            arrive_warp(ct->seg_empty[slot]);
        }
    }
};

// ---------------------------------------------------------------------------
// Matrix products, issued by one elected thread
// ---------------------------------------------------------------------------
template <int DP>
struct Products {
    using Z = Sizes<DP>;
    const PagedArgs& a;
    Control* ct;
    uint32_t smem, tmem;
    uint32_t qk_shape, pv_shape;
    int steps;
    uint32_t weighed = 0;    // parity of each half's weights
    uint32_t cleanings = 0;  // parity of each stage's
    int turn = 0;            // the half that takes the next tile of shared rows

    __device__ Products(const PagedArgs& a, Control* ct, uint32_t smem, uint32_t tmem) : a(a), ct(ct), smem(smem), tmem(tmem) {
        steps = (a.head_dim + 15) / 16;
        qk_shape = bf16_mma_shape(kKeys, false);
        pv_shape = bf16_mma_shape(steps * 16, true);
    }
    template <bool kLong = false>
    __device__ __forceinline__ bool await(const unsigned long long& b, uint32_t parity) {
        const uint32_t bar = smem_addr(&b);
        return mbar_try_wait(bar, parity) || wait_slow<kLong>(bar, parity, ct, a.status);
    }
    __device__ __forceinline__ void commit(const unsigned long long& b) { tmem_commit(smem_addr(&b)); }
    __device__ __forceinline__ bool loaded(uint32_t load) {
        if (!await(ct->full[load % Z::kStages], load / Z::kStages & 1)) return false;
        if (!a.boxes) fence_proxy_async_smem();  // the copies were ordinary writes
        return true;
    }
    __device__ __forceinline__ bool values_loaded(const PagedSegment& g, int t, uint32_t load) {
        if (!loaded(load)) return false;
        const int key0 = (g.tile0 + t) * kKeys, stage = load % Z::kStages;
        if (a.boxes && needs_cleaning(g, key0)) {
            if (!await(ct->cleaned[stage], cleanings >> stage & 1)) return false;
            cleanings ^= 1u << stage;
        }
        return true;
    }
    __device__ __forceinline__ uint32_t stage(uint32_t load) const { return smem + Z::kStage0 + load % Z::kStages * Z::kTile; }
    __device__ __forceinline__ void release(uint32_t load) { commit(ct->empty[load % Z::kStages]); }

    __device__ __forceinline__ void scores(int half, int q_half, uint32_t load) {
        const uint32_t q = swizzled_desc(smem + q_half * Z::kTile, 0), k = swizzled_desc(stage(load), 0);
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
            if (i >= steps) break;
            const uint32_t at = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
            mma_bf16_ss(tmem + half * kKeys, q + at, k + at, qk_shape, i > 0);
        }
        commit(ct->s_full[half]);
    }
    __device__ __forceinline__ bool weigh(int half, uint32_t load, bool accumulate) {
        if (!await(ct->p_full[half], weighed >> half & 1)) return false;
        weighed ^= 1u << half;
        tmem_fence_after_sync();
        const uint32_t v = swizzled_desc(stage(load), 16384);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)
                mma_bf16_ts(tmem + 256 + half * DP, tmem + half * kKeys + part * (kKeys / 2) + i * 8, v + (i * 2048 >> 4), pv_shape,
                            accumulate || part + i > 0);
        return true;
    }

    __device__ void run() {
        uint32_t base = 0;
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!await<true>(ct->seg_full[slot], it / kRing & 1)) return;
            const PagedSegment& g = ct->seg[slot];
            if (!g.live) break;
            const int n = g.tiles;
            const bool shared = g.rows <= 128;
            if (!await(ct->q_full, it & 1)) return;
            fence_proxy_async_smem();
            if (!loaded(k_load(base, 0))) return;
            scores(shared ? turn : 0, 0, k_load(base, 0));
            if (!shared) scores(1, 1, k_load(base, 0));
            release(k_load(base, 0));
            if (shared && n > 1) {
                if (!loaded(k_load(base, 1))) return;
                scores(turn ^ 1, 0, k_load(base, 1));
                release(k_load(base, 1));
            }
            const int ahead = shared ? 2 : 1;  // tiles whose scores are formed before the sums of tile t
            if (n <= ahead) commit(ct->q_empty);
            for (int t = 0; t < n; ++t) {
                const uint32_t v = v_load(base, t, n), k = k_load(base, t + ahead);
                const bool more = t + ahead < n;
                if (!values_loaded(g, t, v) || (more && !loaded(k))) return;
                if (shared) {
                    const int half = (t & 1) ^ turn;
                    if (!weigh(half, v, t >= 2)) return;
                    release(v);
                    if (more) scores(half, 0, k);
                    else commit(ct->o_full[half]);
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!weigh(half, v, t > 0)) return;
                        if (more) scores(half, half, k);
                        else commit(ct->o_full[half]);
                    }
                    release(v);
                }
                if (more) release(k);
                if (more && t + ahead == n - 1) commit(ct->q_empty);
            }
            base += 2 * n;
            if (shared) turn ^= n & 1;
            mbar_arrive(smem_addr(&ct->seg_empty[slot]));
        }
    }
};

// ---------------------------------------------------------------------------
// Softmax and output: one row a thread
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store16(void* p, const uint32_t* w) {  // 16 bytes
    asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

__device__ __forceinline__ void store32(void* p, const uint32_t* w) {  // 32 bytes, aligned to them
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <int DP>
struct Softmax {
    using Z = Sizes<DP>;
    const PagedArgs& a;
    Control* ct;
    uint32_t smem;
    int half, tid;           // thread of the half
    uint32_t s_col, o_col;   // this warp's lanes of tensor memory
    // Parities of this half's waits for scores and for sums and of the halves'
    // exchange, whether there was one yet, and the half that takes the next tile of
    // shared rows.
    uint32_t state = 0;
    static constexpr uint32_t kScores = 1, kSums = 2, kBox = 4, kBoxUsed = 8, kTurn = 16, kFailed = 32;
    __device__ __forceinline__ uint32_t flip(uint32_t bit) {  // its old value
        state ^= bit;
        return (state & bit) ? 0 : 1;
    }
    // Of the current segment:
    float m, l;      // reference (a score) and sum of the weights
    float mc;        // what an exponent subtracts
    bool far;        // some row of the warp is far from zero

    __device__ Softmax(const PagedArgs& a, Control* ct, uint32_t smem, uint32_t tmem) : a(a), ct(ct), smem(smem) {
        half = threadIdx.x >> 7;
        tid = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(tid & ~31) << 16;
        s_col = tmem + lanes + half * kKeys;
        o_col = tmem + lanes + 256 + half * DP;
    }

    // Row of the segment's block that this thread has.
    __device__ __forceinline__ int row_of(const PagedSegment& g) const { return g.rows <= 128 ? tid : half * 128 + tid; }

    // Tile t0's scores into weights.  `first`: O holds nothing yet.
    __device__ __forceinline__ void weights(const PagedSegment& g, int t0, bool masked, bool first) {
        uint32_t w[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_col + 32 * i, w[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_wait_ld(w[i]);
        const float c = a.scale_log2;
        if (masked) {
            const int2 seen = paged_seen(a, g, row_of(g));
            const unsigned from = (unsigned)(seen.x - (g.tile0 + t0) * kKeys), count = (unsigned)(seen.y - seen.x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if ((unsigned)(32 * i + j) - from >= count) w[i][j] = 0xff800000u;
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            top[i] = max3(__uint_as_float(w[i][0]), __uint_as_float(w[i][1]), __uint_as_float(w[i][2]));
#pragma unroll
            for (int j = 3; j < 31; j += 2) top[i] = max3(top[i], __uint_as_float(w[i][j]), __uint_as_float(w[i][j + 1]));
            top[i] = fmaxf(top[i], __uint_as_float(w[i][31]));
        }
        const float t = max3(fmaxf(top[0], top[1]), top[2], top[3]);
        const bool raise = (t - m) * c > kRaise;
        if (__any_sync(kFullMask, raise)) {
            const float to = raise ? t : m;
            const float f = raise ? exp2_fast((m - to) * c) : 1.f;
            m = to;
            l *= f;
            mc = m == -INFINITY ? 0.f : m * c;
            far = __any_sync(kFullMask, !(fabsf(mc) <= kNear));
            if (far) mc = 0.f;
            if (!first) rescale(f);
        }
        if (far) {  // the difference is formed first: it is exact near m
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 32; ++j) w[i][j] = __float_as_uint(__uint_as_float(w[i][j]) - base);
        }
        uint64_t sum[2] = {0, 0};
        const uint64_t c2 = pack2(c, c), mc2 = pack2(-mc, -mc), minus = pack2(-1.f, -1.f);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t p[16], rest[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(w[h][2 * j]), __uint_as_float(w[h][2 * j + 1])), c2, mc2), x, y);
                x = exp2_fast(x);
                y = exp2_fast(y);
                const uint64_t xy = pack2(x, y);
                sum[j & 1] = add2(sum[j & 1], xy);
                p[j] = bf16x2(x, y);
                unpack2(fma2(pack2(__uint_as_float(p[j] << 16), __uint_as_float(p[j] & 0xffff0000u)), minus, xy), x, y);
                rest[j] = bf16x2(x, y);  // of an exact difference
            }
            tmem_st16(s_col + 16 * h, p);
            tmem_st16(s_col + kKeys / 2 + 16 * h, rest);
        }
        float x0, x1, y0, y1;
        unpack2(sum[0], x0, x1);
        unpack2(sum[1], y0, y1);
        l += (x0 + x1) + (y0 + y1);
        tmem_wait_st();
    }

    __device__ __forceinline__ void rescale(float f) {
        const int columns = (a.head_dim + 15) / 16 * 16;
#pragma unroll 1
        for (int j = 0; j < columns; j += 16) {
            uint32_t w[16];
            tmem_ld16(o_col + j, w);
            tmem_wait_ld(w);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
            tmem_st16(o_col + j, w);
        }
        tmem_wait_st();
    }

    // Adds what was taken out of partly masked tiles: infinities and NaN of rows
    // of V that this row sees.  Whole warp; the half's tiles are first, first + step, ...
    __device__ __noinline__ static void add_odd(const PagedArgs& a, const PagedSegment& g, uint32_t o_col, int2 seen, int first,
                                                int step) {
#pragma unroll 1
        for (int j = 0; j < a.head_dim; j += 16) {
            uint32_t w[16];
            tmem_ld16(o_col + j, w);
            tmem_wait_ld(w);
#pragma unroll 1
            for (int t = first; t < g.tiles; t += step) {
                const int key0 = (g.tile0 + t) * kKeys;
                if (!partly_seen(g, key0)) continue;
#pragma unroll 1
                for (int key = max(key0, seen.x); key < min(key0 + kKeys, seen.y); ++key) {
                    if (key >= g.lo_most && key < g.hi_least) key = min(key0 + kKeys, g.hi_least);  // seen by all: left in place
                    if (key >= min(key0 + kKeys, seen.y)) break;
                    const int2 at = paged_slot(a, g.seq, key);
                    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + at.x * a.v_page + at.y * a.v_slot + g.head * a.v_head + j;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = j + i < a.head_dim ? __bfloat162float(v[i]) : 0.f;
                        if (!isfinite(x)) w[i] = __float_as_uint(__uint_as_float(w[i]) + x);
                    }
                }
            }
            __syncwarp();
            tmem_st16(o_col + j, w);
        }
        tmem_wait_st();
    }

    // A row's sums, 32 columns at a time: divided, and written to the output or to
    // the partial results.  Where the halves took the same rows (`both`) the one that
    // had the last tile (`last`) first adds the other's, which come through the
    // queries' second tile (free then): [row][columns], as many columns at a time as
    // there is room for, 16-byte chunks swizzled by the row.
    // Returns the new state, kFailed where a wait gave up.
    __device__ __forceinline__ static uint32_t write(const PagedArgs& a, Control* ct, const PagedSegment& g, uint32_t smem, uint32_t o_col, int row,
                                                  float m, float l, bool both, bool last, uint32_t state) {
        const int tid = threadIdx.x & 127;
        const bool mine = row < g.rows, whole = g.part == kPartWhole;
        const bool some = __any_sync(kFullMask, mine);
        const int lanes = (min(g.rows, 128) + 31) / 32 * 32, wide = max(Z::kTile / 4 / lanes / 32, 1) * 32;
        const uint32_t box = smem + Z::kTile + tid * wide * 4;
        const int flat = g.row0 + row, token = by_group(a, flat);
        const long long part = (2LL * blockIdx.x + g.part) * a.part_rows + row;
        char* to = whole ? static_cast<char*>(a.out) + 2 * ((g.start + token) * a.out_token + (g.head * a.group + flat - token * a.group) * a.out_head)
                         : reinterpret_cast<char*>(a.parts + (part - row) * a.head_dim + row * 4);
        float f0 = 1.f, f1 = 0.f;
#pragma unroll 1
        for (int j = 0; j < a.head_dim; j += 32) {
            uint32_t w[32];
            if (some) {
                tmem_ld32(o_col + j, w);
                tmem_wait_ld(w);
            }
            const uint32_t at = box + (uint32_t)(j % wide) * 4;
            const bool begins = j % wide == 0, ends = (j + 32) % wide == 0 || j + 32 >= a.head_dim;
            if (both && !last) {
                if (begins && (state & kBoxUsed) && !wait(ct->box_free, (state & kBox) ? 0 : 1, ct, a.status)) return kFailed;
                if (j == 0) ct->stats[tid] = make_float2(m, l);
                if (some)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + ((i ^ (tid & 7)) << 4)), "r"(w[4 * i]),
                                     "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                                     : "memory");
                if (ends) {
                    arrive_warp(ct->box_full);
                    state = (state ^ kBox) | kBoxUsed;
                }
                continue;
            }
            if (both && begins && !wait(ct->box_full, (state & kBox) ? 1 : 0, ct, a.status)) return kFailed;
            if (j == 0) {
                if (both) {
                    const float2 other = ct->stats[tid];
                    const float t = fmaxf(m, other.x);
                    f0 = m == -INFINITY ? 0.f : exp2_fast((m - t) * a.scale_log2);
                    f1 = other.x == -INFINITY ? 0.f : exp2_fast((other.x - t) * a.scale_log2);
                    m = t;
                    l = l * f0 + other.y * f1;
                }
                const float z = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
                f0 *= z;
                f1 *= z;
            }
            if (some) {
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f0);
                if (both)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 y = lds128(at + ((i ^ (tid & 7)) << 4));
                        w[4 * i] = __float_as_uint(fmaf(__uint_as_float(y.x), f1, __uint_as_float(w[4 * i])));
                        w[4 * i + 1] = __float_as_uint(fmaf(__uint_as_float(y.y), f1, __uint_as_float(w[4 * i + 1])));
                        w[4 * i + 2] = __float_as_uint(fmaf(__uint_as_float(y.z), f1, __uint_as_float(w[4 * i + 2])));
                        w[4 * i + 3] = __float_as_uint(fmaf(__uint_as_float(y.w), f1, __uint_as_float(w[4 * i + 3])));
                    }
            }
            if (both && ends) {
                arrive_warp(ct->box_free);
                state = (state ^ kBox) | kBoxUsed;
                if (j + 32 >= a.head_dim && (threadIdx.x & 31) == 0) {  // this warp has read all of the other half's
                    __threadfence_block();
                    atomicAdd(&ct->joined, 1);
                }
            }
            if (!mine) continue;
            const int left = a.head_dim - j;  // a multiple of 8
            if (whole && a.out32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t p[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        p[u] = bf16x2(__uint_as_float(w[16 * i + 2 * u]), __uint_as_float(w[16 * i + 2 * u + 1]));
                    if (16 * i < left) store32(to + 2 * j + 32 * i, p);
                }
            } else if (whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t p[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        p[u] = bf16x2(__uint_as_float(w[8 * i + 2 * u]), __uint_as_float(w[8 * i + 2 * u + 1]));
                    if (8 * i < left) store16(to + 2 * j + 16 * i, p);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (4 * i < left) store16(to + (long long)(j / 4 + i) * a.part_rows * 16, w + 4 * i);
            }
        }
        if (!whole && mine && (!both || last)) *reinterpret_cast<float2*>(a.part_stats + 2 * part) = make_float2(m, l);
        return state;
    }

    __device__ void run() {
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!wait<true>(ct->seg_full[slot], it / kRing & 1, ct, a.status)) return;
            const PagedSegment& g = ct->seg[slot];
            if (!g.live) break;
            const bool some = __any_sync(kFullMask, row_of(g) < g.rows);
            // Tiles that every row of this warp sees whole: whole.x <= t < whole.y.
            int2 whole;
            {
                const int row = row_of(g);
                const int2 seen = paged_seen(a, g, row);
                int lo = row < g.rows ? seen.x : 0, hi = row < g.rows ? seen.y : 0x7fffffff;
                if (row < g.rows && seen.x >= seen.y) hi = 0;
                lo = __reduce_max_sync(kFullMask, lo);
                hi = __reduce_min_sync(kFullMask, hi);
                whole = make_int2((lo + kKeys - 1) / kKeys - g.tile0, hi / kKeys - g.tile0);
            }
            m = -INFINITY;
            l = mc = 0.f;
            far = false;
            const int first = g.rows <= 128 ? half ^ (state & kTurn ? 1 : 0) : 0, tiles = g.tiles;
#pragma unroll 1
            for (int t = first; t < tiles; t += g.rows <= 128 ? 2 : 1) {
                if (!wait(ct->s_full[half], flip(kScores), ct, a.status)) return;
                tmem_fence_after_sync();
                if (some) weights(g, t, t < whole.x || t >= whole.y, t == first);
                tmem_fence_before_sync();
                arrive_warp(ct->p_full[half]);
            }
            if (first < tiles) {  // not so for one half of a single tile
                if (!wait(ct->o_full[half], flip(kSums), ct, a.status)) return;
                tmem_fence_after_sync();
                const bool shared = g.rows <= 128;
                if (some && *(volatile int*)&ct->seg[slot].odd_values)
                    add_odd(a, g, o_col, paged_seen(a, g, row_of(g)), first, shared ? 2 : 1);
                state = write(a, ct, g, smem, o_col, row_of(g), m, l, shared && tiles > 1, !shared || ((tiles - 1 - first) & 1) == 0, state);
                if (state & kFailed) return;
            }
            if (g.rows <= 128 && (tiles & 1)) state ^= kTurn;
            tmem_fence_before_sync();
            arrive_warp(ct->seg_empty[slot]);
        }
    }
};

struct Maps {
    CUtensorMap k, v;  // columns, slots, heads, pages
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) paged_mma_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ Maps maps) {
    using Z = Sizes<DP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Control* ct = reinterpret_cast<Control*>(smem + Z::kControl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Z::kStages; ++i) {
            mbar_init(smem_addr(&ct->full[i]), a.boxes ? 1 : 128);
            mbar_init(smem_addr(&ct->empty[i]), 1);
            mbar_init(smem_addr(&ct->started[i]), 1);
            mbar_init(smem_addr(&ct->cleaned[i]), 2);
        }
        mbar_init(smem_addr(&ct->q_full), a.boxes ? 64 : 128);
        mbar_init(smem_addr(&ct->q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ct->s_full[i]), 1);
            mbar_init(smem_addr(&ct->p_full[i]), 4);
            mbar_init(smem_addr(&ct->o_full[i]), 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_addr(&ct->seg_full[i]), 1);
            mbar_init(smem_addr(&ct->seg_empty[i]), kConsumers + (a.boxes ? 2 : 0));
        }
        mbar_init(smem_addr(&ct->box_full), 4);
        mbar_init(smem_addr(&ct->box_free), 4);
        mbar_init(smem_addr(&ct->drained), 1);
        ct->abort = ct->joined = ct->progress = 0;
        fence_barrier_init();
    }
    if (warp == 12) tmem_alloc(smem_addr(&ct->tmem), 512);
    await_previous();  // nothing of the caller's is read or written before
    let_next_start();
    Shares shares;
    if (a.num_seqs > Shares::kSolo) shares.init(a, blockIdx.x, gridDim.x, ct->scratch);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = *(volatile uint32_t*)&ct->tmem, base = smem_addr(smem);

    // 200 + 200 + 56 + 56 registers: the 4 x 128 that the launch has.
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        Softmax<DP>(a, ct, base, tmem).run();
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        Copies<DP> copies(a, ct, base);
        if (!a.boxes) {
            copies.chunks();
        } else if (warp < 10) {
            if (!copies.boxes(warp == 8 ? &maps.k : &maps.v, warp == 9)) copies.landed();
        } else {
            copies.all_cleaning();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 12) {
            if (elect_one()) {
                Products<DP>(a, ct, base, tmem).run();
                // Whatever was issued is done before tensor memory is given back.
                tmem_commit(smem_addr(&ct->drained));
            }
            __syncwarp();
            mbar_wait_bounded(smem_addr(&ct->drained), 0, kWaitLimitNs);
        } else if (warp == 13) {
            PagedMeta meta = {};
            if (a.num_seqs <= Shares::kSolo) shares.init_solo(a, blockIdx.x, gridDim.x);
            for (uint32_t it = 0;; ++it) {
                const int slot = it % kRing;
                PagedSegment g = shares.next(a, &ct->progress);
                if (g.live) {
                    paged_note(meta, g);
                    set_edges(a, g);
                }
                if (it >= kRing && !wait<true>(ct->seg_empty[slot], (it / kRing - 1) & 1, ct, a.status)) break;
                if (lane == 0) ct->seg[slot] = g;
                arrive_warp(ct->seg_full[slot]);
                if (!g.live) break;
            }
            if (lane == 0) static_cast<PagedMeta*>(a.meta)[blockIdx.x] = meta;
        } else if (a.boxes) {
            Copies<DP>(a, ct, base).all_queries();
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    }
    __syncthreads();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int DP>
int run(const PagedArgs& a, const Maps& maps, int ctas, cudaStream_t stream) {
    const auto kernel = paged_mma_kernel<DP>;
    constexpr int smem = Sizes<DP>::kControl + (int)sizeof(Control);
    static SharedOnce once;
    if (!once.allow(kernel, smem)) return cuda_failure();
    return launch_next_shared(kernel, dim3(ctas), kThreads, smem, stream, a, maps);
}

bool encode(CUtensorMap* map, const PagedArgs& a, const void* base, long long page, long long slot, long long head) {
    const int dims[4] = {a.head_dim, a.page_size, a.kv_heads, a.num_pages};
    const long long strides[3] = {slot, head, page};
    const int box[4] = {64, std::min(a.page_size, kKeys), 1, 1};
    return encode_tensor_map_4d_bf16(map, base, dims, strides, box);
}

}  // namespace

int paged_mma_rows() { return kRows; }
int launch_paged_mma(PagedArgs a, int ctas, cudaStream_t stream) {
    Maps maps = {};
    // Boxes of a page's slots: from 8 slots on (a tile is then 32 boxes at most),
    // where pages and tiles fit one another.
    a.boxes = a.page_size >= 8 && (kKeys % a.page_size == 0 || a.page_size % kKeys == 0) &&
              encode(&maps.k, a, a.k, a.k_page, a.k_slot, a.k_head) && encode(&maps.v, a, a.v, a.v_page, a.v_slot, a.v_head);
    a.out32 = a.head_dim % 16 == 0 && ((reinterpret_cast<uintptr_t>(a.out) | (2 * a.out_token) | (2 * a.out_head)) & 31) == 0;
    return a.head_dim <= 64 ? run<64>(a, maps, ctas, stream) : run<128>(a, maps, ctas, stream);
}

}  // namespace usm
