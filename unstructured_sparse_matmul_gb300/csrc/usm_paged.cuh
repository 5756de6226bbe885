// What the kernels over a paged cache share: sequences and positions, and the
// division of attention's work among CTAs.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "usm_args.h"
#include "usm_device.cuh"

namespace usm {

// What a call reads may be written by the kernel before it, which need not have
// ended when this one starts (await_previous() waits for its results): such arrays
// are read by ordinary loads, never through the path for data that nobody writes
// while a kernel lives.

// The new tokens of one sequence.
struct PagedSeq {
    int start;  // its first new token in the calls' arrays
    int n;      // how many
    int len;    // tokens in its cache, the new ones included (>= 0)
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
    PagedSeq s;
    if (a.q_offsets) {
        s.start = min(max(a.q_offsets[b], 0), a.tokens);
        s.n = min(max(a.q_offsets[b + 1], s.start), a.tokens) - s.start;
    } else {
        s.start = b * a.per_seq;
        s.n = a.per_seq;
    }
    const int rows = s.n * a.group;
    if (rows < a.least_rows || rows > a.most_rows) s.n = 0;  // another launch's
    s.len = min(max(a.lengths[b], 0), kPagedMaxLength);
    return s;
}

// x / group, for 0 <= x < 2^31.
__device__ __forceinline__ int by_group(const PagedArgs& a, int x) {
    return (int)((unsigned long long)x * a.group_mul >> a.group_shift);
}

// Rows of attention: new token i of a sequence gives `group` rows for a head of
// keys, i·group + g, one for each query head that reads it.  A block is kRows of
// a sequence's rows; an item is a block with one head of keys; a unit is one tile
// of kKeys keys of an item.
struct PagedBlock {
    int lo, hi;  // keys that some row sees lie in [lo, hi)
    int tile0, tiles;
};

// (A call, by value: in line, in the half dozen places that need it, it is code
// that every launch fetches for the first time.)
template <int kRows, int kKeys>
__device__ __noinline__ PagedBlock paged_block_call(uint32_t group_mul, int group_shift, int causal, int window, int keys, int rows,
                                                    int position, int block) {
    const int first = block * kRows, last = first + min(rows - first, kRows) - 1;
    const int p0 = position + (int)((unsigned long long)first * group_mul >> group_shift);
    const int p1 = position + (int)((unsigned long long)last * group_mul >> group_shift);
    PagedBlock k;
    k.hi = causal ? min(keys, max(p1 + 1, 0)) : keys;
    k.lo = window > 0 && p0 >= window ? p0 - window + 1 : 0;
    if (k.lo >= k.hi) k.lo = k.hi = 0;
    k.tile0 = k.lo / kKeys;
    k.tiles = max((k.hi + kKeys - 1) / kKeys - k.tile0, 1);  // one for a block that sees nothing: it writes zeros
    return k;
}
template <int kRows, int kKeys>
__device__ __forceinline__ PagedBlock paged_block(const PagedArgs& a, const PagedSeq& s, int block) {
    return paged_block_call<kRows, kKeys>(a.group_mul, a.group_shift, a.causal, a.window, min(s.len, a.capacity), s.n * a.group,
                                          s.len - s.n, block);
}

// A CTA's run of tiles of one item.
struct PagedSegment {
    int start, n, len;     // the sequence
    int row0, rows;        // its rows of the block
    int head;              // head of keys
    int seq;
    int lo, hi;            // keys that some row sees
    int tile0, tiles;      // this segment's tiles
    int part;              // kPartWhole, or the slot its partial result goes to
    int ends;              // its last tile is its item's
    int live;              // 0: no further segment
    int odd_values;        // set where a partly masked tile holds infinities or NaN in V
    int hi_least, lo_most; // every row sees the keys in [lo_most, hi_least)
};
constexpr int kPartWhole = -1, kPartLater = 0, kPartFirst = 1;

// What a CTA tells the joining kernel: an item begun in slot kPartFirst goes on
// in the next CTAs' slots kPartLater up to the one with `ends`.
struct alignas(16) PagedMeta {  // read in a piece of 16 bytes and one of 8
    int first_live;        // slot kPartFirst is in use, for this block and head:
    int start, row0, rows;
    int later_live, ends;  // slot kPartLater is in use, and ends its item
    int head, pad;
};

// The CTAs take equal shares of all units in the order (sequence, block, head,
// tile); an item counts kCost units more than it has tiles, before its first.
// init() is called by all kThreads threads, next() by one whole warp.
template <int kRows, int kKeys, int kThreads, int kCost>
struct PagedShares {
    long long left;  // units that remain to this CTA
    int b, block, blocks, head, unit;  // the next one, of its item
    PagedSeq s;
    PagedBlock k;

    __device__ __forceinline__ static int blocks_of(const PagedArgs& a, const PagedSeq& s) {
        return (int)(((unsigned)s.n * (unsigned)a.group + kRows - 1) / kRows);  // below 2^31 rows
    }
    __device__ __forceinline__ static bool many(int blocks) { return blocks > 4; }

    // Units of sequence b (0 past the last), for the calling lane; the whole warp
    // takes part where a sequence has many blocks.
    __device__ __forceinline__ static long long units_of(const PagedArgs& a, int b) {
        PagedSeq s{0, 0, 0};
        if (b < a.num_seqs) s = paged_seq(a, b);
        const int blocks = blocks_of(a, s);
        long long t = 0;
        if (!many(blocks))
#pragma unroll 1
            for (int i = 0; i < blocks; ++i) t += paged_block<kRows, kKeys>(a, s, i).tiles + kCost;
        unsigned rest = __ballot_sync(kFullMask, many(blocks));
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        while (rest) {
            const int from = __ffs(rest) - 1;
            rest &= rest - 1;
            PagedSeq f;
            f.start = 0;
            f.n = __shfl_sync(kFullMask, s.n, from);
            f.len = __shfl_sync(kFullMask, s.len, from);
            const int nb = __shfl_sync(kFullMask, blocks, from);
            long long sum = 0;
#pragma unroll 1
            for (int i = lane; i < nb; i += 32) sum += paged_block<kRows, kKeys>(a, f, i).tiles + kCost;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
            if (lane == from) t = sum;
        }
        return t * a.kv_heads;
    }

    // 64-bit divisions take hundreds of cycles; few need one.
    __device__ __forceinline__ static long long divide(long long x, int y) {
        return x >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
    }

    __device__ static long long warp_scan(long long x) {  // inclusive
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFullMask, x, o);
            if (lane >= o) x += y;
        }
        return x;
    }

    // This CTA's share of `sum` units: its first, and how many (`left`).  False for none.
    __device__ __forceinline__ bool share_of(long long sum, int cta, int ctas, long long& u0) {
        const int active = (int)min((long long)ctas, sum);
        if (cta >= active) return false;
        const long long each = divide(sum, active);
        const int over = (int)(sum - each * active);  // this many CTAs take one more
        u0 = each * cta + min(cta, over);
        left = each + (cta < over ? 1 : 0);
        return true;
    }

    // By one warp, for up to kSolo sequences.
    static constexpr int kSolo = 128;
    __device__ __forceinline__ void init_solo(const PagedArgs& a, int cta, int ctas) {
        long long u0 = 0, sum = 0;
        left = 0;
        b = a.num_seqs;
        block = blocks = head = unit = 0;
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (int search = 0; search < 2; ++search) {
            sum = 0;
#pragma unroll 1
            for (int at = 0; at < a.num_seqs; at += 32) {
                const long long mine = units_of(a, at + lane), scan = sum + warp_scan(mine);
                const unsigned here = __ballot_sync(kFullMask, u0 < scan);
                if (search && here) {
                    const int from = __ffs(here) - 1;
                    b = at + from;
                    find(a, u0 - __shfl_sync(kFullMask, scan - mine, from));
                    return;
                }
                sum = __shfl_sync(kFullMask, scan, 31);
                if (a.num_seqs <= 32 && share_of(sum, cta, ctas, u0)) {  // found in one go
                    const int from = __ffs(__ballot_sync(kFullMask, u0 < scan)) - 1;
                    b = from;
                    find(a, u0 - __shfl_sync(kFullMask, scan - mine, from));
                    return;
                }
            }
            if (search) left = 0;  // not found: the counts changed under the call
            if (search || !share_of(sum, cta, ctas, u0)) return;
        }
    }

    // By all threads, for any number.  scratch: shared, kThreads / 32 + 2 values.
    // Every warp knows the first segment afterwards.
    __device__ __forceinline__ void init(const PagedArgs& a, int cta, int ctas, long long* scratch) {
        constexpr int kWarps = kThreads / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        long long mine = 0, before = 0, u0 = 0;
        if (threadIdx.x == 0) scratch[kWarps] = -1;  // not found: the counts changed under the call
        left = 0;
        b = a.num_seqs;
        block = blocks = head = unit = 0;
        // First the sum over all sequences, then the search for this CTA's share;
        // with up to kThreads sequences every thread still has its own prefix then.
#pragma unroll 1
        for (int search = 0; search < 2; ++search) {
            long long sum = 0;
#pragma unroll 1
            for (int at = 0; at < a.num_seqs; at += kThreads) {
                if (!search || a.num_seqs > kThreads) {
                    mine = units_of(a, at + (int)threadIdx.x);
                    const long long scan = warp_scan(mine);
                    if (lane == 31) scratch[warp] = scan;
                    __syncthreads();
                    // A warp's lanes add up the warps' sums, all and those before it.
                    const long long w = warp_scan(lane < kWarps ? scratch[lane] : 0);
                    before = sum + scan - mine + (warp ? __shfl_sync(kFullMask, w, warp - 1) : 0);
                    sum += __shfl_sync(kFullMask, w, 31);
                    __syncthreads();
                }
                if (search && u0 >= before && u0 < before + mine) {
                    scratch[kWarps] = at + (int)threadIdx.x;
                    scratch[kWarps + 1] = u0 - before;
                }
            }
            if (!search && !share_of(sum, cta, ctas, u0)) return;
        }
        __syncthreads();
        b = (int)scratch[kWarps];
        if (b < 0) left = 0;
        else find(a, scratch[kWarps + 1]);
    }

    // The block, head and tile `skip` units behind sequence b's first; every warp
    // searches for itself.  (Held to what there is, should lengths change under the
    // call: the walk ends whatever it reads.)
    __device__ __forceinline__ void find(const PagedArgs& a, long long skip) {
        s = paged_seq(a, b);
        blocks = blocks_of(a, s);
        const int lane = threadIdx.x & 31;
        long long base = 0;
#pragma unroll 1
        for (int at = 0; at < blocks && blocks > 1; at += 32) {
            const long long w =
                at + lane < blocks ? (long long)(paged_block<kRows, kKeys>(a, s, at + lane).tiles + kCost) * a.kv_heads : 0;
            const long long scan = base + warp_scan(w);
            const unsigned here = __ballot_sync(kFullMask, skip < scan);
            if (here) {
                const int from = __ffs(here) - 1;
                block = at + from;
                skip -= __shfl_sync(kFullMask, scan - w, from);
                break;
            }
            base = __shfl_sync(kFullMask, scan, 31);
        }
        k = paged_block<kRows, kKeys>(a, s, block);
        head = (int)min(divide(skip, k.tiles + kCost), (long long)a.kv_heads - 1);
        unit = (int)min(skip - (long long)head * (k.tiles + kCost), (long long)k.tiles + kCost);
    }

    // On to the next item; whole warp.  beat (may be null): changed with every step.
    __device__ __forceinline__ void advance(const PagedArgs& a, volatile int* beat) {
        unit = 0;
        if (++head < a.kv_heads) return;
        head = 0;
        if (++block == blocks) {
            block = 0;
            const int lane = threadIdx.x & 31;
#pragma unroll 1
            for (++b; b < a.num_seqs; b += 32) {  // past sequences that bring no token
                if (beat) *beat = -b;
                const int n = b + lane < a.num_seqs ? paged_seq(a, b + lane).n : 0;
                const unsigned some = __ballot_sync(kFullMask, n > 0);
                if (some) {
                    b += __ffs(some) - 1;
                    break;
                }
            }
            if (b >= a.num_seqs) {  // the counts changed under the call
                left = 0;
                return;
            }
            s = paged_seq(a, b);
            blocks = blocks_of(a, s);
        }
        k = paged_block<kRows, kKeys>(a, s, block);
    }

    // The next segment; whole warp.
    __device__ __forceinline__ PagedSegment next(const PagedArgs& a, volatile int* beat = nullptr) {
        PagedSegment g;
        g.live = 0;
        g.odd_values = 0;
        while (left > 0) {
            if (unit == k.tiles + kCost) {
                advance(a, beat);
                if (left == 0) break;
            }
            const int take = (int)min((long long)(k.tiles + kCost - unit), left);
            const int begin = max(unit - kCost, 0), end = unit + take - kCost;
            left -= take;
            unit += take;
            if (end <= begin) continue;  // a share that ends before the item's first tile
            g.live = 1;
            g.start = s.start;
            g.n = s.n;
            g.len = s.len;
            g.row0 = block * kRows;
            g.rows = min(kRows, s.n * a.group - g.row0);
            g.head = head;
            g.seq = b;
            g.lo = k.lo;
            g.hi = k.hi;
            g.tile0 = k.tile0 + begin;
            g.tiles = end - begin;
            g.ends = end == k.tiles;
            g.part = begin > 0 ? kPartLater : g.ends ? kPartWhole : kPartFirst;
            break;
        }
        return g;
    }
};

// Keys [lo, hi) that one row of a segment sees; empty for rows past its last.
__device__ __forceinline__ int2 paged_seen(const PagedArgs& a, const PagedSegment& g, int row) {
    if (row >= g.rows) return make_int2(0, 0);
    const int p = g.len - g.n + by_group(a, g.row0 + row);
    const int keys = min(g.len, a.capacity);
    const int hi = a.causal ? min(keys, max(p + 1, 0)) : keys;
    const int lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
    return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}

static_assert(offsetof(PagedMeta, later_live) == 16 && sizeof(PagedMeta) == 32, "read as int4 and int2");

// Notes a segment with a partial result in the CTA's message to the join.
__device__ __forceinline__ void paged_note(PagedMeta& m, const PagedSegment& g) {
    if (g.part == kPartFirst) {
        m.first_live = 1;
        m.start = g.start;
        m.row0 = g.row0;
        m.rows = g.rows;
        m.head = g.head;
    } else if (g.part == kPartLater) {
        m.later_live = 1;
        m.ends = g.ends;
    }
}

// Page and slot of a key.
__device__ __forceinline__ int2 paged_slot(const PagedArgs& a, int seq, int key) {
    const int index = key / a.page_size;
    const int page = a.table[(long long)seq * a.table_stride + index];
    return make_int2(min(max(page, 0), a.num_pages - 1), key - index * a.page_size);
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace usm
