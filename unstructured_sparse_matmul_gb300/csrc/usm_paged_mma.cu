// Attention of new tokens over a paged bf16 cache on the tensor cores (heads of
// up to 128 columns).  Contract and masks: include/usm.h; how the work is
// divided: usm_paged.cuh.
//
// One CTA an SM walks over its share of tiles of 128 keys.  A block has up to
// 256 rows (tokens x the heads that share keys) in two halves of 128, one row a
// lane of tensor memory:
//   S = Q·K^T    both from shared memory, 128 x 128 fp32 in tensor memory;
//   P = 2^(S·c - m·c), a row a thread, in bf16 over S's own columns;
//   O += P·V     P from tensor memory, V from shared memory, fp32 in tensor memory.
// While one half's softmax runs the tensor cores work for the other.  Where a
// block has no more than 128 rows (single tokens, drafts) the halves take the
// same rows over alternate tiles, and their sums are joined at the end.
//
// The reference m of a row is its maximum, but it is raised only when a tile's
// maximum passes it by more than 2^8 in the weights: fp32 sums and bf16 weights keep
// their relative precision, and O is rescaled (a pass over tensor memory) once or
// twice a row instead of in most tiles.
//
// Roles: warps 0-3 and 4-7 softmax and output of the halves, 8-11 copies of
// queries, keys and values (16 bytes a copy, through the page table, rows outside
// the sequence filled with zeros), 12 issues the matrix products, 13 hands out
// the segments.
#include <cuda_bf16.h>

#include <algorithm>

#include "usm_internal.h"
#include "usm_paged.cuh"
#include "usm_tmem.cuh"

namespace usm {
namespace {

constexpr int kRows = 256, kKeys = 128, kThreads = 512;
constexpr int kRing = 4;       // segments handed out ahead
constexpr int kConsumers = 13; // warps that read a segment
constexpr float kRaise = 8.f;  // log2 of the largest weight before a row's reference is raised
// Largest |m·c| for which S·c - m·c is formed by one FMA: the rounding of m·c,
// a common factor of the row's weights, stays below 2^(4096·2^-24).
constexpr float kNear = 4096.f;

using Shares = PagedShares<kRows, kKeys, kThreads>;

template <int DP>  // columns of shared memory: 64 or 128
struct Sizes {
    static constexpr int kTile = DP * 256;              // bytes of 128 rows
    static constexpr int kStages = DP == 128 ? 5 : 10;  // tiles of keys or values in flight
    static constexpr int kStage0 = 2 * kTile;           // behind the two halves' queries
    static constexpr int kControl = kStage0 + kStages * kTile;
};

struct Control {
    unsigned long long full[10], empty[10];  // stages
    unsigned long long q_full, q_empty;
    unsigned long long s_full[2], p_full[2], o_full[2];
    unsigned long long seg_full[kRing], seg_empty[kRing];
    unsigned long long box_full, box_free;  // the halves' exchange
    unsigned long long drained;
    long long scratch[kThreads / 32 + 2];
    PagedSegment seg[kRing];
    float2 stats[128];  // (reference, sum) of the second half's rows
    uint32_t tmem;
    int abort;
};
static_assert(Sizes<128>::kControl + sizeof(Control) <= 227 * 1024, "shared memory");

// Waits are bounded: a wait that gives up says so to all others of the CTA.
__device__ bool wait_slow(uint32_t bar, uint32_t parity, Control* ct, int* status) {
    const unsigned long long t0 = global_timer_ns();
    volatile int* abort = &ct->abort;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            record_status(status, USM_ERR_TIMEOUT);
            return false;
        }
    }
}
// By a whole warp, with one answer.
__device__ __forceinline__ bool wait(const unsigned long long& b, uint32_t parity, Control* ct, int* status) {
    const uint32_t bar = smem_addr(&b);
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) ok = wait_slow(bar, parity, ct, status);
    return __all_sync(kFullMask, ok);
}
__device__ __forceinline__ void arrive_warp(const unsigned long long& b) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&b));
}

// Loads of a segment of n tiles come in the order K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ uint32_t k_load(uint32_t base, int t) { return base + (t == 0 ? 0 : 2 * t - 1); }
__device__ __forceinline__ uint32_t v_load(uint32_t base, int t, int n) { return base + (t == n - 1 ? 2 * n - 1 : 2 * t + 2); }

// Whether some row of the segment's block does not see all of the tile's keys
// that lie in [lo, hi).
struct Edges {
    int hi_least, lo_most;
    bool none;
};
__device__ __forceinline__ Edges edges_of(const PagedArgs& a, const PagedSegment& g) {
    const int2 first = paged_seen(a, g, 0), last = paged_seen(a, g, g.rows - 1);
    return Edges{first.y, last.x, first.y <= first.x || last.y <= last.x};
}
__device__ __forceinline__ bool partly_seen(const Edges& e, const PagedSegment& g, int key0) {
    return e.none || min(key0 + kKeys, g.hi) > e.hi_least || max(key0, g.lo) < e.lo_most;
}

__device__ __forceinline__ bool odd_bf16(uint32_t w) {  // an infinity or NaN in either half
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t without_odd(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// ---------------------------------------------------------------------------
// Copies
// ---------------------------------------------------------------------------
template <int DP>
struct Copies {
    using Z = Sizes<DP>;
    static constexpr int kChunks = DP / 8;           // 16-byte chunks of a row
    static constexpr int kSide = 32 / kChunks;       // rows of a warp's copy
    static constexpr int kSteps = 128 / (4 * kSide); // copies of a warp for a tile

    const PagedArgs& a;
    Control* ct;
    uint32_t smem;
    int warp, lane, chunk, side;
    uint32_t swizzled[2];    // byte offset of the chunk in its panel for rows of either parity of...
    uint32_t issued = 0, retired = 0, stage_in = 0, stage_out = 0;
    unsigned is_query = 0, look = 0;  // of the last 32 groups of copies: queries; values to look at
    unsigned seg_of = 0;              // and two bits each of the ring slot (last 16)

    __device__ Copies(const PagedArgs& a, Control* ct, uint32_t smem) : a(a), ct(ct), smem(smem) {
        warp = (threadIdx.x >> 5) & 3;
        lane = threadIdx.x & 31;
        chunk = lane % kChunks;
        side = lane / kChunks;
    }

    __device__ __forceinline__ int row_of(int step, int side) const { return (step * 4 + warp) * kSide + side; }
    __device__ __forceinline__ uint32_t place(uint32_t tile, int row) const {
        return tile + (chunk >> 3) * 16384 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
    }

    __device__ __forceinline__ static void pending(int n) {  // wait until at most n groups are in flight
        switch (n) {
            case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
            case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
            case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
            case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
            case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
            case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
            case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
            case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
            case 8: asm volatile("cp.async.wait_group 8;" ::: "memory"); break;
            default: asm volatile("cp.async.wait_group 9;" ::: "memory"); break;
        }
    }

    // The oldest group in flight has landed: tell its reader.
    __device__ void retire() {
        pending((int)(issued - retired - 1));
        const unsigned bit = retired & 31;
        const bool query = (is_query >> bit) & 1;
        const uint32_t stage = stage_out % Z::kStages;
        if ((look >> bit) & 1) look_at(stage, (seg_of >> (2 * (retired & 15))) & 3);
        fence_proxy_async_smem();
        arrive_warp(query ? ct->q_full : ct->full[stage]);
        if (!query) ++stage_out;
        ++retired;
    }

    // Values of a partly masked tile: infinities and NaN would reach rows that do
    // not see them (0·inf); they are taken out, and added at the end where seen.
    __device__ void look_at(uint32_t stage, int slot) {
        if (chunk * 8 >= a.head_dim) return;
        const uint32_t tile = smem + Z::kStage0 + stage * Z::kTile;
        for (int step = 0; step < kSteps; ++step) {
            const uint32_t at = place(tile, row_of(step, side));
            uint4 w = lds128(at);
            if (odd_bf16(w.x) || odd_bf16(w.y) || odd_bf16(w.z) || odd_bf16(w.w)) {
                w = make_uint4(without_odd(w.x), without_odd(w.y), without_odd(w.z), without_odd(w.w));
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
                *(volatile int*)&ct->seg[slot].odd_values = 1;
            }
        }
    }

    // Waits for a barrier; until it is free, passes on what has landed.
    __device__ bool acquire(const unsigned long long& b, uint32_t parity) {
        const uint32_t bar = smem_addr(&b);
        while (issued != retired) {
            if (__all_sync(kFullMask, mbar_test_wait(bar, parity))) return true;
            retire();
        }
        return wait(b, parity, ct, a.status);
    }

    __device__ __forceinline__ void commit(bool query, bool look_at_it, int slot) {
        asm volatile("cp.async.commit_group;" ::: "memory");
        const unsigned bit = 1u << (issued & 31);
        is_query = query ? is_query | bit : is_query & ~bit;
        look = look_at_it ? look | bit : look & ~bit;
        const int s = 2 * (issued & 15);
        seg_of = (seg_of & ~(3u << s)) | ((unsigned)slot << s);
        ++issued;
    }

    // 128 rows to `tile`; offset: this lane's row's place (elements; lane = step ·
    // kSide + side), negative for a row of zeros.
    __device__ __forceinline__ void rows(uint32_t tile, const void* base, long long offset) {
        const int D = a.head_dim;
        if (chunk * 8 >= (D + 15) / 16 * 16) chunk = kChunks;  // no column of the products
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            const long long from = __shfl_sync(kFullMask, offset, step * kSide + side);
            if (chunk >= kChunks) continue;
            const bool real = from >= 0 && chunk * 8 < D;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(base) + (real ? from + chunk * 8 : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place(tile, row_of(step, side))), "l"(src),
                         "r"(real ? 16 : 0)
                         : "memory");
        }
    }

    __device__ __forceinline__ long long query_row(const PagedSegment& g, int half) const {
        const int r = 128 * half + row_of(lane / kSide, lane % kSide);
        if (r >= g.rows) return -1;
        const int flat = g.row0 + r, token = flat / a.group;
        return (long long)(g.start + token) * a.q_token + (long long)(g.head * a.group + flat - token * a.group) * a.q_head;
    }

    __device__ __forceinline__ bool tile(const PagedSegment& g, int key0, bool values, bool look_at_it, int slot) {
        const int key = key0 + row_of(lane / kSide, lane % kSide);
        long long offset = -1;
        if (key >= g.lo && key < g.hi) {
            const int2 w = paged_slot(a, g.seq, key);
            offset = values ? w.x * a.v_page + w.y * a.v_slot + g.head * a.v_head
                            : w.x * a.k_page + w.y * a.k_slot + g.head * a.k_head;
        }
        const uint32_t stage = stage_in % Z::kStages;
        if (!acquire(ct->empty[stage], (stage_in / Z::kStages & 1) ^ 1)) return false;
        rows(smem + Z::kStage0 + stage * Z::kTile, values ? a.v : a.k, offset);
        commit(false, look_at_it, slot);
        ++stage_in;
        return true;
    }

    __device__ void run() {
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!acquire(ct->seg_full[slot], it / kRing & 1)) return;
            const PagedSegment g = ct->seg[slot];
            if (!g.live) break;
            if (it > 0 && !acquire(ct->q_empty, (it - 1) & 1)) return;
            rows(smem, a.q, query_row(g, 0));
            if (g.rows > 128) rows(smem + Z::kTile, a.q, query_row(g, 1));
            commit(true, false, slot);
            const Edges e = edges_of(a, g);
            const int n = g.tiles, key0 = g.tile0 * kKeys;
            for (int i = 0; i < 2 * n; ++i) {  // K0 K1 V0 K2 V1 ...
                const bool values = i == 2 * n - 1 || (i > 0 && i % 2 == 0);
                const int t = i == 2 * n - 1 ? n - 1 : values ? i / 2 - 1 : (i + 1) / 2;
                const int at = key0 + t * kKeys;
                if (!tile(g, at, values, values && partly_seen(e, g, at), slot)) return;
            }
            while (issued != retired) retire();
            arrive_warp(ct->seg_empty[slot]);
        }
    }
};

// ---------------------------------------------------------------------------
// Matrix products (one warp; its lane 0 issues)
// ---------------------------------------------------------------------------
template <int DP>
struct Products {
    using Z = Sizes<DP>;
    const PagedArgs& a;
    Control* ct;
    uint32_t smem, tmem;
    uint32_t qk_shape, pv_shape;
    int steps;
    bool lead;
    uint32_t p_uses[2] = {0, 0};

    __device__ Products(const PagedArgs& a, Control* ct, uint32_t smem, uint32_t tmem) : a(a), ct(ct), smem(smem), tmem(tmem) {
        steps = (a.head_dim + 15) / 16;
        qk_shape = bf16_mma_shape(kKeys, false);
        pv_shape = bf16_mma_shape(steps * 16, true);
        lead = (threadIdx.x & 31) == 0;
    }
    __device__ __forceinline__ void commit(const unsigned long long& b) {
        if (lead) tmem_commit(smem_addr(&b));
    }
    __device__ __forceinline__ bool loaded(uint32_t load) {
        return wait(ct->full[load % Z::kStages], load / Z::kStages & 1, ct, a.status);
    }
    __device__ __forceinline__ uint32_t stage(uint32_t load) const { return smem + Z::kStage0 + load % Z::kStages * Z::kTile; }
    __device__ __forceinline__ void release(uint32_t load) { commit(ct->empty[load % Z::kStages]); }

    __device__ __forceinline__ void scores(int half, int q_half, uint32_t load) {
        if (lead) {
            const uint64_t q = swizzled_desc(smem + q_half * Z::kTile, 0), k = swizzled_desc(stage(load), 0);
            for (int i = 0; i < steps; ++i) {
                const uint32_t at = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
                mma_bf16_ss(tmem + half * kKeys, q + at, k + at, qk_shape, i > 0);
            }
        }
        commit(ct->s_full[half]);
    }
    __device__ __forceinline__ bool weigh(int half, uint32_t load, bool accumulate) {
        if (!wait(ct->p_full[half], p_uses[half]++ & 1, ct, a.status)) return false;
        tmem_fence_after_sync();
        if (lead) {
            const uint64_t v = swizzled_desc(stage(load), 16384);
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)
                mma_bf16_ts(tmem + 256 + half * DP, tmem + half * kKeys + i * 8, v + (i * 2048 >> 4), pv_shape, accumulate || i > 0);
        }
        return true;
    }

    __device__ void run() {
        uint32_t base = 0;
        for (uint32_t it = 0;; ++it) {
            const int slot = it % kRing;
            if (!wait(ct->seg_full[slot], it / kRing & 1, ct, a.status)) return;
            if (!ct->seg[slot].live) break;
            const int n = ct->seg[slot].tiles;
            const bool shared = ct->seg[slot].rows <= 128;
            if (!wait(ct->q_full, it & 1, ct, a.status) || !loaded(k_load(base, 0))) return;
            scores(0, 0, k_load(base, 0));
            if (!shared) scores(1, 1, k_load(base, 0));
            release(k_load(base, 0));
            if (shared && n > 1) {
                if (!loaded(k_load(base, 1))) return;
                scores(1, 0, k_load(base, 1));
                release(k_load(base, 1));
            }
            const int ahead = shared ? 2 : 1;  // tiles whose scores are formed before the sums of tile t
            if (n <= ahead) commit(ct->q_empty);
            for (int t = 0; t < n; ++t) {
                const uint32_t v = v_load(base, t, n), k = k_load(base, t + ahead);
                const bool more = t + ahead < n;
                if (!loaded(v) || (more && !loaded(k))) return;
                if (shared) {
                    const int half = t & 1;
                    if (!weigh(half, v, t >= 2)) return;
                    release(v);
                    if (more) scores(half, 0, k);
                    else commit(ct->o_full[half]);
                } else {
#pragma unroll 1
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
            arrive_warp(ct->seg_empty[slot]);
        }
    }
};

// ---------------------------------------------------------------------------
// Softmax and output: one row a thread
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store16(void* p, const uint32_t* w) {  // 32 bytes, 16-byte aligned
    asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

template <int DP>
struct Softmax {
    using Z = Sizes<DP>;
    const PagedArgs& a;
    Control* ct;
    uint32_t smem;
    int half, tid;           // thread of the half
    uint32_t s_col, o_col;   // this warp's lanes of tensor memory
    uint32_t s_uses = 0, o_uses = 0, box_uses = 0;
    // Of the current segment:
    float m, l;  // reference (a score) and sum of the weights
    int2 seen;

    __device__ Softmax(const PagedArgs& a, Control* ct, uint32_t smem, uint32_t tmem) : a(a), ct(ct), smem(smem) {
        half = threadIdx.x >> 7;
        tid = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(tid & ~31) << 16;
        s_col = tmem + lanes + half * kKeys;
        o_col = tmem + lanes + 256 + half * DP;
    }

    // One tile's scores into weights.  `first`: O holds nothing yet.
    __device__ __forceinline__ void weights(int key0, bool masked, bool first) {
        uint32_t w[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_col + 32 * i, w[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_wait_ld(w[i]);
        const float c = a.scale_log2;
        if (masked) {
            const unsigned from = (unsigned)(seen.x - key0), count = (unsigned)(seen.y - seen.x);
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
            if (!first) rescale(f);
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const bool far = !(fabsf(mc) <= kNear);
        uint64_t sum[2] = {0, 0};
        if (!__any_sync(kFullMask, far)) {
            const uint64_t c2 = pack2(c, c), mc2 = pack2(-mc, -mc);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const uint32_t(&s)[32] = w[2 * h + (j >> 4)];
                    const int i = 2 * (j & 15);
                    float x, y;
                    unpack2(fma2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, mc2), x, y);
                    x = exp2_fast(x);
                    y = exp2_fast(y);
                    sum[j & 1] = add2(sum[j & 1], pack2(x, y));
                    p[j] = bf16x2(x, y);
                }
                tmem_st32(s_col + 32 * h, p);
            }
        } else {
            // Far from zero the difference is formed first: it is exact near m.
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const uint32_t(&s)[32] = w[2 * h + (j >> 4)];
                    const int i = 2 * (j & 15);
                    const float x = exp2_fast((__uint_as_float(s[i]) - base) * c);
                    const float y = exp2_fast((__uint_as_float(s[i + 1]) - base) * c);
                    sum[j & 1] = add2(sum[j & 1], pack2(x, y));
                    p[j] = bf16x2(x, y);
                }
                tmem_st32(s_col + 32 * h, p);
            }
        }
        float x0, x1, y0, y1;
        unpack2(sum[0], x0, x1);
        unpack2(sum[1], y0, y1);
        l += (x0 + x1) + (y0 + y1);
        tmem_wait_st();
    }

    __device__ void rescale(float f) {
        const int columns = (a.head_dim + 15) / 16 * 16;
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
            if (32 * j >= columns) break;
            uint32_t w[32];
            tmem_ld32(o_col + 32 * j, w);
            tmem_wait_ld(w);
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
            tmem_st32(o_col + 32 * j, w);
        }
        tmem_wait_st();
    }

    // Adds what was taken out of partly masked tiles (infinities and NaN of rows
    // of V that this row sees) to columns 32·j.. of its sums.
    __device__ void add_odd(const PagedSegment& g, bool shared, int j, uint32_t (&w)[32]) {
        const Edges e = edges_of(a, g);
        for (int t = shared ? half : 0; t < g.tiles; t += shared ? 2 : 1) {
            const int key0 = (g.tile0 + t) * kKeys;
            if (!partly_seen(e, g, key0)) continue;
            for (int key = max(key0, seen.x); key < min(key0 + kKeys, seen.y); ++key) {
                const int2 at = paged_slot(a, g.seq, key);
                const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + at.x * a.v_page + at.y * a.v_slot + g.head * a.v_head;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (32 * j + i >= a.head_dim) break;
                    const float x = __bfloat162float(v[32 * j + i]);
                    if (!isfinite(x)) w[i] = __float_as_uint(__uint_as_float(w[i]) + x);
                }
            }
        }
    }

    // Columns 32·j.. of a row of results: to the output, or to the partial results.
    __device__ __forceinline__ void store(const PagedSegment& g, int row, int j, const uint32_t (&w)[32], float z) {
        const int left = a.head_dim - 32 * j;  // a multiple of 8
        if (g.part == kPartWhole) {
            const int flat = g.row0 + row, token = flat / a.group;
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + (long long)(g.start + token) * a.out_token +
                                (long long)(g.head * a.group + flat - token * a.group) * a.out_head + 32 * j;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (8 * i >= left) break;
                uint32_t p[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    p[u] = bf16x2(__uint_as_float(w[8 * i + 2 * u]) * z, __uint_as_float(w[8 * i + 2 * u + 1]) * z);
                store16(to + 8 * i, p);
            }
        } else {
            float* to = a.parts + ((2LL * blockIdx.x + g.part) * a.part_rows + row) * a.head_dim + 32 * j;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (4 * i >= left) break;
                store16(to + 4 * i, w + 4 * i);
            }
        }
    }

    // Sums of the two halves over the same rows, 32 columns at a time through the
    // queries' second tile (free here: the block has one).
    __device__ bool join_halves(const PagedSegment& g, int row) {
        const bool mine = __any_sync(kFullMask, row < g.rows);  // a warp with rows
        const bool odd = *(volatile int*)&ct->seg[slot].odd_values;
        const uint32_t box = smem + Z::kTile + 4 * tid;  // [32 columns][128 rows]
        float z = 0.f, f0 = 1.f, f1 = 1.f;
        for (int j = 0; j < DP / 32; ++j) {
            if (32 * j >= a.head_dim) break;
            uint32_t w[32];
            if (mine) {
                tmem_ld32(o_col + 32 * j, w);
                tmem_wait_ld(w);
                if (odd && row < g.rows) add_odd(g, true, j, w);
            }
            const uint32_t use = box_uses++;
            if (half == 1) {
                if (use > 0 && !wait(ct->box_free, (use - 1) & 1, ct, a.status)) return false;
                if (j == 0) ct->stats[tid] = make_float2(m, l);
                if (mine)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(box + 512 * i), "r"(w[i]) : "memory");
                arrive_warp(ct->box_full);
                continue;
            }
            if (!wait(ct->box_full, use & 1, ct, a.status)) return false;
            if (mine) {
                if (j == 0) {
                    const float2 other = ct->stats[tid];
                    const float t = fmaxf(m, other.x);
                    f0 = m == -INFINITY ? 0.f : exp2_fast((m - t) * a.scale_log2);
                    f1 = other.x == -INFINITY ? 0.f : exp2_fast((other.x - t) * a.scale_log2);
                    m = t;
                    l = l * f0 + other.y * f1;
                    z = l == 0.f ? 0.f : 1.f / l;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    w[i] = __float_as_uint(__uint_as_float(w[i]) * f0 + __uint_as_float(lds32(box + 512 * i)) * f1);
            }
            arrive_warp(ct->box_free);
            if (row < g.rows) store(g, row, j, w, z);
        }
        return true;
    }

    int slot;

    __device__ void run() {
        for (uint32_t it = 0;; ++it) {
            slot = it % kRing;
            if (!wait(ct->seg_full[slot], it / kRing & 1, ct, a.status)) return;
            const PagedSegment g = ct->seg[slot];
            if (!g.live) break;
            const bool shared = g.rows <= 128;
            const int row = shared ? tid : half * 128 + tid;
            const bool some = __any_sync(kFullMask, row < g.rows);
            seen = paged_seen(a, g, row);
            // Keys that every row of this warp sees.
            int lo = row < g.rows ? seen.x : 0, hi = row < g.rows ? seen.y : 0x7fffffff;
            if (row < g.rows && seen.x >= seen.y) lo = 0x7fffffff;
            lo = __reduce_max_sync(kFullMask, lo);
            hi = __reduce_min_sync(kFullMask, hi);
            if (!shared) arrive_warp(ct->q_empty);
            m = -INFINITY;
            l = 0.f;
            const int first = shared ? half : 0, step = shared ? 2 : 1;
            for (int t = first; t < g.tiles; t += step) {
                if (!wait(ct->s_full[half], s_uses++ & 1, ct, a.status)) return;
                tmem_fence_after_sync();
                const int key0 = (g.tile0 + t) * kKeys;
                if (some) weights(key0, key0 < lo || key0 + kKeys > hi, t == first);
                tmem_fence_before_sync();
                arrive_warp(ct->p_full[half]);
            }
            const bool both = shared && g.tiles > 1;
            if (first < g.tiles) {
                if (!wait(ct->o_full[half], o_uses++ & 1, ct, a.status)) return;
                tmem_fence_after_sync();
            }
            if (both) {
                if (!join_halves(g, row)) return;
            } else if (some && first < g.tiles) {
                const float z = l == 0.f ? 0.f : 1.f / l;
                const bool odd = *(volatile int*)&ct->seg[slot].odd_values;
                for (int j = 0; j < DP / 32; ++j) {
                    if (32 * j >= a.head_dim) break;
                    uint32_t w[32];
                    tmem_ld32(o_col + 32 * j, w);
                    tmem_wait_ld(w);
                    if (row < g.rows) {
                        if (odd) add_odd(g, shared, j, w);
                        store(g, row, j, w, z);
                    }
                }
            }
            if (g.part != kPartWhole && row < g.rows && (!shared || half == 0))
                *reinterpret_cast<float2*>(a.part_stats + 2 * ((2LL * blockIdx.x + g.part) * a.part_rows + row)) = make_float2(m, l);
            tmem_fence_before_sync();
            if (shared) arrive_warp(ct->q_empty);
            arrive_warp(ct->seg_empty[slot]);
        }
    }
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) paged_mma_kernel(const __grid_constant__ PagedArgs a) {
    using Z = Sizes<DP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Control* ct = reinterpret_cast<Control*>(smem + Z::kControl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    let_next_start();
    if (threadIdx.x == 0) {
        for (int i = 0; i < Z::kStages; ++i) {
            mbar_init(smem_addr(&ct->full[i]), 4);
            mbar_init(smem_addr(&ct->empty[i]), 1);
        }
        mbar_init(smem_addr(&ct->q_full), 4);
        mbar_init(smem_addr(&ct->q_empty), 1 + 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ct->s_full[i]), 1);
            mbar_init(smem_addr(&ct->p_full[i]), 4);
            mbar_init(smem_addr(&ct->o_full[i]), 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_addr(&ct->seg_full[i]), 1);
            mbar_init(smem_addr(&ct->seg_empty[i]), kConsumers);
        }
        mbar_init(smem_addr(&ct->box_full), 4);
        mbar_init(smem_addr(&ct->box_free), 4);
        mbar_init(smem_addr(&ct->drained), 1);
        ct->abort = 0;
        fence_barrier_init();
    }
    if (warp == 12) tmem_alloc(smem_addr(&ct->tmem), 512);
    Shares shares;
    shares.init(a, blockIdx.x, gridDim.x, ct->scratch);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = *(volatile uint32_t*)&ct->tmem, base = smem_addr(smem);

    // 192 + 192 + 72 + 56 registers: the 4 x 128 that the launch has.
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        Softmax<DP>(a, ct, base, tmem).run();
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        Copies<DP> copies(a, ct, base);
        copies.run();
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 12) {
            Products<DP>(a, ct, base, tmem).run();
            // Whatever was issued is done before tensor memory is given back.
            if (lane == 0) tmem_commit(smem_addr(&ct->drained));
            __syncwarp();
            mbar_wait_bounded(smem_addr(&ct->drained), 0, kWaitLimitNs);
        } else if (warp == 13) {
            PagedMeta meta = {};
            for (uint32_t it = 0;; ++it) {
                const int slot = it % kRing;
                const PagedSegment g = shares.next(a);
                if (g.live) paged_note(meta, g);
                if (it >= kRing && !wait(ct->seg_empty[slot], (it / kRing - 1) & 1, ct, a.status)) break;
                if (lane == 0) ct->seg[slot] = g;
                arrive_warp(ct->seg_full[slot]);
                if (!g.live) break;
            }
            if (lane == 0) static_cast<PagedMeta*>(a.meta)[blockIdx.x] = meta;
        }
    }
    __syncthreads();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int DP>
int run(const PagedArgs& a, int ctas, cudaStream_t stream) {
    const auto kernel = paged_mma_kernel<DP>;
    constexpr int smem = Sizes<DP>::kControl + (int)sizeof(Control);
    if (!allow_shared(kernel, smem)) return cuda_failure();
    kernel<<<ctas, kThreads, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

}  // namespace

int paged_mma_rows() { return kRows; }
int launch_paged_mma(const PagedArgs& a, int ctas, cudaStream_t stream) {
    return a.head_dim <= 64 ? run<64>(a, ctas, stream) : run<128>(a, ctas, stream);
}

}  // namespace usm
