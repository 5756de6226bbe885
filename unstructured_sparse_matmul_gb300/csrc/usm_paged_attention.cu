// Attention of a chunk of new tokens over a paged cache.  Contract and masks:
// include/usm.h; how the work is divided: usm_paged.cuh.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "usm_internal.h"
#include "usm_paged.cuh"
#include "usm_tmem.cuh"

namespace usm {
namespace {

// Four elements, as they lie in memory and as floats.
__device__ __forceinline__ float4 quad4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ uint2 quad4(const __nv_bfloat16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void quads8(const __nv_bfloat16* p, uint2* x) {  // two at once
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    x[0] = make_uint2(w.x, w.y), x[1] = make_uint2(w.z, w.w);
}
__device__ __forceinline__ float4 floats(float4 x) { return x; }
__device__ __forceinline__ float4 floats(uint2 w) {
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
template <class T>
__device__ __forceinline__ float4 load4(const T* p) {
    return floats(quad4(p));
}
__device__ __forceinline__ void store4(float4 x, float* p) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(float4 x, __nv_bfloat16* p) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(x.x, x.y), bf16x2(x.z, x.w));
}
__device__ __forceinline__ float4 scaled(float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); }
__device__ __forceinline__ float4 add_scaled(float4 x, float4 y, float f) {
    return make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
}

// A row's weight relative to a reference `top`: nothing seen (-inf) gives 0.
__device__ __forceinline__ float weight_of(float m, float top, float scale_log2) {
    return m == -INFINITY ? 0.f : exp2_fast((m - top) * scale_log2);
}

// Query row `row` of a segment, and its row of the output.
template <class T>
__device__ __forceinline__ const T* query_of(const PagedArgs& a, const PagedSegment& g, int row) {
    const int flat = g.row0 + row, token = by_group(a, flat), head = g.head * a.group + flat - token * a.group;
    return (const T*)a.q + (g.start + token) * a.q_token + head * a.q_head;
}
template <class T>
__device__ __forceinline__ T* output_of(const PagedArgs& a, const PagedSegment& g, int row) {
    const int flat = g.row0 + row, token = by_group(a, flat), head = g.head * a.group + flat - token * a.group;
    return (T*)a.out + (g.start + token) * a.out_token + head * a.out_head;
}

// A CTA's walk over its share, in shared memory: its first warp takes the steps.
template <class Shares>
struct Walk {
    alignas(8) char shares[sizeof(Shares)];
    PagedMeta meta;

    __device__ __forceinline__ void begin(const PagedArgs& a, long long* scratch) {
        Shares s;
        if (a.num_seqs > Shares::kSolo) s.init(a, blockIdx.x, gridDim.x, scratch);
        else if (threadIdx.x < 32) s.init_solo(a, blockIdx.x, gridDim.x);
        if (threadIdx.x == 0) {
            memcpy(shares, &s, sizeof s);
            meta = PagedMeta{};
        }
    }
    __device__ __forceinline__ void next(const PagedArgs& a, PagedSegment& seg) {
        Shares s;
        memcpy(&s, shares, sizeof s);
        const PagedSegment g = s.next(a);
        __syncwarp();  // every lane has copied the walk's state
        if (threadIdx.x == 0) {
            memcpy(shares, &s, sizeof s);
            if (g.live) paged_note(meta, g);
            seg = g;
        }
    }
};

// Where columns 4·quad.. of a row of a partial result lie: a warp that has 32 rows
// of a column writes them side by side.
__device__ __forceinline__ float* part_of(float* parts, int part_rows, int head_dim, long long slot, int row, int quad) {
    return parts + (slot * part_rows * (head_dim / 4) + (long long)quad * part_rows + row) * 4;
}
__device__ __forceinline__ float* part_of(const PagedArgs& a, long long slot, int row, int quad) {
    return part_of(a.parts, a.part_rows, a.head_dim, slot, row, quad);
}

// ---------------------------------------------------------------------------
// fp32 caches, many rows, and bf16 heads wider than the matrix kernel takes:
// products on the FMA units.  64 rows of queries stay in shared memory; tiles of
// 64 keys pass through it, fp32 ones copied asynchronously one tile ahead.  Each
// of 256 threads holds 4 rows x 4 keys of the scores and 4 rows x up to 16
// columns of the sums, all in pairs (two FMAs an instruction); 12 wavefronts of
// shared memory feed 64 FMAs of a warp.  Columns come in groups of 64 and, behind
// them, one of 32 (heads of 80 columns do the work of 96, not 128: 376 against 401
// us).  1024 tokens over 4096 keys, 8 heads: 32 TFLOP/s at 128 columns, 25 at 80, 27
// at 64.  Bound by latency and moves, with 8 warps an SM; two CTAs an SM with one
// tile each, or weights stored in pairs, were no faster.
// ---------------------------------------------------------------------------
constexpr int kBlockRows = 64, kBlockKeys = 64, kBlockThreads = 256;
constexpr int kBlockWeights = kBlockKeys + 4;  // pitch of a row of weights
using BlockShares = PagedShares<kBlockRows, kBlockKeys, kBlockThreads, 3>;

// Row pitch of the shared arrays: a multiple of 4 that is 4 modulo 32, so that 8
// consecutive rows start in different groups of banks.
constexpr int block_pitch(int head_dim) { return (head_dim + 31) / 32 * 32 + 4; }
// Tiles of keys and values in shared memory: two where they fit.
constexpr int block_stages(int head_dim) { return head_dim <= 128 ? 2 : 1; }
constexpr int block_smem(int head_dim) {
    return (kBlockRows + 2 * block_stages(head_dim) * kBlockKeys) * block_pitch(head_dim) * 4 + kBlockRows * kBlockWeights * 4;
}

__device__ __forceinline__ void copy4(float* to, const float* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(float* to, const __nv_bfloat16* from, bool there) {
    *reinterpret_cast<float4*>(to) = there ? load4(from) : make_float4(0.f, 0.f, 0.f, 0.f);
}

__device__ __forceinline__ void store2(float x, float y, float* p) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(float x, float y, __nv_bfloat16* p) { *reinterpret_cast<uint32_t*>(p) = bf16x2(x, y); }

// o += P·V for 4 rows of a tile and this thread's columns: 64·c + 4·tx.. of whole
// groups of 64 and, where kWide is odd, 2·tx.. of the 32 behind them.
template <int kWide, bool kGuard>
__device__ __forceinline__ void add_values(const float* p, const float* v, int pitch, int D, int tx, int key0, const int2 (&seen)[4],
                                           uint64_t (&o)[4][kWide]) {
#pragma unroll 2
    for (int key = 0; key < kBlockKeys; key += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + i * kBlockWeights + key);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint64_t y[kWide];
#pragma unroll
            for (int c = 0; c < kWide / 2; ++c) {
                const int col = 64 * c + 4 * tx;
                ulonglong2 w = make_ulonglong2(0, 0);
                if (col < D) w = *reinterpret_cast<const ulonglong2*>(v + (key + u) * pitch + col);
                y[2 * c] = w.x, y[2 * c + 1] = w.y;
            }
            if (kWide % 2) {
                const int col = 32 * (kWide - 1) + 2 * tx;
                y[kWide - 1] = 0;
                if (col < D) y[kWide - 1] = *reinterpret_cast<const uint64_t*>(v + (key + u) * pitch + col);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = u == 0 ? w[i].x : u == 1 ? w[i].y : u == 2 ? w[i].z : w[i].w;
                if (kGuard && (key0 + key + u < seen[i].x || key0 + key + u >= seen[i].y)) continue;
                const uint64_t e2 = pack2(e, e);
#pragma unroll
                for (int c = 0; c < kWide; ++c) o[i][c] = fma2(e2, y[c], o[i][c]);
            }
        }
    }
}

template <class T, int kWide>  // kWide: groups of 32 columns
__global__ void __launch_bounds__(kBlockThreads) paged_block_kernel(const __grid_constant__ PagedArgs a) {
    extern __shared__ float4 smem_raw[];
    __shared__ long long scratch[kBlockThreads / 32 + 2];
    __shared__ PagedSegment seg;
    await_previous();
    let_next_start();
    constexpr int kStages = block_stages(32 * kWide);
    constexpr int kP = kBlockWeights;
    const int D = a.head_dim, pitch = block_pitch(D);
    float* q = reinterpret_cast<float*>(smem_raw);
    float* tiles = q + kBlockRows * pitch;  // [stage][keys, then values][64][pitch]
    float* p = tiles + kStages * 2 * kBlockKeys * pitch;  // probabilities, [row][key]
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, warp = tid >> 5, lane = tid & 31;
    const int quads = D / 4;

    __shared__ Walk<BlockShares> walk;
    walk.begin(a, scratch);
    while (true) {
        __syncthreads();
        if (tid < 32) walk.next(a, seg);
        __syncthreads();
        if (!seg.live) break;
        const PagedSegment& g = seg;
        // A warp copies rows; its lanes find their places, one each.
        for (int r0 = 8 * warp; r0 < 8 * warp + 8; ++r0) {
            const bool there = r0 < g.rows;
            const T* row = there ? query_of<T>(a, g, r0) : (const T*)a.q;
            for (int c = lane; c < quads; c += 32) copy4(q + r0 * pitch + 4 * c, row + 4 * c, there);
        }
        const auto load = [&](int t) {  // a warp: 8 keys and their values
            const int key0 = (g.tile0 + t) * kBlockKeys + 8 * warp, key = key0 + (lane & 7);
            int2 w = make_int2(-1, 0);
            if (key >= g.lo && key < g.hi) w = paged_slot(a, g.seq, key);
            float* to = tiles + (t % kStages) * 2 * kBlockKeys * pitch + 8 * warp * pitch;
#pragma unroll 2
            for (int r = 0; r < 8; ++r) {
                const int page = __shfl_sync(kFullMask, w.x, r), slot = __shfl_sync(kFullMask, w.y, r);
                const bool there = page >= 0;
                const T* k = (const T*)a.k + (there ? page * a.k_page + slot * a.k_slot + g.head * a.k_head : 0);
                const T* v = (const T*)a.v + (there ? page * a.v_page + slot * a.v_slot + g.head * a.v_head : 0);
                for (int c = lane; c < quads; c += 32) {
                    copy4(to + r * pitch + 4 * c, k + 4 * c, there);
                    copy4(to + (kBlockKeys + r) * pitch + 4 * c, v + 4 * c, there);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int2 seen[4];
        float m[4], l[4];
        uint64_t o[4][kWide];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            seen[i] = paged_seen(a, g, ty * 4 + i);
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < kWide; ++j) o[i][j] = 0;
        }
        const int n = g.tiles;
        load(0);
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            const int key0 = (g.tile0 + t) * kBlockKeys;
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
            if (kStages == 2 && t + 1 < n) load(t + 1);
            const float* k = tiles + (t % kStages) * 2 * kBlockKeys * pitch;
            const float* v = k + kBlockKeys * pitch;
            // Scores of rows 4·ty.. and keys tx, tx + 16, ..., even and odd columns apart.
            uint64_t s2[4][4] = {};
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                ulonglong2 qa[4], ka[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qa[i] = *reinterpret_cast<const ulonglong2*>(q + (ty * 4 + i) * pitch + d);
                    ka[i] = *reinterpret_cast<const ulonglong2*>(k + (tx + 16 * i) * pitch + d);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s2[i][j] = fma2(qa[i].y, ka[j].y, fma2(qa[i].x, ka[j].x, s2[i][j]));
            }
            bool partly = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float s[4], top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x, y;
                    unpack2(s2[i][j], x, y);
                    const int key = key0 + tx + 16 * j;
                    s[j] = key >= seen[i].x && key < seen[i].y ? x + y : -INFINITY;
                    top = fmaxf(top, s[j]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, w));
                top = fmaxf(top, m[i]);
                const float f = weight_of(m[i], top, a.scale_log2);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = s[j] == -INFINITY ? 0.f : exp2_fast((s[j] - top) * a.scale_log2);
                    p[(ty * 4 + i) * kP + tx + 16 * j] = e;
                    sum += e;
                }
                l[i] = l[i] * f + sum;  // this thread's keys
                const uint64_t f2 = pack2(f, f);
#pragma unroll
                for (int j = 0; j < kWide; ++j) o[i][j] = mul2(o[i][j], f2);
                partly |= seen[i].x > key0 || seen[i].y < key0 + kBlockKeys;
            }
            __syncwarp();  // a warp's rows of p are its own
            // Where a row does not see the whole tile a weight of 0 takes no value.
            if (__any_sync(kFullMask, partly)) add_values<kWide, true>(p + ty * 4 * kP, v, pitch, D, tx, key0, seen, o);
            else add_values<kWide, false>(p + ty * 4 * kP, v, pitch, D, tx, key0, seen, o);
            if (kStages == 1 && t + 1 < n) {
                __syncthreads();
                load(t + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(kFullMask, l[i], w);
            const int r = ty * 4 + i;
            if (r >= g.rows) continue;
            const bool whole = g.part == kPartWhole;
            const float z = !whole ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
            const long long row = (2LL * blockIdx.x + g.part) * a.part_rows + r;
            T* out = output_of<T>(a, g, r);
#pragma unroll
            for (int c = 0; c < kWide / 2; ++c) {
                const int col = 64 * c + 4 * tx;
                if (col >= D) continue;
                float4 x;
                unpack2(o[i][2 * c], x.x, x.y);
                unpack2(o[i][2 * c + 1], x.z, x.w);
                if (whole) store4(scaled(x, z), out + col);
                else store4(x, part_of(a, 2LL * blockIdx.x + g.part, r, col / 4));
            }
            if (const int col = 32 * (kWide - 1) + 2 * tx; kWide % 2 && col < D) {
                float x, y;
                unpack2(o[i][kWide - 1], x, y);
                if (whole) store2(x * z, y * z, out + col);
                else store2(x, y, part_of(a, 2LL * blockIdx.x + g.part, r, col / 4) + col % 4);
            }
            if (!whole && tx == 0) *reinterpret_cast<float2*>(a.part_stats + 2 * row) = make_float2(m[i], l[i]);
        }
    }
    if (tid == 0) static_cast<PagedMeta*>(a.meta)[blockIdx.x] = walk.meta;
}

// ---------------------------------------------------------------------------
// fp32 caches and wide bf16 heads, few rows (single tokens): every warp takes
// batches of keys straight from memory, kLanes lanes a key, four columns each (wide
// heads: eight).  A batch's scores come first, then the weights, then the sums: a key
// is widened once for all rows, and its registers are free again when the values
// are used.  A lane's partial products of a row are summed across lanes all at once,
// halving the number of values a lane holds with every step, so that a score costs
// about one shuffle; each lane then has one key's weight, which goes back to all for
// the sums.  16 warps an SM keep 64 to 128 KB of keys and values on the way.  Bound
// by HBM with one row (16 tokens over 4096 fp32 keys of 64 columns, 227 MB: 51 us,
// 10 of them start and joining; 32 over 4096 bf16 keys of 256 columns: 5.5 TB/s),
// by instructions with more: 128 fp32 columns 5.0 TB/s with 2 rows, 4.6 with 4, 2.7
// with 8; 256 columns 5.2 with 2 and 4.3 with 4, in bf16 3.5 with 4.  (Row by row
// with keys and values held as floats: 4.2, 2.5, 3.6 and 1.7 with 4, 8, 4 and 4; 2
// rows as 4: 4.5 and 4.4, 192 bf16 columns 2.5 for 4.4; bf16 quads 128 columns
// apart, in loads of 8 bytes: 3.9 with one row.)
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 256, kFewKeys = 128;

// 8, 16, 32 lanes: heads of up to 32, 64, 128 columns, with kQ = 2 up to 256; kR rows.
template <class T, int kLanes, int kQ, int kR>
__global__ void __launch_bounds__(kFewThreads, 2) paged_few_kernel(const __grid_constant__ PagedArgs a) {
    using Shares = PagedShares<kR, kFewKeys, kFewThreads, 2>;
    constexpr int kWarps = kFewThreads / 32, kSide = 32 / kLanes;
    // Loads of keys, and of values, of a batch: what fits the registers.
    constexpr int kRegs = sizeof(T) * kQ;  // of a load
    constexpr int kLoads = kR <= 2 && kRegs <= 4 || kR == 4 && kQ == 1 ? 8 : kR == 4 && kRegs == 8 ? 2 : 4;
    constexpr int kRow = kQ * kLanes;             // quads of columns
    constexpr int kBatch = kLoads * kSide;        // keys
    constexpr int kSteps = kLoads == 8 ? 3 : kLoads / 2;  // that halve the values
    extern __shared__ float4 smem_raw[];          // queries [row][lane]; sums [warp][row][lane]; (reference, sum) [warp][row]
    __shared__ int2 sees[kR];
    __shared__ long long scratch[kWarps + 2];
    __shared__ PagedSegment seg;
    await_previous();
    let_next_start();
    const int D = a.head_dim, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Quad h of a lane, at = h·kLanes + lane in shared memory, is this quad of a row.
    static_assert(kQ == 1 || kLanes == 32);
    const auto quad_of = [](int at) { return sizeof(T) == 2 ? at % 32 * 2 + at / 32 : at; };
    const int side = lane / kLanes, col = 4 * quad_of(lane % kLanes);
    bool there[kQ];
#pragma unroll
    for (int h = 0; h < kQ; ++h) there[h] = col + 128 * h < D;
    float4* queries = smem_raw;
    float4* sums = queries + kR * kRow;
    float2* stats = reinterpret_cast<float2*>(sums + kWarps * kR * kRow);
    // The load whose score this lane ends up with.
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) mine |= (lane & (kLanes >> (i + 1))) ? (kLoads >> (i + 1)) : 0;
    const float c = a.scale_log2;

    __shared__ Walk<Shares> walk;
    walk.begin(a, scratch);
    while (true) {
        __syncthreads();
        if (tid < 32) walk.next(a, seg);
        __syncthreads();
        if (!seg.live) break;
        const PagedSegment& g = seg;
        for (int i = tid; i < kR * kRow; i += kFewThreads) {
            const int r = i / kRow, at = i % kRow, quad = quad_of(at);
            queries[i] = r < g.rows && 4 * quad < D ? load4(query_of<T>(a, g, r) + 4 * quad) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (at == 0) sees[r] = paged_seen(a, g, r);
        }
        __syncthreads();
        float4 o[kR][kQ];
        float m[kR], l[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
#pragma unroll
            for (int h = 0; h < kQ; ++h) o[r][h] = make_float4(0.f, 0.f, 0.f, 0.f);
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
        const int lo = g.lo, hi = g.hi, seq = g.seq;
        const T* kb = (const T*)a.k + g.head * a.k_head + col;
        const T* vb = (const T*)a.v + g.head * a.v_head + col;
        const int first = g.tile0 * kFewKeys + warp * kBatch, end = min((g.tile0 + g.tiles) * kFewKeys, hi);
        const auto slot_of = [&](int base) {  // of this lane's key of a batch
            const int key = base + lane;
            return lane < kBatch && key >= lo && key < end ? paged_slot(a, seq, key) : make_int2(-1, 0);
        };
        int2 next = slot_of(first);
#pragma unroll 1
        for (int base = first; base < end; base += kWarps * kBatch) {
            const int2 w = next;
            next = slot_of(base + kWarps * kBatch);
            decltype(quad4(kb)) k[kLoads][kQ], v[kLoads][kQ];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int page = __shfl_sync(kFullMask, w.x, j * kSide + side), slot = __shfl_sync(kFullMask, w.y, j * kSide + side);
                if constexpr (sizeof(T) == 2) {  // a row's width is a multiple of 16 bytes: both quads are there, or none
                    k[j][0] = v[j][0] = k[j][1] = v[j][1] = {};
                    if (page >= 0 && col < D) {
                        quads8(kb + page * a.k_page + slot * a.k_slot, k[j]);
                        quads8(vb + page * a.v_page + slot * a.v_slot, v[j]);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < kQ; ++h) {
                        k[j][h] = v[j][h] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (page >= 0 && there[h]) {
                            k[j][h] = quad4(kb + page * a.k_page + slot * a.k_slot + 128 * h);
                            v[j][h] = quad4(vb + page * a.v_page + slot * a.v_slot + 128 * h);
                        }
                    }
                }
            }
            float s[kR][kLoads];
#pragma unroll
            for (int h = 0; h < kQ; ++h)
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    const float4 y = floats(k[j][h]);
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        const float4 q = queries[r * kRow + h * kLanes + lane % kLanes];
                        const float x = h == 0 ? q.x * y.x : fmaf(q.x, y.x, s[r][j]);
                        s[r][j] = fmaf(q.w, y.w, fmaf(q.z, y.z, fmaf(q.y, y.y, x)));
                    }
                }
            const int key = base + mine * kSide + side;
            float p[kR];
            bool all = true;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int half = kLoads >> (i + 1), mask = kLanes >> (i + 1);
                    const bool upper = lane & mask;
#pragma unroll
                    for (int j = 0; j < half; ++j) {
                        const float give = upper ? s[r][j] : s[r][j + half], keep = upper ? s[r][j + half] : s[r][j];
                        s[r][j] = keep + __shfl_xor_sync(kFullMask, give, mask);
                    }
                }
#pragma unroll
                for (int mask = kLanes >> (kSteps + 1); mask > 0; mask >>= 1) s[r][0] += __shfl_xor_sync(kFullMask, s[r][0], mask);
                const int2 seen = sees[r];
                const bool use = key >= max(lo, seen.x) && key < min(end, seen.y);
                const float x = use ? s[r][0] : -INFINITY;
                if (__any_sync(kFullMask, x > m[r])) {
                    float top = x;
#pragma unroll
                    for (int mask = 16; mask > 0; mask >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, mask));
                    top = fmaxf(top, m[r]);
                    const float f = weight_of(m[r], top, c);
                    m[r] = top;
                    l[r] *= f;
#pragma unroll
                    for (int h = 0; h < kQ; ++h) o[r][h] = scaled(o[r][h], f);
                }
                const float weight = x == -INFINITY ? 0.f : exp2_fast((x - m[r]) * c);
                l[r] += weight;
                p[r] = use ? weight : -1.f;
                all &= use;
            }
            // Keys that a row does not see (-1) are left out, not weighed by 0.
            const auto add_values = [&](auto guard) {
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    int from = side * kLanes;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) from |= (j & (kLoads >> (i + 1))) ? kLanes >> (i + 1) : 0;
                    float4 y[kQ];
#pragma unroll
                    for (int h = 0; h < kQ; ++h) y[h] = floats(v[j][h]);
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        const float pj = __shfl_sync(kFullMask, p[r], from);
                        if (guard && pj < 0.f) continue;
#pragma unroll
                        for (int h = 0; h < kQ; ++h) o[r][h] = add_scaled(o[r][h], y[h], pj);
                    }
                }
            };
            if (__all_sync(kFullMask, all)) add_values(std::false_type());
            else add_values(std::true_type());
        }
        // Keys of a warp's sides, then the warps.
#pragma unroll
        for (int r = 0; r < kR; ++r) {
#pragma unroll
            for (int mask = kLanes; mask < 32; mask <<= 1) {  // kQ is 1 where there are sides
                o[r][0].x += __shfl_xor_sync(kFullMask, o[r][0].x, mask);
                o[r][0].y += __shfl_xor_sync(kFullMask, o[r][0].y, mask);
                o[r][0].z += __shfl_xor_sync(kFullMask, o[r][0].z, mask);
                o[r][0].w += __shfl_xor_sync(kFullMask, o[r][0].w, mask);
            }
#pragma unroll
            for (int mask = 16; mask > 0; mask >>= 1) l[r] += __shfl_xor_sync(kFullMask, l[r], mask);
            l[r] *= (float)kLoads / kLanes;  // each score is in kLanes / kLoads lanes
            if (side == 0)
#pragma unroll
                for (int h = 0; h < kQ; ++h) sums[(warp * kR + r) * kRow + h * kLanes + lane] = o[r][h];
            if (lane == 0) stats[warp * kR + r] = make_float2(m[r], l[r]);
        }
        __syncthreads();
        for (int i = tid; i < kR * kRow; i += kFewThreads) {
            const int r = i / kRow, at = i % kRow, quad = quad_of(at);
            if (r >= g.rows || 4 * quad >= D) continue;
            float top = -INFINITY, sum = 0.f;
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[w * kR + r].x);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < kWarps; ++w) {
                const float2 st = stats[w * kR + r];
                const float f = weight_of(st.x, top, c);
                sum = fmaf(st.y, f, sum);
                x = add_scaled(x, sums[(w * kR + r) * kRow + at], f);
            }
            if (g.part == kPartWhole) {
                store4(scaled(x, sum == 0.f ? 0.f : 1.f / sum), output_of<T>(a, g, r) + 4 * quad);
            } else {
                const long long row = (2LL * blockIdx.x + g.part) * a.part_rows + r;
                store4(x, part_of(a, 2LL * blockIdx.x + g.part, r, quad));
                if (at == 0) *reinterpret_cast<float2*>(a.part_stats + 2 * row) = make_float2(top, sum);
            }
        }
    }
    if (tid == 0) static_cast<PagedMeta*>(a.meta)[blockIdx.x] = walk.meta;
}

// ---------------------------------------------------------------------------
// Joins the parts of items that several CTAs took: CTA (c, y) of this kernel
// takes rows 16·y.. of the item that CTA c began (of the first launch's CTAs, then
// of the second's).  A thread has four columns of a
// row; neighbours have up to 16 rows of the same columns (256 bytes of a part), and
// where that leaves threads idle a row's parts are dealt out to several.
// ---------------------------------------------------------------------------
// Two waves of CTAs where most of 152 items are cut: 4 to 8 us, bound by the latency
// of message and parts.  (8 rows a CTA 54 us for a prompt that takes 48; 32 the same.)
constexpr int kJoinThreads = 256, kJoinRows = 16;

struct JoinSum {
    float2 stat;  // (reference, sum of weights)
    float4 x;
};
// Adds a part to sums with a reference that is no less.  One without a reference
// saw no key (zeros), or only scores of -inf or NaN: an infinity of V under the
// former's weights of 0, and the latter, are NaN in its sums and go on.
__device__ __forceinline__ void add_part(JoinSum& sum, float2 stat, float4 x, float scale_log2) {
    const float w = weight_of(stat.x, sum.stat.x, scale_log2);
    sum.stat.y = fmaf(stat.y, w, sum.stat.y);
    sum.x = add_scaled(sum.x, x, w);
}
__device__ __forceinline__ void raise_reference(JoinSum& sum, float top, float scale_log2) {
    const float f = weight_of(sum.stat.x, top, scale_log2);
    sum.stat = make_float2(top, sum.stat.y * f);
    sum.x = scaled(sum.x, f);
}

// Where a launch leaves its parts, as PagedArgs has it.
struct Parts {
    float *parts, *stats;
    const PagedMeta* meta;
    int rows, ctas;
};
// (An array: two parameters of the struct's type with a choice between them gave wrong
// members with nvcc 13.0.)
struct BothParts {
    Parts launch[2];
};

template <class T>
__global__ void __launch_bounds__(kJoinThreads, 5)
    paged_join_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ BothParts both) {
    constexpr int kAhead = 4;
    __shared__ float4 sums[kJoinThreads];
    __shared__ float2 stats[kJoinThreads];
    await_previous();
    let_next_start();
    const bool later_launch = blockIdx.x >= both.launch[0].ctas;
    const Parts& p = both.launch[later_launch];
    const PagedMeta* meta = p.meta;
    const int c = blockIdx.x - (later_launch ? both.launch[0].ctas : 0), ctas = p.ctas, lane = threadIdx.x & 31;
    const int4 begin = __ldcg(reinterpret_cast<const int4*>(meta + c));  // first_live, start, row0, rows
    const int head = __ldcg(&meta[c].head);
    int2 later = make_int2(0, 1);  // later_live, ends
    if (c + 1 + lane < ctas) later = __ldcg(reinterpret_cast<const int2*>(&meta[c + 1 + lane].later_live));
    const int row_base = blockIdx.y * kJoinRows, rows = min(begin.w - row_base, kJoinRows);
    if (!begin.x || rows <= 0) return;
    const int head0 = head * a.group;
    // The CTAs c + 1 .. c + count hold the rest.
    int count = 0;
#pragma unroll 1
    for (int at = c + 1; at < ctas; at += 32) {
        if (at > c + 1) {
            later = make_int2(0, 1);
            if (at + lane < ctas) later = __ldcg(reinterpret_cast<const int2*>(&meta[at + lane].later_live));
        }
        const unsigned stop = __ballot_sync(kFullMask, !later.x || later.y);
        if (stop) {
            count = min(at + __ffs(stop) - 1, ctas - 1) - c;
            break;
        }
    }
    const int quads = a.head_dim / 4;
    int side = 1;  // rows side by side
    while (side < kJoinRows && side < rows && 2 * side * quads <= kJoinThreads) side *= 2;
    const int each = side * quads, split = min(kJoinThreads / each, count + 1);  // threads of a share; shares
    const int share = threadIdx.x / each, rest = threadIdx.x - share * each, quad = rest / side;
#pragma unroll 1
    for (int r0 = rest - quad * side; r0 - rest + quad * side < rows; r0 += side) {
        const int r = row_base + r0;
        const bool real = share < split && r0 < rows;
        JoinSum sum = {make_float2(-INFINITY, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        if (real) {
#pragma unroll 1
            for (int i0 = share; i0 <= count; i0 += kAhead * split) {
                float2 stat[kAhead];
                float4 x[kAhead];
                float top = sum.stat.x;
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u * split;
                    stat[u] = make_float2(-INFINITY, 0.f);
                    x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i > count) continue;
                    const long long slot = i == 0 ? 2LL * c + kPartFirst : 2LL * (c + i) + kPartLater;
                    stat[u] = __ldcg(reinterpret_cast<const float2*>(p.stats + 2 * (slot * p.rows + r)));
                    x[u] = __ldcg(reinterpret_cast<const float4*>(part_of(p.parts, p.rows, a.head_dim, slot, r, quad)));
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) top = fmaxf(top, stat[u].x);
                raise_reference(sum, top, a.scale_log2);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) add_part(sum, stat[u], x[u], a.scale_log2);
            }
        }
        if (split > 1) {
            __syncthreads();  // the last rows' sums have been read
            sums[threadIdx.x] = sum.x;
            stats[threadIdx.x] = sum.stat;
            __syncthreads();
            if (share == 0 && real) {
                float top = sum.stat.x;
                for (int u = 1; u < split; ++u) top = fmaxf(top, stats[threadIdx.x + u * each].x);
                raise_reference(sum, top, a.scale_log2);
                for (int u = 1; u < split; ++u) add_part(sum, stats[threadIdx.x + u * each], sums[threadIdx.x + u * each], a.scale_log2);
            }
        }
        if (share > 0 || !real) continue;
        const int flat = begin.z + r, token = by_group(a, flat);
        T* out = (T*)a.out + (begin.y + token) * a.out_token + (head0 + flat - token * a.group) * a.out_head;
        store4(scaled(sum.x, sum.stat.y == 0.f ? 0.f : 1.f / sum.stat.y), out + 4 * quad);
    }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
enum class Form { None, Mma, Block, Few1, Few2, Few4, Few8 };
struct Launch {
    Form form;
    int rows;  // of a block
    int ctas;
    int least, most;  // rows of the sequences that it takes
};
struct Plan {
    Launch first, second;
};
constexpr int kAll = 0x7fffffff, kFewRows = 8;

// bf16 heads of up to 128 columns go to the matrix kernel.  Of the others, sequences with
// up to 8 rows a head of keys are read by few rows at a time: from 9 on the keys
// would be read twice, and the block kernel is as fast.  (Wider heads have room for 4
// rows: they read the keys of 5 to 8 twice, where the block kernel would fill 8 of
// its 64 rows.)  With `equal` shares of tokens all sequences are of one kind; else how many
// tokens each brings is known on the device only, and both kernels are launched, each
// for its own, which costs 3 us where one finds none.  (By the average alone a
// chunk's tokens among idle sequences went through the cache a few rows at a time, and
// single tokens beside a chunk took a block of 64 rows each: a chunk of 1000 beside 16
// tokens over 4096 fp32 keys of 128 columns, 16/2 heads, 964 us, now 736; one of 256 beside
// 63, 16/8 heads of 192 bf16 columns, 4690 us, now 963.)
Plan plan_of(int tokens, int num_seqs, int q_heads, int kv_heads, int head_dim, bool bf16, bool equal) {
    const int sms = sm_count_current_device(), group = q_heads / kv_heads;
    if (bf16 && head_dim <= 128) return {{Form::Mma, paged_mma_rows(), sms, 0, kAll}, {}};
    const long long all = (long long)tokens * group;
    // Rows of a sequence: at most, and on average of those that bring any (one brings a token's at least).
    const long long most = equal ? all / num_seqs : all, average = std::max<long long>(group, (all + num_seqs - 1) / num_seqs);
    Launch few = {Form::Few8, 8, 2 * sms, 0, kAll};
    if (average <= 1) few.form = Form::Few1, few.rows = 1;
    else if (average <= 2) few.form = Form::Few2, few.rows = 2;
    else if (average <= 4 || head_dim > 128) few.form = Form::Few4, few.rows = 4;
    if (most <= kFewRows) return {few, {}};
    const int fit = std::max(1, std::min(2, 220 * 1024 / block_smem(head_dim)));
    Launch block = {Form::Block, kBlockRows, fit * sms, 0, kAll};
    if (equal || group > kFewRows) return {block, {}};
    block.least = kFewRows + 1;
    few.most = kFewRows;
    return {block, few};
}

template <class T, int kWide>
int run_block(PagedArgs a, int ctas, cudaStream_t stream) {
    const auto kernel = paged_block_kernel<T, kWide>;
    const int smem = block_smem(a.head_dim);
    static SharedOnce once;
    if (!once.allow(kernel, block_smem(32 * kWide))) return cuda_failure();
    return launch_next_shared(kernel, dim3(ctas), kBlockThreads, smem, stream, a);
}

template <class T, int kLanes, int kQ, int kR>
int run_few(const PagedArgs& a, int ctas, cudaStream_t stream) {
    const auto kernel = paged_few_kernel<T, kLanes, kQ, kR>;
    constexpr int smem = kR * kLanes * kQ * 16 + kFewThreads / 32 * kR * (kLanes * kQ * 16 + 8);
    static SharedOnce once;
    if (!once.allow(kernel, smem)) return cuda_failure();
    return launch_next_shared(kernel, dim3(ctas), kFewThreads, smem, stream, a);
}
template <int kR>
int run_few(const PagedArgs& a, bool bf16, int ctas, cudaStream_t stream) {
    if constexpr (kR <= 4) {
        if (bf16) return run_few<__nv_bfloat16, 32, 2, kR>(a, ctas, stream);
        if (a.head_dim > 128) return run_few<float, 32, 2, kR>(a, ctas, stream);
    }
    if (a.head_dim <= 32) return run_few<float, 8, 1, kR>(a, ctas, stream);
    return a.head_dim <= 64 ? run_few<float, 16, 1, kR>(a, ctas, stream) : run_few<float, 32, 1, kR>(a, ctas, stream);
}
template <class T>
int run_block(const PagedArgs& a, int ctas, cudaStream_t stream) {
    if constexpr (std::is_same_v<T, float>) {  // bf16 of up to 128 columns: the matrix kernel
        if (a.head_dim <= 32) return run_block<T, 1>(a, ctas, stream);
        if (a.head_dim <= 64) return run_block<T, 2>(a, ctas, stream);
        if (a.head_dim <= 96) return run_block<T, 3>(a, ctas, stream);
        if (a.head_dim <= 128) return run_block<T, 4>(a, ctas, stream);
    }
    if (a.head_dim <= 160) return run_block<T, 5>(a, ctas, stream);
    if (a.head_dim <= 192) return run_block<T, 6>(a, ctas, stream);
    return a.head_dim <= 224 ? run_block<T, 7>(a, ctas, stream) : run_block<T, 8>(a, ctas, stream);
}

template <class T>
int join(const PagedArgs& a, const BothParts& both, cudaStream_t stream) {
    const auto kernel = paged_join_kernel<T>;
    // The same split of an SM's memory as the kernel before it has: to change it the
    // SM would have to drain.
    static SharedOnce once;
    if (!once.allow(kernel, 0)) return cuda_failure();
    const auto& [first, second] = both.launch;
    const int rows = std::max(first.rows, second.rows);
    return launch_next(kernel, dim3(first.ctas + second.ctas, (rows + kJoinRows - 1) / kJoinRows), kJoinThreads, 1, stream, a, both);
}

size_t meta_bytes(int ctas) { return ((size_t)ctas * sizeof(PagedMeta) + 15) / 16 * 16; }

// Rows of a launch's parts, of sequences with `rows` at most; bytes of its workspace.
int part_rows(const Launch& s, long long rows) { return (int)std::min<long long>(s.rows, std::min<long long>(s.most, rows)); }
size_t launch_bytes(const Launch& s, long long rows, int head_dim) {
    if (s.form == Form::None) return 0;
    const size_t parts = (size_t)2 * s.ctas * part_rows(s, rows);
    return meta_bytes(s.ctas) + (parts * (head_dim + 2) * 4 + 15) / 16 * 16;
}

int launch(const Launch& s, const PagedArgs& a, bool bf16, cudaStream_t stream) {
    switch (s.form) {
        case Form::Mma: return launch_paged_mma(a, s.ctas, stream);
        case Form::Few1: return run_few<1>(a, bf16, s.ctas, stream);
        case Form::Few2: return run_few<2>(a, bf16, s.ctas, stream);
        case Form::Few4: return run_few<4>(a, bf16, s.ctas, stream);
        case Form::Few8: return run_few<8>(a, bf16, s.ctas, stream);
        default: return bf16 ? run_block<__nv_bfloat16>(a, s.ctas, stream) : run_block<float>(a, s.ctas, stream);
    }
}

}  // namespace

size_t paged_attention_workspace(int tokens, int num_seqs, int q_heads, int kv_heads, int head_dim, bool bf16, bool equal) {
    const Plan p = plan_of(tokens, num_seqs, q_heads, kv_heads, head_dim, bf16, equal);
    const long long rows = (long long)(equal ? tokens / num_seqs : tokens) * (q_heads / kv_heads);
    return launch_bytes(p.first, rows, head_dim) + launch_bytes(p.second, rows, head_dim);
}

int launch_paged_attention(PagedArgs a, bool bf16, void* workspace, cudaStream_t stream) {
    const bool equal = !a.q_offsets;
    const Plan p = plan_of(a.tokens, a.num_seqs, a.kv_heads * a.group, a.kv_heads, a.head_dim, bf16, equal);
    const long long rows = (long long)(equal ? a.per_seq : a.tokens) * a.group;
    BothParts both = {};
    char* at = static_cast<char*>(workspace);
    for (const Launch* s : {&p.first, &p.second}) {
        if (s->form == Form::None) continue;
        a.least_rows = s->least;
        a.most_rows = s->most;
        a.part_rows = part_rows(*s, rows);
        a.meta = at;
        a.parts = reinterpret_cast<float*>(at + meta_bytes(s->ctas));
        a.part_stats = a.parts + (size_t)2 * s->ctas * a.part_rows * a.head_dim;
        both.launch[s == &p.second] = {a.parts, a.part_stats, static_cast<const PagedMeta*>(a.meta), a.part_rows, s->ctas};
        if (const int code = launch(*s, a, bf16, stream); code != USM_OK) return code;
        at += launch_bytes(*s, rows, a.head_dim);
    }
    return bf16 ? join<__nv_bfloat16>(a, both, stream) : join<float>(a, both, stream);
}

}  // namespace usm
