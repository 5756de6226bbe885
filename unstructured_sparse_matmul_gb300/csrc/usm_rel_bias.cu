// Learned relative position bias of sparse attention, by buckets, and its
// gradient:
//     out[p] = s[p] + T[h][bucket(p)],     dT[h][k] = Σ_{p of head h, bucket(p) = k} dS[p],
// bucket(p) = map[reach + clamp(d, ±reach)], d the key's position less the
// query's.
#include "usm_internal.h"
#include "usm_rel.cuh"
#include "usm_sums.cuh"

namespace usm {
namespace {

__global__ void rel_bucket_kernel(int num_buckets, int reach, int causal, int* __restrict__ map) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i > 2 * reach) return;
    const int d = i - reach;
    const int b = causal ? num_buckets : num_buckets / 2;
    const int n = causal ? max(-d, 0) : abs(d);
    const int e = b / 2;
    int k = n;
    if (n >= e) {
        const double x = log((double)n / e) / log((double)reach / e) * (b - e);
        k = min(b - 1, e + (int)floor(x + 1e-9));
    }
    map[i] = k + (!causal && d > 0 ? b : 0);
}

constexpr int kThreads = 256, kCtas = 3;  // an SM's CTAs (80 registers a thread hold a tile and the walk)
constexpr int kSteps = 4;             // quads of entries a lane has in flight
constexpr int kTile = kSteps * 128;   // entries of a warp's tile

// Entries of a tile in a warp's registers: lane l has entries 128·i + 4·l + u.
// `limit`: entries before it exist (others read as 0).  vec: the array starts on a
// whole quad.  Plain loads of values: the same kernel may write them in place.
template <bool BF>
__device__ __forceinline__ void load_values(const void* p, unsigned tile, unsigned limit, bool vec, int lane,
                                            float (&x)[kSteps][4]) {
    if (vec && tile + kTile <= limit) {
        const char* q = static_cast<const char*>(p) + (size_t)(tile + 4 * lane) * (BF ? 2 : 4);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if constexpr (BF) {
                const uint2 w = *reinterpret_cast<const uint2*>(q + i * 256);
                x[i][0] = __uint_as_float(w.x << 16);
                x[i][1] = __uint_as_float(w.x & 0xffff0000u);
                x[i][2] = __uint_as_float(w.y << 16);
                x[i][3] = __uint_as_float(w.y & 0xffff0000u);
            } else {
                const float4 w = *reinterpret_cast<const float4*>(q + i * 512);
                x[i][0] = w.x;
                x[i][1] = w.y;
                x[i][2] = w.z;
                x[i][3] = w.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const unsigned e = tile + 128 * i + 4 * lane + u;
                if constexpr (BF)
                    x[i][u] = e < limit ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[e] << 16) : 0.f;
                else
                    x[i][u] = e < limit ? static_cast<const float*>(p)[e] : 0.f;
            }
    }
}
__device__ __forceinline__ void load_columns(const int* __restrict__ ci, unsigned tile, unsigned limit, bool vec, int lane,
                                             int (&c)[kSteps][4]) {
    if (vec && tile + kTile <= limit) {
        const int4* q = reinterpret_cast<const int4*>(ci + tile) + lane;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int4 w = __ldg(q + 32 * i);
            c[i][0] = w.x;
            c[i][1] = w.y;
            c[i][2] = w.z;
            c[i][3] = w.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const unsigned e = tile + 128 * i + 4 * lane + u;
                c[i][u] = e < limit ? __ldg(ci + e) : 0;
            }
    }
}

// Asks L2 for a tile's lines (a lane each), while the warp works on the one before.
template <int E>
__device__ __forceinline__ void prefetch_tile(const int* ci, const void* values, unsigned tile, unsigned limit, int lane) {
    constexpr int kLine = 128 / E;
    const unsigned e = lane < 16 ? tile + 32 * lane : tile + kLine * (lane - 16);
    if (e < limit && e < tile + kTile) {
        const void* at = lane < 16 ? static_cast<const void*>(ci + e) : static_cast<const char*>(values) + (size_t)e * E;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
    }
}

// Walks the rows with entries in [p, end) of rows [r, r1).  Lane i holds row
// `first + i`'s offset (31 rows; lane 31 only ends the last), and whatever
// made(row, whether it counts) keeps of it when other rows come to be held.
struct RowWalk {
    const int* ro;
    int r1, nnz, lane;
    unsigned end;
    int first, offset;
    unsigned left;   // held rows from the current one on
    int at;          // lane that holds the current row
    unsigned begin;  // where it begins; past `end` if there is none

    __device__ __forceinline__ void load() {
        offset = min(max(__ldg(ro + min((long long)first + lane, (long long)r1)), 0), nnz);
    }
    // Holds the row that entry p lies in, found among rows [r, r1) by 128 candidates
    // a round.
    __device__ __forceinline__ void find(unsigned p, int r) {
        long long lo = r, n = (long long)r1 - r;
        while (n > 31) {
            const long long step = (n + 127) / 128;
            int tried[4], below = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const long long i = (lane + 32 * k) * step;
                tried[k] = i < n ? __ldg(ro + lo + i) : 0x7fffffff;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) below += __popc(__ballot_sync(kFullMask, tried[k] <= (long long)p));
            const long long skip = max(below - 1, 0) * step;
            lo += skip;
            n = min(step, n - skip);
        }
        first = (int)lo;
        load();
    }
    template <class Made>
    __device__ __forceinline__ void hold(unsigned p, Made made) {
        const unsigned next = __shfl_down_sync(kFullMask, offset, 1);
        const bool some = lane < min(31, r1 - first) && next > (unsigned)offset && next > p;
        made((int)((unsigned)first + lane), some);
        left = __ballot_sync(kFullMask, some);
    }
    template <class Made>
    __device__ __forceinline__ void settle(Made made) {
        while (left == 0) {
            const unsigned p = __shfl_sync(kFullMask, offset, 31);
            if (r1 - first <= 31 || p >= end) {
                begin = 0xffffffffu;
                return;
            }
            first += 31;
            load();
            if ((unsigned)__shfl_sync(kFullMask, offset, 31) <= p && r1 - first > 31) find(p, first);  // rows without entries
            hold(p, made);
        }
        at = __ffs(left) - 1;
        begin = __shfl_sync(kFullMask, offset, at);
    }
    template <class Made>
    __device__ __forceinline__ void start(unsigned p, int r, Made made) {
        find(p, r);
        hold(p, made);
        settle(made);
    }
    template <class Made>
    __device__ __forceinline__ void next(Made made) {
        left &= left - 1;
        settle(made);
    }
};

// Where a column's distance lies in the map: at its start or before (entry 0: every
// key further back), between, or at its end or after (the last entry).
struct Distance {
    bool back, between;
    unsigned entry;
    __device__ __forceinline__ Distance(int col, int start, unsigned last) {
        entry = (unsigned)col - (unsigned)start;
        back = col <= start;
        between = !back && entry < last;
    }
};

// Bound by memory: 8 bytes a nonzero in, 4 out.  Warp w of W takes an equal share
// of the entries, whatever rows they are in, a tile at a time; the search for the
// first tile's rows runs while its loads are in flight.  Most keys are further
// away than the map reaches, and those have one of two values; only groups of 128
// entries that have others look up the map and the table.  8x4096 rows of 410
// entries (161 MB): 37 us in a replayed graph, 6.3 TB/s for every further row; a
// warp to a row took 46, as did 4 CTAs an SM, whose 64 registers spill.
template <bool BT>
__global__ void __launch_bounds__(kThreads, kCtas)
    rel_bias_kernel(int M, int nnz, const int* __restrict__ ro, const int* __restrict__ ci, const float* s,
                    const RelArgs b, float* out, int W, bool vec) {
    const int lane = threadIdx.x & 31, w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (w >= W) return;
    const unsigned quads = ((unsigned)nnz + 3) / 4;
    const unsigned q0 = 4 * (unsigned)((unsigned long long)quads * w / W);
    const unsigned q1 = min((unsigned)nnz, 4 * (unsigned)((unsigned long long)quads * (w + 1) / W));
    const unsigned all0 = min(max(__ldg(ro), 0), nnz), all1 = min(max(__ldg(ro + M), 0), nnz);
    const unsigned p0 = max(q0, all0), p1 = min(q1, all1);
    if (p0 >= p1) return;
    const unsigned last = 2u * (unsigned)b.reach;
    const int bucket0 = rel_bucket(b, 0), bucket1 = rel_bucket(b, (int)last);
    auto table_of = [&](int head) { return static_cast<const char*>(b.table) + (long long)head * b.buckets * (BT ? 2 : 4); };
    RowWalk rows{ro, M, nnz, lane, p1, 0, 0, 0, 0, 0};
    int row_start = 0, row_head = 0;
    auto made = [&](int r, bool some) {
        if (!some) return;
        const int block = r / b.seg_rows;
        row_head = block % b.heads;
        row_start = rel_start(b, block, r - block * b.seg_rows, b.seg_cols > 0 ? __ldg(ci + rows.offset) : 0);
    };
    // The current row's, and its head's.
    int start = 0, head = -1;
    const char* table = nullptr;
    float back = 0.f, ahead = 0.f;
    auto enter = [&]() {
        const int h = __shfl_sync(kFullMask, row_head, rows.at);
        start = __shfl_sync(kFullMask, row_start, rows.at);
        if (h != head) {
            head = h;
            table = table_of(h);
            back = rel_table_entry<BT>(table, bucket0);
            ahead = rel_table_entry<BT>(table, bucket1);
        }
        rows.next(made);
    };
    bool found = false;
#pragma unroll 1
    for (unsigned tile = p0 & ~3u; tile < p1; tile += kTile) {
        int c[kSteps][4];
        float x[kSteps][4];
        load_columns(ci, tile, p1, vec, lane, c);
        load_values<false>(s, tile, p1, vec, lane, x);
        prefetch_tile<4>(ci, s, tile + kTile, p1, lane);
        if (!found) {
            rows.start(p0, 0, made);
            if (rows.begin == 0xffffffffu) return;
            enter();
            found = true;
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const unsigned g = tile + 128 * k, q = g + 4 * lane;
            unsigned lo = g;
            bool more;
            do {  // a head's part of the group (nearly always all of it)
                int from[4] = {start, start, start, start};
                more = false;
                while (rows.begin < g + 128) {
                    if (__shfl_sync(kFullMask, row_head, rows.at) != head) {
                        more = true;
                        break;
                    }
                    const unsigned begin = rows.begin;
                    enter();
#pragma unroll
                    for (int u = 0; u < 4; ++u) from[u] = q + u >= begin ? start : from[u];
                }
                const unsigned n = (more ? rows.begin : g + 128) - lo;
                bool any = false, between[4];
                unsigned entry[4];
                float v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const Distance d(c[k][u], from[u], last);
                    v[u] = d.back ? back : ahead;
                    any = any || d.between;
                    between[u] = d.between;
                    entry[u] = d.entry;
                }
                if (__any_sync(kFullMask, any)) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float near = rel_table_entry<BT>(table, rel_bucket(b, between[u] ? (int)entry[u] : 0));
                        v[u] = between[u] ? near : v[u];
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (q + u - lo < n) x[k][u] += v[u];
                lo += n;
                if (more) enter();
            } while (more);
        }
        if (vec && p0 <= tile && tile + kTile <= p1) {
            float4* to = reinterpret_cast<float4*>(out + tile) + lane;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) to[32 * i] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const unsigned e = tile + 128 * i + 4 * lane + u;
                    if (e >= p0 && e < p1) out[e] = x[i][u];
                }
        }
    }
}

// Head h's entries lie in runs, one a query block; each is cut into Y parts at
// quads, and warp w of the W that CTAs (h, 0) .. (h, J - 1) have takes its equal
// share of the parts.  Every thread sums its entries into its own column of a
// histogram in shared memory ([bucket][thread]: no bank conflicts, no atomics),
// those further away than the map reaches into two sums beside it, and the columns
// are added in a fixed order: which thread takes which entry is fixed too.  The two
// sums get a tile's share at a time and keep what is rounded off (0.3 of 33 us;
// 900 equal entries a thread were off by 8e-6 without, 1e-6 is the bound now).  Bound by
// memory: 8 (or 6) bytes a nonzero.  8x4096 rows of 410 entries in bf16 (81 MB):
// 33 us with the sum of the parts; a warp to a row, a look-up for every entry, 57.
template <bool BF>
__global__ void __launch_bounds__(kThreads, kCtas)
    rel_bias_grad_kernel(int M, int nnz, const int* __restrict__ ro, const int* __restrict__ ci,
                         const void* __restrict__ ds, const RelArgs b, int blocks, int Y, int J, float* __restrict__ part,
                         bool vec) {
    extern __shared__ float hist[];
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = T >> 5;
    for (int k = 0; k < b.buckets; ++k) hist[k * T + t] = 0.f;
    const int head = blockIdx.x / J;
    const long long W = (long long)J * warps, w = (long long)(blockIdx.x % J) * warps + warp;
    const long long parts = head < blocks ? ((blocks - 1 - head) / b.heads + 1LL) * Y : 0;
    const unsigned last = 2u * (unsigned)b.reach;
    LongSum back_sum, ahead_sum;
#pragma unroll 1
    for (long long i = parts * w / W; i < parts * (w + 1) / W; ++i) {
        const int block = (int)(head + i / Y * b.heads), y = (int)(i % Y), r0 = block * b.seg_rows;
        const int r1 = (int)min((long long)M, (long long)r0 + b.seg_rows);
        const unsigned e0 = min(max(__ldg(ro + r0), 0), nnz), e1 = min(max(__ldg(ro + r1), 0), nnz);
        if (e0 >= e1) continue;
        const unsigned f = e0 & ~3u, quads = (e1 - f + 3) / 4;
        const unsigned p0 = max(e0, f + 4 * (unsigned)((unsigned long long)quads * y / Y));
        const unsigned p1 = min(e1, f + 4 * (unsigned)((unsigned long long)quads * (y + 1) / Y));
        if (p0 >= p1) continue;
        RowWalk rows{ro, r1, nnz, lane, p1, 0, 0, 0, 0, 0};
        int row_start = 0, start = 0;
        auto made = [&](int r, bool some) {
            if (some) row_start = rel_start(b, block, r - r0, b.seg_cols > 0 ? __ldg(ci + rows.offset) : 0);
        };
        auto enter = [&]() {
            start = __shfl_sync(kFullMask, row_start, rows.at);
            rows.next(made);
        };
        bool found = false;
#pragma unroll 1
        for (unsigned tile = p0 & ~3u; tile < p1; tile += kTile) {
            int c[kSteps][4];
            float x[kSteps][4];
            load_columns(ci, tile, p1, vec, lane, c);
            load_values<BF>(ds, tile, p1, vec, lane, x);
            prefetch_tile<BF ? 2 : 4>(ci, ds, tile + kTile, p1, lane);
            if (!found) {
                rows.start(p0, r0, made);
                if (rows.begin == 0xffffffffu) break;
                enter();
                found = true;
#pragma unroll
                for (int u = 0; u < 3; ++u)
                    if (tile + 4 * lane + u < p0) x[0][u] = 0.f;
            }
            float back = 0.f, ahead = 0.f;  // the tile's
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const unsigned g = tile + 128 * k, q = g + 4 * lane;
                int from[4] = {start, start, start, start};
                while (rows.begin < g + 128) {
                    const unsigned begin = rows.begin;
                    enter();
#pragma unroll
                    for (int u = 0; u < 4; ++u) from[u] = q + u >= begin ? start : from[u];
                }
                bool any = false, between[4];
                unsigned entry[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const Distance d(c[k][u], from[u], last);
                    if (d.back) back += x[k][u];
                    if (!d.back && !d.between) ahead += x[k][u];
                    any = any || d.between;
                    between[u] = d.between;
                    entry[u] = d.entry;
                }
                if (__any_sync(kFullMask, any)) {
                    int at[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) at[u] = rel_bucket(b, between[u] ? (int)entry[u] : 0) * T + t;
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (between[u]) hist[at[u]] += x[k][u];
                }
            }
            back_sum.add(back);
            ahead_sum.add(ahead);
        }
    }
    hist[rel_bucket(b, 0) * T + t] += back_sum.value();
    hist[rel_bucket(b, (int)last) * T + t] += ahead_sum.value();
    __syncthreads();
    for (int k = warp; k < b.buckets; k += warps) {
        float x = 0.f;
        for (int c = lane; c < T; c += 32) x += hist[k * T + c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
        if (lane == 0) part[(long long)blockIdx.x * b.buckets + k] = x;
    }
}

// dT[h][k] = Σ_j part[h][j][k]: a warp for each (h, k), or for several in large tables.
__global__ void rel_bias_grad_sum_kernel(int heads, int buckets, int J, const float* __restrict__ part,
                                         float* __restrict__ dtable) {
    const int lane = threadIdx.x & 31;
    const long long n = (long long)heads * buckets, step = (long long)gridDim.x * blockDim.x >> 5;
    for (long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < n; i += step) {
        const long long h = i / buckets, k = i % buckets;
        LongSum x;
        for (int j = lane; j < J; j += 32) x.add(part[(h * J + j) * buckets + k]);
        x = x.over_warp();
        if (lane == 0) dtable[i] = x.value();
    }
}

// Threads of a gradient CTA (its histogram is threads × buckets floats, 64 KB
// at most).
int grad_threads(int buckets) { return buckets <= 64 ? 256 : buckets <= 128 ? 128 : buckets <= 256 ? 64 : 32; }

// The gradient's split: CTAs a head, three an SM (of 152) in all or fewer where
// their warps would have less than a tile of entries each, and parts a query
// block, as many as give every warp one.
struct GradSplit {
    int Y, J;
};
GradSplit grad_split(int M, int nnz, int seg_rows, int heads, int buckets) {
    const int warps = grad_threads(buckets) / 32;
    // Query blocks of the first head, which has the most.
    const long long blocks = M > 0 ? ((long long)query_blocks(M, seg_rows) + heads - 1) / heads : 1;
    const long long most = (455LL + heads) / heads * warps, some = nnz / (heads * (long long)kTile) + 1;
    const long long parts = most < some ? most : some;
    GradSplit split;
    split.Y = (int)((parts + blocks - 1) / blocks);
    const long long all = blocks * split.Y, W = all < most ? all : most;
    split.J = (int)((W + warps - 1) / warps);
    return split;
}

}  // namespace

int launch_rel_bucket_build(int num_buckets, int max_distance, bool causal, int* bucket_map, cudaStream_t stream) {
    rel_bucket_kernel<<<(2 * max_distance + 1 + 127) / 128, 128, 0, stream>>>(num_buckets, max_distance, causal ? 1 : 0,
                                                                            bucket_map);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

namespace {
bool quad_aligned(const void* p, bool bf16 = false) { return (reinterpret_cast<uintptr_t>(p) & (bf16 ? 7u : 15u)) == 0; }

template <bool BT>
void launch_bias(int M, int nnz, const int* ro, const int* ci, const float* scores, const RelArgs& bias, float* out,
                 cudaStream_t stream) {
    const bool vec = quad_aligned(ci) && quad_aligned(scores) && quad_aligned(out);
    // A warp has half a tile or more.
    const int most = sm_count_current_device() * kCtas * (kThreads / 32), some = nnz / (kTile / 2) + 1;
    const int W = some < most ? some : most;
    rel_bias_kernel<BT>
        <<<(W + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, stream>>>(M, nnz, ro, ci, scores, bias, out, W, vec);
}
}  // namespace

int launch_rel_bias(int M, int nnz, const int* ro, const int* ci, const float* scores, const RelArgs& bias, float* out,
                    cudaStream_t stream) {
    if (bias.table_bf16)
        launch_bias<true>(M, nnz, ro, ci, scores, bias, out, stream);
    else
        launch_bias<false>(M, nnz, ro, ci, scores, bias, out, stream);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

size_t rel_bias_grad_workspace_bytes(int M, int nnz, int seg_rows, int num_heads, int num_buckets) {
    return (size_t)num_heads * grad_split(M, nnz, seg_rows, num_heads, num_buckets).J * num_buckets * 4;
}

namespace {
template <bool BF>
int launch_grad(int M, int nnz, const int* ro, const int* ci, const void* ds, const RelArgs& bias, float* dtable,
                void* workspace, cudaStream_t stream) {
    const auto [Y, J] = grad_split(M, nnz, bias.seg_rows, bias.heads, bias.buckets);
    const int T = grad_threads(bias.buckets);
    const int smem = bias.buckets * T * 4;
    if (!allow_shared(rel_bias_grad_kernel<BF>, smem)) return cuda_failure();
    float* part = static_cast<float*>(workspace);
    rel_bias_grad_kernel<BF><<<bias.heads * J, T, smem, stream>>>(
        M, nnz, ro, ci, ds, bias, query_blocks(M, bias.seg_rows), Y, J, part,
        quad_aligned(ci) && quad_aligned(ds, BF));
    const long long ctas = ((long long)bias.heads * bias.buckets + 7) / 8;
    rel_bias_grad_sum_kernel<<<(unsigned)(ctas < 1 << 20 ? ctas : 1 << 20), 256, 0, stream>>>(bias.heads, bias.buckets, J,
                                                                                              part, dtable);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}
}  // namespace

int launch_rel_bias_grad(int M, int nnz, const int* ro, const int* ci, const void* dscores, bool bf16,
                         const RelArgs& bias, float* dtable, void* workspace, cudaStream_t stream) {
    const auto launch = bf16 ? launch_grad<true> : launch_grad<false>;
    return launch(M, nnz, ro, ci, dscores, bias, dtable, workspace, stream);
}

}  // namespace usm
