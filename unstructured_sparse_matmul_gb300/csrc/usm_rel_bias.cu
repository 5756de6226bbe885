// Learned relative position bias of sparse attention, by buckets, and its
// gradient:
//     out[p] = s[p] + T[h][bucket(p)],     dT[h][k] = Σ_{p of head h, bucket(p) = k} dS[p],
// bucket(p) = map[reach + clamp(d, ±reach)], d the key's position less the
// query's.
#include "usm_internal.h"
#include "usm_rel.cuh"

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

constexpr int kThreads = 256;
constexpr int kSteps = 4;             // quads of entries a lane has in flight
constexpr int kTile = kSteps * 128;   // entries of a warp's tile

// Four entries from q on (one by one where the array does not start on a quad or
// ends inside it).  Plain loads: the same kernel may write the array in place.
template <bool BF>
__device__ __forceinline__ float load_value(const void* p, unsigned i) {
    if constexpr (BF) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
    return static_cast<const float*>(p)[i];
}
template <bool BF>
__device__ __forceinline__ void load_values(const void* p, unsigned q, unsigned nnz, bool vec, float (&x)[4]) {
    if (vec && q + 4 <= nnz) {
        if constexpr (BF) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + q);
            x[0] = __uint_as_float(w.x << 16);
            x[1] = __uint_as_float(w.x & 0xffff0000u);
            x[2] = __uint_as_float(w.y << 16);
            x[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + q);
            x[0] = w.x;
            x[1] = w.y;
            x[2] = w.z;
            x[3] = w.w;
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = q + u < nnz ? load_value<BF>(p, q + u) : 0.f;
    }
}
__device__ __forceinline__ void load_columns(const int* __restrict__ ci, unsigned q, unsigned nnz, bool vec, int (&c)[4]) {
    if (vec && q + 4 <= nnz) {
        const int4 w = __ldg(reinterpret_cast<const int4*>(ci + q));
        c[0] = w.x;
        c[1] = w.y;
        c[2] = w.z;
        c[3] = w.w;
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) c[u] = q + u < nnz ? __ldg(ci + q + u) : 0;
    }
}

// The rows of a run of entries: lane i holds row `first + i`'s offset and what a
// functor makes of the row (31 rows; lane 31 only ends the last).
struct RowsHeld {
    const int* ro;
    int r1;  // rows before this one
    int nnz, lane;
    int first, offset;

    __device__ __forceinline__ int load(int r) const {
        return min(max(__ldg(ro + min((long long)r + lane, (long long)r1)), 0), nnz);
    }
    // Holds the row that entry p lies in, found among rows [r, r1) by 128 candidates
    // a round.
    __device__ __forceinline__ void find(unsigned p, int r) {
        long long lo = r, n = (long long)r1 - r;
        while (n > 31) {
            const long long step = (n + 127) / 128;
            int at[4], below = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const long long i = (lane + 32 * k) * step;
                at[k] = i < n ? __ldg(ro + lo + i) : 0x7fffffff;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) below += __popc(__ballot_sync(kFullMask, at[k] <= (long long)p));
            const long long skip = max(below - 1, 0) * step;
            lo += skip;
            n = min(step, n - skip);
        }
        first = (int)lo;
        offset = load(first);
    }
    // Calls f(lane that holds the row, begin, end) for each row's part of entries
    // [p, end), which come after what was asked for before.  fresh: other rows are
    // held than made(row, whether it has entries) was last called for.
    template <class Made, class F>
    __device__ __forceinline__ void segments(unsigned p, unsigned end, bool& fresh, Made made, F f) {
        while (true) {
            const unsigned next = __shfl_down_sync(kFullMask, offset, 1);
            const bool row = lane < min(31, r1 - first);
            if (fresh) made(first + lane, row && next > (unsigned)offset);
            fresh = false;
            unsigned left = __ballot_sync(kFullMask, row && next > max((unsigned)offset, p) && (unsigned)offset < end);
            for (; left; left &= left - 1) {
                const int i = __ffs(left) - 1;
                f(i, max((unsigned)__shfl_sync(kFullMask, offset, i), p), min(__shfl_sync(kFullMask, next, i), end));
            }
            const unsigned held = __shfl_sync(kFullMask, offset, 31);
            if (held >= end || r1 - first <= 31) return;
            p = max(p, held);
            first += 31;
            offset = load(first);
            fresh = true;
            if ((unsigned)__shfl_sync(kFullMask, offset, 31) <= p && r1 - first > 31) find(p, first);  // rows without entries
        }
    }
};

// Where column col's distance lies in the map: before or at its start (entry 0:
// every key further back), at its end or after (the last entry), or between.
struct Distance {
    bool back, between;
    unsigned entry;
    __device__ __forceinline__ Distance(int col, int start, unsigned last) {
        entry = (unsigned)col - (unsigned)start;
        back = col <= start;
        between = !back && entry < last;
    }
};

// Bound by memory: 8 bytes a nonzero in, 4 out.  A warp takes a tile of entries,
// whatever rows they are in: its loads go out first, and the search for the
// tile's rows runs while they are in flight.  Each row's part of the tile then
// gets its bias: most keys are further away than the map reaches, and those have
// one of two values that the row's lane holds; only the others look up the map
// and the table.
template <bool BT>
__global__ void __launch_bounds__(kThreads) rel_bias_kernel(int M, int nnz, const int* __restrict__ ro,
                                                            const int* __restrict__ ci, const float* s, const RelArgs b,
                                                            float* out, bool vec) {
    const int lane = threadIdx.x & 31;
    const unsigned tile = (blockIdx.x * (unsigned)(kThreads / 32) + (threadIdx.x >> 5)) * (unsigned)kTile;
    if (tile >= (unsigned)nnz) return;
    int c[kSteps][4];
    float x[kSteps][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        load_columns(ci, tile + 128 * i + 4 * lane, nnz, vec, c[i]);
        load_values<false>(s, tile + 128 * i + 4 * lane, nnz, vec, x[i]);
    }
    const unsigned all0 = min(max(__ldg(ro), 0), nnz), all1 = min(max(__ldg(ro + M), 0), nnz);
    const unsigned p0 = max(tile, all0), p1 = min(tile + kTile, all1);
    if (p0 >= p1) return;
    RowsHeld rows{ro, M, nnz, lane, 0, 0};
    rows.find(p0, 0);
    const unsigned last = 2u * (unsigned)b.reach;
    const int bucket0 = rel_bucket(b, 0), bucket1 = rel_bucket(b, (int)last);
    int start = 0, head = 0;
    float back = 0.f, ahead = 0.f;
    bool fresh = true;
    rows.segments(
        p0, p1, fresh,
        [&](int r, bool some) {
            if (!some) return;
            const int block = r / b.seg_rows;
            head = block % b.heads;
            start = rel_start(b, block, r - block * b.seg_rows, b.seg_cols > 0 ? __ldg(ci + rows.offset) : 0);
            const char* table = static_cast<const char*>(b.table) + (long long)head * b.buckets * (BT ? 2 : 4);
            back = rel_table_entry<BT>(table, bucket0);
            ahead = rel_table_entry<BT>(table, bucket1);
        },
        [&](int i, unsigned s0, unsigned s1) {
            const int from = __shfl_sync(kFullMask, start, i);
            const float far0 = __shfl_sync(kFullMask, back, i), far1 = __shfl_sync(kFullMask, ahead, i);
            const char* table = static_cast<const char*>(b.table) +
                                (long long)__shfl_sync(kFullMask, head, i) * b.buckets * (BT ? 2 : 4);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const unsigned g = tile + 128 * k, q = g + 4 * lane;
                if (g + 128 <= s0 || g >= s1) continue;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const Distance d(c[k][u], from, last);
                    float v = d.back ? far0 : far1;
                    if (d.between) v = rel_table_entry<BT>(table, rel_bucket(b, (int)d.entry));
                    if (q + u - s0 < s1 - s0) x[k][u] += v;
                }
            }
        });
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const unsigned q = tile + 128 * i + 4 * lane;
        if (vec && q >= p0 && q + 4 <= p1) {
            *reinterpret_cast<float4*>(out + q) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (q + u >= p0 && q + u < p1) out[q + u] = x[i][u];
        }
    }
}

// Head h's entries lie in runs, one a query block; each is cut into Y parts at
// quads, and warp w of the W that CTAs (h, 0) .. (h, J - 1) have takes its equal
// share of the parts.  Every thread sums its entries into its own column of a
// histogram in shared memory ([bucket][thread]: no bank conflicts, no atomics),
// those further away than the map reaches into two registers, and the columns are
// added in a fixed order: which thread takes which entry is fixed too.  Bound by
// memory: 8 (or 6) bytes a nonzero.
template <bool BF>
__global__ void __launch_bounds__(kThreads, 3) rel_bias_grad_kernel(int M, int nnz, const int* __restrict__ ro,
                                                                 const int* __restrict__ ci, const void* __restrict__ ds,
                                                                 const RelArgs b, int blocks, int Y, int J,
                                                                 float* __restrict__ part, bool vec) {
    extern __shared__ float hist[];
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = T >> 5;
    for (int k = 0; k < b.buckets; ++k) hist[k * T + t] = 0.f;
    const int head = blockIdx.x / J;
    const long long W = (long long)J * warps, w = (long long)(blockIdx.x % J) * warps + warp;
    const long long parts = head < blocks ? ((blocks - 1 - head) / b.heads + 1LL) * Y : 0;
    const unsigned last = 2u * (unsigned)b.reach;
    float back = 0.f, ahead = 0.f;
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
        RowsHeld rows{ro, r1, nnz, lane, 0, 0};
        int start = 0;
        bool found = false, fresh = true;
#pragma unroll 1
        for (unsigned tile = p0 & ~3u; tile < p1; tile += kTile) {
            int c[kSteps][4];
            float x[kSteps][4];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                load_columns(ci, tile + 128 * k + 4 * lane, p1, vec, c[k]);
                load_values<BF>(ds, tile + 128 * k + 4 * lane, p1, vec, x[k]);
            }
            if (!found) rows.find(p0, r0);
            found = true;
            rows.segments(
                max(tile, p0), min(tile + kTile, p1), fresh,
                [&](int r, bool some) {
                    if (some) start = rel_start(b, block, r - r0, b.seg_cols > 0 ? __ldg(ci + rows.offset) : 0);
                },
                [&](int i, unsigned s0, unsigned s1) {
                    const int from = __shfl_sync(kFullMask, start, i);
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const unsigned g = tile + 128 * k, q = g + 4 * lane;
                        if (g + 128 <= s0 || g >= s1) continue;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const Distance d(c[k][u], from, last);
                            const float v = q + u - s0 < s1 - s0 ? x[k][u] : 0.f;
                            back += d.back ? v : 0.f;
                            ahead += d.back || d.between ? 0.f : v;
                            if (d.between && v != 0.f) hist[rel_bucket(b, (int)d.entry) * T + t] += v;
                        }
                    }
                });
        }
    }
    hist[rel_bucket(b, 0) * T + t] += back;
    hist[rel_bucket(b, (int)last) * T + t] += ahead;
    __syncthreads();
    for (int k = warp; k < b.buckets; k += warps) {
        float x = 0.f;
        for (int c = lane; c < T; c += 32) x += hist[k * T + c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
        if (lane == 0) part[(long long)blockIdx.x * b.buckets + k] = x;
    }
}

// dT[h][k] = Σ_j part[h][j][k]: a warp for each (h, k).
__global__ void rel_bias_grad_sum_kernel(int heads, int buckets, int J, const float* __restrict__ part,
                                         float* __restrict__ dtable) {
    const int lane = threadIdx.x & 31;
    const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (i >= (long long)heads * buckets) return;
    const long long h = i / buckets, k = i % buckets;
    float x = 0.f;
    for (int j = lane; j < J; j += 32) x += part[(h * J + j) * buckets + k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
    if (lane == 0) dtable[i] = x;
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
    const long long blocks = M > 0 ? (query_blocks(M, seg_rows) + heads - 1) / heads : 1;  // of the first head, the most
    const long long most = (456 + heads - 1) / heads * (long long)warps, some = nnz / (heads * (long long)kTile) + 1;
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
    const unsigned per_cta = kThreads / 32 * kTile;
    rel_bias_kernel<BT><<<((unsigned)nnz + per_cta - 1) / per_cta, kThreads, 0, stream>>>(M, nnz, ro, ci, scores, bias, out, vec);
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
    if (!allow_shared(rel_bias_grad_kernel<BF>, smem)) return USM_ERR_CUDA;
    float* part = static_cast<float*>(workspace);
    rel_bias_grad_kernel<BF><<<bias.heads * J, T, smem, stream>>>(
        M, nnz, ro, ci, ds, bias, query_blocks(M, bias.seg_rows), Y, J, part,
        quad_aligned(ci) && quad_aligned(ds, BF));
    const long long warps = (long long)bias.heads * bias.buckets;
    rel_bias_grad_sum_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(bias.heads, bias.buckets, J, part, dtable);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}
}  // namespace

int launch_rel_bias_grad(int M, int nnz, const int* ro, const int* ci, const void* dscores, bool bf16,
                         const RelArgs& bias, float* dtable, void* workspace, cudaStream_t stream) {
    const auto launch = bf16 ? launch_grad<true> : launch_grad<false>;
    return launch(M, nnz, ro, ci, dscores, bias, dtable, workspace, stream);
}

}  // namespace usm
