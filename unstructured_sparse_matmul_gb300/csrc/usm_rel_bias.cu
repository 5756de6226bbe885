// Learned relative position bias of sparse attention, by buckets, and its
// gradient:
//     out[p] = s[p] + T[h][bucket(p)],     dT[h][k] = Σ_{p of head h, bucket(p) = k} dS[p],
// bucket(p) = map[reach + clamp(d, ±reach)], d the key's position less the
// query's.
#include "usm_internal.h"
#include "usm_quads.cuh"
#include "usm_rel.cuh"
#include "usm_rows.cuh"

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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kQuads = 4;         // quads a lane has in flight
constexpr unsigned kLong = 2048;  // entries above which a CTA takes a row

// Columns of quad q (those past the array's end read as 0).
template <bool VEC>
__device__ __forceinline__ void load_columns(const int* __restrict__ ci, unsigned q, unsigned nnz, int (&c)[4]) {
    if (VEC && q + 4 <= nnz) {
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

// Adds the bias to entries [p0, p1) of one row (head and start: the row's), by
// threads t = 0..T-1.
template <bool VEC, bool BT>
__device__ __forceinline__ void bias_entries(const int* __restrict__ ci, unsigned nnz, const float* s, const RelArgs& b,
                                             float* out, int head, int start, unsigned p0, unsigned p1, unsigned t,
                                             unsigned T) {
    const unsigned step = 4 * T;
#pragma unroll 1
    for (unsigned q0 = (p0 & ~3u) + 4 * t; q0 < p1; q0 += kQuads * step) {
        int c[kQuads][4];
        float x[kQuads][4];
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const unsigned q = q0 + i * step;
            if (q < p1) {
                load_columns<VEC>(ci, q, nnz, c[i]);
                load_quad<false, VEC>(s, q, nnz, x[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const unsigned q = q0 + i * step;
            if (q < p1) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    x[i][u] += rel_table<BT>(b, head, rel_bucket(b, rel_entry(c[i][u], start, b.reach)));
                store_quad<false, VEC>(out, q, p0, p1, x[i]);
            }
        }
    }
}

// Bound by memory: 8 bytes a nonzero in, 4 out.  Quads of entries with 16-byte
// accesses, four in flight a lane; the map and the head's row of the table are a
// few hundred bytes that stay in L1.  CTA b of B takes rows [M·b / B, M·(b+1) / B),
// 64 at a time: long ones by the whole CTA, then each warp fetches row after row.
template <bool VEC, bool BT>
__global__ void __launch_bounds__(kThreads) rel_bias_kernel(int M, int nnz, const int* __restrict__ ro,
                                                            const int* __restrict__ ci, const float* s, const RelArgs b,
                                                            float* out) {
    __shared__ RowRun run;
    __shared__ int heads[kRun], starts[kRun];
    const int lane = threadIdx.x & 31;
    const long long r0 = (long long)M * blockIdx.x / gridDim.x, r1 = (long long)M * (blockIdx.x + 1) / gridDim.x;
    for (long long r = r0; r < r1; r += kRun) {
        const int n = (int)min((long long)kRun, r1 - r);
        const bool any_long = run.load(ro, nnz, n, kLong, [&](int i) { return (int)r + i; },
                                       [&](int i, int row) {
                                           const int block = row / b.seg_rows;
                                           heads[i] = block % b.heads;
                                           if (run.begin[i] < run.end[i])
                                               starts[i] = rel_start(b, block, row - block * b.seg_rows, __ldg(ci + run.begin[i]));
                                       });
        if (any_long) {
#pragma unroll 1
            for (int i = 0; i < n; ++i)
                if ((unsigned)(run.end[i] - run.begin[i]) > kLong)
                    bias_entries<VEC, BT>(ci, nnz, s, b, out, heads[i], starts[i], run.begin[i], run.end[i], threadIdx.x, kThreads);
        }
        for (int i = run.fetch(lane); i < n; i = run.fetch(lane))
            if ((unsigned)(run.end[i] - run.begin[i]) <= kLong)
                bias_entries<VEC, BT>(ci, nnz, s, b, out, heads[i], starts[i], run.begin[i], run.end[i], lane, 32);
        __syncthreads();  // the next run's rows overwrite this one's
    }
}

// Piece y of gridDim.y of row x's quads.
__device__ __forceinline__ void piece_range(unsigned p0, unsigned p1, int piece, int pieces, unsigned& b0, unsigned& b1) {
    const unsigned f = p0 & ~3u, quads = (p1 - f + 3) / 4;
    b0 = max(p0, f + 4 * (unsigned)((unsigned long long)quads * piece / pieces));
    b1 = min(p1, f + 4 * (unsigned)((unsigned long long)quads * (piece + 1) / pieces));
}

// Few long rows: CTA (x, y) takes piece y of row x.
template <bool VEC, bool BT>
__global__ void __launch_bounds__(kThreads) rel_bias_pieces_kernel(int nnz, const int* __restrict__ ro,
                                                                   const int* __restrict__ ci, const float* s,
                                                                   const RelArgs b, float* out) {
    const int r = blockIdx.x, block = r / b.seg_rows;
    int p0, p1;
    row_range(ro, r, nnz, p0, p1);
    if (p0 == p1) return;
    unsigned b0, b1;
    piece_range(p0, p1, blockIdx.y, gridDim.y, b0, b1);
    const int start = rel_start(b, block, r - block * b.seg_rows, __ldg(ci + p0));
    bias_entries<VEC, BT>(ci, nnz, s, b, out, block % b.heads, start, b0, b1, threadIdx.x, kThreads);
}

// CTA (h, j) takes part j of J of head h's rows (or of their pieces, where there
// are few long rows).  Every thread sums its entries into its own column of a
// histogram in shared memory ([bucket][thread]: no bank conflicts, no atomics),
// and the columns are added in a fixed order: which thread takes which entry is
// fixed too.  A thread holds the sum of its latest bucket in a register and
// writes it back when the bucket changes: far keys share a bucket, so most of a
// row is a few runs.  Bound by memory: 8 (or 6) bytes a nonzero.
template <bool BF, bool VEC>
__global__ void __launch_bounds__(kThreads) rel_bias_grad_kernel(int M, int nnz, const int* __restrict__ ro,
                                                                 const int* __restrict__ ci, const void* __restrict__ ds,
                                                                 const RelArgs b, int blocks, int pieces, int J,
                                                                 float* __restrict__ part) {
    extern __shared__ float hist[];
    __shared__ RowRun run;
    __shared__ int starts[kRun];
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = T >> 5;
    for (int k = 0; k < b.buckets; ++k) hist[k * T + t] = 0.f;
    const int head = blockIdx.x / J, j = blockIdx.x % J;
    const long long rows = head < blocks ? (long long)((blocks - 1 - head) / b.heads + 1) * b.seg_rows : 0;
    const long long items = rows * pieces, i0 = items * j / J, i1 = items * (j + 1) / J;
    int bucket = 0;
    float sum = 0.f;
    auto entries = [&](int start, unsigned p0, unsigned p1, unsigned at, unsigned threads) {
        const unsigned step = 4 * threads;
#pragma unroll 1
        for (unsigned q0 = (p0 & ~3u) + 4 * at; q0 < p1; q0 += kQuads * step) {
            int c[kQuads][4];
            float x[kQuads][4];
#pragma unroll
            for (int i = 0; i < kQuads; ++i) {
                const unsigned q = q0 + i * step;
                if (q < p1) {
                    load_columns<VEC>(ci, q, nnz, c[i]);
                    load_quad<BF, VEC>(ds, q, nnz, x[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kQuads; ++i) {
                const unsigned q = q0 + i * step;
                if (q >= p1) break;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = rel_bucket(b, rel_entry(c[i][u], start, b.reach));
                    if (q + u < p0 || q + u >= p1) continue;
                    if (k != bucket) {
                        hist[bucket * T + t] += sum;
                        bucket = k;
                        sum = 0.f;
                    }
                    sum += x[i][u];
                }
            }
        }
    };
    for (long long f = i0; f < i1; f += kRun) {
        const int n = (int)min((long long)kRun, i1 - f);
        const bool any_long = run.load(
            ro, nnz, n, kLong,
            [&](int i) {  // item -> row of the head's blocks (the last block may be shorter)
                const long long row = (f + i) / pieces;
                const long long r = (head + row / b.seg_rows * b.heads) * b.seg_rows + row % b.seg_rows;
                return r < M ? (int)r : -1;
            },
            [&](int i, int r) {
                const int block = r / b.seg_rows, p0 = run.begin[i], p1 = run.end[i];
                if (p0 == p1) return;
                starts[i] = rel_start(b, block, r - block * b.seg_rows, __ldg(ci + p0));
                if (pieces > 1) {
                    unsigned b0, b1;
                    piece_range(p0, p1, (int)((f + i) % pieces), pieces, b0, b1);
                    run.begin[i] = b0;
                    run.end[i] = max(b0, b1);
                }
            });
        if (any_long) {
#pragma unroll 1
            for (int i = 0; i < n; ++i)
                if ((unsigned)(run.end[i] - run.begin[i]) > kLong) entries(starts[i], run.begin[i], run.end[i], t, T);
        }
        for (int i = warp; i < n; i += warps)
            if ((unsigned)(run.end[i] - run.begin[i]) <= kLong) entries(starts[i], run.begin[i], run.end[i], lane, 32);
        __syncthreads();  // the next run's rows overwrite this one's
    }
    hist[bucket * T + t] += sum;
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

// Pieces a row is cut into: more where the mean row would keep a CTA busy and
// the rows are too few to fill the GPU.
int row_pieces(int M, int nnz) {
    int pieces = 1;
    while (pieces < 64 && (long long)M * pieces < 2048 && nnz / M / pieces > 1024) pieces *= 2;
    return pieces;
}

// Threads of a gradient CTA (its histogram is threads × buckets floats, 64 KB
// at most) and parts each head's items are cut into.
int grad_threads(int buckets) { return buckets <= 64 ? 256 : buckets <= 128 ? 128 : buckets <= 256 ? 64 : 32; }

int grad_parts(int M, int nnz, int seg_rows, int heads, int buckets) {
    const long long blocks = query_blocks(M, seg_rows);
    const long long items = (blocks + heads - 1) / heads * seg_rows * row_pieces(M, nnz);  // of the first head, the longest
    const int warps = grad_threads(buckets) / 32;
    long long J = (912 + heads - 1) / heads;
    if (J > (items + warps - 1) / warps) J = (items + warps - 1) / warps;
    return (int)(J < 1 ? 1 : J);
}

}  // namespace

int launch_rel_bucket_build(int num_buckets, int max_distance, bool causal, int* bucket_map, cudaStream_t stream) {
    rel_bucket_kernel<<<(2 * max_distance + 1 + 127) / 128, 128, 0, stream>>>(num_buckets, max_distance, causal ? 1 : 0,
                                                                            bucket_map);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

namespace {
template <bool VEC, bool BT>
void launch_bias(int M, int nnz, const int* ro, const int* ci, const float* scores, const RelArgs& bias, float* out,
                 cudaStream_t stream) {
    const int pieces = row_pieces(M, nnz);
    if (pieces > 1) {
        rel_bias_pieces_kernel<VEC, BT><<<dim3(M, pieces), kThreads, 0, stream>>>(nnz, ro, ci, scores, bias, out);
        return;
    }
    const int slots = sm_count_current_device() * 4;
    rel_bias_kernel<VEC, BT><<<M < slots ? M : slots, kThreads, 0, stream>>>(M, nnz, ro, ci, scores, bias, out);
}
}  // namespace

int launch_rel_bias(int M, int nnz, const int* ro, const int* ci, const float* scores, const RelArgs& bias, float* out,
                    cudaStream_t stream) {
    const bool vec = quad_aligned(ci, false) && quad_aligned(scores, false) && quad_aligned(out, false);
    auto call = [&](auto launch) { launch(M, nnz, ro, ci, scores, bias, out, stream); };
    if (bias.table_bf16)
        vec ? call(launch_bias<true, true>) : call(launch_bias<false, true>);
    else
        vec ? call(launch_bias<true, false>) : call(launch_bias<false, false>);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

size_t rel_bias_grad_workspace_bytes(int M, int nnz, int seg_rows, int num_heads, int num_buckets) {
    return (size_t)num_heads * grad_parts(M, nnz, seg_rows, num_heads, num_buckets) * num_buckets * 4;
}

namespace {
template <bool BF, bool VEC>
int launch_grad(int M, int nnz, const int* ro, const int* ci, const void* ds, const RelArgs& bias, float* dtable,
                void* workspace, cudaStream_t stream) {
    const int J = grad_parts(M, nnz, bias.seg_rows, bias.heads, bias.buckets), T = grad_threads(bias.buckets);
    const int smem = bias.buckets * T * 4;
    if (smem > 48 * 1024 && cudaFuncSetAttribute(rel_bias_grad_kernel<BF, VEC>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return USM_ERR_CUDA;
    float* part = static_cast<float*>(workspace);
    rel_bias_grad_kernel<BF, VEC><<<bias.heads * J, T, smem, stream>>>(
        M, nnz, ro, ci, ds, bias, query_blocks(M, bias.seg_rows), row_pieces(M, nnz), J, part);
    const long long warps = (long long)bias.heads * bias.buckets;
    rel_bias_grad_sum_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(bias.heads, bias.buckets, J, part, dtable);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}
}  // namespace

int launch_rel_bias_grad(int M, int nnz, const int* ro, const int* ci, const void* dscores, bool bf16,
                         const RelArgs& bias, float* dtable, void* workspace, cudaStream_t stream) {
    const bool vec = quad_aligned(ci, false) && quad_aligned(dscores, bf16);
    auto call = [&](auto launch) { return launch(M, nnz, ro, ci, dscores, bias, dtable, workspace, stream); };
    if (bf16) return vec ? call(launch_grad<true, true>) : call(launch_grad<true, false>);
    return vec ? call(launch_grad<false, true>) : call(launch_grad<false, false>);
}

}  // namespace usm
