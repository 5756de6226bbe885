// Learned relative position bias of sparse attention, by buckets, and its
// gradient:
//     out[p] = s[p] + T[h][bucket(p)],     dT[h][k] = Σ_{p of head h, bucket(p) = k} dS[p],
// bucket(p) = map[reach + clamp(d, ±reach)], d the key's position less the
// query's.
#include "usm_internal.h"
#include "usm_quads.cuh"
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr unsigned kLong = 2048;  // entries above which a CTA takes a row (or a piece of one)

// Rows are cut into `pieces` equal runs of quads where there are few long ones.
__device__ __forceinline__ void piece_range(unsigned p0, unsigned p1, int piece, int pieces, unsigned& b0, unsigned& b1) {
    b0 = p0;
    b1 = p1;
    if (pieces > 1) {
        const unsigned f = p0 & ~3u, quads = (p1 - f + 3) / 4;
        b0 = max(p0, f + 4 * (unsigned)((unsigned long long)quads * piece / pieces));
        b1 = min(p1, f + 4 * (unsigned)((unsigned long long)quads * (piece + 1) / pieces));
    }
}

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

// Bound by memory: 8 bytes a nonzero in, 4 out.  A warp per row (or piece),
// four entries a lane with 16-byte accesses, two quads in flight; long ones by
// the CTA after its warps are done.  The map and the head's row of the table
// are a few hundred bytes that stay in L1.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) rel_bias_kernel(int M, int nnz, const int* __restrict__ ro,
                                                            const int* __restrict__ ci, const float* s, const RelArgs b,
                                                            int pieces, float* out) {
    __shared__ int waits[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long items = (long long)M * pieces, first = (long long)blockIdx.x * kWarps;
    // Entries of item i by the T threads t = 0..T-1.
    auto item = [&](long long i, unsigned t, unsigned T, bool long_ones) {
        const int r = (int)(i / pieces);
        int p0, p1;
        row_range(ro, r, nnz, p0, p1);
        unsigned b0, b1;
        piece_range(p0, p1, (int)(i - (long long)r * pieces), pieces, b0, b1);
        if (b0 >= b1) return false;
        if (!long_ones && b1 - b0 > kLong) return true;
        const int block = r / b.seg_rows;
        const int start = rel_start(b, block, r - block * b.seg_rows, __ldg(ci + p0));
        const int head = block % b.heads;
        auto quad = [&](unsigned q) {
            int c[4];
            float x[4];
            load_columns<VEC>(ci, q, nnz, c);
            load_quad<false, VEC>(s, q, nnz, x);
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] += rel_table(b, head, rel_bucket(b, rel_entry(c[u], start, b.reach)));
            store_quad<false, VEC>(out, q, b0, b1, x);
        };
#pragma unroll 2
        for (unsigned q = (b0 & ~3u) + 4 * t; q < b1; q += 4 * T) quad(q);
        return false;
    };
    bool is_long = false;
    if (first + warp < items) is_long = item(first + warp, lane, 32, false);
    if (lane == 0) waits[warp] = is_long;
    if (!__syncthreads_or(is_long)) return;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w)
        if (waits[w]) item(first + w, threadIdx.x, kThreads, true);
}

// CTA (h, j) takes part j of J of head h's rows (or pieces).  Every thread sums
// its entries into its own column of a histogram in shared memory ([bucket]
// [thread]: no bank conflicts, no atomics), and the columns are added in a
// fixed order.  A thread holds the sum of its latest bucket in a register and
// writes it back when the bucket changes: far keys share a bucket, so most of a
// row is a few runs.  Bound by memory: 8 (or 6) bytes a nonzero.
template <bool BF, bool VEC>
__global__ void __launch_bounds__(kThreads) rel_bias_grad_kernel(int M, int nnz, const int* __restrict__ ro,
                                                                 const int* __restrict__ ci, const void* __restrict__ ds,
                                                                 const RelArgs b, int blocks, int pieces, int J,
                                                                 float* __restrict__ part) {
    extern __shared__ float hist[];
    __shared__ int waits[kWarps];
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = T >> 5;
    for (int k = 0; k < b.buckets; ++k) hist[k * T + t] = 0.f;
    const int head = blockIdx.x / J, j = blockIdx.x % J;
    const long long rows = head < blocks ? (long long)((blocks - 1 - head) / b.heads + 1) * b.seg_rows : 0;
    const long long items = rows * pieces, i0 = items * j / J, i1 = items * (j + 1) / J;
    int bucket = 0;
    float sum = 0.f;
    auto item = [&](long long i, unsigned at, unsigned step, bool long_ones) {
        const long long row = i / pieces;
        const int in_block = (int)(row % b.seg_rows), block = head + (int)(row / b.seg_rows) * b.heads;
        const long long r = (long long)block * b.seg_rows + in_block;
        if (r >= M) return false;
        int p0, p1;
        row_range(ro, (int)r, nnz, p0, p1);
        unsigned b0, b1;
        piece_range(p0, p1, (int)(i - row * pieces), pieces, b0, b1);
        if (b0 >= b1) return false;
        if (!long_ones && b1 - b0 > kLong) return true;
        const int start = rel_start(b, block, in_block, __ldg(ci + p0));
#pragma unroll 2
        for (unsigned q = (b0 & ~3u) + 4 * at; q < b1; q += 4 * step) {
            int c[4];
            float x[4];
            load_columns<VEC>(ci, q, nnz, c);
            load_quad<BF, VEC>(ds, q, nnz, x);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = rel_bucket(b, rel_entry(c[u], start, b.reach));
                const bool in = q + u >= b0 && q + u < b1;
                if (in && k != bucket) {
                    hist[bucket * T + t] += sum;
                    bucket = k;
                    sum = 0.f;
                }
                if (in) sum += x[u];
            }
        }
        return false;
    };
    for (long long f = i0; f < i1; f += warps) {
        bool is_long = false;
        if (f + warp < i1) is_long = item(f + warp, lane, 32, false);
        if (lane == 0) waits[warp] = is_long;
        if (__syncthreads_or(is_long)) {
#pragma unroll 1
            for (int w = 0; w < warps; ++w)
                if (waits[w]) item(f + w, t, T, true);
            __syncthreads();
        }
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

int launch_rel_bias(int M, int nnz, const int* ro, const int* ci, const float* scores, const RelArgs& bias, float* out,
                    cudaStream_t stream) {
    const int pieces = row_pieces(M, nnz);
    const unsigned grid = (unsigned)(((long long)M * pieces + kWarps - 1) / kWarps);
    if (quad_aligned(ci, false) && quad_aligned(scores, false) && quad_aligned(out, false))
        rel_bias_kernel<true><<<grid, kThreads, 0, stream>>>(M, nnz, ro, ci, scores, bias, pieces, out);
    else
        rel_bias_kernel<false><<<grid, kThreads, 0, stream>>>(M, nnz, ro, ci, scores, bias, pieces, out);
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
