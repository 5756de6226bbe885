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

// A warp per row.
__global__ void rel_bias_kernel(int M, int nnz, const int* __restrict__ ro, const int* __restrict__ ci,
                                const float* s, const RelArgs b, float* out) {
    const int lane = threadIdx.x & 31;
    const long long warps = ((long long)gridDim.x * blockDim.x) >> 5;
    for (long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; r < M; r += warps) {
        int p0, p1;
        row_range(ro, (int)r, nnz, p0, p1);
        if (p0 == p1) continue;
        const int block = (int)r / b.seg_rows;
        const long long shift = rel_shift(b, block, (int)r - block * b.seg_rows, __ldg(ci + p0));
        const int head = block % b.heads;
        for (int p = p0 + lane; p < p1; p += 32)
            out[p] = s[p] + rel_table(b, head, rel_bucket(b, rel_entry(__ldg(ci + p), shift, b.reach)));
    }
}

// CTA (h, j) takes part j of J of head h's rows; every thread sums its entries
// into its own column of a histogram in shared memory ([bucket][thread]: no
// bank conflicts, no atomics), and the columns are added in a fixed order.
__global__ void rel_bias_grad_kernel(int M, int nnz, const int* __restrict__ ro, const int* __restrict__ ci,
                                     const void* __restrict__ ds, int bf16, const RelArgs b, int J, float* part) {
    extern __shared__ float hist[];
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31;
    for (int k = 0; k < b.buckets; ++k) hist[k * T + t] = 0.f;
    const int head = blockIdx.x / J, j = blockIdx.x % J;
    const int blocks = (M + b.seg_rows - 1) / b.seg_rows;
    const long long rows = head < blocks ? (long long)((blocks - 1 - head) / b.heads + 1) * b.seg_rows : 0;
    const long long i0 = rows * j / J, i1 = rows * (j + 1) / J;
    for (long long i = i0 + (t >> 5); i < i1; i += T >> 5) {
        const int block = head + (int)(i / b.seg_rows) * b.heads;
        const int in_block = (int)(i % b.seg_rows);
        const long long r = (long long)block * b.seg_rows + in_block;
        if (r >= M) continue;
        int p0, p1;
        row_range(ro, (int)r, nnz, p0, p1);
        if (p0 == p1) continue;
        const long long shift = rel_shift(b, block, in_block, __ldg(ci + p0));
        for (int p = p0 + lane; p < p1; p += 32) {
            const int k = rel_bucket(b, rel_entry(__ldg(ci + p), shift, b.reach));
            const float v = bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(ds) + p) << 16)
                                 : __ldg(static_cast<const float*>(ds) + p);
            hist[k * T + t] += v;
        }
    }
    __syncthreads();
    for (int k = t >> 5; k < b.buckets; k += T >> 5) {
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

constexpr int kGradThreads = 64;

// Parts each head's rows are cut into.
int grad_parts(int M, int seg_rows, int num_heads) {
    const long long blocks = query_blocks(M, seg_rows);
    const long long rows = (blocks + num_heads - 1) / num_heads * seg_rows;  // of the first head, the longest
    long long J = (1216 + num_heads - 1) / num_heads;
    if (J > rows) J = rows;
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
    long long blocks = ((long long)M * 32 + 255) / 256;
    const long long cap = 16LL * sm_count_current_device();
    if (blocks > cap) blocks = cap;
    rel_bias_kernel<<<(int)blocks, 256, 0, stream>>>(M, nnz, ro, ci, scores, bias, out);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

size_t rel_bias_grad_workspace_bytes(int M, int, int seg_rows, int num_heads, int num_buckets) {
    return (size_t)num_heads * grad_parts(M, seg_rows, num_heads) * num_buckets * 4;
}

int launch_rel_bias_grad(int M, int nnz, const int* ro, const int* ci, const void* dscores, bool bf16,
                         const RelArgs& bias, float* dtable, void* workspace, cudaStream_t stream) {
    const int J = grad_parts(M, bias.seg_rows, bias.heads);
    const int smem = bias.buckets * kGradThreads * 4;
    if (smem > 48 * 1024 && cudaFuncSetAttribute(rel_bias_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 smem) != cudaSuccess)
        return USM_ERR_CUDA;
    float* part = static_cast<float*>(workspace);
    rel_bias_grad_kernel<<<bias.heads * J, kGradThreads, smem, stream>>>(M, nnz, ro, ci, dscores, bf16 ? 1 : 0, bias, J,
                                                                         part);
    const long long warps = (long long)bias.heads * bias.buckets;
    rel_bias_grad_sum_kernel<<<(int)((warps + 7) / 8), 256, 0, stream>>>(bias.heads, bias.buckets, J, part, dtable);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

}  // namespace usm
