// Softmax maps over CSR rows and their gradients:
//     differential map   A = P1 - λ P2,
//     its gradient       dS1 = P1 (dA - c1), dS2 = -λ P2 (dA - c2), dλ = -Σ_rows c2, ck = Σ_row Pk dA,
//     softmax gradient   dS = P (dP - Σ_row P dP),
// Pk = exp(sk - mk) / Σ exp(sk - mk) over the row's stored entries.
#include <cmath>

#include "usm_internal.h"
#include "usm_rel.cuh"

namespace usm {
namespace {

__device__ __forceinline__ float load_elem(const void* p, int bf16, long long i) {
    return bf16 ? __uint_as_float((uint32_t) static_cast<const unsigned short*>(p)[i] << 16)
                : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_elem(void* p, int bf16, long long i, float v) {
    if (bf16)
        static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v);
    else
        static_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
    return x;
}

// What exponents are measured from: the row's maximum, or 0 where it is -inf
// (every entry masked), so that exp(-inf - 0) = 0 and the row's map is zero.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// 1/z, or 0 for a row without weight; NaN stays NaN.
__device__ __forceinline__ float inverse(float z) { return z == 0.f ? 0.f : 1.f / z; }
// e·d, 0 where the entry is masked (whatever d is there).
__device__ __forceinline__ float masked_mul(float s, float e, float d) { return s == -INFINITY ? 0.f : e * d; }

// A warp per row; TWO maps or one, GRAD or the map itself.
template <bool TWO, bool GRAD>
__global__ void softmax_map_kernel(const MapArgs a) {
    const int lane = threadIdx.x & 31;
    const long long warps = ((long long)gridDim.x * blockDim.x) >> 5;
    for (long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; r < a.M; r += warps) {
        int p0, p1;
        row_range(a.row_offsets, (int)r, a.nnz, p0, p1);
        if (p0 == p1) {
            if (GRAD && TWO && a.row_c2 && lane == 0) a.row_c2[r] = 0.f;
            continue;
        }
        const float lam = TWO ? __ldg(a.lambda + (int)r / a.seg_rows % a.heads) : 0.f;
        float m1 = -INFINITY, m2 = -INFINITY;
        for (int p = p0 + lane; p < p1; p += 32) {
            m1 = fmaxf(m1, a.s1[p]);
            if (TWO) m2 = fmaxf(m2, a.s2[p]);
        }
        m1 = base_of(warp_max(m1));
        if (TWO) m2 = base_of(warp_max(m2));
        float z1 = 0.f, z2 = 0.f, c1 = 0.f, c2 = 0.f;
        for (int p = p0 + lane; p < p1; p += 32) {
            const float x1 = a.s1[p], e1 = __expf(x1 - m1);
            const float d = GRAD ? load_elem(a.dout, a.dout_bf16, p) : 0.f;
            z1 += e1;
            if (GRAD) c1 += masked_mul(x1, e1, d);
            if (TWO) {
                const float x2 = a.s2[p], e2 = __expf(x2 - m2);
                z2 += e2;
                if (GRAD) c2 += masked_mul(x2, e2, d);
            }
        }
        const float r1 = inverse(warp_sum(z1)), r2 = TWO ? inverse(warp_sum(z2)) : 0.f;
        if (GRAD) {
            c1 = warp_sum(c1) * r1;
            if (TWO) c2 = warp_sum(c2) * r2;
            if (TWO && a.row_c2 && lane == 0) a.row_c2[r] = c2;
        }
        for (int p = p0 + lane; p < p1; p += 32) {
            const float x1 = a.s1[p], e1 = __expf(x1 - m1) * r1;
            const float x2 = TWO ? a.s2[p] : 0.f, e2 = TWO ? __expf(x2 - m2) * r2 : 0.f;
            if (GRAD) {
                const float d = load_elem(a.dout, a.dout_bf16, p);
                store_elem(a.out1, a.out_bf16, p, masked_mul(x1, e1, d - c1));
                if (TWO) store_elem(a.out2, a.out_bf16, p, -lam * masked_mul(x2, e2, d - c2));
            } else {
                store_elem(a.out1, a.out_bf16, p, e1 - lam * e2);
            }
        }
    }
}

// dλ[h] = -Σ c2 over head h's rows: a CTA per head, a fixed order.
__global__ void lambda_grad_kernel(int M, int heads, int seg_rows, const float* __restrict__ row_c2,
                                   float* __restrict__ dlambda) {
    __shared__ float warp_part[8];
    const int head = blockIdx.x, t = threadIdx.x;
    const int blocks = (M + seg_rows - 1) / seg_rows;
    const long long rows = head < blocks ? (long long)((blocks - 1 - head) / heads + 1) * seg_rows : 0;
    float x = 0.f;
    for (long long i = t; i < rows; i += blockDim.x) {
        const long long r = (head + i / seg_rows * heads) * seg_rows + i % seg_rows;
        if (r < M) x += row_c2[r];
    }
    x = warp_sum(x);
    if ((t & 31) == 0) warp_part[t >> 5] = x;
    __syncthreads();
    if (t == 0) {
        float y = 0.f;
        for (int w = 0; w < 8; ++w) y += warp_part[w];
        dlambda[head] = -y;
    }
}

template <bool TWO, bool GRAD>
int launch_map(const MapArgs& a, cudaStream_t stream) {
    long long blocks = ((long long)a.M * 32 + 255) / 256;
    const long long cap = 16LL * sm_count_current_device();
    if (blocks > cap) blocks = cap;
    softmax_map_kernel<TWO, GRAD><<<(int)blocks, 256, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

}  // namespace

int launch_diff_softmax(const MapArgs& a, cudaStream_t stream) { return launch_map<true, false>(a, stream); }

int launch_row_softmax_grad(const MapArgs& a, cudaStream_t stream) { return launch_map<false, true>(a, stream); }

int launch_diff_softmax_grad(const MapArgs& a, float* dlambda, cudaStream_t stream) {
    const int r = launch_map<true, true>(a, stream);
    if (r != USM_OK || !dlambda) return r;
    lambda_grad_kernel<<<a.heads, 256, 0, stream>>>(a.M, a.heads, a.seg_rows, a.row_c2, dlambda);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

}  // namespace usm
