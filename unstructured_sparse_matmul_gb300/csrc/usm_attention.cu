// Sparse attention of few query rows in one pass (single tokens over a cache):
//     C[r] = Σ_p (P1[p] - λ P2[p]) V[c_p],   sk[p] = scale·(Qk[r]·Kk[c_p]) + bias(p).
#include <cmath>

#include "usm_internal.h"
#include "usm_rel.cuh"

namespace usm {
namespace {

template <bool BF>
__device__ __forceinline__ float elem(const void* p, long long i) {
    if constexpr (BF) return __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(p) + i) << 16);
    return __ldg(static_cast<const float*>(p) + i);
}

// A CTA per row: a warp per entry for the scores; then each thread owns
// output columns and walks the entries with the running sums of both maps.
template <bool BF, bool TWO>
__global__ void attention_kernel(const AttnArgs a) {
    constexpr int T = 128, W = T / 32;
    __shared__ float sc[2][T];
    __shared__ int sk[T];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int r = blockIdx.x;
    int p0, p1;
    row_range(a.row_offsets, r, a.nnz, p0, p1);
    const int block = r / a.seg_rows;
    long long shift = 0;
    if (a.bias.table && p0 < p1) shift = rel_shift(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + p0));
    float m[2] = {-INFINITY, -INFINITY}, z[2] = {0.f, 0.f}, acc[2][4] = {};
    for (int b = p0; b < p1; b += T) {
        const int n = min(T, p1 - b);
        __syncthreads();
        for (int i = warp; i < n; i += W) {
            const int c0 = __ldg(a.col_indices + b + i);
            const int c = min(max(c0, 0), a.K - 1);
            float x1 = 0.f, x2 = 0.f;
            for (int d = lane; d < a.D; d += 32) {
                x1 += elem<BF>(a.Q, (long long)r * a.ldq + d) * elem<BF>(a.Km, (long long)c * a.ldk + d);
                if (TWO) x2 += elem<BF>(a.Q2, (long long)r * a.ldq2 + d) * elem<BF>(a.K2, (long long)c * a.ldk2 + d);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                x1 += __shfl_xor_sync(kFullMask, x1, o);
                x2 += __shfl_xor_sync(kFullMask, x2, o);
            }
            if (lane == 0) {
                const float bias = a.bias.table ? rel_table(a.bias, block % a.heads,
                                                            rel_bucket(a.bias, rel_entry(c0, shift, a.bias.reach)))
                                                : 0.f;
                sc[0][i] = x1 * a.scale + bias;
                sc[1][i] = TWO ? x2 * a.scale + bias : -INFINITY;
                sk[i] = c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < (TWO ? 2 : 1); ++k) {
            float top = m[k];
            for (int i = 0; i < n; ++i) top = fmaxf(top, sc[k][i]);
            const float f = m[k] == -INFINITY ? 0.f : __expf(m[k] - top);
            z[k] *= f;
            for (int j = 0; j < 4; ++j) acc[k][j] *= f;
            m[k] = top;
            const float base = top == -INFINITY ? 0.f : top;
            for (int i = 0; i < n; ++i) {
                if (sc[k][i] == -INFINITY) continue;
                const float e = __expf(sc[k][i] - base);
                z[k] += e;
                for (int j = 0; j < 4; ++j) {
                    const int col = t + j * T;
                    if (col < a.N) acc[k][j] += e * elem<BF>(a.V, (long long)sk[i] * a.ldv + col);
                }
            }
        }
    }
    const float lam = TWO ? __ldg(a.lambda + block % a.heads) : 0.f;
    for (int j = 0; j < 4; ++j) {
        const int col = t + j * T;
        if (col >= a.N) break;
        float o = z[0] == 0.f ? 0.f : acc[0][j] / z[0];
        if (TWO && z[1] != 0.f) o -= lam * (acc[1][j] / z[1]);
        a.C[(long long)r * a.ldc + col] = o;
    }
}

}  // namespace

int launch_attention(const AttnArgs& a, bool bf16, cudaStream_t stream) {
    const bool two = a.lambda != nullptr;
    if (bf16)
        two ? attention_kernel<true, true><<<a.M, 128, 0, stream>>>(a)
            : attention_kernel<true, false><<<a.M, 128, 0, stream>>>(a);
    else
        two ? attention_kernel<false, true><<<a.M, 128, 0, stream>>>(a)
            : attention_kernel<false, false><<<a.M, 128, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

}  // namespace usm
