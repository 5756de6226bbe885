// Softmax maps over CSR rows and their gradients:
//     differential map   A = P1 - λ P2,
//     its gradient       dS1 = P1 (dA - c1), dS2 = -λ P2 (dA - c2), dλ = -Σ_rows c2, ck = Σ_row Pk dA,
//     softmax gradient   dS = P (dP - Σ_row P dP),
// Pk = exp(sk - mk) / zk, mk the row's maximum, zk = Σ exp(sk - mk) over its
// stored entries.
//
// Bound by memory: 8 to 12 bytes a nonzero in, 2 to 8 out, each once.  A row is
// read once into registers (four quads a lane: 512 entries a warp, 4096 a CTA),
// its maximum and then its sums are reduced over the lanes, and the results are
// written from the registers.  Entries past those are summed as they are read,
// with a running maximum, and read a second time (from L2) for the output.
// A warp takes a row; rows over kLong entries wait until the warps of the CTA
// are done and are then taken by the whole CTA, so a long row among short ones
// costs an eighth of its time.  Where rows are long throughout, or few, a CTA
// or a cluster of up to 8 takes each row (launch_map), the CTAs joining their
// maxima and sums through distributed shared memory.
#include <cmath>
#include <type_traits>

#include "usm_cluster.cuh"
#include "usm_internal.h"
#include "usm_quads.cuh"
#include "usm_rel.cuh"

namespace usm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kQuads = 4;             // quads a lane keeps in registers
constexpr unsigned kLong = 2048;      // entries above which a CTA takes the row

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

// What exponents are measured from: the maximum, or 0 where it is -inf (every
// entry masked), so that exp(-inf - 0) = 0 and the row's map is zero.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// 1/z, or 0 for a row without weight; NaN stays NaN.
__device__ __forceinline__ float inverse(float z) { return z == 0.f ? 0.f : 1.f / z; }
// w·d, or 0 under a weight of 0 (a masked entry) whatever d is there.
__device__ __forceinline__ float weighted(float w, float d) { return w == 0.f ? 0.f : w * d; }

// Sums of one map over (part of) a row: the maximum m, z = Σ exp(s - m) and
// c = Σ exp(s - m)·d.
struct Stat {
    float m, z, c;
};

// Shared memory of a CTA that takes a row: one slot a warp, and the CTA's.
struct BlockStats {
    float top[2][kWarps];
    float sum[2][2][kWarps];
    float whole[2][3];
};

// One row [p0, p1).  BLOCK: by the CTA (or its cluster's), else by the warp.
template <bool TWO, bool GRAD, bool DIN, bool OUT, bool VEC, bool BLOCK>
__device__ __forceinline__ void map_row(const MapArgs& a, int r, unsigned p0, unsigned p1, BlockStats& sh, int ctas,
                                        int rank) {
    constexpr int MAPS = TWO ? 2 : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned nnz = a.nnz;
    // Thread t of T takes quads t, t + T, ... of the row.
    const unsigned T = BLOCK ? kThreads * ctas : 32, t = BLOCK ? rank * kThreads + threadIdx.x : lane;
    const unsigned q0 = (p0 & ~3u) + 4 * t, step = 4 * T;
    const float* s[2] = {a.s1, a.s2};

    // Scores of quad q; entries of neighbouring rows become -inf.  Only the
    // row's first quad (thread 0's) can hold entries before it.
    auto load_scores = [&](unsigned q, bool first, float (&x)[MAPS][4]) {
#pragma unroll
        for (int k = 0; k < MAPS; ++k) load_quad<false, VEC>(s[k], q, nnz, x[k]);
        const int left = (int)(p1 - q);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool out = u >= left || (first && q + u < p0);
#pragma unroll
            for (int k = 0; k < MAPS; ++k)
                if (out) x[k][u] = -INFINITY;
        }
    };

    float x[kQuads][MAPS][4], d[GRAD ? kQuads : 1][4];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        const unsigned q = q0 + i * step;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int k = 0; k < MAPS; ++k) x[i][k][u] = -INFINITY;
            if constexpr (GRAD) d[i][u] = 0.f;
        }
        if (q < p1) {
            load_scores(q, i == 0, x[i]);
            if constexpr (GRAD) load_quad<DIN, VEC>(a.dout, q, nnz, d[i]);
        }
    }
    // Quads past the registers: a running maximum and sums.
    const unsigned tail = q0 + kQuads * step;
    Stat run[MAPS];
#pragma unroll
    for (int k = 0; k < MAPS; ++k) run[k] = {-INFINITY, 0.f, 0.f};
#pragma unroll 1
    for (unsigned q = tail; q < p1; q += step) {
        float y[MAPS][4], dy[4];
        load_scores(q, false, y);
        if constexpr (GRAD) load_quad<DIN, VEC>(a.dout, q, nnz, dy);
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            const float top = fmaxf(fmaxf(fmaxf(y[k][0], y[k][1]), fmaxf(y[k][2], y[k][3])), run[k].m);
            const float base = base_of(top), f = exp_flush(run[k].m - base);
            run[k].z *= f;
            run[k].c *= f;
            run[k].m = top;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float e = exp_flush(y[k][u] - base);
                run[k].z += e;
                if constexpr (GRAD) run[k].c += weighted(e, dy[u]);
            }
        }
    }

    // Maximum over the warp or CTA.
    float m[MAPS];
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        float top = run[k].m;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            top = fmaxf(top, fmaxf(fmaxf(x[i][k][0], x[i][k][1]), fmaxf(x[i][k][2], x[i][k][3])));
        m[k] = warp_max(top);
        if (BLOCK && lane == 0) sh.top[k][warp] = m[k];
    }
    if constexpr (BLOCK) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < MAPS; ++k)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m[k] = fmaxf(m[k], sh.top[k][w]);
    }
    // Weights (in the scores' registers) and their sums.
    float z[MAPS], c[MAPS], inv[MAPS];
    auto dot = [&](int k, bool guarded) {
        float sum = 0.f;
        if constexpr (GRAD) {
#pragma unroll
            for (int i = 0; i < kQuads; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    sum = guarded && x[i][k][u] == 0.f ? sum : fmaf(x[i][k][u], d[i][u], sum);
        }
        return sum;
    };
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        const float base = base_of(m[k]), f = exp_flush(run[k].m - base);
        z[k] = run[k].z * f;
        run[k].c *= f;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[i][k][u] = exp_flush(x[i][k][u] - base);
                z[k] += x[i][k][u];
            }
        z[k] = warp_sum(z[k]);
        c[k] = 0.f;
        if constexpr (GRAD) c[k] = warp_sum(run[k].c + dot(k, BLOCK));
        if (BLOCK && lane == 0) {
            sh.sum[k][0][warp] = z[k];
            sh.sum[k][1][warp] = c[k];
        }
    }
    // A dout that is not finite makes c so too, even under weights of 0: such a
    // row (and every row of a CTA) guards each product.
    bool guarded = BLOCK;
    if constexpr (GRAD && !BLOCK) {
#pragma unroll
        for (int k = 0; k < MAPS; ++k) guarded = guarded || !(fabsf(c[k]) < INFINITY);
        if (guarded) {
#pragma unroll
            for (int k = 0; k < MAPS; ++k) c[k] = warp_sum(run[k].c + dot(k, true));
        }
    }
    if constexpr (BLOCK) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            z[k] = c[k] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                z[k] += sh.sum[k][0][w];
                if constexpr (GRAD) c[k] += sh.sum[k][1][w];
            }
        }
    }
    float own[MAPS];  // what this CTA's weights are multiplied by to be the row's
#pragma unroll
    for (int k = 0; k < MAPS; ++k) own[k] = 1.f;
    if (BLOCK && ctas > 1) {
        if (threadIdx.x == 0) {
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                sh.whole[k][0] = m[k];
                sh.whole[k][1] = z[k];
                sh.whole[k][2] = c[k];
            }
        }
        cluster_sync();
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY;
            for (int i = 0; i < ctas; ++i) top = fmaxf(top, load_cluster(smem_addr(&sh.whole[k][0]), i));
            const float base = base_of(top);
            z[k] = c[k] = 0.f;
            for (int i = 0; i < ctas; ++i) {
                const float f = exp_flush(load_cluster(smem_addr(&sh.whole[k][0]), i) - base);
                z[k] += f * load_cluster(smem_addr(&sh.whole[k][1]), i);
                if constexpr (GRAD) c[k] += weighted(f, load_cluster(smem_addr(&sh.whole[k][2]), i));
            }
            own[k] = exp_flush(m[k] - base);
        }
        cluster_sync();  // no CTA goes on to overwrite, or leave, what another reads
    }
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        inv[k] = inverse(z[k]);
        if constexpr (GRAD) c[k] *= inv[k];
        inv[k] *= own[k];
    }
    if (GRAD && TWO && a.row_c2 && (BLOCK ? rank == 0 && threadIdx.x == 0 : lane == 0)) a.row_c2[r] = c[MAPS - 1];
    if constexpr (TWO) inv[1] *= -__ldg(a.lambda + r / a.seg_rows % a.heads);

    // The results of one quad from its weights (and dout).  Gradients are
    // w·(inv·d - inv·c).
    auto finish = [&](unsigned q, const float (&w)[MAPS][4], const float (&dy)[4]) {
        float y[4];
        if constexpr (GRAD) {
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                const float ic = -inv[k] * c[k];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float g = fmaf(inv[k], dy[u], ic);
                    y[u] = guarded ? weighted(w[k][u], g) : w[k][u] * g;
                }
                store_quad<OUT, VEC>(k == 0 ? a.out1 : a.out2, q, p0, p1, y);
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] = fmaf(w[0][u], inv[0], w[MAPS - 1][u] * inv[MAPS - 1]);
            store_quad<OUT, VEC>(a.out1, q, p0, p1, y);
        }
    };
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        const unsigned q = q0 + i * step;
        if (q < p1) finish(q, x[i], d[GRAD ? i : 0]);
    }
#pragma unroll 1
    for (unsigned q = tail; q < p1; q += step) {
        float y[MAPS][4], dy[4];
        load_scores(q, false, y);
        if constexpr (GRAD) load_quad<DIN, VEC>(a.dout, q, nnz, dy);
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            const float base = base_of(m[k]);
#pragma unroll
            for (int u = 0; u < 4; ++u) y[k][u] = exp_flush(y[k][u] - base);
        }
        finish(q, y, dy);
    }
}

// A warp per row; long rows by the CTA.
template <bool TWO, bool GRAD, bool DIN, bool OUT, bool VEC>
__global__ void __launch_bounds__(kThreads, TWO && GRAD ? 3 : 4) warp_rows_kernel(const MapArgs a) {
    __shared__ BlockStats sh;
    __shared__ int waits[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long first = (long long)blockIdx.x * kWarps;
    int p0 = 0, p1 = 0;
    const int r = (int)min(first + warp, (long long)a.M - 1);
    const bool live = first + warp < a.M;
    if (live) row_range(a.row_offsets, r, a.nnz, p0, p1);
    const bool is_long = (unsigned)(p1 - p0) > kLong;
    if (lane == 0) waits[warp] = is_long;
    if (live && !is_long) {
        if (p0 < p1)
            map_row<TWO, GRAD, DIN, OUT, VEC, false>(a, r, p0, p1, sh, 1, 0);
        else if (GRAD && TWO && a.row_c2 && lane == 0)
            a.row_c2[r] = 0.f;
    }
    if (!__syncthreads_or(is_long)) return;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
        if (!waits[w]) continue;
        row_range(a.row_offsets, (int)first + w, a.nnz, p0, p1);
        map_row<TWO, GRAD, DIN, OUT, VEC, true>(a, (int)first + w, p0, p1, sh, 1, 0);
    }
}

// A CTA, or a cluster, per row.
template <bool TWO, bool GRAD, bool DIN, bool OUT, bool VEC>
__global__ void __launch_bounds__(kThreads) block_rows_kernel(const MapArgs a) {
    __shared__ BlockStats sh;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    int p0, p1;
    row_range(a.row_offsets, r, a.nnz, p0, p1);
    if (p0 == p1) {
        if (GRAD && TWO && a.row_c2 && rank == 0 && threadIdx.x == 0) a.row_c2[r] = 0.f;
        return;
    }
    map_row<TWO, GRAD, DIN, OUT, VEC, true>(a, r, p0, p1, sh, ctas, rank);
}

// dλ[h] = -Σ c2 over head h's rows: a CTA per head, a fixed order.
__global__ void __launch_bounds__(1024) lambda_grad_kernel(int M, int blocks, int heads, int seg_rows,
                                                           const float* __restrict__ row_c2,
                                                           float* __restrict__ dlambda) {
    __shared__ float warp_part[32];
    const int head = blockIdx.x, t = threadIdx.x, lane = t & 31;
    float x = 0.f;
    for (long long b = head; b < blocks; b += heads) {
        const long long r0 = b * seg_rows;
        const int n = (int)min((long long)seg_rows, M - r0);
        for (int i = t; i < n; i += 1024) x += row_c2[r0 + i];
    }
    x = warp_sum(x);
    if (lane == 0) warp_part[t >> 5] = x;
    __syncthreads();
    if (t < 32) {
        x = warp_sum(warp_part[lane]);
        if (lane == 0) dlambda[head] = -x;
    }
}

template <bool TWO, bool GRAD, bool DIN, bool OUT, bool VEC>
int launch_rows(const MapArgs& a, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    const int mean = a.nnz / a.M;
    // A CTA a row where most rows are long, or where rows are too few to fill
    // the SMs with a warp each; a cluster where they are too few for CTAs.
    if (mean > (int)kLong || (mean > 128 * kQuads && a.M < kWarps * sms)) {
        int ctas = 1;
        while (ctas < 8 && (long long)a.M * ctas < 2LL * sms && mean / ctas > kThreads * 4 * kQuads / 2) ctas *= 2;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = ctas;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((long long)a.M * ctas));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, block_rows_kernel<TWO, GRAD, DIN, OUT, VEC>, a) == cudaSuccess ? USM_OK
                                                                                                      : USM_ERR_CUDA;
    }
    warp_rows_kernel<TWO, GRAD, DIN, OUT, VEC><<<(unsigned)(((long long)a.M + kWarps - 1) / kWarps), kThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

template <bool TWO, bool GRAD>
int launch_map(const MapArgs& a, cudaStream_t stream) {
    const bool vec = quad_aligned(a.s1, false) && (!TWO || quad_aligned(a.s2, false)) &&
                     (!GRAD || quad_aligned(a.dout, a.dout_bf16)) && quad_aligned(a.out1, a.out_bf16) &&
                     (!(GRAD && TWO) || quad_aligned(a.out2, a.out_bf16));
    auto pick = [&](auto din, auto out) {
        constexpr bool D = decltype(din)::value, O = decltype(out)::value;
        return vec ? launch_rows<TWO, GRAD, D, O, true>(a, stream) : launch_rows<TWO, GRAD, D, O, false>(a, stream);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    if (GRAD && a.dout_bf16) return a.out_bf16 ? pick(std::bool_constant<GRAD>{}, Yes{}) : pick(std::bool_constant<GRAD>{}, No{});
    return a.out_bf16 ? pick(No{}, Yes{}) : pick(No{}, No{});
}

}  // namespace

int launch_diff_softmax(const MapArgs& a, cudaStream_t stream) { return launch_map<true, false>(a, stream); }

int launch_row_softmax_grad(const MapArgs& a, cudaStream_t stream) { return launch_map<false, true>(a, stream); }

int launch_diff_softmax_grad(const MapArgs& a, float* dlambda, cudaStream_t stream) {
    const int r = launch_map<true, true>(a, stream);
    if (r != USM_OK || !dlambda) return r;
    lambda_grad_kernel<<<a.heads, 1024, 0, stream>>>(a.M, query_blocks(a.M, a.seg_rows), a.heads, a.seg_rows,
                                                       a.row_c2, dlambda);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

}  // namespace usm
