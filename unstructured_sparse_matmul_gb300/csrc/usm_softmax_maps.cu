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
// A CTA takes a run of rows: the long ones first, with all its warps, then its
// warps fetch the others one by one, so that neither a long row nor a long run
// of luck keeps seven warps waiting.  (A warp and a row each, with a barrier at
// the end for the long ones: half of all warp time at that barrier, 58 us at
// 8x4096 rows of 410.)  Where long rows are too few to fill the GPU, a cluster
// of up to 8 CTAs takes each (launch_rows), joined through distributed shared
// memory.  Arithmetic is in pairs (f32x2) where it can be: with eight to twelve
// bytes an entry, a kernel of more than about 16 instructions an entry and lane
// would be bound by issue slots instead.
#include <cmath>
#include <type_traits>

#include "usm_cluster.cuh"
#include "usm_internal.h"
#include "usm_quads.cuh"
#include "usm_rel.cuh"
#include "usm_rows.cuh"

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

// 1/z, or 0 for a row without weight; NaN stays NaN.
__device__ __forceinline__ float inverse(float z) { return z == 0.f ? 0.f : 1.f / z; }
// w·d, or 0 under a weight of 0 (a masked entry) whatever d is there.
__device__ __forceinline__ float weighted(float w, float d) { return w == 0.f ? 0.f : w * d; }

constexpr float kLog2e = 1.4426950408889634f;

// exp(s - m) as 2^(s·log2 e - shift), shift = m·log2 e: one fused product and the
// hardware's exponential.  The rounding of the shift is the same factor in every
// weight of the row and in their sum.  Scores so large that s·log2 e overflows
// are first brought near zero (off = m, shift = 0); a maximum of -inf (every
// entry masked) has shift 0, so that all weights are 0.
struct Base {
    float off, shift;
    __device__ __forceinline__ explicit Base(float m) {
        const bool huge = fabsf(m) > 1e37f && m != -INFINITY;
        off = huge ? m : 0.f;
        shift = huge || m == -INFINITY ? 0.f : m * kLog2e;
    }
    __device__ __forceinline__ bool huge() const { return off != 0.f; }
};
__device__ __forceinline__ float exp2_flush(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float weight_of(float s, const Base& b) {
    return exp2_flush(fmaf(s - b.off, kLog2e, -b.shift));
}

// Sums of one map over (part of) a row: the maximum m, z = Σ exp(s - m) and
// c = Σ exp(s - m)·d.
struct Stat {
    float m, z, c;
};

// Shared memory of a CTA: one slot a warp, and what its cluster reads.
struct BlockStats {
    float top[2][kWarps];
    float sum[2][2][kWarps];
    float whole_top[2];
    float whole[2][2];
};

// One row [p0, p1).  BLOCK: by the CTA (or its cluster's), else by the warp.
template <bool TWO, bool GRAD, bool DIN, bool OUT, bool VEC, bool BLOCK>
__device__ __forceinline__ void map_row(const MapArgs& a, int r, float lam, unsigned p0, unsigned p1, BlockStats& sh,
                                        int ctas, int rank) {
    constexpr int MAPS = TWO ? 2 : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned nnz = a.nnz;
    // Thread t of T takes quads t, t + T, ... of the row.
    const unsigned T = BLOCK ? kThreads * ctas : 32, t = BLOCK ? rank * kThreads + threadIdx.x : lane;
    const unsigned q0 = (p0 & ~3u) + 4 * t, step = 4 * T;
    const unsigned qw = (p0 & ~3u) + (BLOCK ? 4 * (t & ~31u) : 0);  // the warp's first quad
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
            const float f = top == -INFINITY ? 0.f : __expf(run[k].m - top);
            run[k].z *= f;
            run[k].c *= f;
            run[k].m = top;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float e = __expf(y[k][u] - (top == -INFINITY ? 0.f : top));
                run[k].z += e;
                if constexpr (GRAD) run[k].c += weighted(e, dy[u]);
            }
        }
    }

    // Maximum over the warp, the CTA, the cluster.
    float m[MAPS];
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        float top = run[k].m;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            if (qw + i * step < p1)
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
        if (ctas > 1) {
            if (threadIdx.x < MAPS) sh.whole_top[threadIdx.x] = threadIdx.x ? m[MAPS - 1] : m[0];
            cluster_sync();
#pragma unroll
            for (int k = 0; k < MAPS; ++k)
                for (int i = 0; i < ctas; ++i) m[k] = fmaxf(m[k], load_cluster(smem_addr(&sh.whole_top[k]), i));
        }
    }
    // Weights (in the scores' registers) and their sums.
    float z[MAPS], c[MAPS], inv[MAPS];
    auto dot = [&](int k, bool guarded) {
        float2 sum = make_float2(0.f, 0.f);
        if constexpr (GRAD) {
#pragma unroll
            for (int i = 0; i < kQuads; ++i)
                if (qw + i * step < p1) {
#pragma unroll
                    for (int u = 0; u < 4; u += 2) {
                        float2 w = make_float2(x[i][k][u], x[i][k][u + 1]), v = make_float2(d[i][u], d[i][u + 1]);
                        if (guarded) {
                            if (w.x == 0.f) v.x = 0.f;
                            if (w.y == 0.f) v.y = 0.f;
                        }
                        sum = __ffma2_rn(w, v, sum);
                    }
                }
        }
        return sum.x + sum.y;
    };
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        const Base base(m[k]);
        const float f = weight_of(run[k].m, base);
        z[k] = run[k].z * f;
        run[k].c *= f;
        const float2 scale = make_float2(kLog2e, kLog2e), shift = make_float2(-base.shift, -base.shift);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            if (qw + i * step < p1) {
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    float2 y = make_float2(x[i][k][u], x[i][k][u + 1]);
                    if (base.huge()) y = make_float2(y.x - base.off, y.y - base.off);
                    y = __ffma2_rn(y, scale, shift);
                    y = make_float2(exp2_flush(y.x), exp2_flush(y.y));
                    x[i][k][u] = y.x;
                    x[i][k][u + 1] = y.y;
                    sum = __fadd2_rn(sum, y);
                }
            }
        z[k] = warp_sum(z[k] + (sum.x + sum.y));
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
        if (ctas > 1) {
            if (threadIdx.x == 0) {
#pragma unroll
                for (int k = 0; k < MAPS; ++k) {
                    sh.whole[k][0] = z[k];
                    sh.whole[k][1] = c[k];
                }
            }
            cluster_sync();
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                z[k] = c[k] = 0.f;
                for (int i = 0; i < ctas; ++i) {
                    z[k] += load_cluster(smem_addr(&sh.whole[k][0]), i);
                    if constexpr (GRAD) c[k] += load_cluster(smem_addr(&sh.whole[k][1]), i);
                }
            }
            cluster_sync();  // no CTA leaves what another may still read
        }
    }
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        inv[k] = inverse(z[k]);
        if constexpr (GRAD) c[k] *= inv[k];
    }
    if (GRAD && TWO && a.row_c2 && (BLOCK ? rank == 0 && threadIdx.x == 0 : lane == 0)) a.row_c2[r] = c[MAPS - 1];
    if constexpr (TWO) inv[1] *= -lam;

    // The results of one quad from its weights (and dout).  Gradients are
    // w·(inv·d - inv·c).
    auto finish = [&](unsigned q, const float (&w)[MAPS][4], const float (&dy)[4]) {
        float y[4];
        if constexpr (GRAD) {
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                const float ic = -inv[k] * c[k];
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    const float2 g = __ffma2_rn(make_float2(inv[k], inv[k]), make_float2(dy[u], dy[u + 1]), make_float2(ic, ic));
                    const float2 v = __fmul2_rn(make_float2(w[k][u], w[k][u + 1]), g);
                    y[u] = v.x;
                    y[u + 1] = v.y;
                    if (guarded) {
                        if (w[k][u] == 0.f) y[u] = 0.f;
                        if (w[k][u + 1] == 0.f) y[u + 1] = 0.f;
                    }
                }
                store_quad<OUT, VEC>(k == 0 ? a.out1 : a.out2, q, p0, p1, y);
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
                float2 v = __fmul2_rn(make_float2(w[MAPS - 1][u], w[MAPS - 1][u + 1]), make_float2(inv[MAPS - 1], inv[MAPS - 1]));
                v = __ffma2_rn(make_float2(w[0][u], w[0][u + 1]), make_float2(inv[0], inv[0]), v);
                y[u] = v.x;
                y[u + 1] = v.y;
            }
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
            const Base base(m[k]);
#pragma unroll
            for (int u = 0; u < 4; ++u) y[k][u] = weight_of(y[k][u], base);
        }
        finish(q, y, dy);
    }
}

// Rows [M·b / B, M·(b+1) / B) of CTA b of B, 64 at a time: rows over `long_at`
// entries by the whole CTA, then each warp fetches row after row.
template <bool TWO, bool GRAD, bool DIN, bool OUT, bool VEC>
__global__ void __launch_bounds__(kThreads, TWO && GRAD ? 3 : 4) row_runs_kernel(const MapArgs a, unsigned long_at) {
    __shared__ BlockStats sh;
    __shared__ RowRun run;
    __shared__ float lams[kRun];
    const int lane = threadIdx.x & 31;
    const long long r0 = (long long)a.M * blockIdx.x / gridDim.x, r1 = (long long)a.M * (blockIdx.x + 1) / gridDim.x;
    for (long long r = r0; r < r1; r += kRun) {
        const int n = (int)min((long long)kRun, r1 - r);
        const bool any_long =
            run.load(a.row_offsets, a.nnz, n, long_at, [&](int i) { return (int)r + i; },
                     [&](int i, int row) {
                         if (TWO) lams[i] = __ldg(a.lambda + row / a.seg_rows % a.heads);
                     });
        if (any_long) {
#pragma unroll 1
            for (int i = 0; i < n; ++i)
                if ((unsigned)(run.end[i] - run.begin[i]) > long_at)
                    map_row<TWO, GRAD, DIN, OUT, VEC, true>(a, (int)r + i, TWO ? lams[i] : 0.f, run.begin[i], run.end[i], sh, 1, 0);
        }
        for (int i = run.fetch(lane); i < n; i = run.fetch(lane)) {
            const unsigned p0 = run.begin[i], p1 = run.end[i];
            if (p0 == p1) {
                if (GRAD && TWO && a.row_c2 && lane == 0) a.row_c2[r + i] = 0.f;
            } else if (p1 - p0 <= long_at) {
                map_row<TWO, GRAD, DIN, OUT, VEC, false>(a, (int)r + i, TWO ? lams[i] : 0.f, p0, p1, sh, 1, 0);
            }
        }
        __syncthreads();  // the next run's rows overwrite this one's
    }
}

// A cluster per row.
template <bool TWO, bool GRAD, bool DIN, bool OUT, bool VEC>
__global__ void __launch_bounds__(kThreads) cluster_rows_kernel(const MapArgs a) {
    __shared__ BlockStats sh;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    int p0, p1;
    row_range(a.row_offsets, r, a.nnz, p0, p1);
    if (p0 == p1) {
        if (GRAD && TWO && a.row_c2 && rank == 0 && threadIdx.x == 0) a.row_c2[r] = 0.f;
        return;
    }
    const float lam = TWO ? __ldg(a.lambda + r / a.seg_rows % a.heads) : 0.f;
    map_row<TWO, GRAD, DIN, OUT, VEC, true>(a, r, lam, p0, p1, sh, ctas, rank);
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
    // Clusters where rows are long (their CTAs hold over half a CTA's registers'
    // worth each) and too few to give every SM one.
    int ctas = 1;
    while (ctas < 8 && (long long)a.M * ctas < 2LL * sms && mean / ctas > kThreads * 4 * kQuads / 2) ctas *= 2;
    if (ctas > 1) {
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
        return cudaLaunchKernelEx(&cfg, cluster_rows_kernel<TWO, GRAD, DIN, OUT, VEC>, a) == cudaSuccess ? USM_OK
                                                                                                        : USM_ERR_CUDA;
    }
    // A CTA each while there are fewer rows than CTA slots (a CTA then takes rows
    // that a warp would have to walk twice), else one wave of CTAs.
    const int slots = sms * (TWO && GRAD ? 3 : 4);
    const bool few = a.M <= slots;
    row_runs_kernel<TWO, GRAD, DIN, OUT, VEC>
        <<<few ? a.M : slots, kThreads, 0, stream>>>(a, few ? 32 * 4 * kQuads : kLong);
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
