// Softmax maps over CSR rows and their gradients:
//     differential map   A = P1 - λ P2,
//     its gradient       dS1 = P1 (dA - c1), dS2 = -λ P2 (dA - c2), dλ = -Σ_rows c2, ck = Σ_row Pk dA,
//     softmax gradient   dS = P (dP - Σ_row P dP),
// Pk = exp(sk - mk) / zk, mk the row's maximum, zk = Σ exp(sk - mk) over its
// stored entries.
//
// Bound by memory: 8 to 12 bytes a nonzero in, 2 to 8 out, each once.  Every warp
// takes the rows that begin in an equal share of the entries and streams them
// through a ring in shared memory (usm_stream.cuh), so copies are in flight all
// the time whatever the rows' arithmetic and lengths do.  An SM's shared memory
// holds the rings of 8 to 16 warps, few to cover the latency of a row's
// arithmetic, which is what is left to wait for (figures: the differential map of
// 8x4096 rows of 410 entries in a replayed graph):
//   - A row is walked twice in the ring (weights and their sums; results), four
//     entries a lane, in pairs of fp32 (f32x2).  Loops are short: rows read into
//     registers, unrolled, measured 47 to 58 us where these took 45 and, with what
//     follows, 37.  (Weights written back to the ring instead of formed twice save
//     0.6 us, but the scores with them, which a second try needs.)
//   - Two rows of about a length are taken at once, by half a warp each (42.7 to
//     39.7 us), or four short ones.
//   - The maximum is not looked for (45 to 42 us): exponents are measured from
//     the largest of a few entries (at the row's ends and in its middle), which
//     gives the same quotients.  An
//     exponent x = s·log2 e - m·log2 e is off by half a step, 2^-20 for |x| up to
//     32 (7e-7 of the weight); a row whose sum is not in [1/4, 2^31) is done again
//     from its maximum: rows with masks at all those places, with values that are
//     not finite, or with scores so far from zero that the rounding of m·log2 e
//     leaves the exponents' range (all rows again: 51 us).
//   - Rows that do not fit the ring are first taken by the whole CTA (rows of even
//     lengths: 33 us); where most rows are long, a CTA takes each, or a cluster of
//     up to 8 (launch_rows).
#include <cmath>
#include <type_traits>

#include "usm_cluster.cuh"
#include "usm_internal.h"
#include "usm_stream.cuh"
#include "usm_sums.cuh"

namespace usm {
namespace {

constexpr int kSteps = 16;  // entries of a long row a thread keeps in registers
constexpr int kTail = 16;   // and has in flight of the others (82 rows of 16384 entries among 2048: 27 us; 8: 29, 4: 33)

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

// 1/z (within one step of 2^-23), or 0 for a row without weight; NaN stays NaN.
__device__ __forceinline__ float inverse(float z) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(z));
    return z == 0.f ? 0.f : y;
}
// w·d, or 0 under a weight of 0 (a masked entry) whatever d is there.
__device__ __forceinline__ float weighted(float w, float d) { return w == 0.f ? 0.f : w * d; }

constexpr float kLog2e = 1.4426950408889634f;

// exp(s - m) as 2^(s·log2 e - shift), shift = m·log2 e: one fused product and the
// hardware's exponential.  The rounding of the shift is the same factor in every
// weight of the row and in their sum: up to |m| = kNear it is half a step of 2 at
// most, a factor between 1/2 and 2; from about 1e9 on the factor would be infinite
// or 0.  Scores with a maximum beyond kNear are therefore first brought near zero
// (off = m, shift = 0: one more rounding, relative to s - m).  A maximum of -inf
// (every entry masked) has shift 0, so that all weights are 0.
constexpr float kNear = 0x1p24f;
struct Base {
    float off, shift;
    __device__ __forceinline__ explicit Base(float m) {
        const bool far = fabsf(m) > kNear && m != -INFINITY;
        off = far ? m : 0.f;
        shift = far || m == -INFINITY ? 0.f : m * kLog2e;
    }
    __device__ __forceinline__ bool far() const { return off != 0.f; }
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

// Shared memory of a CTA that takes a row: one slot a warp, and what its cluster
// reads.
template <int WARPS>
struct BlockStats {
    float top[2][WARPS];
    float sum[2][2][WARPS];
    float whole_top[2];
    float whole[2][2];
};

// A long row [p0, p1) by the CTA's WARPS warps, or its cluster's: 16 entries a
// thread in registers, the rest read twice.
template <bool TWO, bool GRAD, bool DIN, bool OUT, int WARPS>
__device__ __forceinline__ void block_row(const MapArgs& a, int r, float lam, int p0, int p1, BlockStats<WARPS>& sh, int ctas,
                                        int rank) {
    constexpr int MAPS = TWO ? 2 : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Thread t of T takes entries t, t + T, ... of the row.
    const int T = WARPS * 32 * ctas, t = rank * WARPS * 32 + threadIdx.x;
    const int n = p1 - p0, nw = n - (t - lane);  // entries of the row, and from the warp's first one on
    const float* s[2] = {a.s1 + p0, TWO ? a.s2 + p0 : nullptr};
    const void* dout = GRAD ? static_cast<const char*>(a.dout) + (long long)p0 * (DIN ? 2 : 4) : nullptr;
    void* out[2] = {static_cast<char*>(a.out1) + (long long)p0 * (OUT ? 2 : 4),
                    GRAD && TWO ? static_cast<char*>(a.out2) + (long long)p0 * (OUT ? 2 : 4) : nullptr};

    // Steps come in pairs; a pair without an entry in the warp is skipped.
    float2 x[MAPS][kSteps / 2], d[GRAD ? kSteps / 2 : 1];
#pragma unroll
    for (int i = 0; i < kSteps / 2; ++i) {
        const int e = t + 2 * i * T;
        if (2 * i * T < nw) {
#pragma unroll
            for (int k = 0; k < MAPS; ++k)
                x[k][i] = make_float2(e < n ? s[k][e] : -INFINITY, e + T < n ? s[k][e + T] : -INFINITY);
            if constexpr (GRAD)
                d[i] = make_float2(e < n ? load_global<DIN>(dout, e) : 0.f, e + T < n ? load_global<DIN>(dout, e + T) : 0.f);
        }
    }
    // Entries past the registers, kTail at a time: a running maximum and sums.
    const unsigned tail = t + kSteps * T, un = n;  // unsigned: a tail's end may pass 2^31
    Stat run[MAPS];
#pragma unroll
    for (int k = 0; k < MAPS; ++k) run[k] = {-INFINITY, 0.f, 0.f};
    auto load_tail = [&](unsigned e, float (&y)[MAPS][kTail], float (&dy)[kTail]) {
#pragma unroll
        for (int u = 0; u < kTail; ++u) {
            const bool in = e + u * T < un;
#pragma unroll
            for (int k = 0; k < MAPS; ++k) y[k][u] = in ? s[k][e + u * T] : -INFINITY;
            dy[u] = GRAD && in ? load_global<DIN>(dout, e + u * T) : 0.f;
        }
    };
#pragma unroll 1
    for (unsigned e = tail; e < un; e += kTail * T) {
        float y[MAPS][kTail], dy[kTail];
        load_tail(e, y, dy);
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = run[k].m;
#pragma unroll
            for (int u = 0; u < kTail; ++u) top = fmaxf(top, y[k][u]);
            const float base = top == -INFINITY ? 0.f : top, f = __expf(run[k].m - base);
            run[k].z *= f;
            run[k].c *= f;
            run[k].m = top;
#pragma unroll
            for (int u = 0; u < kTail; ++u) {
                const float w = __expf(y[k][u] - base);
                run[k].z += w;
                if constexpr (GRAD) run[k].c += weighted(w, dy[u]);
            }
        }
    }

    // Maximum over the warp, the CTA, the cluster.
    float m[MAPS];
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        float top = run[k].m;
#pragma unroll
        for (int i = 0; i < kSteps / 2; ++i)
            if (2 * i * T < nw) top = fmaxf(top, fmaxf(x[k][i].x, x[k][i].y));
        m[k] = warp_max(top);
        if (lane == 0) sh.top[k][warp] = m[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MAPS; ++k)
#pragma unroll
        for (int w = 0; w < WARPS; ++w) m[k] = fmaxf(m[k], sh.top[k][w]);
    if (ctas > 1) {
        if (threadIdx.x < MAPS) sh.whole_top[threadIdx.x] = threadIdx.x ? m[MAPS - 1] : m[0];
        cluster_sync();
#pragma unroll
        for (int k = 0; k < MAPS; ++k)
            for (int i = 0; i < ctas; ++i) m[k] = fmaxf(m[k], load_cluster(smem_addr(&sh.whole_top[k]), i));
    }
    // Weights (in the scores' registers) and their sums.
    float z[MAPS], c[MAPS], inv[MAPS];
    auto dot = [&](int k) {
        float2 sum = make_float2(0.f, 0.f);
        if constexpr (GRAD) {
#pragma unroll
            for (int i = 0; i < kSteps / 2; ++i)
                if (2 * i * T < nw) {
                    float2 v = d[i];
                    if (x[k][i].x == 0.f) v.x = 0.f;
                    if (x[k][i].y == 0.f) v.y = 0.f;
                    sum = __ffma2_rn(x[k][i], v, sum);
                }
        }
        return sum.x + sum.y;
    };
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        const Base base(m[k]);
        if (base.far()) {
#pragma unroll
            for (int i = 0; i < kSteps / 2; ++i)
                if (2 * i * T < nw) x[k][i] = make_float2(x[k][i].x - base.off, x[k][i].y - base.off);
        }
        const float f = weight_of(run[k].m, base);
        z[k] = run[k].z * f;
        run[k].c *= f;
        const float2 scale = make_float2(kLog2e, kLog2e), shift = make_float2(-base.shift, -base.shift);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kSteps / 2; ++i)
            if (2 * i * T < nw) {
                const float2 y = __ffma2_rn(x[k][i], scale, shift);
                x[k][i] = make_float2(exp2_flush(y.x), exp2_flush(y.y));
                sum = __fadd2_rn(sum, x[k][i]);
            }
        z[k] = warp_sum(z[k] + (sum.x + sum.y));
        c[k] = 0.f;
        if constexpr (GRAD) c[k] = warp_sum(run[k].c + dot(k));
        if (lane == 0) {
            sh.sum[k][0][warp] = z[k];
            sh.sum[k][1][warp] = c[k];
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        z[k] = c[k] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
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
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        inv[k] = inverse(z[k]);
        if constexpr (GRAD) c[k] *= inv[k];
    }
    if (GRAD && TWO && a.row_c2 && rank == 0 && threadIdx.x == 0) a.row_c2[r] = c[MAPS - 1];
    if constexpr (TWO) inv[1] *= -lam;

    // The results of two entries from their weights (and dout).  Gradients are
    // w·(inv·d - inv·c).
    auto finish = [&](unsigned e, const float2 (&w)[MAPS], float2 dy) {
        if constexpr (GRAD) {
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                const float ic = -inv[k] * c[k];
                float2 y = __fmul2_rn(w[k], __ffma2_rn(make_float2(inv[k], inv[k]), dy, make_float2(ic, ic)));
                if (w[k].x == 0.f) y.x = 0.f;
                if (w[k].y == 0.f) y.y = 0.f;
                if (e < un) store_entry<OUT>(out[k], e, y.x);
                if (e + T < un) store_entry<OUT>(out[k], e + T, y.y);
            }
        } else {
            float2 y = __fmul2_rn(w[MAPS - 1], make_float2(inv[MAPS - 1], inv[MAPS - 1]));
            y = __ffma2_rn(w[0], make_float2(inv[0], inv[0]), y);
            if (e < un) store_entry<OUT>(out[0], e, y.x);
            if (e + T < un) store_entry<OUT>(out[0], e + T, y.y);
        }
    };
#pragma unroll
    for (int i = 0; i < kSteps / 2; ++i)
        if (2 * i * T < nw) {
            float2 w[MAPS];
#pragma unroll
            for (int k = 0; k < MAPS; ++k) w[k] = x[k][i];
            finish(t + 2 * i * T, w, d[GRAD ? i : 0]);
        }
#pragma unroll 1
    for (unsigned e = tail; e < un; e += kTail * T) {
        float y[MAPS][kTail], dy[kTail];
        load_tail(e, y, dy);
#pragma unroll
        for (int u = 0; u < kTail; u += 2) {
            float2 w[MAPS];
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                const Base base(m[k]);
                w[k] = make_float2(weight_of(y[k][u], base), weight_of(y[k][u + 1], base));
            }
            finish(e + u * T, w, make_float2(dy[u], dy[u + 1]));
        }
    }
}

// Out of line in the kernel below: long rows are rare there.
template <bool TWO, bool GRAD, bool DIN, bool OUT, int WARPS>
__device__ __noinline__ void long_row(const MapArgs& a, int r, float lam, int p0, int p1, BlockStats<WARPS>& sh) {
    block_row<TWO, GRAD, DIN, OUT, WARPS>(a, r, lam, p0, p1, sh, 1, 0);
}

// A row [p0, p1), which lies in the warp's ring, by the
// warp, half or a quarter of it (width 32, 16 or 8, the same for all lanes; each
// part has its own row, which may be empty: false), walked twice: for weights and
// their sums, and for results.  MAX: exponents are measured from the row's maximum; else
// from the largest of a few entries, and false if that does not do (nothing is
// changed then).
template <bool TWO, bool GRAD, bool DIN, bool OUT, bool MAX, class S>
__device__ __forceinline__ bool ring_row(const MapArgs& a, const S& st, int width, int r, float lam, int p0, int p1, bool vec) {
    constexpr int MAPS = TWO ? 2 : 1;
    const int base = threadIdx.x & 31 & -width, lane = threadIdx.x & (width - 1);
    const unsigned step = 4 * width;
    const RowQuads rq(p0, p1, lane);
    const unsigned first = rq.qs + 4 * lane;
    // Lane 4 looks at the row's middle (padding may be on the left).
    const unsigned probe = lane == 4 && rq.qs < rq.qe ? rq.qs + (((rq.qe - rq.qs) >> 1) & ~3u) : first;

    float m[MAPS], xe[MAPS];
    const float de = GRAD && rq.has_edge ? lds_entry<DIN>(st.at(MAPS, rq.edge)) : 0.f;
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        xe[k] = rq.has_edge ? lds_f32(st.at(k, rq.edge)) : -INFINITY;
        m[k] = xe[k];
#pragma unroll 1
        for (unsigned q = MAX ? first : probe; q < rq.qe; q += step) {
            float2 lo, hi;
            lds_quad<false>(st.at(k, q), lo, hi);
            m[k] = fmaxf(m[k], fmaxf(fmaxf(lo.x, lo.y), fmaxf(hi.x, hi.y)));
            if (!MAX) break;
        }
        if (MAX) {
            m[k] = warp_max(m[k]);
            // A maximum of -inf (every entry masked) leaves the scores as they are, and
            // scores with one beyond kNear are brought near zero first.
            if (!(fabsf(m[k]) <= kNear)) {
                if (m[k] != -INFINITY) {
                    xe[k] -= m[k];
#pragma unroll 1
                    for (unsigned q = first; q < rq.qe; q += step) {
                        float2 lo, hi;
                        lds_quad<false>(st.at(k, q), lo, hi);
                        sts_quad(st.at(k, q), make_float2(lo.x - m[k], lo.y - m[k]), make_float2(hi.x - m[k], hi.y - m[k]));
                    }
                }
                m[k] = 0.f;
            }
        } else {
            m[k] = fmaxf(__shfl_sync(kFullMask, m[k], base), __shfl_sync(kFullMask, m[k], base + 4));
        }
    }

    // Weights exp(s - m) = 2^(s·log2 e - m·log2 e), and their sums.
    float z[MAPS], c[MAPS], inv[MAPS];
    float2 zs[MAPS], cs[MAPS], shift[MAPS];
    const float2 scale = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        const float sh = -m[k] * kLog2e;
        shift[k] = make_float2(sh, sh);
        xe[k] = exp2_flush(fmaf(xe[k], kLog2e, sh));
        zs[k] = make_float2(xe[k], 0.f);
        cs[k] = make_float2(GRAD ? __fmul_rn(xe[k], de) : 0.f, 0.f);
    }
    // (Formed again for the results: cheaper than writing them back.)
    auto weights = [&](int k, unsigned q, float2& lo, float2& hi) {
        lds_quad<false>(st.at(k, q), lo, hi);
        lo = __ffma2_rn(lo, scale, shift[k]);
        hi = __ffma2_rn(hi, scale, shift[k]);
        lo = make_float2(exp2_flush(lo.x), exp2_flush(lo.y));
        hi = make_float2(exp2_flush(hi.x), exp2_flush(hi.y));
    };
#pragma unroll 1
    for (unsigned q = first; q < rq.qe; q += step) {
        float2 d0, d1;
        if constexpr (GRAD) lds_quad<DIN>(st.at(MAPS, q), d0, d1);
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float2 lo, hi;
            weights(k, q, lo, hi);
            zs[k] = __fadd2_rn(zs[k], __fadd2_rn(lo, hi));
            if constexpr (GRAD) cs[k] = __ffma2_rn(hi, d1, __ffma2_rn(lo, d0, cs[k]));
        }
    }
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        z[k] = zs[k].x + zs[k].y;
        c[k] = cs[k].x + cs[k].y;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o < 8 || o < width)
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                z[k] += __shfl_xor_sync(kFullMask, z[k], o);
                if constexpr (GRAD) c[k] += __shfl_xor_sync(kFullMask, c[k], o);
            }
    // A dout that is not finite makes c so too, even under weights of 0: such a
    // row leaves those products out.
    bool fine = true, guarded = false;
    auto at_weight = [&](float2 w, float2 v) { return make_float2(w.x == 0.f ? 0.f : v.x, w.y == 0.f ? 0.f : v.y); };
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        fine = fine && z[k] >= 0.25f && z[k] < 0x1p31f;
        if constexpr (GRAD) guarded = guarded || !(fabsf(c[k]) < 0x1p100f);
    }
    if (GRAD && __any_sync(kFullMask, guarded)) {
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float2 sum = make_float2(xe[k] != 0.f ? __fmul_rn(xe[k], de) : 0.f, 0.f);
#pragma unroll 1
            for (unsigned q = first; q < rq.qe; q += step) {
                float2 d0, d1, lo, hi;
                lds_quad<DIN>(st.at(MAPS, q), d0, d1);
                weights(k, q, lo, hi);
                sum = __ffma2_rn(hi, at_weight(hi, d1), __ffma2_rn(lo, at_weight(lo, d0), sum));
            }
            float x = sum.x + sum.y;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                if (o < 8 || o < width) x += __shfl_xor_sync(kFullMask, x, o);
            if (guarded) c[k] = x;
            fine = fine && fabsf(c[k]) < 0x1p100f;
        }
    }
    if (!MAX && !fine) return false;
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        inv[k] = inverse(z[k]);
        if constexpr (GRAD) c[k] *= inv[k];
    }
    if (GRAD && TWO && a.row_c2 && lane == 0) a.row_c2[r] = c[MAPS - 1];
    if constexpr (TWO) inv[1] *= -lam;

    // Results.  Gradients are w·(inv·d - inv·c).
    auto map = [&](const float2 (&w)[MAPS]) {
        const float2 y = __fmul2_rn(w[MAPS - 1], make_float2(inv[MAPS - 1], inv[MAPS - 1]));
        return TWO ? __ffma2_rn(w[0], make_float2(inv[0], inv[0]), y) : y;
    };
    // slow: outputs off 16 bytes, or products to leave out (told apart in the loop it
    // costs the others 2 us of 37).
    auto results = [&](auto slow) {
        auto grad = [&](int k, float2 w, float2 d) {
            const float ic = -inv[k] * c[k];
            if (slow() && guarded) d = at_weight(w, d);
            const float2 y = __fmul2_rn(w, __ffma2_rn(make_float2(inv[k], inv[k]), d, make_float2(ic, ic)));
            return slow() && guarded ? at_weight(w, y) : y;
        };
        if (rq.has_edge) {
            if constexpr (GRAD) {
                store_entry<OUT>(a.out1, rq.edge, grad(0, make_float2(xe[0], 0.f), make_float2(de, 0.f)).x);
                if constexpr (TWO) store_entry<OUT>(a.out2, rq.edge, grad(1, make_float2(xe[1], 0.f), make_float2(de, 0.f)).x);
            } else {
                float2 w[MAPS];
#pragma unroll
                for (int k = 0; k < MAPS; ++k) w[k] = make_float2(xe[k], 0.f);
                store_entry<OUT>(a.out1, rq.edge, map(w).x);
            }
        }
#pragma unroll 1
        for (unsigned q = first; q < rq.qe; q += step) {
            float2 lo[MAPS], hi[MAPS];
#pragma unroll
            for (int k = 0; k < MAPS; ++k) weights(k, q, lo[k], hi[k]);
            if constexpr (GRAD) {
                float2 d0, d1;
                lds_quad<DIN>(st.at(MAPS, q), d0, d1);
                store_quad<OUT>(a.out1, q, grad(0, lo[0], d0), grad(0, hi[0], d1), !slow() || vec);
                if constexpr (TWO) store_quad<OUT>(a.out2, q, grad(1, lo[1], d0), grad(1, hi[1], d1), !slow() || vec);
            } else {
                store_quad<OUT>(a.out1, q, map(lo), map(hi), !slow() || vec);
            }
        }
    };
    if (!vec || guarded)
        results(std::true_type{});
    else
        results(std::false_type{});
    return true;
}

// The same from the row's maximum, out of line: rarely needed.
template <bool TWO, bool GRAD, bool DIN, bool OUT, class S>
__device__ __noinline__ void max_row(const MapArgs& a, const S& st, int r, float lam, int p0, int p1, bool vec) {
    ring_row<TWO, GRAD, DIN, OUT, true>(a, st, 32, r, lam, p0, p1, vec);
}

template <bool TWO, bool GRAD, bool DIN>
using MapStream = Stream<4, TWO ? 4 : (GRAD ? (DIN ? 2 : 4) : 0), TWO && GRAD ? (DIN ? 2 : 4) : 0>;

constexpr int kWarps = 4, kThreads = kWarps * 32;

// CTAs an SM that the rings leave room for, at most 6 (80 registers a thread).
template <class S>
constexpr int ctas_per_sm() {
    constexpr int n = 224 * 1024 / (kWarps * S::kBytes + 1536);
    return n > 6 ? 6 : n;
}

// Warp g of G takes the rows that begin in share g of the entries.  vec: the
// outputs start on whole quads.
template <bool TWO, bool GRAD, bool DIN, bool OUT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<MapStream<TWO, GRAD, DIN>>())
    stream_rows_kernel(const MapArgs a, int G, bool aligned, bool vec) {
    if (TWO && GRAD && a.row_c2) let_next_start();
    using S = MapStream<TWO, GRAD, DIN>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ BlockStats<kWarps> sh;
    __shared__ int bounds[kWarps + 1];
    __shared__ unsigned is_long[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.x * kWarps + warp;
    const int t0 = share_begin(a.nnz, min(g, G), G), t1 = share_begin(a.nnz, min(g + 1, G), G);
    S st;
    st.src[0] = reinterpret_cast<const unsigned char*>(a.s1);
    st.src[1] = static_cast<const unsigned char*>(TWO ? (const void*)a.s2 : a.dout);
    st.src[2] = static_cast<const unsigned char*>(a.dout);
    st.base = smem_addr(smem) + warp * S::kBytes;
    st.nnz = a.nnz;
    st.lane = lane;
    st.aligned = aligned;
    st.whole = aligned ? a.nnz / kChunk : 0;
    st.issued = 0;
    st.limit = (int)(((long long)t1 + kChunk - 1) / kChunk);
    st.seek(t0);  // the copies need not wait for the search
    int r0, r1;
    first_rows_from(a.row_offsets, a.M, t0, t1, lane, r0, r1);
    RowWalk walk{a.row_offsets, a.M, a.nnz, lane, -64, 0};
    int p0, p1;
    bool any_long = false;
    if (r0 < r1) {
        const int end = min(max(__ldg(a.row_offsets + r1), 0), a.nnz);
        walk.hold(r0, 2);
        st.extend((int)(((long long)end + kChunk - 1) / kChunk));
        any_long = walk.any_over(r0, r1);
    }
    if (lane == 0) {
        bounds[warp] = r0;
        if (warp == kWarps - 1) bounds[kWarps] = r1;
    }
    // Long rows by the CTA, while the rings fill.
    if (__syncthreads_or(any_long)) {
        const int past = bounds[kWarps];
        RowWalk all{a.row_offsets, a.M, a.nnz, lane, -64, 0};
#pragma unroll 1
        for (int r = bounds[0]; r < past;) {
            const int rows = min(past - r, kThreads);
            bool some = false, mine = false;
            if (threadIdx.x < rows) {
                row_range(a.row_offsets, r + threadIdx.x, a.nnz, p0, p1);
                some = p0 < p1;
                mine = some && !ring_holds(p0, p1);
            }
            const unsigned mask = __ballot_sync(kFullMask, mine);
            if (lane == 0) is_long[warp] = mask;
            some = __syncthreads_or(some);
#pragma unroll 1
            for (int w = 0; w < kWarps; ++w)
#pragma unroll 1
                for (unsigned left = is_long[w]; left; left &= left - 1) {
                    const int row = r + w * 32 + __ffs(left) - 1;
                    row_range(a.row_offsets, row, a.nnz, p0, p1);
                    long_row<TWO, GRAD, DIN, OUT, kWarps>(a, row, TWO ? __ldg(a.lambda + row / a.seg_rows % a.heads) : 0.f,
                                                          p0, p1, sh);
                }
            __syncthreads();  // is_long is read
            r += rows;
            // Runs of rows without entries are passed by a search, the same in every
            // warp: `all` is where the others' are.
            if (!some && r < past) r = all.with_entries(r, past);
        }
    }
    float lam = 0.f;
    long long block_end = 0;  // lam is the head's of the rows before this one
#pragma unroll 1
    for (int r = r0; r < r1;) {
        // Two rows of about a length by half a warp each: a row's fixed part (its sums
        // over lanes, first entries, edges) is half its instructions otherwise, as
        // much as another 450 entries (differences of up to 128, 256 and 512 entries
        // measured 41.0, 39.7 and 41.1 us).
        // Four short rows by a quarter each (32768 rows of 64: gradient 29 us, 32 by
        // halves; 1M rows of 8: map 150 us, 236 by halves).
        walk.hold(r, 4);
        const int begin = walk.offset(r), mid = max(walk.offset(r, 1), begin), far = max(walk.offset(r, 2), mid);
        const bool pair = r + 1 < r1 && ring_holds(begin, far) && abs((mid - begin) - (far - mid)) < 256;
        p0 = begin;
        p1 = mid;
        int end = mid, width = 32, part = 0;
        if (pair) {
            width = 16;
            part = lane >> 4;
            end = far;
            p0 = part ? mid : begin;
            p1 = part ? far : mid;
            if (far - begin <= 128 && r + 3 < r1) {
                const int third = max(walk.offset(r, 3), far), fourth = max(walk.offset(r, 4), third);
                if (fourth - begin <= 256) {
                    width = 8;
                    part = lane >> 3;
                    end = fourth;
                    p0 = part == 0 ? begin : part == 1 ? mid : part == 2 ? far : third;
                    p1 = part == 0 ? mid : part == 1 ? far : part == 2 ? third : fourth;
                }
            }
        }
        if (begin == end) {
            r = walk.with_entries(r, r1);
            continue;
        }
        const int row = r + part;
        r += 32 / width;
        if (!ring_holds(begin, end)) continue;  // a long row
        st.need(begin, end);
        if (TWO && row >= block_end) {
            const int block = row / a.seg_rows;
            block_end = (block + 1LL) * a.seg_rows;
            lam = __ldg(a.lambda + block % a.heads);
        }
        bool done = ring_row<TWO, GRAD, DIN, OUT, false>(a, st, width, row, lam, p0, p1, vec);
        done = done || p0 == p1;
        const unsigned leaders = width == 8 ? 0x01010101u : width == 16 ? 0x10001u : 1u;
        for (unsigned again = __ballot_sync(kFullMask, !done) & leaders; again; again &= again - 1) {
            const int from = __ffs(again) - 1;
            max_row<TWO, GRAD, DIN, OUT>(a, st, __shfl_sync(kFullMask, row, from), __shfl_sync(kFullMask, lam, from),
                                         __shfl_sync(kFullMask, p0, from), __shfl_sync(kFullMask, p1, from), vec);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // copies of rows left to the CTA
}

// A CTA or a cluster to a row.
template <bool TWO, bool GRAD, bool DIN, bool OUT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) cluster_rows_kernel(const MapArgs a) {
    if (TWO && GRAD && a.row_c2) let_next_start();
    __shared__ BlockStats<WARPS> sh;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    int p0, p1;
    row_range(a.row_offsets, r, a.nnz, p0, p1);
    if (p0 == p1) return;
    const float lam = TWO ? __ldg(a.lambda + r / a.seg_rows % a.heads) : 0.f;
    block_row<TWO, GRAD, DIN, OUT, WARPS>(a, r, lam, p0, p1, sh, ctas, rank);
}

// dλ[h] = -Σ c2 over head h's rows (those with entries: the others have no c2): a
// cluster per head, a fixed order, in two fp32 numbers, since rows may cancel.  CTAs
// are small, so that they fit beside those of the kernel before (with 1024 threads
// they start after it: 3 us later).
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) lambda_grad_kernel(const MapArgs a, int blocks, float* __restrict__ dlambda) {
    __shared__ LongSum warp_part[kSumThreads / 32], whole;
    await_previous();
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int head = blockIdx.x / ctas, t = threadIdx.x, lane = t & 31;
    LongSum x;
    // Rows of all of the head's blocks, one after the other.
    const long long rows = head < blocks ? ((blocks - 1 - head) / a.heads + 1LL) * a.seg_rows : 0;
    // Four rows a thread in flight.
    for (long long i0 = rank * kSumThreads + t; i0 < rows; i0 += 4 * kSumThreads * ctas) {
        float c2[4];
        bool some[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const unsigned i = (unsigned)min(i0 + u * kSumThreads * ctas, rows - 1);
            const unsigned block = i / (unsigned)a.seg_rows, row = i - block * a.seg_rows;
            const long long r = (head + (long long)block * a.heads) * a.seg_rows + row, at = min(r, a.M - 1LL);
            some[u] = i0 + u * kSumThreads * ctas < rows && r < a.M && __ldg(a.row_offsets + at) < __ldg(a.row_offsets + at + 1);
            c2[u] = a.row_c2[at];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) x.add(some[u] ? c2[u] : 0.f);
    }
    x = x.over_warp();
    if (lane == 0) warp_part[t >> 5] = x;
    __syncthreads();
    if (t < 32) {
        x = lane < kSumThreads / 32 ? warp_part[lane] : LongSum{};
        x = x.over_warp();
        if (lane == 0) whole = x;
    }
    if (ctas > 1) cluster_sync();
    if (rank == 0 && t == 0) {
        for (int i = 1; i < ctas; ++i)
            x.add(LongSum{load_cluster(smem_addr(&whole.hi), i), load_cluster(smem_addr(&whole.lo), i)});
        dlambda[head] = -x.value();
    }
    if (ctas > 1) cluster_sync();  // no CTA leaves what another may still read
}

template <bool TWO, bool GRAD, bool DIN, bool OUT>
int launch_rows(const MapArgs& a, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    const int mean = a.nnz / a.M;
    // Rows that rings mostly do not hold: a CTA of 4 warps a row (8192 rows of 2048:
    // map 53 us, gradient 74, softmax gradient 44; by 8 warps 80, 105 and 72, through
    // the rings 75, 134 and 69; even at means of about 1500 for the map and 1200 for
    // gradients).  Of 8 warps where rows are few, and a cluster of CTAs while those
    // are too few too and keep at least half their registers' worth each.
    if (mean > (GRAD ? 1280 : 1536)) {
        const int warps = a.M >= 4 * sms ? 4 : 8;
        int ctas = 1;
        while (ctas < 8 && (long long)a.M * ctas < 2LL * sms && mean / ctas > warps * 32 * kSteps / 2) ctas *= 2;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = ctas;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((long long)a.M * ctas));
        cfg.blockDim = dim3(warps * 32);
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const auto kernel = warps == 4 ? cluster_rows_kernel<TWO, GRAD, DIN, OUT, 4> : cluster_rows_kernel<TWO, GRAD, DIN, OUT, 8>;
        return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? USM_OK : cuda_failure();
    }
    // As many warps as there is room for their rings, of at least 256 entries each.
    using S = MapStream<TWO, GRAD, DIN>;
    constexpr int smem = kWarps * S::kBytes;
    const int most = sms * ctas_per_sm<S>() * kWarps, some = a.nnz / 256, G = some < 1 ? 1 : some < most ? some : most;
    const bool aligned = aligned_for_stream(a.s1) && aligned_for_stream(a.s2) && aligned_for_stream(a.dout);
    const bool vec = aligned_for_stream(a.out1) && aligned_for_stream(a.out2);
    const auto kernel = stream_rows_kernel<TWO, GRAD, DIN, OUT>;
    if (!allow_shared(kernel, smem)) return cuda_failure();
    kernel<<<(G + kWarps - 1) / kWarps, kThreads, smem, stream>>>(a, G, aligned, vec);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

template <bool TWO, bool GRAD>
int launch_map(const MapArgs& a, cudaStream_t stream) {
    if constexpr (GRAD) {
        if (a.dout_bf16)
            return a.out_bf16 ? launch_rows<TWO, true, true, true>(a, stream) : launch_rows<TWO, true, true, false>(a, stream);
    }
    return a.out_bf16 ? launch_rows<TWO, GRAD, false, true>(a, stream) : launch_rows<TWO, GRAD, false, false>(a, stream);
}

}  // namespace

int launch_diff_softmax(const MapArgs& a, cudaStream_t stream) { return launch_map<true, false>(a, stream); }

int launch_row_softmax_grad(const MapArgs& a, cudaStream_t stream) { return launch_map<false, true>(a, stream); }

int launch_diff_softmax_grad(const MapArgs& a, float* dlambda, cudaStream_t stream) {
    const int r = launch_map<true, true>(a, stream);
    if (r != USM_OK || !dlambda) return r;
    const int blocks = query_blocks(a.M, a.seg_rows);
    const long long rows = (blocks + a.heads - 1LL) / a.heads * a.seg_rows;  // of the first head, the most
    int ctas = 1;
    while (ctas < 8 && rows > 4LL * kSumThreads * ctas && (long long)a.heads * ctas < (1 << 24)) ctas *= 2;
    return launch_next(lambda_grad_kernel, a.heads * ctas, kSumThreads, ctas, stream, a, blocks, dlambda);
}

}  // namespace usm
