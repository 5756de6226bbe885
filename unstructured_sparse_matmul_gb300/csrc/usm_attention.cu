// Sparse attention of few query rows in one pass (single tokens over a cache):
//     C[r] = Σ_p (P1[p] - λ P2[p]) V[c_p],   sk[p] = scale·(Qk[r]·Kk[c_p]) + bias(p),
// Pk the softmax of sk over the row's entries.
//
// One pass over the entries with a running maximum and sum for each map: with
// m the maximum so far, z = Σ exp(s - m) and o = Σ exp(s - m) V are scaled by
// exp(m - m') when the maximum rises to m'; at the end C = o1/z1 - λ o2/z2.
//
// A cluster of 1, 2, 4 or 8 CTAs works on one row.  Its warps take windows of
// 32 entries in turn.  LPR lanes hold a key row (16 bytes a lane, CH times), so
// a warp reads G = 32/LPR key rows a step and S steps at once, all loads of
// K1, K2 and V in flight before the first product: what bounds the kernel is
// how fast listed rows of 128 to 512 bytes come from HBM or L2.  The S partial
// dot products a lane holds are reduced together (a transposing butterfly: S - 1
// shuffles and log2(LPR / S) more), which leaves a score of its own in every
// lane group.  Lanes, warps and CTAs each keep their own maximum and sums and
// are joined in a fixed order at the end, the CTAs through distributed shared
// memory: no workspace, no atomics.
#include <cmath>

#include "usm_cluster.cuh"
#include "usm_internal.h"
#include "usm_rel.cuh"

namespace usm {
namespace {

constexpr int kWarps = 4;

// 16 bytes of a row, `left` of its elements still inside the row's width
// (RAGGED: fewer than a whole piece at the end are read one by one).
template <bool BF, bool RAGGED>
__device__ __forceinline__ uint4 load_piece(const unsigned char* at, int left) {
    constexpr int E = BF ? 8 : 4;
    if (left >= E) return __ldg(reinterpret_cast<const uint4*>(at));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if constexpr (RAGGED) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < left) {
                if constexpr (BF)
                    w[e / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(at) + e) << (16 * (e & 1));
                else
                    w[e] = __ldg(reinterpret_cast<const unsigned int*>(at) + e);
            }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF>
__device__ __forceinline__ float dot_piece(uint4 a, uint4 b, float x) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF) {
            x = fma_bf16(lo16(aw[i]), lo16(bw[i]), x);
            x = fma_bf16(hi16(aw[i]), hi16(bw[i]), x);
        } else {
            x = fmaf(__uint_as_float(aw[i]), __uint_as_float(bw[i]), x);
        }
    }
    return x;
}

// Sums over the LPR lanes of a group of the S values each lane holds: lane l
// gets the sum of value l / (LPR / S).
template <int LPR, int S>
__device__ __forceinline__ float reduce_steps(float (&x)[S], int l) {
#pragma unroll
    for (int n = S / 2, o = LPR / 2; n > 0; n /= 2, o /= 2) {
        const bool up = (l & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = up ? x[i + n] : x[i], other = up ? x[i] : x[i + n];
            x[i] = mine + __shfl_xor_sync(kFullMask, other, o);
        }
    }
    float v = x[0];
#pragma unroll
    for (int o = LPR / S / 2; o > 0; o /= 2) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

template <bool BF, bool TWO, int LPR, int CH, bool RAGGED>
__global__ void __launch_bounds__(kWarps * 32, TWO || CH > 1 ? 3 : 4) attention_kernel(const AttnArgs a) {
    constexpr int E = BF ? 8 : 4, ES = BF ? 2 : 4;  // elements of a 16-byte piece; element bytes
    constexpr int G = 32 / LPR;                     // rows a step
    constexpr int S = CH > 1 ? 4 : 8;               // steps at once
    constexpr int R = LPR / S;                      // lanes that hold the same score
    constexpr int B = S * G;                        // entries at once
    constexpr int NC = LPR * CH * E;                // columns a row can have
    constexpr int MAPS = TWO ? 2 : 1;
    __shared__ float part[MAPS][kWarps][NC];
    __shared__ float stat[MAPS][kWarps][2];  // maximum and sum of each warp
    __shared__ float whole[MAPS][NC + 2];    // the CTA's: sums, maximum, sum of weights

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane / LPR, l = lane % LPR;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    int p0, p1;
    row_range(a.row_offsets, r, a.nnz, p0, p1);
    const int block = r / a.seg_rows;
    if (p0 == p1) {  // the same in every CTA of the cluster
        if (rank == 0)
            for (int j = threadIdx.x; j < a.N; j += kWarps * 32) a.C[(long long)r * a.ldc + j] = 0.f;
        return;
    }
    const int start =
        a.bias.table ? rel_start(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + p0)) : 0;

    uint4 q1[CH], q2[CH];
    int left_d[CH], left_n[CH];  // elements of the lane's pieces inside D and N
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e0 = (c * LPR + l) * E;
        left_d[c] = a.D - e0;
        left_n[c] = a.N - e0;
        q1[c] = load_piece<BF, RAGGED>(static_cast<const unsigned char*>(a.Q) + ((long long)r * a.ldq + e0) * ES, left_d[c]);
        if (TWO)
            q2[c] =
                load_piece<BF, RAGGED>(static_cast<const unsigned char*>(a.Q2) + ((long long)r * a.ldq2 + e0) * ES, left_d[c]);
    }
    const unsigned char* k1 = static_cast<const unsigned char*>(a.Km) + l * 16;
    const unsigned char* k2 = static_cast<const unsigned char*>(a.K2) + l * 16;
    const unsigned char* vv = static_cast<const unsigned char*>(a.V) + l * 16;

    float m[MAPS], z[MAPS], o[MAPS][CH * E];
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        m[k] = -INFINITY;
        z[k] = 0.f;
#pragma unroll
        for (int i = 0; i < CH * E; ++i) o[k][i] = 0.f;
    }

    const long long step = 32LL * kWarps * ctas;
    long long w = p0 + 32LL * (rank * kWarps + warp);
    int col = w + lane < p1 ? __ldg(a.col_indices + w + lane) : 0;
    for (; w < p1; w += step) {
        const int n = (int)min(32LL, p1 - w);
        const int next = w + step + lane < p1 ? __ldg(a.col_indices + w + step + lane) : 0;
#pragma unroll 1
        for (int b = 0; b < n; b += B) {
            // Entry of step t in this lane group: b + t·G + g.
            uint4 kw1[S][CH], kw2[TWO ? S : 1][CH], vw[S][CH];
#pragma unroll
            for (int t = 0; t < S; ++t) {
                const int j = b + t * G + g;
                const int c0 = __shfl_sync(kFullMask, col, j & 31);
                const long long c = min(max(c0, 0), a.K - 1);
                const bool in = j < n;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int ld = in ? left_d[i] : 0;
                    kw1[t][i] = load_piece<BF, RAGGED>(k1 + c * a.ldk * ES + i * LPR * 16, ld);
                    if (TWO) kw2[t][i] = load_piece<BF, RAGGED>(k2 + c * a.ldk2 * ES + i * LPR * 16, ld);
                }
            }
#pragma unroll
            for (int t = 0; t < S; ++t) {
                const int j = b + t * G + g;
                const int c0 = __shfl_sync(kFullMask, col, j & 31);
                const long long c = min(max(c0, 0), a.K - 1);
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    vw[t][i] = load_piece<BF, RAGGED>(vv + c * a.ldv * ES + i * LPR * 16, j < n ? left_n[i] : 0);
            }
            // This lane's score: entry b + (l / R)·G + g, R lanes each.
            const int j = b + l / R * G + g;
            const int c0 = __shfl_sync(kFullMask, col, j & 31);
            float bias = 0.f;
            if (a.bias.table)
                bias = rel_table(a.bias, block % a.heads, rel_bucket(a.bias, rel_entry(c0, start, a.bias.reach)));
            float e[MAPS];
            bool used = false;
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                float x[S];
#pragma unroll
                for (int t = 0; t < S; ++t) {
                    x[t] = 0.f;
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        x[t] = k == 0 ? dot_piece<BF>(q1[i], kw1[t][i], x[t]) : dot_piece<BF>(q2[i], kw2[TWO ? t : 0][i], x[t]);
                }
                const float dot = reduce_steps<LPR, S>(x, l);
                const float s = j < n ? dot * a.scale + bias : -INFINITY;
                used = used || s != -INFINITY;
                float top = s;
#pragma unroll
                for (int d = 16; d >= R; d /= 2) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
                if (top > m[k]) {  // the same in every lane
                    const float f = __expf(m[k] - top);
                    z[k] *= f;
#pragma unroll
                    for (int i = 0; i < CH * E; ++i) o[k][i] *= f;
                    m[k] = top;
                }
                e[k] = __expf(s - (m[k] == -INFINITY ? 0.f : m[k]));
                if (l % R == 0) z[k] += e[k];
            }
            // Values under entries that every map masks are not used.
            if (__any_sync(kFullMask, !used && j < n)) {
#pragma unroll
                for (int t = 0; t < S; ++t) {
                    const bool u = __shfl_sync(kFullMask, (int)used, g * LPR + t * R) != 0;
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        if (!u) vw[t][i] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
#pragma unroll
            for (int t = 0; t < S; ++t) {
                float et[MAPS];
#pragma unroll
                for (int k = 0; k < MAPS; ++k) et[k] = __shfl_sync(kFullMask, e[k], g * LPR + t * R);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const uint32_t vx[4] = {vw[t][i].x, vw[t][i].y, vw[t][i].z, vw[t][i].w};
#pragma unroll
                    for (int u = 0; u < E; ++u) {
                        const float v = __uint_as_float(!BF ? vx[u % 4] : (u & 1) ? vx[u / 2] & 0xffff0000u : vx[u / 2] << 16);
#pragma unroll
                        for (int k = 0; k < MAPS; ++k) o[k][i * E + u] = fmaf(et[k], v, o[k][i * E + u]);
                    }
                }
            }
        }
        col = next;
    }

    // The warp's lanes, then the CTA's warps, then the cluster's CTAs.
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) z[k] += __shfl_xor_sync(kFullMask, z[k], d);
        if (lane == 0) {
            stat[k][warp][0] = m[k];
            stat[k][warp][1] = z[k];
        }
#pragma unroll
        for (int i = 0; i < CH * E; ++i) {
            float x = o[k][i];
#pragma unroll
            for (int d = LPR; d < 32; d *= 2) x += __shfl_xor_sync(kFullMask, x, d);
            if (g == 0) part[k][warp][(i / E * LPR + l) * E + i % E] = x;
        }
    }
    __syncthreads();
    const float lam = TWO ? __ldg(a.lambda + block % a.heads) : 0.f;
    // Joins n partial sums of one map, each relative to a maximum of its own:
    // their common maximum and the weight of each.
    auto weight = [](float m_i, float top) { return m_i == -INFINITY ? 0.f : __expf(m_i - top); };
    for (int j = threadIdx.x; j < a.N; j += kWarps * 32) {
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, s = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) top = fmaxf(top, stat[k][i][0]);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float f = weight(stat[k][i][0], top);
                x += f * part[k][i][j];
                s += f * stat[k][i][1];
            }
            if (ctas == 1) {
                if (s != 0.f) res += (k == 0 ? 1.f : -lam) * (x / s);
            } else {
                whole[k][j] = x;
                if (j == 0) {
                    whole[k][NC] = top;
                    whole[k][NC + 1] = s;
                }
            }
        }
        if (ctas == 1) a.C[(long long)r * a.ldc + j] = res;
    }
    if (ctas == 1) return;
    cluster_sync();
    // Runs of 32 columns are dealt to the CTAs in turn.
    for (int j = threadIdx.x; j < a.N; j += kWarps * 32) {
        if (j / 32 % ctas != rank) continue;
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, s = 0.f;
            for (int i = 0; i < ctas; ++i) top = fmaxf(top, load_cluster(smem_addr(&whole[k][NC]), i));
            for (int i = 0; i < ctas; ++i) {
                const float f = weight(load_cluster(smem_addr(&whole[k][NC]), i), top);
                x += f * load_cluster(smem_addr(&whole[k][j]), i);
                s += f * load_cluster(smem_addr(&whole[k][NC + 1]), i);
            }
            if (s != 0.f) res += (k == 0 ? 1.f : -lam) * (x / s);
        }
        a.C[(long long)r * a.ldc + j] = res;
    }
    cluster_sync();  // no CTA leaves while another may read its sums
}

template <bool BF, bool TWO, int LPR, int CH, bool RAGGED>
int launch_shape(const AttnArgs& a, cudaStream_t stream) {
    // CTAs a row: more until the rows fill the SMs or a row's windows of 32
    // entries (on average) no longer give every warp one.
    const int sms = sm_count_current_device();
    const long long windows = (a.nnz / a.M + 31) / 32;
    int ctas = 1;
    while (ctas < 8 && (long long)a.M * ctas < 4LL * sms && (long long)ctas * kWarps < windows) ctas *= 2;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.M * ctas));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_kernel<BF, TWO, LPR, CH, RAGGED>, a) == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

template <bool BF, bool TWO, bool RAGGED>
int launch_width(const AttnArgs& a, cudaStream_t stream) {
    const int bytes = (a.D > a.N ? a.D : a.N) * (BF ? 2 : 4);
    if (bytes <= 128) return launch_shape<BF, TWO, 8, 1, RAGGED>(a, stream);
    if (bytes <= 256) return launch_shape<BF, TWO, 16, 1, RAGGED>(a, stream);
    if (bytes <= 512) return launch_shape<BF, TWO, 32, 1, RAGGED>(a, stream);
    return launch_shape<BF, TWO, 32, 2, RAGGED>(a, stream);
}

template <bool BF, bool TWO>
int launch_ragged(const AttnArgs& a, cudaStream_t stream) {
    constexpr int E = BF ? 8 : 4;
    return a.D % E == 0 && a.N % E == 0 ? launch_width<BF, TWO, false>(a, stream) : launch_width<BF, TWO, true>(a, stream);
}

}  // namespace

int launch_attention(const AttnArgs& a, bool bf16, cudaStream_t stream) {
    const bool two = a.lambda != nullptr;
    if (bf16) return two ? launch_ragged<true, true>(a, stream) : launch_ragged<true, false>(a, stream);
    return two ? launch_ragged<false, true>(a, stream) : launch_ragged<false, false>(a, stream);
}

}  // namespace usm
