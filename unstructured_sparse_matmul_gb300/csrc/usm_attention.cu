// Sparse attention of few query rows in one pass (single tokens over a cache):
//     C[r] = Σ_p (P1[p] - λ P2[p]) V[c_p],   sk[p] = scale·(Qk[r]·Kk[c_p]) + bias(p),
// Pk the softmax of sk over the row's entries.
//
// One pass over the entries with a running maximum and sum for each map: with
// m the maximum so far, z = Σ exp(s - m) and o = Σ exp(s - m) V are scaled by
// exp(m - m') when the maximum rises to m'; at the end C = o1/z1 - λ o2/z2.
//
// What bounds it is how fast listed rows of 64 to 1024 bytes come from HBM, so
// copies must be in flight all the time, whatever the arithmetic does.  A
// cluster of 1, 2, 4 or 8 CTAs works on one row; its warps take windows of 8 or
// 16 entries in turn, each warp with a ring of stages of its own in shared
// memory that TMA fills with the windows' rows of K1, K2 and V (four listed
// rows an instruction, in slabs of 128 bytes a row, 16-byte pieces swizzled by
// the row so that lanes reading one piece of different rows meet no bank
// conflict).  No barrier but the stage's own, in the warp that owns it.
// Scores: 32 / window lanes to an entry, each summing its share of the pieces.
// Output: LV lanes to a row of V, four columns a lane (NP times), 32 / LV
// entries at once, weights broadcast by shuffles; products in fp32 pairs.
// Lanes, warps and CTAs each keep their own maximum and sums and are joined in
// a fixed order at the end, the CTAs through distributed shared memory: no
// workspace, no atomics.
#include <cmath>

#include "usm_cluster.cuh"
#include "usm_internal.h"
#include "usm_rel.cuh"

namespace usm {
namespace {

#ifndef USM_ATTN_WARPS
#define USM_ATTN_WARPS 4
#endif
#ifndef USM_ATTN_RING
#define USM_ATTN_RING 100
#endif
constexpr int kWarps = USM_ATTN_WARPS, kThreads = kWarps * 32;
constexpr int kMaxStages = 4;

// How the rows lie in a stage (the same for every warp).
struct Stages {
    int log2_window;  // entries a window: 8 or 16
    int count;        // stages a warp
    int slabs_d;      // slabs of a row of K1 or K2, and of V
    int slabs_n;
};

template <bool BF>
__device__ __forceinline__ void dot_piece(uint4 a, uint4 b, float& x, float& y) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; i += BF ? 1 : 2) {
        if constexpr (BF) {
            x = fma_bf16(lo16(aw[i]), lo16(bw[i]), x);
            y = fma_bf16(hi16(aw[i]), hi16(bw[i]), y);
        } else {
            x = fmaf(__uint_as_float(aw[i]), __uint_as_float(bw[i]), x);
            y = fmaf(__uint_as_float(aw[i + 1]), __uint_as_float(bw[i + 1]), y);
        }
    }
}

template <bool BF, bool TWO, int LV, int NP>
__global__ void __launch_bounds__(kThreads)
    attention_kernel(const __grid_constant__ CUtensorMap map_k1, const __grid_constant__ CUtensorMap map_k2,
                     const __grid_constant__ CUtensorMap map_v, const AttnArgs a, const Stages st) {
    constexpr int ES = BF ? 2 : 4;   // element bytes
    constexpr int G = 32 / LV;       // rows of V a step
    constexpr int NC = LV * NP * 4;  // columns a row of V can have
    constexpr int MAPS = TWO ? 2 : 1;
    extern __shared__ unsigned char smem_base[];
    __shared__ float part[MAPS][kWarps][NC];
    __shared__ float stat[MAPS][kWarps][2];  // maximum and sum of each warp
    __shared__ float whole[MAPS][NC + 2];    // the CTA's: sums, maximum, sum of weights
    __shared__ int cols_ring[kWarps][kMaxStages][16];
    __shared__ uint64_t bars[kWarps][kMaxStages];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    int p0, p1;
    row_range(a.row_offsets, r, a.nnz, p0, p1);
    const int block = r / a.seg_rows;
    if (p0 == p1) {  // the same in every CTA of the cluster
        if (rank == 0)
            for (int j = threadIdx.x; j < a.N; j += kThreads) a.C[(long long)r * a.ldc + j] = 0.f;
        return;
    }
    const int window = 1 << st.log2_window, slab = window * 128;
    const int slabs = MAPS * st.slabs_d + st.slabs_n, stage_bytes = slabs * slab;
    // Slabs start on 1024 bytes (the swizzle's period).
    unsigned char* smem = smem_base + ((1024 - (smem_addr(smem_base) & 1023)) & 1023);
    const uint32_t ring = smem_addr(smem) + warp * st.count * stage_bytes;
    unsigned char* q_at = smem + kWarps * st.count * stage_bytes;  // Q1 and Q2 in whole slabs, zeros past D
    const uint32_t q_addr = smem_addr(q_at);

    // This warp's windows: first, first + stride, ...
    const long long windows = ((long long)(p1 - p0) + window - 1) >> st.log2_window;
    const long long first = rank * kWarps + warp, stride = (long long)ctas * kWarps;
    auto load_col = [&](long long w) {  // column of entry `lane` of window w (the last one's past the end)
        const long long b = p0 + (w << st.log2_window);
        return w < windows && lane < window ? __ldg(a.col_indices + min(b + lane, (long long)p1 - 1)) : 0;
    };
    auto issue = [&](long long w, int s, int col) {
        const uint32_t bar = smem_addr(&bars[warp][s]);
        const int n = (int)min((long long)window, p1 - p0 - (w << st.log2_window)), quads = (n + 3) / 4;
        if (lane < window) cols_ring[warp][s][lane] = col;
        col = min(max(col, 0), a.K - 1);
        const int per = st.log2_window - 2;  // lanes: quad = lane mod window/4, slabs by the rest
        const int quad = lane & ((1 << per) - 1);
        const int y0 = __shfl_sync(kFullMask, col, 4 * quad), y1 = __shfl_sync(kFullMask, col, 4 * quad + 1);
        const int y2 = __shfl_sync(kFullMask, col, 4 * quad + 2), y3 = __shfl_sync(kFullMask, col, 4 * quad + 3);
        if (lane == 0) mbar_arrive_expect_tx(bar, quads * 512 * slabs);
        __syncwarp();
        if (quad < quads) {
            for (int i = lane >> per; i < slabs; i += 32 >> per) {
                const int k2 = i - st.slabs_d, v = i - MAPS * st.slabs_d;
                const CUtensorMap* map = v >= 0 ? &map_v : k2 >= 0 ? &map_k2 : &map_k1;
                const int x = v >= 0 ? v : k2 >= 0 ? k2 : i;
                tma_gather_rows4(ring + s * stage_bytes + i * slab + quad * 512, map, x * (128 / ES), y0, y1, y2, y3, bar);
            }
        }
    };
    int ahead[kMaxStages];
#pragma unroll
    for (int s = 0; s < kMaxStages; ++s) ahead[s] = s < st.count ? load_col(first + s * stride) : 0;
    if (lane < st.count) mbar_init(smem_addr(&bars[warp][lane]), 1);
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&map_v);
        if (a.D > 0) prefetch_tensor_map(&map_k1);
        if (TWO && a.D > 0) prefetch_tensor_map(&map_k2);
    }
    fence_barrier_init();
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kMaxStages; ++s)
        if (s < st.count && first + s * stride < windows) issue(first + s * stride, s, ahead[s]);

    const int start =
        a.bias.table ? rel_start(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + p0)) : 0;
    const int head = block % a.heads;
    for (int i = threadIdx.x; i < MAPS * st.slabs_d * 128 / ES; i += kThreads) {
        const int per = st.slabs_d * 128 / ES, k = i / per, d = i - k * per;
        const long long at = (long long)r * (k ? a.ldq2 : a.ldq) + d;
        const void* q = k ? a.Q2 : a.Q;
        if constexpr (BF)
            reinterpret_cast<uint16_t*>(q_at)[i] = d < a.D ? __ldg(static_cast<const uint16_t*>(q) + at) : (uint16_t)0;
        else
            reinterpret_cast<float*>(q_at)[i] = d < a.D ? __ldg(static_cast<const float*>(q) + at) : 0.f;
    }
    __syncthreads();

    const int entry = lane & (window - 1), share = lane >> st.log2_window, shares = 32 >> st.log2_window;
    const int pieces = (a.D * ES + 15) / 16;
    const int g = lane / LV, l = lane % LV;
    float m[MAPS], z[MAPS];
    float2 o[MAPS][NP][2];
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        m[k] = -INFINITY;
        z[k] = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) o[k][i][0] = o[k][i][1] = make_float2(0.f, 0.f);
    }
    // Where the lane's columns lie in a row of V: slab and byte within its 128.
    int v_slab[NP], v_byte[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int byte = (i * LV + l) * 4 * ES;
        v_slab[i] = (MAPS * st.slabs_d + min(byte / 128, st.slabs_n - 1)) * slab;
        v_byte[i] = byte % 128;
    }

    bool alive = true;
    int s = 0, phase = 0;
    for (long long w = first; w < windows; w += stride) {
        const int next = load_col(w + st.count * stride);
        const uint32_t stage = ring + s * stage_bytes;
        if (!__all_sync(kFullMask, mbar_wait_bounded(smem_addr(&bars[warp][s]), phase, kWaitLimitNs))) {
            alive = false;
            break;
        }
        const int n = (int)min((long long)window, p1 - p0 - (w << st.log2_window));
        const bool in = entry < n;
        float bias = 0.f;
        if (a.bias.table)
            bias = rel_table(a.bias, head, rel_bucket(a.bias, rel_entry(cols_ring[warp][s][entry], start, a.bias.reach)));
        float e[MAPS];
        bool used = false;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float x = 0.f, y = 0.f;
            const uint32_t at = stage + k * st.slabs_d * slab + entry * 128, q = q_addr + k * st.slabs_d * 128;
#pragma unroll 4
            for (int c = share; c < pieces; c += shares)
                dot_piece<BF>(lds128(at + (c >> 3) * slab + (((c ^ entry) & 7) << 4)), lds128(q + c * 16), x, y);
            x += y;
            for (int d = window; d < 32; d *= 2) x += __shfl_xor_sync(kFullMask, x, d);
            const float sc = in ? x * a.scale + bias : -INFINITY;
            used = used || sc != -INFINITY;
            float top = sc;
#pragma unroll
            for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
            if (top > m[k]) {  // the same in every lane
                const float f = __expf(m[k] - top);
                z[k] *= f;
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) o[k][i][h] = __fmul2_rn(o[k][i][h], make_float2(f, f));
                m[k] = top;
            }
            e[k] = __expf(sc - (m[k] == -INFINITY ? 0.f : m[k]));
            if (share == 0) z[k] += e[k];
        }
        // Entries that every map masks do not use their row of V, nor do those
        // that only fill up the last step.
        const bool guard = __any_sync(kFullMask, in && !used) || n % G != 0;
        const int steps = (n + G - 1) / G;
#pragma unroll 4
        for (int t = 0; t < steps; ++t) {
            const int en = t * G + g;
            float2 et[MAPS];
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                const float f = __shfl_sync(kFullMask, e[k], en);
                et[k] = make_float2(f, f);
            }
            const bool take = !guard || __shfl_sync(kFullMask, (int)used, en) != 0;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const uint32_t at = stage + v_slab[i] + en * 128 + (v_byte[i] ^ ((en & 7) << 4));
                float2 v0, v1;
                if constexpr (BF) {
                    const uint2 vw = lds64(at);
                    v0 = make_float2(__uint_as_float(vw.x << 16), __uint_as_float(vw.x & 0xffff0000u));
                    v1 = make_float2(__uint_as_float(vw.y << 16), __uint_as_float(vw.y & 0xffff0000u));
                } else {
                    const uint4 vw = lds128(at);
                    v0 = make_float2(__uint_as_float(vw.x), __uint_as_float(vw.y));
                    v1 = make_float2(__uint_as_float(vw.z), __uint_as_float(vw.w));
                }
                if (!take) v0 = v1 = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < MAPS; ++k) {
                    o[k][i][0] = __ffma2_rn(et[k], v0, o[k][i][0]);
                    o[k][i][1] = __ffma2_rn(et[k], v1, o[k][i][1]);
                }
            }
        }
        __syncwarp();  // every lane is done with the stage
        if (w + st.count * stride < windows) {
            fence_proxy_async_smem();
            issue(w + st.count * stride, s, next);
        }
        if (++s == st.count) {
            s = 0;
            phase ^= 1;
        }
    }
    if (!alive && lane == 0) {
        // A copy never landed: say so, and wait (bounded) for those in flight,
        // so that none lands after the CTA has gone.  The row is incomplete.
        record_status(a.status, USM_ERR_TIMEOUT);
        for (int i = 0; i < st.count; ++i) {
            mbar_wait_bounded(smem_addr(&bars[warp][i]), 0, 1000000ull);
            mbar_wait_bounded(smem_addr(&bars[warp][i]), 1, 1000000ull);
        }
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
        for (int i = 0; i < NP; ++i) {
            float x[4] = {o[k][i][0].x, o[k][i][0].y, o[k][i][1].x, o[k][i][1].y};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int d = LV; d < 32; d *= 2) x[u] += __shfl_xor_sync(kFullMask, x[u], d);
                if (g == 0) part[k][warp][(i * LV + l) * 4 + u] = x[u];
            }
        }
    }
    __syncthreads();
    const float lam = TWO ? __ldg(a.lambda + head) : 0.f;
    // Joins partial sums of one map, each relative to a maximum of its own.
    auto weight = [](float m_i, float top) { return m_i == -INFINITY ? 0.f : __expf(m_i - top); };
    for (int j = threadIdx.x; j < a.N; j += kThreads) {
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, sum = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) top = fmaxf(top, stat[k][i][0]);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float f = weight(stat[k][i][0], top);
                x += f * part[k][i][j];
                sum += f * stat[k][i][1];
            }
            if (ctas == 1) {
                if (sum != 0.f) res += (k == 0 ? 1.f : -lam) * (x / sum);
            } else {
                whole[k][j] = x;
                if (j == 0) {
                    whole[k][NC] = top;
                    whole[k][NC + 1] = sum;
                }
            }
        }
        if (ctas == 1) a.C[(long long)r * a.ldc + j] = res;
    }
    if (ctas == 1) return;
    cluster_sync();
    // Runs of 32 columns are dealt to the CTAs in turn.
    for (int j = threadIdx.x; j < a.N; j += kThreads) {
        if (j / 32 % ctas != rank) continue;
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, sum = 0.f;
            for (int i = 0; i < ctas; ++i) top = fmaxf(top, load_cluster(smem_addr(&whole[k][NC]), i));
            for (int i = 0; i < ctas; ++i) {
                const float f = weight(load_cluster(smem_addr(&whole[k][NC]), i), top);
                x += f * load_cluster(smem_addr(&whole[k][j]), i);
                sum += f * load_cluster(smem_addr(&whole[k][NC + 1]), i);
            }
            if (sum != 0.f) res += (k == 0 ? 1.f : -lam) * (x / sum);
        }
        a.C[(long long)r * a.ldc + j] = res;
    }
    cluster_sync();  // no CTA leaves while another may read its sums
}

template <bool BF, bool TWO, int LV, int NP>
int launch_shape(const AttnArgs& a, cudaStream_t stream) {
    constexpr int ES = BF ? 2 : 4;
    Stages st;
    st.slabs_d = (a.D * ES + 127) / 128;
    st.slabs_n = (a.N * ES + 127) / 128;
    const int slabs = (TWO ? 2 : 1) * st.slabs_d + st.slabs_n;
    // 16 entries a window while that keeps a stage at 16 KB, else 8; stages a
    // warp until the rings fill about 100 KB (two CTAs an SM).
    st.log2_window = slabs <= 8 ? 4 : 3;
    const int stage_bytes = slabs * 128 << st.log2_window;
    st.count = USM_ATTN_RING * 1024 / (kWarps * stage_bytes);
    st.count = st.count < 2 ? 2 : st.count > kMaxStages ? kMaxStages : st.count;
    const int smem = 1024 + kWarps * st.count * stage_bytes + (TWO ? 2 : 1) * st.slabs_d * 128;

    CUtensorMap maps[3];
    if (!encode_gather_map(&maps[2], a.V, BF, a.K, a.N, a.ldv)) return USM_ERR_CUDA;
    maps[0] = maps[1] = maps[2];
    if (a.D > 0 && !encode_gather_map(&maps[0], a.Km, BF, a.K, a.D, a.ldk)) return USM_ERR_CUDA;
    if (TWO && a.D > 0 && !encode_gather_map(&maps[1], a.K2, BF, a.K, a.D, a.ldk2)) return USM_ERR_CUDA;

    // CTAs a row: more until the rows fill the SMs or a row's windows (on
    // average) no longer give every warp one.
    const int sms = sm_count_current_device();
    const long long windows = (a.nnz / a.M >> st.log2_window) + 1;
    int ctas = 1;
    while (ctas < 8 && (long long)a.M * ctas < 4LL * sms && (long long)ctas * kWarps < windows) ctas *= 2;
    if (cudaFuncSetAttribute(attention_kernel<BF, TWO, LV, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return USM_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.M * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_kernel<BF, TWO, LV, NP>, maps[0], maps[1], maps[2], a, st) == cudaSuccess
               ? USM_OK
               : USM_ERR_CUDA;
}

template <bool BF, bool TWO>
int launch_width(const AttnArgs& a, cudaStream_t stream) {
    if (a.N <= 32) return launch_shape<BF, TWO, 8, 1>(a, stream);
    if (a.N <= 64) return launch_shape<BF, TWO, 16, 1>(a, stream);
    if (a.N <= 128) return launch_shape<BF, TWO, 32, 1>(a, stream);
    if (a.N <= 256) return launch_shape<BF, TWO, 32, 2>(a, stream);
    if constexpr (BF) return launch_shape<BF, TWO, 32, 4>(a, stream);
    return USM_ERR_UNSUPPORTED;
}

}  // namespace

int launch_attention(const AttnArgs& a, bool bf16, cudaStream_t stream) {
    const bool two = a.lambda != nullptr;
    if (bf16) return two ? launch_width<true, true>(a, stream) : launch_width<true, false>(a, stream);
    return two ? launch_width<false, true>(a, stream) : launch_width<false, false>(a, stream);
}

}  // namespace usm
