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
// cluster of 1, 2, 4 or 8 CTAs works on one row; its warps take windows of 16
// entries in turn, each warp with a ring of stages of its own in shared memory
// that TMA fills with the windows' rows of K1, K2 and V (four listed rows an
// instruction, in slabs of 128 bytes a row, 16-byte pieces swizzled by the row
// so that reading one piece of different rows meets no bank conflict).  No
// barrier but the stage's own, in the warp that owns it.
//
// Products.  bf16: matrix instructions (16 x 8 x 16), which take the operands
// as they lie and leave the issue slots to the copies: on CUDA cores a window
// takes five times the instructions and the kernel 2.4 times as long.  fp32:
// CUDA cores.  Lanes, warps and CTAs each keep their own maximum and sums and
// are joined in a fixed order at the end, the CTAs through distributed shared
// memory: no workspace, no atomics.
#include <cmath>

#include "usm_cluster.cuh"
#include "usm_internal.h"
#include "usm_rel.cuh"

namespace usm {
namespace {

constexpr int kMaxWarps = 4, kMaxStages = 4, kWindow = 16;

// A warp's ring of stages, and how a window's rows lie in a stage: slab i of a
// row of K1, then K2, then V (128 bytes of each of the 16 rows).
struct Stages {
    int warps;    // warps a CTA
    int count;    // stages a warp
    int slabs_d;  // slabs of a row of K1 or K2, and of V
    int slabs_n;
};
constexpr int kSlab = kWindow * 128;

struct GatherMaps {
    CUtensorMap k1, k2, v;
};

// Sums of a CTA's warps: o by column, the maximum and the sum of weights.
template <int MAPS, int NC>
struct Joined {
    float part[MAPS][kMaxWarps][NC];
    float stat[MAPS][kMaxWarps][2];
    float whole[MAPS][NC + 2];
};

// One warp's windows of its row and the ring their rows are copied into.
struct Ring {
    uint32_t base, stage_bytes, bars;  // shared addresses; bytes a stage
    int (*cols)[kWindow];              // columns of each stage's entries
    int p0, p1, lane, count, slabs_d, slabs, maps;
    long long windows, first, stride;  // the warp's windows: first, first + stride, ...

    __device__ __forceinline__ int size(long long w) const {
        return (int)min((long long)kWindow, p1 - p0 - w * kWindow);
    }
    // Column of entry `lane` of window w (the last entry's past the row's end).
    __device__ __forceinline__ int load_col(const int* __restrict__ ci, long long w) const {
        return w < windows && lane < kWindow ? __ldg(ci + min(p0 + w * kWindow + lane, (long long)p1 - 1)) : 0;
    }
    // Copies window w's rows into stage s: lane = quad of entries + 4·slab.
    __device__ __forceinline__ void issue(const GatherMaps& m, long long w, int s, int col, int K, int slab_cols) const {
        const int quads = (size(w) + 3) / 4, quad = lane & 3;
        if (lane < kWindow) cols[s][lane] = col;
        col = min(max(col, 0), K - 1);
        const int y0 = __shfl_sync(kFullMask, col, 4 * quad), y1 = __shfl_sync(kFullMask, col, 4 * quad + 1);
        const int y2 = __shfl_sync(kFullMask, col, 4 * quad + 2), y3 = __shfl_sync(kFullMask, col, 4 * quad + 3);
        if (lane == 0) mbar_arrive_expect_tx(bars + 8 * s, quads * 512 * slabs);
        __syncwarp();
        if (quad < quads) {
            for (int i = lane >> 2; i < slabs; i += 8) {
                const int k2 = i - slabs_d, v = i - maps * slabs_d;
                const CUtensorMap* map = v >= 0 ? &m.v : k2 >= 0 ? &m.k2 : &m.k1;
                const int x = v >= 0 ? v : k2 >= 0 ? k2 : i;
                tma_gather_rows4(base + s * stage_bytes + i * kSlab + quad * 512, map, x * slab_cols, y0, y1, y2, y3,
                                 bars + 8 * s);
            }
        }
    }
};

// Weight of a partial sum with maximum m_i under the common maximum.
__device__ __forceinline__ float join_weight(float m_i, float top) { return m_i == -INFINITY ? 0.f : __expf(m_i - top); }

// The CTA's warps (in `sh`), then the cluster's CTAs, and the row of C.
template <int MAPS, int NC>
__device__ __forceinline__ void join(Joined<MAPS, NC>& sh, const AttnArgs& a, int r, int head, int warps, int ctas,
                                     int rank) {
    __syncthreads();
    const int threads = warps * 32;
    const float lam = MAPS > 1 ? __ldg(a.lambda + head) : 0.f;
    for (int j = threadIdx.x; j < a.N; j += threads) {
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, sum = 0.f;
            for (int i = 0; i < warps; ++i) top = fmaxf(top, sh.stat[k][i][0]);
            for (int i = 0; i < warps; ++i) {
                const float f = join_weight(sh.stat[k][i][0], top);
                x += f * sh.part[k][i][j];
                sum += f * sh.stat[k][i][1];
            }
            if (ctas == 1) {
                if (sum != 0.f) res += (k == 0 ? 1.f : -lam) * (x / sum);
            } else {
                sh.whole[k][j] = x;
                if (j == 0) {
                    sh.whole[k][NC] = top;
                    sh.whole[k][NC + 1] = sum;
                }
            }
        }
        if (ctas == 1) a.C[(long long)r * a.ldc + j] = res;
    }
    if (ctas == 1) return;
    cluster_sync();
    // Runs of 32 columns are dealt to the CTAs in turn.
    for (int j = threadIdx.x; j < a.N; j += threads) {
        if (j / 32 % ctas != rank) continue;
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, sum = 0.f;
            for (int i = 0; i < ctas; ++i) top = fmaxf(top, load_cluster(smem_addr(&sh.whole[k][NC]), i));
            for (int i = 0; i < ctas; ++i) {
                const float f = join_weight(load_cluster(smem_addr(&sh.whole[k][NC]), i), top);
                x += f * load_cluster(smem_addr(&sh.whole[k][j]), i);
                sum += f * load_cluster(smem_addr(&sh.whole[k][NC + 1]), i);
            }
            if (sum != 0.f) res += (k == 0 ? 1.f : -lam) * (x / sum);
        }
        a.C[(long long)r * a.ldc + j] = res;
    }
    cluster_sync();  // no CTA leaves while another may read its sums
}

__device__ __forceinline__ void load_matrix4(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at));
}
__device__ __forceinline__ void load_matrix4_trans(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at));
}
// Rows 0-7 of D = A·B + C (16 x 8 x 16, bf16 in, fp32 sums); rows 8-15 of A are
// zero, so are theirs.
__device__ __forceinline__ void mma_upper(float& c0, float& c1, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
    [[maybe_unused]] float z2, z3;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%9,%9};"
        : "+f"(c0), "+f"(c1), "=f"(z2), "=f"(z3)
        : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// Everything both kernels do before their first window; false for a row
// without entries (its output is written).
template <int MAPS>
__device__ __forceinline__ bool start_row(const GatherMaps& maps, const AttnArgs& a, const Stages& st, Ring& ring,
                                          unsigned char* smem, uint64_t* bars, int (*cols)[kWindow], int r, int ctas,
                                          int rank, int slab_cols) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    row_range(a.row_offsets, r, a.nnz, ring.p0, ring.p1);
    if (ring.p0 == ring.p1) {  // the same in every CTA of the cluster
        if (rank == 0)
            for (int j = threadIdx.x; j < a.N; j += st.warps * 32) a.C[(long long)r * a.ldc + j] = 0.f;
        return false;
    }
    ring.lane = lane;
    ring.maps = MAPS;
    ring.count = st.count;
    ring.slabs_d = st.slabs_d;
    ring.slabs = MAPS * st.slabs_d + st.slabs_n;
    ring.stage_bytes = ring.slabs * kSlab;
    ring.base = smem_addr(smem) + warp * st.count * ring.stage_bytes;
    ring.bars = smem_addr(bars);
    ring.cols = cols;
    ring.windows = ((long long)(ring.p1 - ring.p0) + kWindow - 1) / kWindow;
    ring.first = rank * st.warps + warp;
    ring.stride = (long long)ctas * st.warps;
    int ahead[kMaxStages];
#pragma unroll
    for (int s = 0; s < kMaxStages; ++s)
        ahead[s] = s < st.count ? ring.load_col(a.col_indices, ring.first + s * ring.stride) : 0;
    if (lane < st.count) mbar_init(ring.bars + 8 * lane, 1);
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&maps.v);
        if (a.D > 0) prefetch_tensor_map(&maps.k1);
        if (MAPS > 1 && a.D > 0) prefetch_tensor_map(&maps.k2);
    }
    fence_barrier_init();
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kMaxStages; ++s)
        if (s < st.count && ring.first + s * ring.stride < ring.windows)
            ring.issue(maps, ring.first + s * ring.stride, s, ahead[s], a.K, slab_cols);
    return true;
}

// A copy never landed: say so, and wait (bounded) for those in flight, so that
// none lands after the CTA has gone.  The row is incomplete.
__device__ __forceinline__ void give_up(const AttnArgs& a, const Ring& ring) {
    if (ring.lane == 0) {
        record_status(a.status, USM_ERR_TIMEOUT);
        for (int i = 0; i < ring.count; ++i) {
            mbar_wait_bounded(ring.bars + 8 * i, 0, 1000000ull);
            mbar_wait_bounded(ring.bars + 8 * i, 1, 1000000ull);
        }
    }
    __syncwarp();
}

// bf16.  With lane = 4·row + t, a matrix instruction gives the lane elements
// (row, 2t) and (row, 2t + 1) of its result and takes from it elements
// (row, 2t), (row, 2t + 1), (row, 2t + 8), (row, 2t + 9) of its left operand.
// Scores: the left operand holds q in each of rows 0-7, so every lane gets the
// scores of entries 2t, 2t + 1, 2t + 8 and 2t + 9: just those whose weights it
// passes to the product with V.  There the left operand's rows 0-2 hold map 1's
// weights and rows 3-5 map 2's, each split into three bf16 numbers whose sum is
// the fp32 weight (bits 1-8, 9-16 and 17-24), so a lane works on the map and the
// part of its row alone, and nothing is exchanged but two shuffles for the
// maximum.  Each window's products with V start from zero and are added to the
// running sums in fp32: matrix instructions do not round their sums to nearest.
// NT: tiles of 8 columns of V.
template <bool TWO, int NT>
__global__ void __launch_bounds__(kMaxWarps * 32)
    attention_bf16_kernel(const __grid_constant__ GatherMaps maps, const AttnArgs a, const Stages st) {
    constexpr int MAPS = TWO ? 2 : 1, NC = NT * 8;
    extern __shared__ unsigned char smem_base[];
    __shared__ Joined<MAPS, NC> sh;
    __shared__ int cols[kMaxWarps][kMaxStages][kWindow];
    __shared__ uint64_t bars[kMaxWarps][kMaxStages];
    // Slabs start on 1024 bytes (the swizzle's period).
    unsigned char* smem = smem_base + ((1024 - (smem_addr(smem_base) & 1023)) & 1023);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    Ring ring;
    if (!start_row<MAPS>(maps, a, st, ring, smem, bars[warp], cols[warp], r, ctas, rank, 64)) return;
    const int block = r / a.seg_rows, head = block % a.heads;
    const int start =
        a.bias.table ? rel_start(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + ring.p0)) : 0;

    // q, in steps of 16 dimensions: for each t the two words the lane passes.
    const int ksteps = (a.D + 15) / 16;
    uint32_t* qs = reinterpret_cast<uint32_t*>(smem + st.warps * st.count * ring.stage_bytes);
    for (int i = threadIdx.x; i < MAPS * ksteps * 8; i += st.warps * 32) {
        const int k = i / (ksteps * 8), w = i - k * ksteps * 8;
        const int d = w / 8 * 16 + (w & 7) / 2 * 2 + (w & 1) * 8;
        const uint16_t* q = static_cast<const uint16_t*>(k ? a.Q2 : a.Q) + (long long)r * (k ? a.ldq2 : a.ldq);
        const uint32_t lo = d < a.D ? __ldg(q + d) : 0, hi = d + 1 < a.D ? __ldg(q + d + 1) : 0;
        qs[i] = lo | hi << 16;
    }
    __syncthreads();

    const int row = lane >> 2, t = lane & 3;
    const int mine = TWO && row >= 3, part = row - 3 * mine;  // the lane's map, and its part of the weights
    const bool weighs = row < 3 * MAPS;
    // Operand tiles of 8 rows and 16 bytes: lane i addresses row i % 8 of tile i / 8.
    const int tile = lane >> 3, tile_row = lane & 7;
    const uint32_t k_row = (tile_row + 8 * (tile >> 1)) * 128, v_row = (tile_row + 8 * (tile & 1)) * 128;
    const uint32_t k_piece = tile & 1, v_piece = tile >> 1;
    const uint32_t q_addr = smem_addr(qs) + t * 8;

    float m = -INFINITY, z = 0.f;  // the lane's map's
    float o[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = 0.f;
    bool alive = true;
    int s = 0, phase = 0;
    for (long long w = ring.first; w < ring.windows; w += ring.stride) {
        const int next = ring.load_col(a.col_indices, w + ring.count * ring.stride);
        const uint32_t stage = ring.base + s * ring.stage_bytes;
        if (!__all_sync(kFullMask, mbar_wait_bounded(ring.bars + 8 * s, phase, kWaitLimitNs))) {
            alive = false;
            break;
        }
        // Dot products: 4 of each map in every lane.
        float x[MAPS][4];
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
#pragma unroll
            for (int u = 0; u < 4; ++u) x[k][u] = 0.f;
            const uint32_t at = stage + k * st.slabs_d * kSlab + k_row, q = q_addr + k * ksteps * 32;
#pragma unroll 4
            for (int c = 0; c < ksteps; ++c) {
                uint32_t b[4];
                load_matrix4(at + (c >> 2) * kSlab + ((((c & 3) * 2 + k_piece) ^ tile_row) << 4), b);
                const uint2 qw = lds64(q + c * 32);
                mma_upper(x[k][0], x[k][1], qw.x, qw.y, b[0], b[1]);
                mma_upper(x[k][2], x[k][3], qw.x, qw.y, b[2], b[3]);
            }
        }
        // Scores of the lane's map; entries that no map uses.
        const int n = ring.size(w);
        float sc[4];
        unsigned unused = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int en = 2 * t + (u & 1) + (u >> 1) * 8;
            float bias = 0.f;
            if (a.bias.table)
                bias = rel_table(a.bias, head, rel_bucket(a.bias, rel_entry(ring.cols[s][en], start, a.bias.reach)));
            float y[MAPS];
            bool none = true;
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                y[k] = en < n ? fmaf(x[k][u], a.scale, bias) : -INFINITY;
                none = none && y[k] == -INFINITY;
            }
            sc[u] = mine ? y[MAPS - 1] : y[0];
            if (none) unused |= 1u << en;
        }
        float top = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
        if (top > m) {
            const float f = __expf(m - top);
            z *= f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                o[i][0] *= f;
                o[i][1] *= f;
            }
            m = top;
        }
        const float base = m == -INFINITY ? 0.f : m;
        float e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            e[u] = __expf(sc[u] - base);
            z += e[u];
        }
        // The lane's part of its weights: 8 bits each, rounded to nearest.
        uint32_t w0 = pack_bf16(e[0], e[1]), w1 = pack_bf16(e[2], e[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (part > h) {
                e[0] -= __uint_as_float(w0 << 16);
                e[1] -= __uint_as_float(w0 & 0xffff0000u);
                e[2] -= __uint_as_float(w1 << 16);
                e[3] -= __uint_as_float(w1 & 0xffff0000u);
                w0 = pack_bf16(e[0], e[1]);
                w1 = pack_bf16(e[2], e[3]);
            }
        }
        if (!weighs) w0 = w1 = 0;
        // Rows of V under entries that no map uses (and past the row's end) may
        // hold anything: they become zeros.
        if (__any_sync(kFullMask, unused != 0)) {
            unused |= __shfl_xor_sync(kFullMask, unused, 1);
            unused |= __shfl_xor_sync(kFullMask, unused, 2);
            for (; unused; unused &= unused - 1) {
                const uint32_t at = stage + MAPS * st.slabs_d * kSlab + (__ffs(unused) - 1) * 128;
                for (int i = lane; i < st.slabs_n * 8; i += 32)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + (i >> 3) * kSlab + (i & 7) * 16), "r"(0)
                                 : "memory");
            }
            __syncwarp();
        }
        const uint32_t v_at = stage + MAPS * st.slabs_d * kSlab + v_row;
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            if (i * 16 >= a.N) break;
            uint32_t b[4];
            load_matrix4_trans(v_at + (i >> 2) * kSlab + ((((i & 3) * 2 + v_piece) ^ tile_row) << 4), b);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float c0 = 0.f, c1 = 0.f;
                mma_upper(c0, c1, w0, w1, b[2 * h], b[2 * h + 1]);
                o[2 * i + h][0] += c0;
                o[2 * i + h][1] += c1;
            }
        }
        __syncwarp();  // every lane is done with the stage
        if (w + ring.count * ring.stride < ring.windows) {
            fence_proxy_async_smem();
            ring.issue(maps, w + ring.count * ring.stride, s, next, a.K, 64);
        }
        if (++s == ring.count) {
            s = 0;
            phase ^= 1;
        }
    }
    if (!alive) give_up(a, ring);

    z += __shfl_xor_sync(kFullMask, z, 1);
    z += __shfl_xor_sync(kFullMask, z, 2);
    const bool writes = row == 0 || (TWO && row == 3);
    if (writes && t == 0) {
        sh.stat[mine][warp][0] = m;
        sh.stat[mine][warp][1] = z;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float mid = __shfl_down_sync(kFullMask, o[i][u], 4), low = __shfl_down_sync(kFullMask, o[i][u], 8);
            if (writes) sh.part[mine][warp][i * 8 + 2 * t + u] = o[i][u] + (mid + low);
        }
    join(sh, a, r, head, st.warps, ctas, rank);
}

// fp32 on CUDA cores.  Scores: two lanes to an entry, each summing every other
// piece of 16 bytes.  Output: LV lanes to a row of V, four columns a lane (NP
// times), 32 / LV entries at once, weights broadcast by shuffles.
template <bool TWO, int LV, int NP>
__global__ void __launch_bounds__(kMaxWarps * 32)
    attention_f32_kernel(const __grid_constant__ GatherMaps maps, const AttnArgs a, const Stages st) {
    constexpr int G = 32 / LV;       // rows of V a step
    constexpr int NC = LV * NP * 4;  // columns a row of V can have
    constexpr int MAPS = TWO ? 2 : 1;
    extern __shared__ unsigned char smem_base[];
    __shared__ Joined<MAPS, NC> sh;
    __shared__ int cols[kMaxWarps][kMaxStages][kWindow];
    __shared__ uint64_t bars[kMaxWarps][kMaxStages];
    unsigned char* smem = smem_base + ((1024 - (smem_addr(smem_base) & 1023)) & 1023);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    Ring ring;
    if (!start_row<MAPS>(maps, a, st, ring, smem, bars[warp], cols[warp], r, ctas, rank, 32)) return;
    const int block = r / a.seg_rows, head = block % a.heads;
    const int start =
        a.bias.table ? rel_start(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + ring.p0)) : 0;
    // Q1 and Q2 in whole slabs, zeros past D.
    float* qs = reinterpret_cast<float*>(smem + st.warps * st.count * ring.stage_bytes);
    for (int i = threadIdx.x; i < MAPS * st.slabs_d * 32; i += st.warps * 32) {
        const int per = st.slabs_d * 32, k = i / per, d = i - k * per;
        const float* q = static_cast<const float*>(k ? a.Q2 : a.Q) + (long long)r * (k ? a.ldq2 : a.ldq);
        qs[i] = d < a.D ? __ldg(q + d) : 0.f;
    }
    __syncthreads();

    const int entry = lane & (kWindow - 1), share = lane / kWindow;
    const int pieces = (a.D + 3) / 4;
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
        const int byte = (i * LV + l) * 16;
        v_slab[i] = (MAPS * st.slabs_d + min(byte / 128, st.slabs_n - 1)) * kSlab;
        v_byte[i] = byte % 128;
    }
    bool alive = true;
    int s = 0, phase = 0;
    for (long long w = ring.first; w < ring.windows; w += ring.stride) {
        const int next = ring.load_col(a.col_indices, w + ring.count * ring.stride);
        const uint32_t stage = ring.base + s * ring.stage_bytes;
        if (!__all_sync(kFullMask, mbar_wait_bounded(ring.bars + 8 * s, phase, kWaitLimitNs))) {
            alive = false;
            break;
        }
        const int n = ring.size(w);
        const bool in = entry < n;
        float bias = 0.f;
        if (a.bias.table)
            bias = rel_table(a.bias, head, rel_bucket(a.bias, rel_entry(ring.cols[s][entry], start, a.bias.reach)));
        float e[MAPS];
        bool used = false;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float2 x = make_float2(0.f, 0.f), y = x;
            const uint32_t at = stage + k * st.slabs_d * kSlab + entry * 128, q = smem_addr(qs) + k * st.slabs_d * 128;
#pragma unroll 4
            for (int c = share; c < pieces; c += 2) {
                const uint4 kw = lds128(at + (c >> 3) * kSlab + (((c ^ entry) & 7) << 4)), qw = lds128(q + c * 16);
                x = __ffma2_rn(make_float2(__uint_as_float(kw.x), __uint_as_float(kw.y)),
                               make_float2(__uint_as_float(qw.x), __uint_as_float(qw.y)), x);
                y = __ffma2_rn(make_float2(__uint_as_float(kw.z), __uint_as_float(kw.w)),
                               make_float2(__uint_as_float(qw.z), __uint_as_float(qw.w)), y);
            }
            float dot = (x.x + x.y) + (y.x + y.y);
            dot += __shfl_xor_sync(kFullMask, dot, kWindow);
            const float sc = in ? fmaf(dot, a.scale, bias) : -INFINITY;
            used = used || sc != -INFINITY;
            float top = sc;
#pragma unroll
            for (int d = 1; d < kWindow; d *= 2) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
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
                const uint4 vw = lds128(stage + v_slab[i] + en * 128 + (v_byte[i] ^ ((en & 7) << 4)));
                float2 v0 = make_float2(__uint_as_float(vw.x), __uint_as_float(vw.y));
                float2 v1 = make_float2(__uint_as_float(vw.z), __uint_as_float(vw.w));
                if (!take) v0 = v1 = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < MAPS; ++k) {
                    o[k][i][0] = __ffma2_rn(et[k], v0, o[k][i][0]);
                    o[k][i][1] = __ffma2_rn(et[k], v1, o[k][i][1]);
                }
            }
        }
        __syncwarp();  // every lane is done with the stage
        if (w + ring.count * ring.stride < ring.windows) {
            fence_proxy_async_smem();
            ring.issue(maps, w + ring.count * ring.stride, s, next, a.K, 32);
        }
        if (++s == ring.count) {
            s = 0;
            phase ^= 1;
        }
    }
    if (!alive) give_up(a, ring);

#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) z[k] += __shfl_xor_sync(kFullMask, z[k], d);
        if (lane == 0) {
            sh.stat[k][warp][0] = m[k];
            sh.stat[k][warp][1] = z[k];
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float x[4] = {o[k][i][0].x, o[k][i][0].y, o[k][i][1].x, o[k][i][1].y};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int d = LV; d < 32; d *= 2) x[u] += __shfl_xor_sync(kFullMask, x[u], d);
                if (g == 0) sh.part[k][warp][(i * LV + l) * 4 + u] = x[u];
            }
        }
    }
    join(sh, a, r, head, st.warps, ctas, rank);
}

template <bool BF, bool TWO, class Kernel>
int launch_kernel(Kernel kernel, const AttnArgs& a, cudaStream_t stream) {
    constexpr int ES = BF ? 2 : 4, MAPS = TWO ? 2 : 1;
    Stages st;
    st.slabs_d = (a.D * ES + 127) / 128;
    st.slabs_n = (a.N * ES + 127) / 128;
    // A stage is 0.25 to 48 KB.  Four warps a CTA while two stages each fit in
    // about 96 KB (so that two CTAs fit an SM), else two; as many stages as fit.
    const int stage_bytes = (MAPS * st.slabs_d + st.slabs_n) * kSlab;
    st.warps = stage_bytes <= 12 * 1024 ? 4 : 2;
    st.count = 96 * 1024 / (st.warps * stage_bytes);
    st.count = st.count < 2 ? 2 : st.count > kMaxStages ? kMaxStages : st.count;
    const int smem = 1024 + st.warps * st.count * stage_bytes + MAPS * st.slabs_d * 128;

    GatherMaps maps;
    if (!encode_gather_map(&maps.v, a.V, BF, a.K, a.N, a.ldv)) return USM_ERR_CUDA;
    maps.k1 = maps.k2 = maps.v;
    if (a.D > 0 && !encode_gather_map(&maps.k1, a.Km, BF, a.K, a.D, a.ldk)) return USM_ERR_CUDA;
    if (TWO && a.D > 0 && !encode_gather_map(&maps.k2, a.K2, BF, a.K, a.D, a.ldk2)) return USM_ERR_CUDA;

    // CTAs a row: more until the rows fill the SMs or a row's windows (on
    // average) no longer give every warp one.
    const int sms = sm_count_current_device();
    const long long windows = a.nnz / a.M / kWindow + 1;
    int ctas = 1;
    while (ctas < 8 && (long long)a.M * ctas < 4LL * sms && (long long)ctas * st.warps < windows) ctas *= 2;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return USM_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.M * ctas));
    cfg.blockDim = dim3(st.warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a, st) == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

template <bool TWO>
int launch_bf16(const AttnArgs& a, cudaStream_t stream) {
    if (a.N <= 64) return launch_kernel<true, TWO>(attention_bf16_kernel<TWO, 8>, a, stream);
    if (a.N <= 128) return launch_kernel<true, TWO>(attention_bf16_kernel<TWO, 16>, a, stream);
    if (a.N <= 256) return launch_kernel<true, TWO>(attention_bf16_kernel<TWO, 32>, a, stream);
    return launch_kernel<true, TWO>(attention_bf16_kernel<TWO, 64>, a, stream);
}

template <bool TWO>
int launch_f32(const AttnArgs& a, cudaStream_t stream) {
    if (a.N <= 32) return launch_kernel<false, TWO>(attention_f32_kernel<TWO, 8, 1>, a, stream);
    if (a.N <= 64) return launch_kernel<false, TWO>(attention_f32_kernel<TWO, 16, 1>, a, stream);
    if (a.N <= 128) return launch_kernel<false, TWO>(attention_f32_kernel<TWO, 32, 1>, a, stream);
    return launch_kernel<false, TWO>(attention_f32_kernel<TWO, 32, 2>, a, stream);
}

}  // namespace

int launch_attention(const AttnArgs& a, bool bf16, cudaStream_t stream) {
    const bool two = a.lambda != nullptr;
    if (bf16) return two ? launch_bf16<true>(a, stream) : launch_bf16<false>(a, stream);
    return two ? launch_f32<true>(a, stream) : launch_f32<false>(a, stream);
}

}  // namespace usm
