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
// that asynchronous 16-byte copies fill with the windows' rows of K1, K2 and V:
// no barrier, and a warp's copies run ahead of its arithmetic by the ring.  A
// stage holds slabs of 128 bytes of each row, the 16-byte pieces of row i moved
// by i mod 8, so that reading one piece of eight rows meets no bank conflict.
// (TMA's gather of four rows an instruction was slower, 163 us against the
// figures below: each such instruction costs the warp about 14 issue slots,
// eight asynchronous copies that move as much about 16 for a whole window.)
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

constexpr int kMaxStages = 4, kWindow = 16;

// A stage holds, slab after slab (128 bytes of each of the 16 rows), SD slabs of
// K1, SD of K2 with two maps, and SN of V.
constexpr int kSlab = kWindow * 128;
template <bool TWO, int SD, int SN>
constexpr int kStageBytes = ((TWO ? 2 : 1) * SD + SN) * kSlab;

// Warps a CTA: four while two stages each fit in 96 KB (two CTAs an SM), else
// two; as many stages as fit there, 2 to kMaxStages.
constexpr int ring_warps(int stage_bytes) { return stage_bytes <= 12 * 1024 ? 4 : 2; }
constexpr int ring_stages(int stage_bytes) {
    const int n = 96 * 1024 / (ring_warps(stage_bytes) * stage_bytes);
    return n < 2 ? 2 : n > kMaxStages ? kMaxStages : n;
}

// Sums of a CTA's warps: o by column, the maximum and the sum of weights.
template <int MAPS, int NC, int WARPS>
struct Joined {
    float part[MAPS][WARPS][NC];
    float stat[MAPS][WARPS][2];
    float whole[MAPS][NC + 2];
};

__device__ __forceinline__ void copy_piece(uint32_t dst, const unsigned char* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most LEFT of the thread's groups are in flight.
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// One warp's windows of its row, and the ring their rows are copied into.  A
// lane copies one 16-byte piece (lane mod 8) of a row (lane / 8, of four at
// once) in every slab.
template <bool TWO, int SD, int SN, int ES>
struct Ring {
    static constexpr int kBytes = kStageBytes<TWO, SD, SN>, kWarps = ring_warps(kBytes), kCount = ring_stages(kBytes);
    uint32_t base;                      // shared address
    int (*cols)[kWindow];               // columns of each stage's entries
    int p0, p1, lane;
    int windows, first, stride;         // the warp's windows: first, first + stride, ... < windows
    int bytes_d[SD], bytes_n[SN];       // bytes of the lane's piece inside D and N: the rest become zeros, unread
    const unsigned char *k1, *k2, *v;   // the operands, at the lane's piece

    __device__ __forceinline__ int size(int w) const { return min(kWindow, p1 - (p0 + w * kWindow)); }
    // Column of entry `lane` of window w (the last entry's past the row's end).
    __device__ __forceinline__ int load_col(const int* __restrict__ ci, int w) const {
        return w < windows && lane < kWindow ? __ldg(ci + p0 + w * kWindow + min(lane, size(w) - 1)) : 0;
    }
    // Copies window w's rows into stage s (one group, empty past the last window).
    __device__ __forceinline__ void issue(const AttnArgs& a, int w, int s, int col) const {
        if (w < windows) {
            if (lane < kWindow) cols[s][lane] = col;
            col = min(max(col, 0), a.K - 1);
            const int n = size(w);
            const uint32_t dst = base + s * kBytes + (lane >> 3) * 128;
#pragma unroll
            for (int i = 0; i < kWindow / 4; ++i) {
                const int row = i * 4 + (lane >> 3);
                const long long c = (long long)__shfl_sync(kFullMask, col, row) * ES;
                if (i * 4 >= n) break;
                const uint32_t at = dst + i * 512 + (((lane ^ row) & 7) << 4);
                const unsigned char *r1 = k1 + c * a.ldk, *rv = v + c * a.ldv;
#pragma unroll
                for (int j = 0; j < SD; ++j) copy_piece(at + j * kSlab, r1 + j * 128, bytes_d[j]);
                if constexpr (TWO) {
                    const unsigned char* r2 = k2 + c * a.ldk2;
#pragma unroll
                    for (int j = 0; j < SD; ++j) copy_piece(at + (SD + j) * kSlab, r2 + j * 128, bytes_d[j]);
                }
#pragma unroll
                for (int j = 0; j < SN; ++j) copy_piece(at + ((TWO ? 2 : 1) * SD + j) * kSlab, rv + j * 128, bytes_n[j]);
            }
        }
        copies_commit();
    }
};

// Weight of a partial sum with maximum m_i under the common maximum.
__device__ __forceinline__ float join_weight(float m_i, float top) { return m_i == -INFINITY ? 0.f : __expf(m_i - top); }

// The CTA's warps (in `sh`), then the cluster's CTAs, and the row of C.
template <int MAPS, int NC, int WARPS>
__device__ __forceinline__ void join(Joined<MAPS, NC, WARPS>& sh, const AttnArgs& a, int r, int head, int ctas, int rank) {
    __syncthreads();
    constexpr int threads = WARPS * 32;
    const float lam = MAPS > 1 ? __ldg(a.lambda + head) : 0.f;
    for (int j = threadIdx.x; j < a.N; j += threads) {
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, sum = 0.f;
            for (int i = 0; i < WARPS; ++i) top = fmaxf(top, sh.stat[k][i][0]);
            for (int i = 0; i < WARPS; ++i) {
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
// Rows 0-7 of A·B + (c0, c1) (16 x 8 x 16, bf16 in, fp32 sums); rows 8-15 of A
// are zero, and theirs are dropped.
__device__ __forceinline__ float2 mma_upper(float2 c, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
    float2 d;
    [[maybe_unused]] float d2, d3;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%9,%10,%11,%11};"
        : "=f"(d.x), "=f"(d.y), "=f"(d2), "=f"(d3)
        : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(0.f));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// Everything both kernels do before their first window; false for a row
// without entries (its output is written).
template <bool TWO, int SD, int SN, int ES>
__device__ __forceinline__ bool start_row(const AttnArgs& a, Ring<TWO, SD, SN, ES>& ring, unsigned char* smem,
                                          int (*cols)[Ring<TWO, SD, SN, ES>::kCount][kWindow], int r, int ctas, int rank) {
    using R = Ring<TWO, SD, SN, ES>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    row_range(a.row_offsets, r, a.nnz, ring.p0, ring.p1);
    if (ring.p0 == ring.p1) {  // the same in every CTA of the cluster
        if (rank == 0)
            for (int j = threadIdx.x; j < a.N; j += R::kWarps * 32) a.C[(long long)r * a.ldc + j] = 0.f;
        return false;
    }
    ring.lane = lane;
    ring.base = smem_addr(smem) + warp * R::kCount * R::kBytes;
    ring.cols = cols[warp];
    ring.windows = (ring.p1 - ring.p0 - 1) / kWindow + 1;
    ring.first = rank * R::kWarps + warp;
    ring.stride = ctas * R::kWarps;
    const int piece = (lane & 7) * 16;
#pragma unroll
    for (int j = 0; j < SD; ++j) ring.bytes_d[j] = min(max(a.D * ES - j * 128 - piece, 0), 16);
#pragma unroll
    for (int j = 0; j < SN; ++j) ring.bytes_n[j] = min(max(a.N * ES - j * 128 - piece, 0), 16);
    ring.k1 = static_cast<const unsigned char*>(a.Km) + piece;
    ring.k2 = static_cast<const unsigned char*>(a.K2) + piece;
    ring.v = static_cast<const unsigned char*>(a.V) + piece;
    int ahead[R::kCount];
#pragma unroll
    for (int s = 0; s < R::kCount; ++s) ahead[s] = ring.load_col(a.col_indices, ring.first + s * ring.stride);
#pragma unroll 1
    for (int s = 0; s < R::kCount; ++s) {
        int col = ahead[0];
#pragma unroll
        for (int i = 1; i < R::kCount; ++i) col = s == i ? ahead[i] : col;
        ring.issue(a, ring.first + s * ring.stride, s, col);
    }
    return true;
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
template <bool TWO, int SD, int SN>
__global__ void __launch_bounds__(ring_warps(kStageBytes<TWO, SD, SN>) * 32) attention_bf16_kernel(const AttnArgs a) {
    constexpr int MAPS = TWO ? 2 : 1, NT = SN * 8, NC = NT * 8;  // tiles of 8 columns of V
    constexpr int kSteps = SD * 4;                               // steps of 16 dimensions
    using R = Ring<TWO, SD, SN, 2>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Joined<MAPS, NC, R::kWarps> sh;
    __shared__ int cols[R::kWarps][R::kCount][kWindow];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    R ring;
    if (!start_row(a, ring, smem, cols, r, ctas, rank)) return;
    const int block = r / a.seg_rows, head = block % a.heads;
    const int start =
        a.bias.table ? rel_start(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + ring.p0)) : 0;

    // q in steps of 16 dimensions (zeros past D): for each t the two words the lane passes.
    uint32_t* qs = reinterpret_cast<uint32_t*>(smem + R::kWarps * R::kCount * R::kBytes);
    for (int i = threadIdx.x; i < MAPS * kSteps * 8; i += R::kWarps * 32) {
        const int k = i / (kSteps * 8), w = i % (kSteps * 8);
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
    float2 o[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i] = make_float2(0.f, 0.f);
    int s = 0;
#pragma unroll 1
    for (int w = ring.first; w < ring.windows; w += ring.stride) {
        const int next = ring.load_col(a.col_indices, w + R::kCount * ring.stride);
        const uint32_t stage = ring.base + s * R::kBytes;
        copies_wait<R::kCount - 1>();
        __syncwarp();  // every lane's copies have landed
        // Dot products: 4 of each map in every lane.
        float2 x[MAPS][2];
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            x[k][0] = x[k][1] = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int c = 0; c < kSteps; ++c) {
                uint32_t b[4];
                load_matrix4(stage + k_row + (k * SD + c / 4) * kSlab + (((c % 4 * 2 + k_piece) ^ tile_row) << 4), b);
                const uint2 qw = lds64(q_addr + (k * kSteps + c) * 32);
                x[k][0] = mma_upper(x[k][0], qw.x, qw.y, b[0], b[1]);
                x[k][1] = mma_upper(x[k][1], qw.x, qw.y, b[2], b[3]);
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
                const float dot = u & 1 ? x[k][u >> 1].y : x[k][u >> 1].x;
                y[k] = en < n ? fmaf(dot, a.scale, bias) : -INFINITY;
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
            for (int i = 0; i < NT; ++i) o[i] = __fmul2_rn(o[i], make_float2(f, f));
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
                const uint32_t at = stage + MAPS * SD * kSlab + (__ffs(unused) - 1) * 128;
                for (int i = lane; i < SN * 8; i += 32)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + (i >> 3) * kSlab + (i & 7) * 16), "r"(0)
                                 : "memory");
            }
            __syncwarp();
        }
        const uint32_t v_at = stage + MAPS * SD * kSlab + v_row;
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            uint32_t b[4];
            load_matrix4_trans(v_at + i / 4 * kSlab + (((i % 4 * 2 + v_piece) ^ tile_row) << 4), b);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                o[2 * i + h] = __fadd2_rn(o[2 * i + h],
                                          mma_upper(make_float2(0.f, 0.f), w0, w1, b[2 * h], b[2 * h + 1]));
        }
        __syncwarp();  // every lane is done with the stage
        ring.issue(a, w + R::kCount * ring.stride, s, next);
        s = s + 1 == R::kCount ? 0 : s + 1;
    }

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
            const float high = u ? o[i].y : o[i].x;
            const float mid = __shfl_down_sync(kFullMask, high, 4), low = __shfl_down_sync(kFullMask, high, 8);
            if (writes) sh.part[mine][warp][i * 8 + 2 * t + u] = high + (mid + low);
        }
    join(sh, a, r, head, ctas, rank);
}

// fp32 on CUDA cores.  Scores: two lanes to an entry, each summing every other
// piece of 16 bytes.  Output: LV lanes to a row of V, four columns a lane (NP
// times), 32 / LV entries at once, weights broadcast by shuffles.
template <bool TWO, int SD, int SN>
__global__ void __launch_bounds__(ring_warps(kStageBytes<TWO, SD, SN>) * 32) attention_f32_kernel(const AttnArgs a) {
    constexpr int MAPS = TWO ? 2 : 1;
    constexpr int LV = SN >= 4 ? 32 : SN * 8, NP = SN * 8 / LV;
    constexpr int G = 32 / LV;       // rows of V a step
    constexpr int NC = LV * NP * 4;  // columns of the slabs
    using R = Ring<TWO, SD, SN, 4>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Joined<MAPS, NC, R::kWarps> sh;
    __shared__ int cols[R::kWarps][R::kCount][kWindow];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    R ring;
    if (!start_row(a, ring, smem, cols, r, ctas, rank)) return;
    const int block = r / a.seg_rows, head = block % a.heads;
    const int start =
        a.bias.table ? rel_start(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + ring.p0)) : 0;
    // Q1 and Q2 in whole slabs, zeros past D.
    float* qs = reinterpret_cast<float*>(smem + R::kWarps * R::kCount * R::kBytes);
    for (int i = threadIdx.x; i < MAPS * SD * 32; i += R::kWarps * 32) {
        const int k = i / (SD * 32), d = i % (SD * 32);
        const float* q = static_cast<const float*>(k ? a.Q2 : a.Q) + (long long)r * (k ? a.ldq2 : a.ldq);
        qs[i] = d < a.D ? __ldg(q + d) : 0.f;
    }
    __syncthreads();

    const int entry = lane & (kWindow - 1), share = lane / kWindow;
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
        v_slab[i] = (MAPS * SD + byte / 128) * kSlab;
        v_byte[i] = byte % 128;
    }
    int s = 0;
#pragma unroll 1
    for (int w = ring.first; w < ring.windows; w += ring.stride) {
        const int next = ring.load_col(a.col_indices, w + R::kCount * ring.stride);
        const uint32_t stage = ring.base + s * R::kBytes;
        copies_wait<R::kCount - 1>();
        __syncwarp();  // every lane's copies have landed
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
            const uint32_t at = stage + k * SD * kSlab + entry * 128, q = smem_addr(qs) + k * SD * 128 + share * 16;
            const int flip = (entry ^ share) & 7;
#pragma unroll 8
            for (int c = 0; c < SD * 8; c += 2) {
                const uint4 kw = lds128(at + (c >> 3) * kSlab + (((c & 7) ^ flip) << 4)), qw = lds128(q + c * 16);
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
        ring.issue(a, w + R::kCount * ring.stride, s, next);
        s = s + 1 == R::kCount ? 0 : s + 1;
    }

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
    join(sh, a, r, head, ctas, rank);
}

template <bool BF, bool TWO, int SD, int SN>
int launch_slabs(const AttnArgs& a, cudaStream_t stream) {
    using R = Ring<TWO, SD, SN, BF ? 2 : 4>;
    constexpr int smem = R::kWarps * R::kCount * R::kBytes + (TWO ? 2 : 1) * SD * 128;
    constexpr auto kernel = [] {
        if constexpr (BF)
            return attention_bf16_kernel<TWO, SD, SN>;
        else
            return attention_f32_kernel<TWO, SD, SN>;
    }();
    // CTAs a row: more until the rows fill the SMs or a row's windows (on
    // average) no longer give every warp one.
    const int sms = sm_count_current_device();
    const long long windows = a.nnz / a.M / kWindow + 1;
    int ctas = 1;
    while (ctas < 8 && (long long)a.M * ctas < 4LL * sms && (long long)ctas * R::kWarps < windows) ctas *= 2;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return USM_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.M * ctas));
    cfg.blockDim = dim3(R::kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

// Slabs: 1, 2, 4 or 8 of K, and as many or twice as many of V.
template <bool BF, bool TWO>
int launch_type(const AttnArgs& a, cudaStream_t stream) {
    constexpr int per = BF ? 64 : 32;
    const int d = (a.D + per - 1) / per, n = (a.N + per - 1) / per;
    if (d <= 1 && n <= 1) return launch_slabs<BF, TWO, 1, 1>(a, stream);
    if (d <= 1 && n <= 2) return launch_slabs<BF, TWO, 1, 2>(a, stream);
    if (d <= 2 && n <= 2) return launch_slabs<BF, TWO, 2, 2>(a, stream);
    if (d <= 2 && n <= 4) return launch_slabs<BF, TWO, 2, 4>(a, stream);
    if (d <= 4 && n <= 4) return launch_slabs<BF, TWO, 4, 4>(a, stream);
    if (d <= 4 && n <= 8) return launch_slabs<BF, TWO, 4, 8>(a, stream);
    return launch_slabs<BF, TWO, 8, 8>(a, stream);
}

}  // namespace

int launch_attention(const AttnArgs& a, bool bf16, cudaStream_t stream) {
    const bool two = a.lambda != nullptr;
    if (bf16) return two ? launch_type<true, true>(a, stream) : launch_type<true, false>(a, stream);
    return two ? launch_type<false, true>(a, stream) : launch_type<false, false>(a, stream);
}

}  // namespace usm
