// Sparse attention of few query rows in one pass (single tokens over a cache):
//     C[r] = Σ_p (P1[p] - λ P2[p]) V[c_p],   sk[p] = scale·(Qk[r]·Kk[c_p]) + bias(p),
// Pk the softmax of sk over the row's entries.
//
// One pass over the entries with a running maximum and sum for each map: with
// m the maximum so far, z = Σ exp(s - m) and o = Σ exp(s - m) V are scaled by
// exp(m - m') when the maximum rises to m'; at the end C = o1/z1 - λ o2/z2.
//
// What bounds it is how fast listed rows of 64 to 1024 bytes come from HBM, so
// copies must be in flight all the time, whatever the arithmetic does.  A warp
// takes its entries in windows of 16 and has a ring of stages of its own in
// shared memory that asynchronous 16-byte copies fill with the windows' rows of
// K1, K2, V and Q: no barrier, and its copies run ahead of its arithmetic by the
// ring.  A stage holds slabs of 128 bytes of each row, the 16-byte pieces of row
// i moved by i mod 8, so that reading one piece of eight rows meets no bank
// conflict.  (TMA's gather of four rows an instruction measured 163 us where
// these copies took 128: each such instruction costs the warp about 14 issue
// slots, a window's copies 16 and their addresses.)
//
// Two ways of dealing the work out.  Few entries: a cluster of 1, 2, 4 or 8
// CTAs to a row, its warps taking the row's windows in turn, joined through
// distributed shared memory: one launch, no workspace.  Many: every warp of a
// grid that fills the GPU once takes the same number of consecutive entries,
// whatever rows they belong to; a row inside one warp's share is finished there,
// the others' parts go to the workspace and a second kernel joins them.  No
// atomics, and a fixed order, either way.
//
// Products.  bf16: matrix instructions (16 x 8 x 16), which take the operands as
// they lie: on CUDA cores a window took three times the instructions and the
// kernel 201 us instead of 163.  fp32: CUDA cores.
#include <cmath>

#include "usm_cluster.cuh"
#include "usm_internal.h"
#include "usm_rel.cuh"

namespace usm {
namespace {

constexpr int kMaxStages = 4, kWindow = 16;
// A stage holds, slab after slab (128 bytes of each of the 16 rows), SD slabs of
// K1, SD of K2 with two maps, and SN of V; then the row's Q1 and Q2.
constexpr int kSlab = kWindow * 128;
template <bool TWO, int SD, int SN>
constexpr int kStageBytes = ((TWO ? 2 : 1) * SD + SN) * kSlab + (TWO ? 2 : 1) * SD * 128;

// Warps a CTA: four while a stage is at most 12 KB, else two; as many stages as
// fit in 66 KB (three CTAs an SM), 2 to kMaxStages.
constexpr int ring_warps(int stage_bytes) { return stage_bytes <= 12 * 1024 ? 4 : 2; }
constexpr int ring_stages(int stage_bytes) {
    const int n = 66 * 1024 / (ring_warps(stage_bytes) * stage_bytes);
    return n < 2 ? 2 : n > kMaxStages ? kMaxStages : n;
}

__device__ __forceinline__ void copy_piece(uint32_t dst, const unsigned char* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most LEFT of the thread's groups are in flight.
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Up to 16 entries of one row: [p, p + n) of row r.
struct Window {
    int r, p, n;
};

// The ring a warp's windows are copied into.  A lane copies one 16-byte piece
// (lane mod 8) of a row (lane / 8, of four at once) in every slab.
template <bool TWO, int SD, int SN, int ES>
struct Ring {
    static constexpr int kMaps = TWO ? 2 : 1;
    static constexpr int kBytes = kStageBytes<TWO, SD, SN>, kWarps = ring_warps(kBytes), kCount = ring_stages(kBytes);
    static constexpr int kSmem = kWarps * kCount * kBytes;
    uint32_t base;                         // shared address
    int (*cols)[kWindow];                  // columns of each stage's entries
    int lane;
    int bytes_d[SD], bytes_n[SN];          // bytes of the lane's piece inside D and N: the rest become zeros, unread
    const unsigned char *k1, *k2, *v;      // the operands, at the lane's piece
    unsigned pitch_k, pitch_k2, pitch_v;   // their rows, in pieces of 16 bytes

    __device__ __forceinline__ void init(const AttnArgs& a, unsigned char* smem, int (*all_cols)[kCount][kWindow]) {
        const int warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        base = smem_addr(smem) + warp * kCount * kBytes;
        cols = all_cols[warp];
        const int piece = (lane & 7) * 16;
#pragma unroll
        for (int j = 0; j < SD; ++j) bytes_d[j] = min(max(a.D * ES - j * 128 - piece, 0), 16);
#pragma unroll
        for (int j = 0; j < SN; ++j) bytes_n[j] = min(max(a.N * ES - j * 128 - piece, 0), 16);
        k1 = static_cast<const unsigned char*>(a.Km) + piece;
        k2 = static_cast<const unsigned char*>(a.K2) + piece;
        v = static_cast<const unsigned char*>(a.V) + piece;
        pitch_k = (unsigned)(a.ldk * ES / 16);
        pitch_k2 = (unsigned)(a.ldk2 * ES / 16);
        pitch_v = (unsigned)(a.ldv * ES / 16);
    }
    // Column of entry `lane` of a window (the last entry's past its end).
    __device__ __forceinline__ int load_col(const AttnArgs& a, const Window& w) const {
        return w.n > 0 && lane < kWindow ? __ldg(a.col_indices + w.p + min(lane, w.n - 1)) : 0;
    }
    // Copies a window's rows into stage s (one group, empty for no entries).
    __device__ __forceinline__ void issue(const AttnArgs& a, const Window& w, int s, int col) const {
        if (w.n > 0) {
            if (lane < kWindow) cols[s][lane] = col;
            col = min(max(col, 0), a.K - 1);
            const uint32_t stage = base + s * kBytes, dst = stage + (lane >> 3) * 128;
#pragma unroll
            for (int i = 0; i < kWindow / 4; ++i) {
                const int row = i * 4 + (lane >> 3);
                const unsigned c = (unsigned)__shfl_sync(kFullMask, col, row);
                if (i * 4 >= w.n) break;
                const uint32_t at = dst + i * 512 + (((lane ^ row) & 7) << 4);
                const unsigned char *r1 = k1 + 16 * ((unsigned long long)c * pitch_k),
                                    *rv = v + 16 * ((unsigned long long)c * pitch_v);
#pragma unroll
                for (int j = 0; j < SD; ++j) copy_piece(at + j * kSlab, r1 + j * 128, bytes_d[j]);
                if constexpr (TWO) {
                    const unsigned char* r2 = k2 + 16 * ((unsigned long long)c * pitch_k2);
#pragma unroll
                    for (int j = 0; j < SD; ++j) copy_piece(at + (SD + j) * kSlab, r2 + j * 128, bytes_d[j]);
                }
#pragma unroll
                for (int j = 0; j < SN; ++j) copy_piece(at + (kMaps * SD + j) * kSlab, rv + j * 128, bytes_n[j]);
            }
            // Q: piece i of the SD·8 of each map by lane i.
#pragma unroll
            for (int i = 0; i < (kMaps * SD * 8 + 31) / 32; ++i) {
                const int x = i * 32 + lane, k = x / (SD * 8), d = x % (SD * 8) * 16;
                if (x < kMaps * SD * 8) {
                    const unsigned char* q = k ? static_cast<const unsigned char*>(a.Q2) + (long long)w.r * a.ldq2 * ES
                                               : static_cast<const unsigned char*>(a.Q) + (long long)w.r * a.ldq * ES;
                    copy_piece(stage + (kMaps * SD + SN) * kSlab + x * 16, q + d, min(max(a.D * ES - d, 0), 16));
                }
            }
        }
        copies_commit();
    }
};

// What a row's bias needs.
struct RowBias {
    int head, start;
    __device__ __forceinline__ void set(const AttnArgs& a, int r, int p0) {
        const int block = r / a.seg_rows;
        head = block % a.heads;
        start = a.bias.table ? rel_start(a.bias, block, r - block * a.seg_rows, __ldg(a.col_indices + p0)) : 0;
    }
    __device__ __forceinline__ float at(const AttnArgs& a, int col) const {
        return a.bias.table ? rel_table(a.bias, head, rel_bucket(a.bias, rel_entry(col, start, a.bias.reach))) : 0.f;
    }
};

// Not volatile, so that loads and products interleave: what keeps them between
// the waits is that their address comes from pinned() and their results go
// through it.
__device__ __forceinline__ void load_matrix4(uint32_t at, uint32_t (&x)[4]) {
    asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
        : "r"(at));
}
__device__ __forceinline__ void load_matrix4_trans(uint32_t at, uint32_t (&x)[4]) {
    asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
        : "r"(at));
}
// The value as of here: nothing that makes it moves below, nothing that uses
// it above.
__device__ __forceinline__ uint32_t pinned(uint32_t x) {
    asm volatile("" : "+r"(x)::"memory");
    return x;
}
__device__ __forceinline__ uint32_t load_word(uint32_t at) {
    uint32_t x;
    asm("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at));
    return x;
}
__device__ __forceinline__ float2 pinned(float2 x) {
    asm volatile("" : "+f"(x.x), "+f"(x.y)::"memory");
    return x;
}
// Rows 0-7 of A·B + (c0, c1) (16 x 8 x 16, bf16 in, fp32 sums); rows 8-15 of A
// are zero, and theirs are dropped.
__device__ __forceinline__ float2 mma_upper(float2 c, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
    float2 d;
    [[maybe_unused]] float d2, d3;
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%9,%10,%11,%11};"
        : "=f"(d.x), "=f"(d.y), "=f"(d2), "=f"(d3)
        : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(0.f));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
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
struct RowBf16 {
    static constexpr int kElem = 2, kMaps = TWO ? 2 : 1, NT = SN * 8, kColumns = NT * 8, kSteps = SD * 4;
    using R = Ring<TWO, SD, SN, kElem>;
    float m, z;  // the lane's map's
    float2 o[NT];

    __device__ __forceinline__ int row() const { return (threadIdx.x & 31) >> 2; }
    __device__ __forceinline__ int mine() const { return TWO && row() >= 3; }  // the lane's map

    __device__ __forceinline__ void reset() {
        m = -INFINITY;
        z = 0.f;
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i] = make_float2(0.f, 0.f);
    }

    __device__ __forceinline__ void window(const AttnArgs& a, const R& ring, int s, int n, const RowBias& bias) {
        const uint32_t stage = pinned(ring.base + s * R::kBytes);
        const int lane = threadIdx.x & 31, t = lane & 3;
        const int part = row() - 3 * mine();  // of the weights
        // Operand tiles of 8 rows and 16 bytes: lane i addresses row i % 8 of tile i / 8.
        const int tile = lane >> 3, tile_row = lane & 7;
        const uint32_t k_row = (tile_row + 8 * (tile >> 1)) * 128, v_row = (tile_row + 8 * (tile & 1)) * 128;
        const uint32_t k_piece = tile & 1, v_piece = tile >> 1;
        // Dot products: 4 of each map in every lane.
        float2 x[kMaps][2];
#pragma unroll
        for (int k = 0; k < kMaps; ++k) {
            x[k][0] = x[k][1] = make_float2(0.f, 0.f);
            const uint32_t q = stage + (kMaps * SD + SN) * kSlab + k * SD * 128 + t * 4;
#pragma unroll 4
            for (int c = 0; c < kSteps; ++c) {
                uint32_t b[4];
                load_matrix4(stage + k_row + (k * SD + c / 4) * kSlab + (((c % 4 * 2 + k_piece) ^ tile_row) << 4), b);
                const uint32_t q0 = load_word(q + c * 32), q1 = load_word(q + c * 32 + 16);
                x[k][0] = mma_upper(x[k][0], q0, q1, b[0], b[1]);
                x[k][1] = mma_upper(x[k][1], q0, q1, b[2], b[3]);
            }
        }
        // Scores of the lane's map; entries that no map uses.
        float sc[4];
        unsigned unused = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int en = 2 * t + (u & 1) + (u >> 1) * 8;
            const float add = bias.at(a, ring.cols[s][en]);
            float y[kMaps];
            bool none = true;
#pragma unroll
            for (int k = 0; k < kMaps; ++k) {
                const float dot = u & 1 ? x[k][u >> 1].y : x[k][u >> 1].x;
                y[k] = en < n ? fmaf(dot, a.scale, add) : -INFINITY;
                none = none && y[k] == -INFINITY;
            }
            sc[u] = mine() ? y[kMaps - 1] : y[0];
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
        if (row() >= 3 * kMaps) w0 = w1 = 0;
        // Rows of V under entries that no map uses (and past the window's end)
        // may hold anything: they become zeros.
        if (__any_sync(kFullMask, unused != 0)) {
            unused |= __shfl_xor_sync(kFullMask, unused, 1);
            unused |= __shfl_xor_sync(kFullMask, unused, 2);
            for (; unused; unused &= unused - 1) {
                const uint32_t at = stage + kMaps * SD * kSlab + (__ffs(unused) - 1) * 128;
                for (int i = lane; i < SN * 8; i += 32)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at + (i >> 3) * kSlab + (i & 7) * 16), "r"(0)
                                 : "memory");
            }
            __syncwarp();
        }
        const uint32_t v_at = pinned(stage + kMaps * SD * kSlab + v_row);
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            uint32_t b[4];
            load_matrix4_trans(v_at + i / 4 * kSlab + (((i % 4 * 2 + v_piece) ^ tile_row) << 4), b);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                o[2 * i + h] = __fadd2_rn(o[2 * i + h],
                                          mma_upper(make_float2(0.f, 0.f), w0, w1, b[2 * h], b[2 * h + 1]));
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i] = pinned(o[i]);
    }

    // The warp's maximum and sums of each map, to part[map][column] and stat[map].
    __device__ __forceinline__ void emit(float* part, size_t map_stride, float (*stat)[2]) {
        const int t = threadIdx.x & 3;
        z += __shfl_xor_sync(kFullMask, z, 1);
        z += __shfl_xor_sync(kFullMask, z, 2);
        const bool writes = row() == 0 || (TWO && row() == 3);
        if (writes && t == 0) {
            stat[mine()][0] = m;
            stat[mine()][1] = z;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float2 x = o[i];
            x.x += __shfl_down_sync(kFullMask, o[i].x, 4) + __shfl_down_sync(kFullMask, o[i].x, 8);
            x.y += __shfl_down_sync(kFullMask, o[i].y, 4) + __shfl_down_sync(kFullMask, o[i].y, 8);
            if (writes) *reinterpret_cast<float2*>(part + mine() * map_stride + i * 8 + 2 * t) = x;
        }
    }
};

// fp32 on CUDA cores.  Scores: two lanes to an entry, each summing every other
// piece of 16 bytes.  Output: LV lanes to a row of V, four columns a lane (NP
// times), 32 / LV entries at once, weights broadcast by shuffles.
template <bool TWO, int SD, int SN>
struct RowF32 {
    static constexpr int kElem = 4, kMaps = TWO ? 2 : 1, kColumns = SN * 32;
    static constexpr int LV = SN >= 4 ? 32 : SN * 8, NP = SN * 8 / LV, G = 32 / LV;
    using R = Ring<TWO, SD, SN, kElem>;
    float m[kMaps], z[kMaps];
    float2 o[kMaps][NP][2];

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int k = 0; k < kMaps; ++k) {
            m[k] = -INFINITY;
            z[k] = 0.f;
#pragma unroll
            for (int i = 0; i < NP; ++i) o[k][i][0] = o[k][i][1] = make_float2(0.f, 0.f);
        }
    }

    __device__ __forceinline__ void window(const AttnArgs& a, const R& ring, int s, int n, const RowBias& bias) {
        const uint32_t stage = ring.base + s * R::kBytes;
        const int lane = threadIdx.x & 31;
        const int entry = lane & (kWindow - 1), share = lane / kWindow;
        const int g = lane / LV, l = lane % LV;
        const bool in = entry < n;
        const float add = bias.at(a, ring.cols[s][entry]);
        float e[kMaps];
        bool used = false;
#pragma unroll
        for (int k = 0; k < kMaps; ++k) {
            float2 x = make_float2(0.f, 0.f), y = x;
            const uint32_t at = stage + k * SD * kSlab + entry * 128;
            const uint32_t q = stage + (kMaps * SD + SN) * kSlab + k * SD * 128 + share * 16;
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
            const float sc = in ? fmaf(dot, a.scale, add) : -INFINITY;
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
            float2 et[kMaps];
#pragma unroll
            for (int k = 0; k < kMaps; ++k) {
                const float f = __shfl_sync(kFullMask, e[k], en);
                et[k] = make_float2(f, f);
            }
            const bool take = !guard || __shfl_sync(kFullMask, (int)used, en) != 0;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int byte = (i * LV + l) * 16;
                const uint4 vw = lds128(stage + (kMaps * SD + byte / 128) * kSlab + en * 128 + ((byte % 128) ^ ((en & 7) << 4)));
                float2 v0 = make_float2(__uint_as_float(vw.x), __uint_as_float(vw.y));
                float2 v1 = make_float2(__uint_as_float(vw.z), __uint_as_float(vw.w));
                if (!take) v0 = v1 = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kMaps; ++k) {
                    o[k][i][0] = __ffma2_rn(et[k], v0, o[k][i][0]);
                    o[k][i][1] = __ffma2_rn(et[k], v1, o[k][i][1]);
                }
            }
        }
    }

    __device__ __forceinline__ void emit(float* part, size_t map_stride, float (*stat)[2]) {
        const int lane = threadIdx.x & 31, g = lane / LV, l = lane % LV;
#pragma unroll
        for (int k = 0; k < kMaps; ++k) {
#pragma unroll
            for (int d = 16; d > 0; d /= 2) z[k] += __shfl_xor_sync(kFullMask, z[k], d);
            if (lane == 0) {
                stat[k][0] = m[k];
                stat[k][1] = z[k];
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float x[4] = {o[k][i][0].x, o[k][i][0].y, o[k][i][1].x, o[k][i][1].y};
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int d = LV; d < 32; d *= 2) x[u] += __shfl_xor_sync(kFullMask, x[u], d);
                if (g == 0)
                    *reinterpret_cast<float4*>(part + k * map_stride + (i * LV + l) * 4) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
    }
};

// Weight of a partial sum with maximum m_i under the common maximum.
__device__ __forceinline__ float join_weight(float m_i, float top) { return m_i == -INFINITY ? 0.f : __expf(m_i - top); }

// -------------------------------------------------------- a cluster to a row
template <class Row>
__global__ void __launch_bounds__(Row::R::kWarps * 32) attention_cluster_kernel(const AttnArgs a) {
    using R = typename Row::R;
    constexpr int MAPS = Row::kMaps, NC = Row::kColumns, W = R::kWarps, threads = W * 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float part[W][MAPS][NC];
    __shared__ float stat[W][MAPS][2];
    __shared__ float whole[MAPS][NC + 2];  // the CTA's: sums, maximum, sum of weights
    __shared__ int cols[W][R::kCount][kWindow];
    const int warp = threadIdx.x >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int r = blockIdx.x / ctas;
    int p0, p1;
    row_range(a.row_offsets, r, a.nnz, p0, p1);
    float* crow = a.C + (long long)r * a.ldc;
    if (p0 == p1) {  // the same in every CTA of the cluster
        if (rank == 0)
            for (int j = threadIdx.x; j < a.N; j += threads) crow[j] = 0.f;
        return;
    }
    R ring;
    ring.init(a, smem, cols);
    // The warp's windows: first, first + stride, ...
    const int windows = (p1 - p0 - 1) / kWindow + 1, first = rank * W + warp, stride = ctas * W;
    auto at = [&](int w) {
        return w < windows ? Window{r, p0 + w * kWindow, min(kWindow, p1 - (p0 + w * kWindow))} : Window{r, 0, 0};
    };
    int ahead[R::kCount];
#pragma unroll
    for (int s = 0; s < R::kCount; ++s) ahead[s] = ring.load_col(a, at(first + s * stride));
#pragma unroll
    for (int s = 0; s < R::kCount; ++s) ring.issue(a, at(first + s * stride), s, ahead[s]);
    RowBias bias;
    bias.set(a, r, p0);
    const float lam = MAPS > 1 ? __ldg(a.lambda + bias.head) : 0.f;
    Row row;
    row.reset();
    int s = 0;
#pragma unroll 1
    for (int w = first; w < windows; w += stride) {
        const Window then = at(w + R::kCount * stride);
        const int next = ring.load_col(a, then);
        copies_wait<R::kCount - 1>();
        __syncwarp();  // every lane's copies have landed
        row.window(a, ring, s, min(kWindow, p1 - (p0 + w * kWindow)), bias);
        __syncwarp();  // every lane is done with the stage
        ring.issue(a, then, s, next);
        s = s + 1 == R::kCount ? 0 : s + 1;
    }
    row.emit(&part[warp][0][0], NC, stat[warp]);
    __syncthreads();

    // The CTA's warps.
    for (int j = threadIdx.x; j < a.N; j += threads) {
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, sum = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) top = fmaxf(top, stat[i][k][0]);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float f = join_weight(stat[i][k][0], top);
                x += f * part[i][k][j];
                sum += f * stat[i][k][1];
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
        if (ctas == 1) crow[j] = res;
    }
    if (ctas == 1) return;
    // The cluster's CTAs: runs of 32 columns are dealt to them in turn.
    cluster_sync();
    for (int j = threadIdx.x; j < a.N; j += threads) {
        if (j / 32 % ctas != rank) continue;
        float res = 0.f;
#pragma unroll
        for (int k = 0; k < MAPS; ++k) {
            float top = -INFINITY, x = 0.f, sum = 0.f;
            for (int i = 0; i < ctas; ++i) top = fmaxf(top, load_cluster(smem_addr(&whole[k][NC]), i));
            for (int i = 0; i < ctas; ++i) {
                const float f = join_weight(load_cluster(smem_addr(&whole[k][NC]), i), top);
                x += f * load_cluster(smem_addr(&whole[k][j]), i);
                sum += f * load_cluster(smem_addr(&whole[k][NC + 1]), i);
            }
            if (sum != 0.f) res += (k == 0 ? 1.f : -lam) * (x / sum);
        }
        crow[j] = res;
    }
    cluster_sync();  // no CTA leaves while another may read its sums
}

// ------------------------------------------------- equal shares of all entries
// Share g of G is entries [first(g), first(g + 1)) of the E = nnz.
__device__ __forceinline__ int share_first(int nnz, int g, int G) { return (int)((long long)nnz * g / G); }
__device__ __forceinline__ int share_of(int p, int nnz, int G) { return (int)((((long long)p + 1) * G - 1) / nnz); }

// A share's parts of rows that other shares hold parts of too: part 0 of the row
// that began before the share, part 1 of the row that goes on after it (a row
// that does both is part 0).  In the workspace a part is, for each map, the sums
// of its columns, the maximum and the sum of weights.
__device__ __forceinline__ float* part_at(float* parts, int g, int which, int maps, int columns) {
    return parts + ((long long)g * 2 + which) * maps * (columns + 2);
}

// The warp's walk over its share: windows of consecutive rows.
struct Walk {
    const int* ro;
    int nnz, M, r, p, row_end, end;  // at entry p of row r, which ends at row_end; the share ends at `end`

    // The last of rows [lo, M) that starts at or before entry p (32 candidates a
    // round).
    __device__ __forceinline__ int row_of(int lo) const {
        for (int n = M - lo; n > 1;) {
            const int step = (int)((n + 31LL) / 32), lane = threadIdx.x & 31;
            const bool in = (long long)lane * step < n;
            const unsigned before = __ballot_sync(kFullMask, in && __ldg(ro + lo + (in ? lane * step : 0)) <= p);
            const int skip = before ? (31 - __clz(before)) * step : 0;
            lo += skip;
            n = min(step, n - skip);
        }
        return lo;
    }
    // To the first row at or after r that has entries from p on.
    __device__ __forceinline__ void settle() {
        if (p < end && r < M) {
            int b;
            row_range(ro, r, nnz, b, row_end);
            p = max(p, b);
            if (p >= row_end) {  // over the rows without entries
                r = row_of(r);
                row_range(ro, r, nnz, b, row_end);
            }
            if (p >= b && p < min(row_end, end)) return;
        }
        p = end;
    }
    // The window here, and on to the next one.
    __device__ __forceinline__ Window take() {
        if (p >= end) return {0, 0, 0};
        const int stop = min(row_end, end);
        const Window w{r, p, min(kWindow, stop - p)};
        p += w.n;
        if (p >= row_end) {
            ++r;
            settle();
        }
        return w;
    }
};

template <class Row>
__global__ void __launch_bounds__(Row::R::kWarps * 32)
    attention_shares_kernel(const AttnArgs a, float* parts, int* cut_rows, int G) {
    let_next_start();
    using R = typename Row::R;
    constexpr int MAPS = Row::kMaps, NC = Row::kColumns, W = R::kWarps;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float part[W][MAPS][NC];
    __shared__ float stat[W][MAPS][2];
    __shared__ int cols[W][R::kCount][kWindow];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.x * W + warp;
    if (g >= G) return;  // no barriers below: warps work alone
    const int begin = share_first(a.nnz, g, G);
    Walk walk{a.row_offsets, a.nnz, a.M, 0, begin, 0, share_first(a.nnz, g + 1, G)};
    walk.r = walk.row_of(0);
    walk.settle();

    R ring;
    ring.init(a, smem, cols);
    Window queue[R::kCount];
#pragma unroll
    for (int s = 0; s < R::kCount; ++s) {
        queue[s] = walk.take();
        const int col = ring.load_col(a, queue[s]);
        ring.issue(a, queue[s], s, col);
    }
    Row row;
    RowBias bias;
    bias.head = bias.start = 0;
    int s = 0, at_row = -1, p0 = 0, p1 = 0, cut = -1;
#pragma unroll 1
    while (true) {
        const Window w = queue[0];
        if (w.n == 0) break;
        const Window then = walk.take();
        const int next = ring.load_col(a, then);
#pragma unroll
        for (int i = 0; i + 1 < R::kCount; ++i) queue[i] = queue[i + 1];
        queue[R::kCount - 1] = then;
        if (w.r != at_row) {
            at_row = w.r;
            row_range(a.row_offsets, w.r, a.nnz, p0, p1);
            bias.set(a, w.r, p0);
            row.reset();
        }
        copies_wait<R::kCount - 1>();
        __syncwarp();  // every lane's copies have landed
        row.window(a, ring, s, w.n, bias);
        __syncwarp();  // every lane is done with the stage
        ring.issue(a, then, s, next);
        s = s + 1 == R::kCount ? 0 : s + 1;
        if (queue[0].n != 0 && queue[0].r == w.r) continue;
        // The last of the share's windows of this row.
        row.emit(&part[warp][0][0], NC, stat[warp]);
        __syncwarp();
        const bool began = p0 >= begin, ends = w.p + w.n == p1;
        if (began && ends) {
            const float lam = MAPS > 1 ? __ldg(a.lambda + bias.head) : 0.f;
            for (int j = lane; j < a.N; j += 32) {
                float res = 0.f;
#pragma unroll
                for (int k = 0; k < MAPS; ++k)
                    if (stat[warp][k][1] != 0.f) res += (k == 0 ? 1.f : -lam) * (part[warp][k][j] / stat[warp][k][1]);
                a.C[(long long)w.r * a.ldc + j] = res;
            }
        } else {
            float* to = part_at(parts, g, began ? 1 : 0, MAPS, a.N);
            if (began) cut = w.r;
#pragma unroll
            for (int k = 0; k < MAPS; ++k) {
                for (int j = lane; j < a.N; j += 32) to[k * (a.N + 2) + j] = part[warp][k][j];
                if (lane < 2) to[k * (a.N + 2) + a.N + lane] = stat[warp][k][lane];
            }
        }
        __syncwarp();  // part and stat are free again
    }
    if (lane == 0) cut_rows[g] = cut;
}

// Joins the parts of rows that several shares hold and writes zeros to the rows
// without entries: columns 32c..32c+31 by CTA (i, c), eight threads to a column,
// each joining every eighth part.  BY_ROWS, for no more rows than shares: CTA
// (r, c) looks after row r.  Else CTA (g, c), g < G, after the row that goes on
// after share g, if one does, and the CTAs past G after 256 rows each.  (256 rows
// of 1824 shares: 5 us by shares, most of whose CTAs find nothing to do, 4 by
// rows.)
template <int MAPS, bool BY_ROWS>
__global__ void __launch_bounds__(256)
    attention_join_kernel(const AttnArgs a, const float* parts, const int* cut_rows, int G) {
    __shared__ float sums[8][MAPS][3][32];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, j = blockIdx.y * 32 + lane;
    int g0 = blockIdx.x, r = blockIdx.x, p0, p1;
    if constexpr (BY_ROWS) row_range(a.row_offsets, r, a.nnz, p0, p1);
    await_previous();  // in every CTA: the kernel must not end before the one it follows
    if constexpr (BY_ROWS) {
        if (p0 == p1) {
            if (grp == 0 && j < a.N) a.C[(long long)r * a.ldc + j] = 0.f;
            return;
        }
        g0 = share_of(p0, a.nnz, G);
    } else {
        if (g0 >= G) {
            const long long r0 = (g0 - G) * 256LL + grp * 32;
            bool empty = false;
            if (blockIdx.y == 0 && r0 + lane < a.M) {
                row_range(a.row_offsets, (int)r0 + lane, a.nnz, p0, p1);
                empty = p0 == p1;
            }
            for (unsigned rows = __ballot_sync(kFullMask, empty); rows; rows &= rows - 1)
                for (int c = lane; c < a.N; c += 32) a.C[(r0 + __ffs(rows) - 1) * a.ldc + c] = 0.f;
            return;
        }
        r = cut_rows[g0];
        if (r < 0) return;
        row_range(a.row_offsets, r, a.nnz, p0, p1);
    }
    const int g1 = p0 < p1 ? share_of(p1 - 1, a.nnz, G) : g0;
    if (BY_ROWS && g0 == g1) return;
    const int col = min(j, a.N - 1);
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        float top = -INFINITY, x = 0.f, z = 0.f;
        for (int g = g0 + grp; g <= g1; g += 8) {
            const float* from = part_at(const_cast<float*>(parts), g, g == g0, MAPS, a.N) + k * (a.N + 2);
            const float m = from[a.N], t = fmaxf(top, m), f = join_weight(top, t), h = join_weight(m, t);
            x = x * f + h * from[col];
            z = z * f + h * from[a.N + 1];
            top = t;
        }
        sums[grp][k][0][lane] = top;
        sums[grp][k][1][lane] = x;
        sums[grp][k][2][lane] = z;
    }
    __syncthreads();
    if (grp != 0 || j >= a.N) return;
    float res = 0.f;
#pragma unroll
    for (int k = 0; k < MAPS; ++k) {
        float top = -INFINITY, x = 0.f, z = 0.f;
        for (int i = 0; i < 8; ++i) top = fmaxf(top, sums[i][k][0][lane]);
        for (int i = 0; i < 8; ++i) {
            const float f = join_weight(sums[i][k][0][lane], top);
            x += f * sums[i][k][1][lane];
            z += f * sums[i][k][2][lane];
        }
        const float w = k == 0 ? 1.f : -__ldg(a.lambda + r / a.seg_rows % a.heads);
        if (z != 0.f) res += w * (x / z);
    }
    a.C[(long long)r * a.ldc + j] = res;
}

// ---------------------------------------------------------------- launches
// Shares pay once the rows' bytes take longer than the second launch and the
// parts' way through memory cost: measured even at about 12 MB.
constexpr long long kShareBytes = 12LL << 20;

bool takes_shares(const AttnArgs& a, int es) {
    return (long long)a.nnz * ((a.lambda ? 2 : 1) * a.D + a.N) * es >= kShareBytes;
}

// Warps that share the entries: as many as 152 SMs hold at once (three CTAs an
// SM; two or one of the widest rows), at least 64 entries each.
template <class Row>
int share_count(int nnz) {
    const int G = 152 * (Row::R::kSmem <= 66 * 1024 ? 3 : Row::R::kSmem <= 100 * 1024 ? 2 : 1) * Row::R::kWarps;
    return nnz / 64 < G ? nnz / 64 : G;
}

template <class Row>
struct Launch {
    static size_t workspace(const AttnArgs& a) {
        if (!takes_shares(a, Row::kElem)) return 0;
        return (size_t)share_count<Row>(a.nnz) * (2 * Row::kMaps * (a.N + 2) + 1) * 4;
    }

    static int run(const AttnArgs& a, void* workspace, cudaStream_t stream) {
        using R = typename Row::R;
        const int sms = sm_count_current_device();
        if (takes_shares(a, Row::kElem)) {
            const int G = share_count<Row>(a.nnz);
            float* parts = static_cast<float*>(workspace);
            int* cut_rows = reinterpret_cast<int*>(parts + (size_t)G * 2 * Row::kMaps * (a.N + 2));
            const auto kernel = attention_shares_kernel<Row>;
            if (!allow_shared(kernel, R::kSmem)) return cuda_failure();
            kernel<<<(G + R::kWarps - 1) / R::kWarps, R::kWarps * 32, R::kSmem, stream>>>(a, parts, cut_rows, G);
            if (cudaGetLastError() != cudaSuccess) return USM_ERR_CUDA;
            const unsigned strips = (a.N + 31) / 32;
            if (a.M <= G)
                return launch_next(attention_join_kernel<Row::kMaps, true>, dim3(a.M, strips), 256, 1, stream, a,
                                   (const float*)parts, (const int*)cut_rows, G);
            return launch_next(attention_join_kernel<Row::kMaps, false>,
                               dim3((unsigned)(G + ((long long)a.M + 255) / 256), strips), 256, 1, stream, a,
                               (const float*)parts, (const int*)cut_rows, G);
        }
        // CTAs a row: more until the rows fill the SMs or a row's windows (on
        // average) no longer give every warp one.
        const long long windows = a.nnz / a.M / kWindow + 1;
        int ctas = 1;
        while (ctas < 8 && (long long)a.M * ctas < 4LL * sms && (long long)ctas * R::kWarps < windows) ctas *= 2;
        const auto kernel = attention_cluster_kernel<Row>;
        if (!allow_shared(kernel, R::kSmem)) return cuda_failure();
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = ctas;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((long long)a.M * ctas));
        cfg.blockDim = dim3(R::kWarps * 32);
        cfg.dynamicSmemBytes = R::kSmem;
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? USM_OK : cuda_failure();
    }
};

// Calls f with the Launch of the widths: 1, 2, 4 or 8 slabs of K, and as many
// or twice as many of V.
template <template <bool, int, int> class Row, bool TWO, class F>
auto with_slabs(const AttnArgs& a, F f) {
    constexpr int per = 128 / Row<TWO, 1, 1>::kElem;
    const int d = (a.D + per - 1) / per, n = (a.N + per - 1) / per;
    if (d <= 1 && n <= 1) return f(Launch<Row<TWO, 1, 1>>{});
    if (d <= 1 && n <= 2) return f(Launch<Row<TWO, 1, 2>>{});
    if (d <= 2 && n <= 2) return f(Launch<Row<TWO, 2, 2>>{});
    if (d <= 2 && n <= 4) return f(Launch<Row<TWO, 2, 4>>{});
    if (d <= 4 && n <= 4) return f(Launch<Row<TWO, 4, 4>>{});
    if (d <= 4 && n <= 8) return f(Launch<Row<TWO, 4, 8>>{});
    return f(Launch<Row<TWO, 8, 8>>{});
}

template <class F>
auto with_launch(const AttnArgs& a, bool bf16, F f) {
    if (bf16) return a.lambda ? with_slabs<RowBf16, true>(a, f) : with_slabs<RowBf16, false>(a, f);
    return a.lambda ? with_slabs<RowF32, true>(a, f) : with_slabs<RowF32, false>(a, f);
}

}  // namespace

size_t attention_workspace_bytes(const AttnArgs& a, bool bf16) {
    return with_launch(a, bf16, [&](auto l) { return l.workspace(a); });
}

int launch_attention(const AttnArgs& a, bool bf16, void* workspace, cudaStream_t stream) {
    return with_launch(a, bf16, [&](auto l) { return l.run(a, workspace, stream); });
}

}  // namespace usm
