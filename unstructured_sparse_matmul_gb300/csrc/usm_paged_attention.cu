// Attention of a chunk of new tokens over a paged cache.  Contract and masks:
// include/usm.h; how the work is divided: usm_paged.cuh.
#include <cuda_bf16.h>

#include <algorithm>

#include "usm_internal.h"
#include "usm_paged.cuh"

namespace usm {
namespace {

// ---------------------------------------------------------------------------
// fp32 products on the FMA units: fp32 caches, and bf16 heads wider than the
// matrix kernel takes.  kRows rows of queries stay in shared memory; tiles of
// 64 keys pass through it.  Each of 256 threads holds 4 rows x 4 keys of the
// scores and 4 rows x up to 16 columns of the sums.
// ---------------------------------------------------------------------------
constexpr int kBlockRows = 64, kBlockKeys = 64, kBlockThreads = 256;
using BlockShares = PagedShares<kBlockRows, kBlockKeys, kBlockThreads, 2>;

template <class T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float4 x, float* p) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(float4 x, __nv_bfloat16* p) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x.w), "f"(x.z));
    *reinterpret_cast<uint2*>(p) = w;
}

// Row pitch of the shared arrays: a multiple of 4 that is 4 modulo 32, so that 8
// consecutive rows start in different groups of banks.
constexpr int block_pitch(int head_dim) { return (head_dim + 31) / 32 * 32 + 4; }
constexpr int block_smem(int head_dim) {
    return (kBlockRows + 2 * kBlockKeys) * block_pitch(head_dim) * 4 + kBlockRows * (kBlockKeys + 4) * 4;
}

// Reference of a row's exponents and its weight relative to another's: both
// -inf (nothing seen) gives 0.
__device__ __forceinline__ float weight_of(float m, float top, float scale_log2) {
    return m == -INFINITY ? 0.f : exp2_fast((m - top) * scale_log2);
}

template <class T, int kWide>  // kWide: groups of 64 columns
__global__ void __launch_bounds__(kBlockThreads) paged_block_kernel(const PagedArgs a) {
    extern __shared__ float4 smem_raw[];
    __shared__ long long scratch[kBlockThreads / 32 + 2];
    __shared__ PagedSegment seg;
    let_next_start();
    const int D = a.head_dim, pitch = block_pitch(D);
    float* q = reinterpret_cast<float*>(smem_raw);
    float* k = q + kBlockRows * pitch;
    float* v = k + kBlockKeys * pitch;
    float* p = v + kBlockKeys * pitch;  // probabilities, [row][key]
    constexpr int kP = kBlockKeys + 4;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int quads = D / 4;

    BlockShares shares;
    shares.init(a, blockIdx.x, gridDim.x, scratch);
    PagedMeta meta = {};
    while (true) {
        __syncthreads();
        if (tid < 32) {
            const PagedSegment g = shares.next(a);
            if (g.live) paged_note(meta, g);
            if (tid == 0) seg = g;
        }
        __syncthreads();
        if (!seg.live) break;
        const PagedSegment g = seg;
        for (int i = tid; i < kBlockRows * quads; i += kBlockThreads) {
            const int r = i / quads, c = i - r * quads;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < g.rows) {
                const int flat = g.row0 + r, token = flat / a.group, head = g.head * a.group + flat - token * a.group;
                x = load4((const T*)a.q + (g.start + token) * a.q_token + head * a.q_head + 4 * c);
            }
            *reinterpret_cast<float4*>(q + r * pitch + 4 * c) = x;
        }
        int2 seen[4];
        float m[4], l[4], o[4][4 * kWide];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            seen[i] = paged_seen(a, g, ty * 4 + i);
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4 * kWide; ++j) o[i][j] = 0.f;
        }
        for (int t = 0; t < g.tiles; ++t) {
            const int key0 = (g.tile0 + t) * kBlockKeys;
            __syncthreads();  // the last tile's readers are done
            for (int i = tid; i < kBlockKeys * quads; i += kBlockThreads) {
                const int r = i / quads, c = i - r * quads, key = key0 + r;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (key >= g.lo && key < g.hi) {
                    const int2 w = paged_slot(a, g.seq, key);
                    x = load4((const T*)a.k + w.x * a.k_page + w.y * a.k_slot + g.head * a.k_head + 4 * c);
                    y = load4((const T*)a.v + w.x * a.v_page + w.y * a.v_slot + g.head * a.v_head + 4 * c);
                }
                *reinterpret_cast<float4*>(k + r * pitch + 4 * c) = x;
                *reinterpret_cast<float4*>(v + r * pitch + 4 * c) = y;
            }
            __syncthreads();
            // Scores of rows 4·ty.. and keys tx, tx + 16, ...
            float s[4][4] = {};
            for (int d = 0; d < D; d += 4) {
                float4 qa[4], ka[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qa[i] = *reinterpret_cast<const float4*>(q + (ty * 4 + i) * pitch + d);
                    ka[i] = *reinterpret_cast<const float4*>(k + (tx + 16 * i) * pitch + d);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(qa[i].w, ka[j].w, fmaf(qa[i].z, ka[j].z, fmaf(qa[i].y, ka[j].y, fmaf(qa[i].x, ka[j].x, s[i][j]))));
            }
            bool partly = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + tx + 16 * j;
                    if (key < seen[i].x || key >= seen[i].y) s[i][j] = -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, w));
                top = fmaxf(top, m[i]);
                const float f = weight_of(m[i], top, a.scale_log2);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = s[i][j] == -INFINITY ? 0.f : exp2_fast((s[i][j] - top) * a.scale_log2);
                    p[(ty * 4 + i) * kP + tx + 16 * j] = e;
                    sum += e;
                }
                l[i] = l[i] * f + sum;  // this thread's keys
#pragma unroll
                for (int j = 0; j < 4 * kWide; ++j) o[i][j] *= f;
                partly |= seen[i].x > key0 || seen[i].y < key0 + kBlockKeys;
            }
            __syncwarp();  // a warp's rows of p are its own
            // Where a row does not see the whole tile a weight of 0 takes no value.
            const bool guard = __any_sync(kFullMask, partly);
            for (int key = 0; key < kBlockKeys; key += 4) {
                float4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + (ty * 4 + i) * kP + key);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
#pragma unroll
                    for (int c = 0; c < kWide; ++c) {
                        const int col = 64 * c + 4 * tx;
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (col < D) y = *reinterpret_cast<const float4*>(v + (key + u) * pitch + col);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e = u == 0 ? w[i].x : u == 1 ? w[i].y : u == 2 ? w[i].z : w[i].w;
                            if (guard) {
                                const int at = key0 + key + u;
                                const bool use = at >= seen[i].x && at < seen[i].y;
                                if (use) {
                                    o[i][4 * c] = fmaf(e, y.x, o[i][4 * c]);
                                    o[i][4 * c + 1] = fmaf(e, y.y, o[i][4 * c + 1]);
                                    o[i][4 * c + 2] = fmaf(e, y.z, o[i][4 * c + 2]);
                                    o[i][4 * c + 3] = fmaf(e, y.w, o[i][4 * c + 3]);
                                }
                            } else {
                                o[i][4 * c] = fmaf(e, y.x, o[i][4 * c]);
                                o[i][4 * c + 1] = fmaf(e, y.y, o[i][4 * c + 1]);
                                o[i][4 * c + 2] = fmaf(e, y.z, o[i][4 * c + 2]);
                                o[i][4 * c + 3] = fmaf(e, y.w, o[i][4 * c + 3]);
                            }
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(kFullMask, l[i], w);
            const int r = ty * 4 + i;
            if (r >= g.rows) continue;
            if (g.part == kPartWhole) {
                const int flat = g.row0 + r, token = flat / a.group, head = g.head * a.group + flat - token * a.group;
                const float z = l[i] == 0.f ? 0.f : 1.f / l[i];
                T* out = (T*)a.out + (g.start + token) * a.out_token + head * a.out_head;
#pragma unroll
                for (int c = 0; c < kWide; ++c) {
                    const int col = 64 * c + 4 * tx;
                    if (col < D)
                        store4(make_float4(o[i][4 * c] * z, o[i][4 * c + 1] * z, o[i][4 * c + 2] * z, o[i][4 * c + 3] * z),
                               out + col);
                }
            } else {
                const long long row = (2LL * blockIdx.x + g.part) * a.part_rows + r;
#pragma unroll
                for (int c = 0; c < kWide; ++c) {
                    const int col = 64 * c + 4 * tx;
                    if (col < D)
                        store4(make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]),
                               a.parts + row * D + col);
                }
                if (tx == 0) *reinterpret_cast<float2*>(a.part_stats + 2 * row) = make_float2(m[i], l[i]);
            }
        }
    }
    if (tid == 0) static_cast<PagedMeta*>(a.meta)[blockIdx.x] = meta;
}

// ---------------------------------------------------------------------------
// Joins the parts of items that several CTAs took: CTA (c, y) of this kernel
// takes rows 8·y.. of the item that CTA c began, a warp each.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

template <class T>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const PagedArgs a, int ctas) {
    await_previous();
    const PagedMeta* meta = static_cast<const PagedMeta*>(a.meta);
    const int c = blockIdx.x, lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
    const PagedMeta first = meta[c];
    if (!first.first_live || r >= first.rows) return;
    // The CTAs c + 1 .. c + count hold the rest.
    int count = 0;
    for (int at = c + 1; at < ctas; at += 32) {
        const int i = at + lane;
        const bool last = i >= ctas || !meta[i].later_live || meta[i].ends;
        const unsigned stop = __ballot_sync(kFullMask, last);
        if (stop) {
            count = min(at + __ffs(stop) - 1, ctas - 1) - c;
            break;
        }
    }
    if (!meta[c + count].later_live) return;  // not a message of this call: nothing to join
    const int D = a.head_dim;
    const auto row_of = [&](int i) { return (i == 0 ? 2LL * c + kPartFirst : 2LL * (c + i) + kPartLater) * a.part_rows + r; };
    const auto stat_of = [&](int i) { return *reinterpret_cast<const float2*>(a.part_stats + 2 * row_of(i)); };
    float top = -INFINITY;
    for (int i = lane; i <= count; i += 32) top = fmaxf(top, stat_of(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
    float sum = 0.f;
    float4 x[2] = {};
    for (int i = 0; i <= count; ++i) {
        const float2 st = stat_of(i);
        const float w = weight_of(st.x, top, a.scale_log2);
        sum = fmaf(st.y, w, sum);
        const float* part = a.parts + row_of(i) * D;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = 128 * j + 4 * lane;
            if (col < D && st.x != -INFINITY) {
                const float4 y = *reinterpret_cast<const float4*>(part + col);
                x[j].x = fmaf(y.x, w, x[j].x);
                x[j].y = fmaf(y.y, w, x[j].y);
                x[j].z = fmaf(y.z, w, x[j].z);
                x[j].w = fmaf(y.w, w, x[j].w);
            }
        }
    }
    const int flat = first.row0 + r, token = flat / a.group, head = first.head * a.group + flat - token * a.group;
    T* out = (T*)a.out + (first.start + token) * a.out_token + head * a.out_head;
    const float z = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = 128 * j + 4 * lane;
        if (col < D) store4(make_float4(x[j].x * z, x[j].y * z, x[j].z * z, x[j].w * z), out + col);
    }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
struct Shape {
    bool mma;
    int rows;  // of a block
    int ctas;
};
Shape shape_of(int head_dim, bool bf16) {
    if (bf16 && head_dim <= 128) return Shape{true, paged_mma_rows(), sm_count_current_device()};
    const int fit = std::max(1, std::min(4, 220 * 1024 / block_smem(head_dim)));
    return Shape{false, kBlockRows, fit * sm_count_current_device()};
}

int part_rows(int tokens, int q_heads, int kv_heads, int rows) {
    return (int)std::min<long long>(rows, (long long)tokens * (q_heads / kv_heads));
}

// bf16 heads of up to 128 columns go to the matrix kernel.
template <class T, int kWide>
int run_block(PagedArgs a, int ctas, cudaStream_t stream) {
    const auto kernel = paged_block_kernel<T, kWide>;
    const int smem = block_smem(a.head_dim);
    if (!allow_shared(kernel, smem)) return cuda_failure();
    kernel<<<ctas, kBlockThreads, smem, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

size_t meta_bytes(int ctas) { return ((size_t)ctas * sizeof(PagedMeta) + 15) / 16 * 16; }

}  // namespace

size_t paged_attention_workspace(int tokens, int q_heads, int kv_heads, int head_dim, bool bf16) {
    const Shape s = shape_of(head_dim, bf16);
    const size_t rows = (size_t)2 * s.ctas * part_rows(tokens, q_heads, kv_heads, s.rows);
    return meta_bytes(s.ctas) + rows * head_dim * 4 + rows * 8;
}

int launch_paged_attention(PagedArgs a, bool bf16, void* workspace, cudaStream_t stream) {
    const Shape s = shape_of(a.head_dim, bf16);
    a.part_rows = (int)std::min<long long>(s.rows, (long long)(a.q_offsets ? a.tokens : a.per_seq) * a.group);
    a.meta = workspace;
    a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + meta_bytes(s.ctas));
    a.part_stats = a.parts + (size_t)2 * s.ctas * a.part_rows * a.head_dim;
    int code;
    if (s.mma) code = launch_paged_mma(a, s.ctas, stream);
    else switch ((a.head_dim + 63) / 64) {
        case 1: code = bf16 ? run_block<__nv_bfloat16, 1>(a, s.ctas, stream) : run_block<float, 1>(a, s.ctas, stream); break;
        case 2: code = bf16 ? run_block<__nv_bfloat16, 2>(a, s.ctas, stream) : run_block<float, 2>(a, s.ctas, stream); break;
        case 3: code = bf16 ? run_block<__nv_bfloat16, 3>(a, s.ctas, stream) : run_block<float, 3>(a, s.ctas, stream); break;
        default: code = bf16 ? run_block<__nv_bfloat16, 4>(a, s.ctas, stream) : run_block<float, 4>(a, s.ctas, stream); break;
    }
    if (code != USM_OK) return code;
    // The join asks for the same split of an SM's memory as the kernel before it: to
    // change it the SM has to drain.
    if (!allow_shared(paged_join_kernel<__nv_bfloat16>, 0) || !allow_shared(paged_join_kernel<float>, 0)) return cuda_failure();
    const dim3 grid(s.ctas, (a.part_rows + kJoinWarps - 1) / kJoinWarps);
    if (bf16) return launch_next(paged_join_kernel<__nv_bfloat16>, grid, kJoinWarps * 32, 1, stream, a, s.ctas);
    return launch_next(paged_join_kernel<float>, grid, kJoinWarps * 32, 1, stream, a, s.ctas);
}

}  // namespace usm
