// Appending keys and values to a paged cache with the rotation by position
// applied on the way, and the table of rotations.  Contracts: include/usm.h.
//
// A thread holds the rotation of one unit (two 16-byte chunks of a head's row:
// the two halves of eight or four pairs) in registers and walks over heads of
// its token with it, so the table is read once a token and not once a head, and
// queries, keys and values go through in one launch.  Bound: HBM, each element
// read and written once: 16384 tokens of 32 + 8 + 8 heads of 128 columns (405 MB) take
// 65 us, 6.2 TB/s; 32 tokens 2.6 us.
#include <cuda_bf16.h>

#include <algorithm>

#include "usm_internal.h"
#include "usm_paged.cuh"

namespace usm {
namespace {

__global__ void rope_table_kernel(int positions, int half, double exponent, float* __restrict__ table) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)positions * half) return;
    const int p = (int)(i / half), j = (int)(i - (long long)p * half);
    double s, c;
    sincos(p * exp2(exponent * j), &s, &c);
    table[(long long)p * 2 * half + j] = (float)c;
    table[(long long)p * 2 * half + half + j] = (float)s;
}

// Where a new token stands, and its slots in the cache (null: not stored).
struct Place {
    int position;
    bool known;  // belongs to a sequence
    long long k, v;  // offsets of its slot, elements; -1: none
};

__device__ Place place_of(const AppendArgs& a, int token) {
    Place w{0, false, -1, -1};
    int b;
    int start, n;
    if (a.q_offsets) {
        // The last sequence that begins at or before the token (those without
        // tokens share their successor's offset).
        int lo = 0, hi = a.num_seqs;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (a.q_offsets[mid] <= token) lo = mid + 1;
            else hi = mid;
        }
        b = lo - 1;
        if (b < 0) return w;
        start = max(a.q_offsets[b], 0);
        const int end = min(a.q_offsets[b + 1], a.tokens);
        if (token < start || token >= end) return w;
        n = end - start;
    } else {
        b = token / a.per_seq;
        start = b * a.per_seq;
        n = a.per_seq;
    }
    const int len = min(max(a.lengths[b], 0), kPagedMaxLength);
    w.known = true;
    w.position = len - n + (token - start);
    if (w.position < 0 || w.position >= a.capacity) return w;
    const int index = w.position / a.page_size;
    const int page = a.table[(long long)b * a.table_stride + index];
    if ((unsigned)page >= (unsigned)a.num_pages) return w;
    const int slot = w.position - index * a.page_size;
    w.k = page * a.kc_page + slot * a.kc_slot;
    w.v = page * a.vc_page + slot * a.vc_slot;
    return w;
}

template <class T>
struct Chunk;  // 16 bytes of a row
template <>
struct Chunk<float> {
    static constexpr int E = 4;
    __device__ static void widen(const uint4& w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    __device__ static uint4 narrow(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int E = 8;
    __device__ static void widen(const uint4& w, float (&x)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 narrow(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// Unit u of a row: chunks `first` and `second` (-1: none), and which are turned.
struct Unit {
    int first, second;
    bool turn_first, turn_second;  // halves: the two chunks turn together
};
template <int E>
__device__ __forceinline__ Unit unit_of(const AppendArgs& a, int u) {
    const int chunks = a.head_dim / E;
    Unit w;
    const int half = a.rot / 2 / E;
    if (!a.interleaved && u < half) {
        w.first = u;
        w.second = u + half;
        w.turn_first = w.turn_second = true;
        return w;
    }
    w.first = 2 * u;
    w.second = 2 * u + 1 < chunks ? 2 * u + 1 : -1;
    w.turn_first = a.interleaved && w.first * E < a.rot;
    w.turn_second = a.interleaved && w.second >= 0 && w.second * E < a.rot;
    return w;
}

constexpr int kAppendThreads = 256;
constexpr int kInFlight = 4;  // heads whose chunks are loaded before the first is turned

// One row's two chunks at a time, kInFlight rows in flight.
// blockDim: (units, heads walked side by side, tokens).
template <class T>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
    using C = Chunk<T>;
    constexpr int E = C::E;
    await_previous();
    let_next_start();
    const int u = threadIdx.x;
    const unsigned step = blockDim.y;
    const int token = blockIdx.x * blockDim.z + threadIdx.z;
    if (token >= a.tokens) return;
    const Unit w = unit_of<E>(a, u);
    const Place at = place_of(a, token);
    if (!at.known) return;

    float cos[E], sin[E];  // the unit's E pairs
    if (w.turn_first || w.turn_second) {
        const float* row = a.rope + (long long)min(max(at.position, 0), a.rope_positions - 1) * a.rot;
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (u * E + i < a.rot / 2) {
                c = *reinterpret_cast<const float4*>(row + u * E + i);
                s = *reinterpret_cast<const float4*>(row + a.rot / 2 + u * E + i);
            }
            cos[i] = c.x, cos[i + 1] = c.y, cos[i + 2] = c.z, cos[i + 3] = c.w;
            sin[i] = s.x, sin[i + 1] = s.y, sin[i + 2] = s.z, sin[i + 3] = s.w;
        }
    }

    // Heads in the order q, k, v; up to 2^31, so that the last steps pass it.
    const unsigned q_heads = a.q ? a.q_heads : 0, kv_heads = a.kv_heads, heads = q_heads + (at.k >= 0 ? 2 * kv_heads : 0);
    for (unsigned h0 = threadIdx.y; h0 < heads; h0 += kInFlight * step) {
        uint4 x[kInFlight], y[kInFlight];
        T* to[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const unsigned h = h0 + i * step;
            if (h < heads) {
                const T* from;
                if (h < q_heads) {
                    from = (const T*)a.q + token * a.q_token + h * a.q_head;
                    to[i] = (T*)a.q_out + token * a.q_out_token + h * a.q_out_head;
                } else if (h < q_heads + kv_heads) {
                    from = (const T*)a.k + token * a.k_token + (h - q_heads) * a.k_head;
                    to[i] = (T*)a.k_cache + at.k + (h - q_heads) * a.kc_head;
                } else {
                    from = (const T*)a.v + token * a.v_token + (h - q_heads - kv_heads) * a.v_head;
                    to[i] = (T*)a.v_cache + at.v + (h - q_heads - kv_heads) * a.vc_head;
                }
                x[i] = *reinterpret_cast<const uint4*>(from + w.first * E);
                if (w.second >= 0) y[i] = *reinterpret_cast<const uint4*>(from + w.second * E);
            }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const unsigned h = h0 + i * step;
            if (h >= heads) break;
            if (h < q_heads + kv_heads && (w.turn_first || w.turn_second)) {
                float p[E], r[E];
                C::widen(x[i], p);
                if (w.second >= 0) C::widen(y[i], r);
                if (!a.interleaved) {
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        const float x1 = p[j], x2 = r[j];
                        p[j] = x1 * cos[j] - x2 * sin[j];
                        r[j] = x2 * cos[j] + x1 * sin[j];
                    }
                    x[i] = C::narrow(p);
                    y[i] = C::narrow(r);
                } else {
#pragma unroll
                    for (int j = 0; j < E / 2; ++j) {
                        const float x1 = p[2 * j], x2 = p[2 * j + 1];
                        p[2 * j] = x1 * cos[j] - x2 * sin[j];
                        p[2 * j + 1] = x2 * cos[j] + x1 * sin[j];
                        const float z1 = r[2 * j], z2 = r[2 * j + 1];
                        r[2 * j] = z1 * cos[E / 2 + j] - z2 * sin[E / 2 + j];
                        r[2 * j + 1] = z2 * cos[E / 2 + j] + z1 * sin[E / 2 + j];
                    }
                    x[i] = C::narrow(p);
                    if (w.turn_second) y[i] = C::narrow(r);
                }
            }
            *reinterpret_cast<uint4*>(to[i] + w.first * E) = x[i];
            if (w.second >= 0) *reinterpret_cast<uint4*>(to[i] + w.second * E) = y[i];
        }
    }
}

// Rotations whose halves are not whole chunks: a thread turns one pair (or copies
// one element) of a row at a time.  Correct for every even rot.
template <class T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen(float x) {
    return x;
}
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 x) {
    return __bfloat162float(x);
}
__device__ __forceinline__ void narrow(float x, float* to) { *to = x; }
__device__ __forceinline__ void narrow(float x, __nv_bfloat16* to) { *to = __float2bfloat16_rn(x); }

template <class T>
__global__ void __launch_bounds__(kAppendThreads) append_pairs_kernel(const __grid_constant__ AppendArgs a) {
    await_previous();
    let_next_start();
    const int token = blockIdx.x;
    const Place at = place_of(a, token);
    if (!at.known) return;
    const int half = a.rot / 2, items = half + a.head_dim - a.rot;  // pairs, then single elements
    const int q_heads = a.q ? a.q_heads : 0, heads = q_heads + (at.k >= 0 ? 2 * a.kv_heads : 0);
    const float* row = a.rope + (long long)min(max(at.position, 0), a.rope_positions - 1) * a.rot;
    for (long long i = threadIdx.x; i < (long long)heads * items; i += blockDim.x) {
        const int h = (int)(i / items), j = (int)(i - (long long)h * items);
        const T* from;
        T* to;
        bool turn = true;
        if (h < q_heads) {
            from = (const T*)a.q + token * a.q_token + h * a.q_head;
            to = (T*)a.q_out + token * a.q_out_token + h * a.q_out_head;
        } else if (h < q_heads + a.kv_heads) {
            from = (const T*)a.k + token * a.k_token + (h - q_heads) * a.k_head;
            to = (T*)a.k_cache + at.k + (h - q_heads) * a.kc_head;
        } else {
            from = (const T*)a.v + token * a.v_token + (h - q_heads - a.kv_heads) * a.v_head;
            to = (T*)a.v_cache + at.v + (h - q_heads - a.kv_heads) * a.vc_head;
            turn = false;
        }
        if (j >= half) {
            to[half + j] = from[half + j];
            continue;
        }
        const int j1 = a.interleaved ? 2 * j : j, j2 = a.interleaved ? 2 * j + 1 : j + half;
        const T t1 = from[j1], t2 = from[j2];
        if (!turn) {
            to[j1] = t1;
            to[j2] = t2;
            continue;
        }
        const float c = row[j], s = row[half + j], x1 = widen(t1), x2 = widen(t2);
        narrow(x1 * c - x2 * s, to + j1);
        narrow(x2 * c + x1 * s, to + j2);
    }
}

template <class T>
int append(const AppendArgs& a, cudaStream_t stream) {
    constexpr int E = Chunk<T>::E;
    const int heads = a.q_heads + 2 * a.kv_heads;
    // Whole chunks turn where a pair's halves lie in two of them, or in one; the
    // table's rows are read by 16 bytes.
    const bool whole = a.rot == 0 || (a.interleaved ? a.rot % E == 0 && a.rot % 8 == 0 : a.rot % (2 * E) == 0);
    if (!whole) {
        return launch_next_shared(append_pairs_kernel<T>, dim3(a.tokens), kAppendThreads, 0, stream, a);
    }
    const int units = (a.head_dim / E + 1) / 2;  // at most 32
    // Heads side by side: few tokens are spread over more threads.
    int side = 1;
    while (side < 32 && side * units < kAppendThreads && side < heads &&
           (long long)a.tokens * units * side < 4LL * 2048 * sm_count_current_device() / kInFlight)
        side *= 2;
    while (side * units > kAppendThreads) side /= 2;
    const int tokens = std::max(1, std::min(64, kAppendThreads / (side * units)));
    const unsigned grid = (unsigned)(((long long)a.tokens + tokens - 1) / tokens);
    return launch_next_shared(append_kernel<T>, dim3(grid), dim3(units, side, tokens), 0, stream, a);
}

}  // namespace

int launch_rope_table(int positions, int rot, double base, float* table, cudaStream_t stream) {
    const long long n = (long long)positions * (rot / 2);
    rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(positions, rot / 2, -2.0 * log2(base) / rot, table);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

int launch_paged_append(const AppendArgs& a, bool bf16, cudaStream_t stream) {
    return bf16 ? append<__nv_bfloat16>(a, stream) : append<float>(a, stream);
}

}  // namespace usm
