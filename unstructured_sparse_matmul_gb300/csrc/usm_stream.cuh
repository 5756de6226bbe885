// CSR value arrays streamed through shared memory, a warp at a time.
//
// A warp works on consecutive rows, whose entries are consecutive too: what it
// reads of every array is one run.  It has a ring of kRing entries in shared
// memory for each array (entry p lies at p mod kRing) that asynchronous copies
// fill kChunk entries at a time, up to a ring ahead of the row it works on: the
// copies do not wait for the row's arithmetic, nor for where rows begin and end.
#pragma once

#include "usm_device.cuh"
#include "usm_rel.cuh"

namespace usm {

constexpr int kChunk = 512, kRing = 4 * kChunk;
// Whether entries [p0, p1), one at least, fit the ring together: up to 1537 of them
// do wherever they start, up to 2048 at the start of a chunk.
__device__ __forceinline__ bool ring_holds(int p0, int p1) {
    return (unsigned)(p1 - 1) / kChunk - (unsigned)p0 / kChunk < kRing / kChunk;
}

// Streams up to three arrays of E0, E1, E2 bytes an element (0: none).
template <int E0, int E1, int E2>
struct Stream {
    static constexpr int kBytes = kRing * (E0 + E1 + E2);  // shared memory a warp
    const unsigned char* src[3];
    uint32_t base;  // shared address of the warp's rings
    int nnz, lane;
    bool aligned;   // every array starts on 16 bytes
    int whole;      // chunks before this one are whole (none, if not aligned)
    int issued;     // chunks before this one are copied or in flight
    int limit;      // chunks from this one on are not needed

    __device__ __forceinline__ uint32_t at(int array, uint32_t p) const {
        const uint32_t i = p & (kRing - 1);
        return array == 0 ? base + i * E0 : array == 1 ? base + kRing * E0 + i * E1 : base + kRing * (E0 + E1) + i * E2;
    }

    // Chunk `chunk` of one array: whole, or (EDGE) where the array may end inside
    // it or starts off 16 bytes.
    template <int E, bool EDGE>
    __device__ __forceinline__ void copy(int array, int chunk) const {
        if constexpr (E > 0) {
            constexpr int PER = 16 / E;  // entries a copy
            const uint32_t p0 = (uint32_t)chunk * kChunk + lane * PER, to = at(array, p0);
            const unsigned char* from = src[array] + (unsigned long long)p0 * E;
#pragma unroll
            for (int i = 0; i < kChunk / PER / 32; ++i) {
                if constexpr (!EDGE) {
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to + i * 512), "l"(from + i * 512)
                                 : "memory");
                } else {
                    const long long left = ((long long)nnz - p0 - i * 32 * PER) * E;
                    const int bytes = (int)min(max(left, 0LL), 16LL);  // past the end: zeros, unread
                    if (aligned) {
                        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to + i * 512),
                                     "l"(from + i * 512), "r"(bytes)
                                     : "memory");
                    } else {
                        for (int u = 0; u < bytes; u += E) {
                            if constexpr (E == 4)
                                asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + i * 512 + u),
                                             "r"(*reinterpret_cast<const uint32_t*>(from + i * 512 + u))
                                             : "memory");
                            else
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + i * 512 + u),
                                             "h"(*reinterpret_cast<const uint16_t*>(from + i * 512 + u))
                                             : "memory");
                        }
                    }
                }
            }
        }
    }
    __device__ __noinline__ void copy_edge(int chunk) const {
        copy<E0, true>(0, chunk);
        copy<E1, true>(1, chunk);
        copy<E2, true>(2, chunk);
    }
    // The next chunk (an empty set of copies past the limit).
    __device__ __forceinline__ void issue() {
        if (issued < limit) {
            if (issued < whole) {
                copy<E0, false>(0, issued);
                copy<E1, false>(1, issued);
                copy<E2, false>(2, issued);
            } else {
                copy_edge(issued);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++issued;
    }
    // Starts at entry p, with a full ring ahead of it.
    __device__ __forceinline__ void seek(int p) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        issued = p / kChunk;
#pragma unroll 1
        for (int i = 0; i < kRing / kChunk; ++i) issue();
    }
    // Moves the limit up; chunks that the old one kept out are still to be copied.
    __device__ __forceinline__ void extend(int new_limit) {
        issued = min(issued, limit);
        limit = new_limit;
    }
    // Makes entries [p0, p1) (one at least, no more than fit) readable by every
    // lane; runs come in order, and the ring before p0 is given up.
    __device__ __forceinline__ void need(int p0, int p1) {
        const int c0 = p0 / kChunk;
        if (c0 >= issued || c0 + kRing / kChunk < issued) seek(p0);  // rows were left out
        if (c0 + kRing / kChunk > issued) {
            __syncwarp();  // every lane is done with what is overwritten
            do issue();
            while (c0 + kRing / kChunk > issued);
        }
        const int left = issued - 1 - (p1 - 1) / kChunk;
        if (left == 0)
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (left == 1)
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        else if (left == 2)
            asm volatile("cp.async.wait_group 2;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 3;" ::: "memory");
        __syncwarp();
    }
};

__device__ __forceinline__ float lds_f32(uint32_t at) { return __uint_as_float(lds32(at)); }
// Four entries (4q .. 4q + 3) or one, widened.
template <bool BF>
__device__ __forceinline__ void lds_quad(uint32_t at, float2& lo, float2& hi) {
    if constexpr (BF) {
        const uint2 w = lds64(at);
        lo = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        hi = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    } else {
        const uint4 w = lds128(at);
        lo = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        hi = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
}
template <bool BF>
__device__ __forceinline__ float lds_entry(uint32_t at) {
    return BF ? __uint_as_float((uint32_t)lds16(at) << 16) : lds_f32(at);
}
__device__ __forceinline__ void sts_quad(uint32_t at, float2 lo, float2 hi) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(lo.x), "f"(lo.y), "f"(hi.x), "f"(hi.y) : "memory");
}
// Entries p .. p + 3 (p a multiple of 4) of a global array, whole quads; vec: it
// starts on 16 (bf16: 8) bytes.  bf16 rounds to nearest even.
template <bool BF>
__device__ __forceinline__ void store_quad(void* p, long long i, float2 lo, float2 hi, bool vec) {
    if constexpr (BF) {
        uint16_t* q = static_cast<uint16_t*>(p) + i;
        uint32_t a, b;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(lo.y), "f"(lo.x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(hi.y), "f"(hi.x));
        if (vec) {
            *reinterpret_cast<uint2*>(q) = make_uint2(a, b);
        } else {
            q[0] = (uint16_t)a;
            q[1] = (uint16_t)(a >> 16);
            q[2] = (uint16_t)b;
            q[3] = (uint16_t)(b >> 16);
        }
    } else {
        float* q = static_cast<float*>(p) + i;
        if (vec) {
            *reinterpret_cast<float4*>(q) = make_float4(lo.x, lo.y, hi.x, hi.y);
        } else {
            q[0] = lo.x;
            q[1] = lo.y;
            q[2] = hi.x;
            q[3] = hi.y;
        }
    }
}
template <bool BF>
__device__ __forceinline__ float load_global(const void* p, long long i) {
    if constexpr (BF) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
    return static_cast<const float*>(p)[i];
}
template <bool BF>
__device__ __forceinline__ void store_entry(void* p, long long i, float v) {
    if constexpr (BF)
        static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v);
    else
        static_cast<float*>(p)[i] = v;
}

// How a row [p0, p1) lies in quads: whole ones [qs, qe), and up to three entries
// on either side, one each for lanes 0-2 (head) and 4-6 (tail).
struct RowQuads {
    unsigned qs, qe, edge;
    bool has_edge;
    __device__ __forceinline__ RowQuads(unsigned p0, unsigned p1, int lane) {
        qs = (p0 + 3u) & ~3u;
        qe = p1 & ~3u;
        const unsigned head = min(qs, p1) - p0, tail_at = max(qe, qs), tail = p1 > tail_at ? p1 - tail_at : 0u;
        edge = lane < 4 ? p0 + lane : tail_at + lane - 4;
        has_edge = lane < 4 ? (unsigned)lane < head : (unsigned)lane - 4u < tail;
    }
};

// First rows r0 and r1 whose offset is at least t0 and t1 (in [0, M]), by 32
// candidates a round, both at once.
__device__ __forceinline__ void first_rows_from(const int* __restrict__ ro, int M, int t0, int t1, int lane, int& r0,
                                                int& r1) {
    int lo[2] = {0, 0}, hi[2] = {M, M};  // offsets before lo are below the target, hi's is not (or hi is M)
    const int target[2] = {t0, t1};
    while (lo[0] < hi[0] || lo[1] < hi[1]) {
        int step[2], v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            step[k] = (int)(((unsigned)(hi[k] - lo[k]) + 31u) / 32u);
            v[k] = __ldg(ro + min((long long)lo[k] + (long long)lane * step[k], (long long)M));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool candidate = (long long)lo[k] + (long long)lane * step[k] < hi[k];
            const unsigned below = __ballot_sync(kFullMask, candidate && v[k] < target[k]);
            if (below == 0) {
                hi[k] = lo[k];
            } else {
                const int last = lo[k] + (31 - __clz(below)) * step[k];
                hi[k] = (int)min((long long)hi[k], (long long)last + step[k]);
                lo[k] = last + 1;
            }
        }
    }
    r0 = lo[0];
    r1 = lo[1];
}

// Lanes hold 32 consecutive row offsets, read off them one by one.  M may be as
// large as 2^31 - 1: no row number past M is formed.
struct RowWalk {
    const int* ro;
    int M, nnz, lane, at, held;  // held: offset of row at + lane
    // Offsets of rows r .. r + n (n < 32) can be read.
    __device__ __forceinline__ void hold(int r, int n) {
        if ((unsigned)r - (unsigned)at > (unsigned)(31 - n)) {
            at = r;
            held = min(max(__ldg(ro + min((long long)r + lane, (long long)M)), 0), nnz);
        }
    }
    // Offset of row r + ahead (the last one's past M).
    __device__ __forceinline__ int offset(int r, int ahead = 0) const { return __shfl_sync(kFullMask, held, r - at + ahead); }
    // The first row from r on (r < r1) that has entries, or r1.  Runs of rows
    // without any are passed by a search.
    __device__ __forceinline__ int with_entries(int r, int r1) {
        while (true) {
            hold(r, 1);
            const int next = __shfl_down_sync(kFullMask, held, 1);
            const unsigned some = __ballot_sync(kFullMask, lane < 31 && lane >= r - at && next > held);
            if (some) return min(at + __ffs(some) - 1, r1);
            const int p = offset(at, 31);
            if (r1 - at <= 31 || p >= nnz) return r1;
            r = at + 31;
            hold(r, 31);
            if (offset(r, 31) > p) continue;
            if (r1 - r <= 31) return r1;
            int after, same;
            first_rows_from(ro, M, p + 1, p + 1, lane, after, same);
            r = max(after - 1, r + 31);
            if (r >= r1) return r1;
        }
    }
    // Whether one of rows r0 .. r1 - 1 does not fit the ring.
    __device__ __forceinline__ bool any_over(int r0, int r1) {
        bool over = false;
        for (int r = with_entries(r0, r1); r < r1;) {
            hold(r, 31);
            const int next = __shfl_down_sync(kFullMask, held, 1);
            over = over || (lane < min(31, r1 - at) && next > held && !ring_holds(held, next));
            if (r1 - at <= 31) break;
            r = with_entries(at + 31, r1);
        }
        return over;
    }
};

// Share g of G of nnz entries.
__device__ __forceinline__ int share_begin(int nnz, int g, int G) { return (int)((long long)nnz * g / G); }

inline bool aligned_for_stream(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace usm
