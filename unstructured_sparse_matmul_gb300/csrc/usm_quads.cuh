// Rows of CSR value arrays read and written four entries at a time.  A row
// [p0, p1) starts anywhere, so its quads are those of the whole array (entries
// 4q .. 4q+3) that meet the row: a quad at either end holds entries of its
// neighbours too, which are masked after the load and never written.
#pragma once

#include "usm_device.cuh"

namespace usm {

// Entries q .. q+3 of an array of nnz (those past the end read as 0).  VEC:
// the array starts on a 16-byte (fp32) or 8-byte (bf16) boundary.  Plain
// loads: the array may be written in place by the same kernel.
template <bool BF, bool VEC>
__device__ __forceinline__ void load_quad(const void* p, unsigned q, unsigned nnz, float (&x)[4]) {
    if (VEC && q + 4 <= nnz) {
        if constexpr (BF) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + q);
            x[0] = __uint_as_float(w.x << 16);
            x[1] = __uint_as_float(w.x & 0xffff0000u);
            x[2] = __uint_as_float(w.y << 16);
            x[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + q);
            x[0] = w.x;
            x[1] = w.y;
            x[2] = w.z;
            x[3] = w.w;
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        x[u] = 0.f;
        if (q + u < nnz) {
            if constexpr (BF)
                x[u] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[q + u] << 16);
            else
                x[u] = static_cast<const float*>(p)[q + u];
        }
    }
}

// Writes the entries of quad q that lie in [p0, p1); bf16 rounds to nearest even.
template <bool BF, bool VEC>
__device__ __forceinline__ void store_quad(void* p, unsigned q, unsigned p0, unsigned p1, const float (&x)[4]) {
    if (VEC && q >= p0 && q + 4 <= p1) {
        if constexpr (BF) {
            uint2 w;
            w.x = f32_to_bf16_rne(x[0]) | ((uint32_t)f32_to_bf16_rne(x[1]) << 16);
            w.y = f32_to_bf16_rne(x[2]) | ((uint32_t)f32_to_bf16_rne(x[3]) << 16);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + q) = w;
        } else {
            *reinterpret_cast<float4*>(static_cast<float*>(p) + q) = make_float4(x[0], x[1], x[2], x[3]);
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (q + u >= p0 && q + u < p1) {
            if constexpr (BF)
                static_cast<uint16_t*>(p)[q + u] = f32_to_bf16_rne(x[u]);
            else
                static_cast<float*>(p)[q + u] = x[u];
        }
    }
}

// Whether an array can be read and written in quads.
inline bool quad_aligned(const void* p, bool bf16) { return (reinterpret_cast<uintptr_t>(p) & (bf16 ? 7u : 15u)) == 0; }

}  // namespace usm
