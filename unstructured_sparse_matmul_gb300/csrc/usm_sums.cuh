// Sums of many terms in two fp32 numbers: hi + lo, lo the sum of what rounding
// took from hi at each addition (the error of an addition is an fp32 number
// itself; Knuth, The Art of Computer Programming, vol. 2, 4.2.2).  n terms are off
// by about n·2^-48 of their absolute sum instead of n·2^-24.  An addition takes 7
// fp32 instructions; additions in 64 bits run at about 1/60 of their rate here.
#pragma once

#include "usm_device.cuh"

namespace usm {

struct LongSum {
    float hi = 0.f, lo = 0.f;

    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    __device__ __forceinline__ void add(const LongSum& other) {
        add(other.hi);
        lo += other.lo;
    }
    // Infinite and NaN sums stay as plain additions leave them (lo is NaN then).
    __device__ __forceinline__ float value() const { return lo == lo ? hi + lo : hi; }
    // Sum over the warp's lanes, in lane 0.
    __device__ __forceinline__ LongSum over_warp() const {
        LongSum x = *this;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            LongSum y;
            y.hi = __shfl_xor_sync(kFullMask, x.hi, o);
            y.lo = __shfl_xor_sync(kFullMask, x.lo, o);
            x.add(y);
        }
        return x;
    }
};

}  // namespace usm
