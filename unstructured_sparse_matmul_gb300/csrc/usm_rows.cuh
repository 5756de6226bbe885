// A run of up to kRun CSR rows that a CTA shares out to its warps: their
// extents, and a counter the warps fetch row after row from.
#pragma once

#include "usm_device.cuh"
#include "usm_rel.cuh"

namespace usm {

constexpr int kRun = 64;

struct RowRun {
    int begin[kRun], end[kRun];
    int next;

    // Loads rows row_of(0) .. row_of(n - 1) (-1: none) and starts the counter; true
    // if one has over long_at entries.  `more(i, row)` runs in row i's thread.  A
    // barrier: every thread of the CTA calls it, after every warp is done with
    // the previous run.
    template <class RowOf, class More>
    __device__ __forceinline__ bool load(const int* __restrict__ ro, int nnz, int n, unsigned long_at, RowOf row_of,
                                         More more) {
        bool is_long = false;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int r = row_of(i);
            int p0 = 0, p1 = 0;
            if (r >= 0) row_range(ro, r, nnz, p0, p1);
            begin[i] = p0;
            end[i] = p1;
            is_long = is_long || (unsigned)(p1 - p0) > long_at;
            if (r >= 0) more(i, r);
        }
        if (threadIdx.x == 0) next = 0;
        return __syncthreads_or(is_long);
    }
    // The warp's next row of the run (the run's size or more: none is left).
    __device__ __forceinline__ int fetch(int lane) {
        int i = 0;
        if (lane == 0) i = atomicAdd(&next, 1);
        return __shfl_sync(kFullMask, i, 0);
    }
};

}  // namespace usm
