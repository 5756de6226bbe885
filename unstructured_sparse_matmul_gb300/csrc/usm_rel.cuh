// Query blocks, positions and the relative position bias, as the
// sparse-attention kernels read them (include/usm.h, usm_rel_bias).
#pragma once

#include "usm_args.h"
#include "usm_device.cuh"

namespace usm {

// The column at which row r's part of the bucket map starts: column col reads
// entry clamp(col - start, 0, 2·reach), since its relative position is col less
// the row's key block's first column and its query position.  Those can add up
// past 32 bits (and q_offset may be negative); a start outside [-2^30, 2^31)
// gives every column the same entry as the nearest start inside does.
__device__ __forceinline__ int rel_start(const RelArgs& b, int block, int row_in_block, int first_col) {
    long long start = (long long)row_in_block - b.reach;
    if (b.q_offset) start += __ldg(b.q_offset + block);
    if (b.seg_cols > 0) start += (long long)(first_col / b.seg_cols) * b.seg_cols;
    return (int)min(max(start, -(1LL << 30)), 0x7fffffffLL);
}

__device__ __forceinline__ int rel_entry(int col, int start, int reach) {
    return col < start ? 0 : (int)min((unsigned)col - (unsigned)start, 2u * (unsigned)reach);
}

__device__ __forceinline__ int rel_bucket(const RelArgs& b, int entry) {
    return min(max(__ldg(b.map + entry), 0), b.buckets - 1);
}

// Entry `bucket` of a head's row of the table.
template <bool BF>
__device__ __forceinline__ float rel_table_entry(const void* row, int bucket) {
    if constexpr (BF)
        return __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(row) + bucket) << 16);
    return __ldg(static_cast<const float*>(row) + bucket);
}
__device__ __forceinline__ float rel_table(const RelArgs& b, int head, int bucket) {
    const char* row = static_cast<const char*>(b.table) + (long long)head * b.buckets * (b.table_bf16 ? 2 : 4);
    return b.table_bf16 ? rel_table_entry<true>(row, bucket) : rel_table_entry<false>(row, bucket);
}

// Entries [s, e) of row r, clamped into [0, nnz) whatever row_offsets holds.
__device__ __forceinline__ void row_range(const int* __restrict__ ro, int r, int nnz, int& s, int& e) {
    s = min(max(__ldg(ro + r), 0), nnz);
    e = min(max(__ldg(ro + r + 1), s), nnz);
}

}  // namespace usm
