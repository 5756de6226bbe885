// Query blocks, positions and the relative position bias, as the
// sparse-attention kernels read them (include/usm.h, usm_rel_bias).
#pragma once

#include "usm_args.h"
#include "usm_device.cuh"

namespace usm {

// What a column of row r is measured from: d = column - shift is its relative
// position.  64 bits: the block's first column and the query position (both up
// to 2^31, q_offset any int) add up.
__device__ __forceinline__ long long rel_shift(const RelArgs& b, int block, int row_in_block, int first_col) {
    long long shift = row_in_block;
    if (b.q_offset) shift += __ldg(b.q_offset + block);
    if (b.seg_cols > 0) shift += (long long)(first_col / b.seg_cols) * b.seg_cols;
    return shift;
}

// Entry of the bucket map (and of tables laid out like it) for column col.
__device__ __forceinline__ int rel_entry(int col, long long shift, int reach) {
    const long long d = col - shift;
    return (int)min(max(d, -(long long)reach), (long long)reach) + reach;
}

__device__ __forceinline__ int rel_bucket(const RelArgs& b, int entry) {
    return min(max(__ldg(b.map + entry), 0), b.buckets - 1);
}

__device__ __forceinline__ float rel_table(const RelArgs& b, int head, int bucket) {
    const long long i = (long long)head * b.buckets + bucket;
    if (b.table_bf16) return __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(b.table) + i) << 16);
    return __ldg(static_cast<const float*>(b.table) + i);
}

// Entries [s, e) of row r, clamped into [0, nnz) whatever row_offsets holds.
__device__ __forceinline__ void row_range(const int* __restrict__ ro, int r, int nnz, int& s, int& e) {
    s = min(max(__ldg(ro + r), 0), nnz);
    e = min(max(__ldg(ro + r + 1), s), nnz);
}

}  // namespace usm
