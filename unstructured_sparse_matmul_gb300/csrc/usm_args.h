// Arguments the kernels receive by value (plain data, shared by the host
// launch code and the device code).
#pragma once

#include <stdint.h>

namespace usm {

struct SpmmArgs {
    int M, K, N, nnz;
    const int* row_offsets;
    const int* col_indices;
    const void* values;
    const int* perm;  // may be null (identity order)
    int seg_rows;     // rows per diagonal block of the schedule (> 0)
    float* C;
    long long ldc;
    int* status;
    int tiles_per_block = 0;  // row tiles per diagonal block (set by the launcher)
};

struct SddmmArgs {
    int M, K, D, nnz;
    const int* row_offsets;
    const int* col_indices;
    const int* perm;
    int seg_rows;
    const void* X;
    long long ldx;
    void* out;           // final output (single strip) or fp32 partials (several strips)
    long long out_stride;  // elements between strips of partials
    int out_bf16;        // final output element type is bf16
    int rows_per_warp;
    int* status;
    const void* scale;   // null, or the mask's values: out[p] is multiplied by scale[p]
    int scale_bf16;      // scale elements are bf16 (else fp32)
    int tiles_per_block = 0;  // row tiles per diagonal block (set by the launcher)
};

// A relative position bias (usm_rel_bias) and the query blocks it applies to.
struct RelArgs {
    const void* table;  // null: no bias
    int table_bf16;
    int heads, buckets;
    const int* map;
    int reach;            // max_distance
    int seg_cols;         // <= 0: one key block
    const int* q_offset;  // may be null
    int seg_rows;         // > 0
};

// Softmax maps over CSR rows and their gradients.  s2, lambda: null with one map.
struct MapArgs {
    int M, nnz;
    const int* row_offsets;
    const float* s1;
    const float* s2;
    const float* lambda;
    int heads, seg_rows;  // > 0
    const void* dout;     // gradients only
    int dout_bf16;
    void* out1;           // the map, or the gradient of s1
    void* out2;           // the gradient of s2
    int out_bf16;
    float* row_c2;        // gradients with two maps: c2 of each row, or null
};

struct AttnArgs {
    int M, K, D, N, nnz;
    const int* row_offsets;
    const int* col_indices;
    const void *Q, *Km, *Q2, *K2, *V;  // Q2, K2: null with one map
    long long ldq, ldk, ldq2, ldk2, ldv;
    float scale;
    const float* lambda;
    int heads, seg_rows;
    RelArgs bias;
    float* C;
    long long ldc;
};

}  // namespace usm
