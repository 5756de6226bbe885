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

constexpr int kPagedMaxSeqs = 1 << 30;    // sequences of a call (walks over them step past the last, searches add two)
constexpr int kPagedMaxLength = 1 << 30;  // tokens of a sequence (positions and their differences stay in 32 bits)

// Attention of new tokens over a paged cache, as usm_paged_cache lays it out.
struct PagedArgs {
    const void *q, *k, *v;
    void* out;
    long long q_token, q_head, out_token, out_head;  // strides, elements
    long long k_page, k_slot, k_head, v_page, v_slot, v_head;
    const int* table;
    const int* lengths;
    const int* q_offsets;  // may be null: per_seq tokens each
    int table_stride, num_pages, page_size;
    int capacity;          // positions that the table has room for
    int num_seqs, tokens, per_seq;
    int kv_heads, group, head_dim;
    uint32_t group_mul;    // x / group = x·group_mul >> group_shift for 0 <= x < 2^31
    int group_shift;
    float scale_log2;      // scale·log2 e
    int causal, window;
    int table_pages;       // entries of a sequence's row of the table
    int out32;             // rows of the output are 32-byte aligned and that much at least
    int boxes;             // keys and values come by TMA, a box of a page's slots at a time
    int least_rows, most_rows;  // rows (tokens·group) of the sequences that the launch takes
    int part_rows;         // rows of a partial result
    float* parts;          // [2·ctas][head_dim / 4][part_rows][4], then [2·ctas][part_rows][2]
    float* part_stats;     // (reference, sum) of each row
    void* meta;            // PagedMeta[ctas]
    int* status;
};

struct AppendArgs {
    const void *k, *v, *q;  // q: null for none
    void *k_cache, *v_cache, *q_out;
    long long k_token, k_head, v_token, v_head, q_token, q_head, q_out_token, q_out_head;
    long long kc_page, kc_slot, kc_head, vc_page, vc_slot, vc_head;
    const int* table;
    const int* lengths;
    const int* q_offsets;
    int table_stride, num_pages, page_size, capacity;
    int num_seqs, tokens, per_seq;
    int kv_heads, q_heads, head_dim;
    const float* rope;
    int rope_positions, rot, interleaved;
};

}  // namespace usm
