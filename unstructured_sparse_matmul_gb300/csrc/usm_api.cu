// C ABI of the library: argument checks, dispatch, status word, tensor maps.
// The declarations and their contracts are in include/usm.h.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "usm_device.cuh"
#include "usm_internal.h"

namespace usm {

// One status word per device (a __device__ variable exists once in every
// device context that loads this module).
__device__ int g_status_word;

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];
std::once_flag g_encode_once;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_ctx_once;
PFN_cuCtxGetCurrent_v4000 g_ctx_get_current = nullptr;
PFN_cuCtxGetId_v12000 g_ctx_get_id = nullptr;
std::mutex g_symbol_mutex;

void* driver_entry(const char* name, unsigned version) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion(name, &fn, version, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        return fn;
    return nullptr;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

__global__ void wait_timeout_selftest_kernel(long long limit_ns, int* status) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&bar), 1);
        fence_barrier_init();
    }
    __syncthreads();
    // Nothing ever arrives on this barrier: the wait must give up by itself.
    if (threadIdx.x == 0 && !mbar_wait_bounded(smem_addr(&bar), 0, (unsigned long long)limit_ns))
        record_status(status, USM_ERR_TIMEOUT);
}

}  // namespace

unsigned long long current_context_id() {
    std::call_once(g_ctx_once, [] {
        g_ctx_get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(driver_entry("cuCtxGetCurrent", 4000));
        g_ctx_get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(driver_entry("cuCtxGetId", 12000));
    });
    if (!g_ctx_get_current || !g_ctx_get_id) return 0;
    CUcontext ctx = nullptr;
    if (g_ctx_get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
    unsigned long long id = 0;
    if (g_ctx_get_id(ctx, &id) != CUDA_SUCCESS) return 0;
    return id;
}

void* SymbolAddressCache::get() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(g_symbol_mutex);
    const unsigned long long ctx = current_context_id();
    if (ctx != 0 && ctx == ctx_[dev] && addr_[dev] != nullptr) return addr_[dev];
    // First use in this context (or no context current yet): the lookup
    // makes the device's primary context current and may load the module.
    void* addr = nullptr;
    if (cudaGetSymbolAddress(&addr, symbol_) != cudaSuccess || addr == nullptr) return nullptr;
    ctx_[dev] = current_context_id();
    addr_[dev] = addr;
    return addr;
}

namespace {
SymbolAddressCache g_status_cache(&g_status_word);
}  // namespace

int* status_word_for_current_device() { return static_cast<int*>(g_status_cache.get()); }

int sm_count_current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    int n = g_sm_count[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 148;
    g_sm_count[dev].store(n, std::memory_order_relaxed);
    return n;
}

namespace {
bool find_encode() {
    std::call_once(g_encode_once, [] {
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(driver_entry("cuTensorMapEncodeTiled", 12000));
    });
    return g_encode != nullptr;
}
}  // namespace

bool encode_tensor_map_4d_bf16(CUtensorMap* map, const void* base, const int (&extents)[4], const long long (&strides)[3],
                               const int (&box)[4]) {
    if (!find_encode()) return false;
    cuuint64_t dims[4], bytes[3];
    cuuint32_t boxes[4];
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) dims[i] = (cuuint64_t)extents[i], boxes[i] = (cuuint32_t)box[i];
    // A dimension of one is never stepped over, but its stride has to be a valid one.
    for (int i = 0; i < 3; ++i) bytes[i] = extents[i + 1] > 1 ? (cuuint64_t)strides[i] * 2 : (cuuint64_t)extents[0] * 2;
    return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, bytes, boxes, unit,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tensor_map_2d(CUtensorMap* map, const void* base, bool bf16, long long rows,
                          long long cols, long long ld_elems, int box_cols, int box_rows) {
    if (!find_encode()) return false;
    const int es = bf16 ? 2 : 4;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld_elems * es)};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

int launch_wait_timeout_selftest(long long limit_ns, int* status, cudaStream_t stream) {
    wait_timeout_selftest_kernel<<<1, 32, 0, stream>>>(limit_ns, status);
    return cudaGetLastError() == cudaSuccess ? USM_OK : USM_ERR_CUDA;
}

}  // namespace usm

using namespace usm;

namespace {
std::atomic<int> g_override_rows{0}, g_override_tiles{0}, g_override_splits{0};
}  // namespace

namespace usm {
ScheduleOverride schedule_override() {
    return {g_override_rows.load(std::memory_order_relaxed), g_override_tiles.load(std::memory_order_relaxed),
            g_override_splits.load(std::memory_order_relaxed)};
}
}  // namespace usm

extern "C" {

int csr_spmm(int M, int K, int N, int nnz, const int* row_offsets, const int* col_indices,
             const void* values, const int* row_swizzle, int seg_rows, const void* B, int ldb, float* C,
             int ldc, usm_dtype dtype, void* stream) {
    if (M < 0 || K < 0 || N < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    if (dtype != USM_F32 && dtype != USM_BF16) return USM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return USM_OK;
    if (ldc < N) return USM_ERR_INVALID_ARG;
    if (!C || !row_offsets) return USM_ERR_INVALID_ARG;
    if (!aligned16(C) || (ldc % 4) != 0) return USM_ERR_ALIGNMENT;
    if (nnz > 0 && K == 0) return USM_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (nnz == 0) return launch_fill_f32(C, M, N, ldc, st);
    if (!col_indices || !values || !B) return USM_ERR_INVALID_ARG;
    if (ldb < N) return USM_ERR_INVALID_ARG;
    const int es = dtype == USM_BF16 ? 2 : 4;
    if (!aligned16(B) || ((long long)ldb * es) % 16 != 0) return USM_ERR_ALIGNMENT;
    int* status = status_word_for_current_device();
    if (!status) return USM_ERR_CUDA;
    SpmmArgs a{M, K, N, nnz, row_offsets, col_indices, values, row_swizzle, effective_seg(M, seg_rows), C, ldc,
               status};
    return launch_spmm(a, B, ldb, dtype == USM_BF16, st);
}

int csr_spmm_row_softmax(int M, int K, int N, int nnz, const int* row_offsets, const int* col_indices,
                         const float* scores, const int* row_swizzle, int seg_rows, const void* B, int ldb, float* C,
                         int ldc, usm_dtype dtype, void* stream) {
    if (M < 0 || K < 0 || N < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    if (dtype != USM_F32 && dtype != USM_BF16) return USM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return USM_OK;
    if (ldc < N) return USM_ERR_INVALID_ARG;
    if (!C || !row_offsets) return USM_ERR_INVALID_ARG;
    if (!aligned16(C) || (ldc % 4) != 0) return USM_ERR_ALIGNMENT;
    if (nnz > 0 && K == 0) return USM_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (nnz == 0) return launch_fill_f32(C, M, N, ldc, st);
    if (!col_indices || !scores || !B) return USM_ERR_INVALID_ARG;
    if (ldb < N) return USM_ERR_INVALID_ARG;
    const int es = dtype == USM_BF16 ? 2 : 4;
    if (!aligned16(B) || ((long long)ldb * es) % 16 != 0) return USM_ERR_ALIGNMENT;
    int* status = status_word_for_current_device();
    if (!status) return USM_ERR_CUDA;
    SpmmArgs a{M, K, N, nnz, row_offsets, col_indices, scores, row_swizzle, effective_seg(M, seg_rows), C, ldc,
               status};
    return launch_spmm(a, B, ldb, dtype == USM_BF16, st, true);
}

size_t csr_sddmm_workspace_bytes(int M, int K, int D, int nnz, usm_dtype in_dtype) {
    if (M <= 0 || K < 0 || D <= 0 || nnz <= 0) return 0;
    return sddmm_workspace_bytes(M, K, D, nnz, in_dtype == USM_BF16);
}

int csr_sddmm(int M, int K, int D, int nnz, const int* row_offsets, const int* col_indices,
              const int* row_swizzle, int seg_rows, const void* X, int ldx, const void* Y, int ldy, void* out,
              usm_dtype in_dtype, usm_dtype out_dtype, void* workspace, size_t workspace_bytes,
              void* stream) {
    if (M < 0 || K < 0 || D < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    if ((in_dtype != USM_F32 && in_dtype != USM_BF16) || (out_dtype != USM_F32 && out_dtype != USM_BF16))
        return USM_ERR_INVALID_ARG;
    if (M == 0 || nnz == 0) return USM_OK;
    if (!out || !row_offsets || !col_indices) return USM_ERR_INVALID_ARG;
    if (K == 0) return USM_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (D == 0) return launch_fill_out(out, nnz, out_dtype == USM_BF16, st);
    if (!X || !Y || ldx < D || ldy < D) return USM_ERR_INVALID_ARG;
    const int es = in_dtype == USM_BF16 ? 2 : 4;
    if (!aligned16(X) || !aligned16(Y) || ((long long)ldx * es) % 16 != 0 ||
        ((long long)ldy * es) % 16 != 0)
        return USM_ERR_ALIGNMENT;
    const size_t need = sddmm_workspace_bytes(M, K, D, nnz, in_dtype == USM_BF16);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return USM_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return USM_ERR_ALIGNMENT;
    int* status = status_word_for_current_device();
    if (!status) return USM_ERR_CUDA;
    SddmmArgs a{M, K, D, nnz, row_offsets, col_indices, row_swizzle, effective_seg(M, seg_rows), X, ldx, out, 0,
                out_dtype == USM_BF16 ? 1 : 0, 1, status};
    return launch_sddmm(a, Y, ldy, in_dtype == USM_BF16, workspace, workspace_bytes, st);
}

size_t row_swizzle_workspace_bytes(int M, int K) {
    if (M <= 0 || K < 0) return 0;
    return swizzle_workspace_bytes(M, K);
}

int row_swizzle_build(int M, int K, int seg_rows, const int* row_offsets, int* swizzle_out,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || K < 0) return USM_ERR_INVALID_ARG;
    if (M == 0) return USM_OK;
    if (!row_offsets || !swizzle_out) return USM_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < swizzle_workspace_bytes(M, K)) return USM_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 3u) != 0) return USM_ERR_ALIGNMENT;
    return launch_row_swizzle(M, K, seg_rows, row_offsets, swizzle_out, workspace, workspace_bytes,
                              as_stream(stream));
}

namespace {
size_t align256(size_t b) { return (b + 255) / 256 * 256; }
// Leading dimension of the transposed Y the general SDDMM builds (16-byte rows).
long long yt_ld(int D, bool bf16) {
    const int per = bf16 ? 8 : 4;
    return ((long long)D + per - 1) / per * per;
}
size_t general_yt_bytes(int K, int D, bool bf16, int y_transposed) {
    if (y_transposed || K <= 0 || D <= 0) return 0;
    return align256((size_t)K * (size_t)yt_ld(D, bf16) * (bf16 ? 2 : 4));
}
}  // namespace

size_t csr_sddmm_general_workspace_bytes(int M, int K, int D, int nnz, usm_dtype in_dtype, int y_transposed) {
    if (M <= 0 || K < 0 || D <= 0 || nnz <= 0) return 0;
    const bool bf = in_dtype == USM_BF16;
    return general_yt_bytes(K, D, bf, y_transposed) + sddmm_workspace_bytes(M, K, D, nnz, bf);
}

int csr_sddmm_general(int M, int K, int D, int nnz, const int* row_offsets, const int* col_indices,
                      const void* values, const int* row_swizzle, int seg_rows, const void* X, int ldx,
                      const void* Y, int ldy,
                      int y_transposed, void* out, usm_dtype in_dtype, usm_dtype out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
    if (M < 0 || K < 0 || D < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    if ((in_dtype != USM_F32 && in_dtype != USM_BF16) || (out_dtype != USM_F32 && out_dtype != USM_BF16))
        return USM_ERR_INVALID_ARG;
    if (y_transposed != 0 && y_transposed != 1) return USM_ERR_INVALID_ARG;
    if (M == 0 || nnz == 0) return USM_OK;
    if (!out || !row_offsets || !col_indices) return USM_ERR_INVALID_ARG;
    if (K == 0) return USM_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (D == 0) return launch_fill_out(out, nnz, out_dtype == USM_BF16, st);
    const bool bf = in_dtype == USM_BF16;
    const int es = bf ? 2 : 4;
    if (!X || !Y || ldx < D) return USM_ERR_INVALID_ARG;
    if (y_transposed ? ldy < D : ldy < K) return USM_ERR_INVALID_ARG;
    if (!aligned16(X) || ((long long)ldx * es) % 16 != 0) return USM_ERR_ALIGNMENT;
    if (y_transposed && (!aligned16(Y) || ((long long)ldy * es) % 16 != 0)) return USM_ERR_ALIGNMENT;
    const size_t yt_bytes = general_yt_bytes(K, D, bf, y_transposed);
    const size_t part_bytes = sddmm_workspace_bytes(M, K, D, nnz, bf);
    const size_t need = yt_bytes + part_bytes;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return USM_ERR_WORKSPACE;
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return USM_ERR_ALIGNMENT;
    int* status = status_word_for_current_device();
    if (!status) return USM_ERR_CUDA;
    const void* Yk = Y;
    long long ldyk = ldy;
    if (!y_transposed) {
        ldyk = yt_ld(D, bf);
        const int r = launch_dense_transpose(Y, ldy, D, K, bf, workspace, ldyk, st);
        if (r != USM_OK) return r;
        Yk = workspace;
    }
    if (ldyk > 0x7fffffffLL) return USM_ERR_UNSUPPORTED;
    SddmmArgs a{M, K, D, nnz, row_offsets, col_indices, row_swizzle, effective_seg(M, seg_rows), X, ldx, out, 0,
                out_dtype == USM_BF16 ? 1 : 0, 1, status, values, bf ? 1 : 0};
    void* part = part_bytes ? static_cast<unsigned char*>(workspace) + yt_bytes : nullptr;
    return launch_sddmm(a, Yk, (int)ldyk, bf, part, part_bytes, st);
}

int csr_row_softmax(int M, int nnz, const int* row_offsets, const float* scores, void* out, usm_dtype out_dtype,
                    void* stream) {
    if (M < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    if (out_dtype != USM_F32 && out_dtype != USM_BF16) return USM_ERR_INVALID_ARG;
    if (M == 0 || nnz == 0) return USM_OK;
    if (!row_offsets || !scores || !out) return USM_ERR_INVALID_ARG;
    return launch_row_softmax(M, nnz, row_offsets, scores, out, out_dtype == USM_BF16, as_stream(stream));
}

namespace {
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool dtype_ok(usm_dtype d) { return d == USM_F32 || d == USM_BF16; }
size_t dtype_size(usm_dtype d) { return d == USM_BF16 ? 2 : 4; }

// Checks of a usm_rel_bias; `table`: whether its table is read.
int check_bias(const usm_rel_bias* b, bool table) {
    if (!b || b->num_heads <= 0 || b->num_buckets <= 0 || b->max_distance <= 0 || !b->bucket_map)
        return USM_ERR_INVALID_ARG;
    if (table && (!b->table || !dtype_ok(b->table_dtype))) return USM_ERR_INVALID_ARG;
    if (b->num_buckets > USM_REL_BIAS_MAX_BUCKETS || b->max_distance > USM_REL_BIAS_MAX_DISTANCE)
        return USM_ERR_UNSUPPORTED;
    if (!aligned_to(b->bucket_map, 4) || !aligned_to(b->q_offset, 4) ||
        (table && !aligned_to(b->table, dtype_size(b->table_dtype))))
        return USM_ERR_ALIGNMENT;
    return USM_OK;
}

RelArgs rel_args(const usm_rel_bias* b, int M, int seg_rows) {
    return {b->table,    b->table_dtype == USM_BF16, b->num_heads, b->num_buckets, b->bucket_map, b->max_distance,
            b->seg_cols, b->q_offset,                effective_seg(M, seg_rows)};
}

constexpr int kPagedMaxHeadDim = 256;

// One cache's array: `extent` x stride, for pages, slots and heads.
int check_cache_array(const usm_paged_cache& c, const void* p, long long page, long long slot, long long head) {
    const long long es = (long long)dtype_size(c.dtype);
    if (!p) return USM_ERR_INVALID_ARG;
    const struct {
        int extent;
        long long stride;
    } dims[3] = {{c.num_pages, page}, {c.page_size, slot}, {c.kv_heads, head}};
    for (const auto& d : dims)
        if (d.extent > 1 && d.stride < c.head_dim) return USM_ERR_INVALID_ARG;
    for (const auto& d : dims)
        if (d.extent > 1 && d.stride * es % 16 != 0) return USM_ERR_ALIGNMENT;
    return aligned16(p) ? USM_OK : USM_ERR_ALIGNMENT;
}

// A paged cache and the number of its call's tokens; `heads`: rows of a token.
// Pointers are looked at where there are tokens to work on.
int check_paged(const usm_paged_cache& c, int tokens, long long heads) {
    if (tokens < 0 || c.num_seqs < 0 || c.kv_heads <= 0 || c.head_dim <= 0 || c.num_pages <= 0 || c.page_size <= 0 ||
        c.table_pages < 0 || !dtype_ok(c.dtype))
        return USM_ERR_INVALID_ARG;
    if (c.head_dim > kPagedMaxHeadDim || c.num_seqs > kPagedMaxSeqs || tokens * heads >= 1LL << 31) return USM_ERR_UNSUPPORTED;
    if (c.head_dim * dtype_size(c.dtype) % 16 != 0) return USM_ERR_ALIGNMENT;
    if (tokens == 0 || c.num_seqs == 0) return USM_OK;
    if (!c.lengths || (c.table_pages > 0 && !c.page_table)) return USM_ERR_INVALID_ARG;
    if (c.num_seqs > 1 && c.table_stride < c.table_pages) return USM_ERR_INVALID_ARG;
    if (!c.q_offsets && tokens % c.num_seqs != 0) return USM_ERR_INVALID_ARG;
    if (!aligned_to(c.lengths, 4) || !aligned_to(c.page_table, 4) || !aligned_to(c.q_offsets, 4)) return USM_ERR_ALIGNMENT;
    const int code = check_cache_array(c, c.k, c.k_page_stride, c.k_slot_stride, c.k_head_stride);
    return code != USM_OK ? code : check_cache_array(c, c.v, c.v_page_stride, c.v_slot_stride, c.v_head_stride);
}

// Rows of the call's tokens; written ones must not lie over one another.
int check_tokens(const usm_tokens* t, const usm_paged_cache& c, int tokens, int heads, bool written) {
    if (!t || !t->data) return USM_ERR_INVALID_ARG;
    const long long es = (long long)dtype_size(c.dtype), least = written ? c.head_dim : 0;
    if ((tokens > 1 && t->token_stride < least) || (heads > 1 && t->head_stride < least)) return USM_ERR_INVALID_ARG;
    if ((tokens > 1 && t->token_stride * es % 16 != 0) || (heads > 1 && t->head_stride * es % 16 != 0))
        return USM_ERR_ALIGNMENT;
    return aligned16(t->data) ? USM_OK : USM_ERR_ALIGNMENT;
}

// Positions that a sequence's row of the page table has slots for.
int capacity_of(const usm_paged_cache& c) {
    const long long n = (long long)c.table_pages * c.page_size;
    return n < kPagedMaxLength ? (int)n : kPagedMaxLength;
}
}  // namespace

int rel_bucket_build(int num_buckets, int max_distance, int causal, int* bucket_map, void* stream) {
    if (causal != 0 && causal != 1) return USM_ERR_INVALID_ARG;
    if (causal ? num_buckets < 2 : (num_buckets < 4 || num_buckets % 2 != 0)) return USM_ERR_INVALID_ARG;
    if (max_distance <= (causal ? num_buckets : num_buckets / 2) / 2) return USM_ERR_INVALID_ARG;
    if (num_buckets > USM_REL_BIAS_MAX_BUCKETS || max_distance > USM_REL_BIAS_MAX_DISTANCE)
        return USM_ERR_UNSUPPORTED;
    if (!bucket_map) return USM_ERR_INVALID_ARG;
    if (!aligned_to(bucket_map, 4)) return USM_ERR_ALIGNMENT;
    return launch_rel_bucket_build(num_buckets, max_distance, causal == 1, bucket_map, as_stream(stream));
}

int csr_rel_bias(int M, int K, int nnz, const int* row_offsets, const int* col_indices, const float* scores,
                 int seg_rows, const usm_rel_bias* bias, float* out, void* stream) {
    if (M < 0 || K < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    const int c = check_bias(bias, true);
    if (c != USM_OK) return c;
    if (M == 0 || nnz == 0) return USM_OK;
    if (K == 0 || !row_offsets || !col_indices || !scores || !out) return USM_ERR_INVALID_ARG;
    if (!aligned_to(scores, 4) || !aligned_to(out, 4) || !aligned_to(col_indices, 4)) return USM_ERR_ALIGNMENT;
    return launch_rel_bias(M, nnz, row_offsets, col_indices, scores, rel_args(bias, M, seg_rows), out,
                           as_stream(stream));
}

size_t csr_rel_bias_grad_workspace_bytes(int M, int nnz, int seg_rows, int num_heads, int num_buckets) {
    if (M <= 0 || nnz <= 0 || num_heads <= 0 || num_buckets <= 0 || num_buckets > USM_REL_BIAS_MAX_BUCKETS) return 0;
    return rel_bias_grad_workspace_bytes(M, nnz, effective_seg(M, seg_rows), num_heads, num_buckets);
}

int csr_rel_bias_grad(int M, int K, int nnz, const int* row_offsets, const int* col_indices, const void* dscores,
                      usm_dtype dscores_dtype, int seg_rows, const usm_rel_bias* bias, float* dtable,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || K < 0 || nnz < 0 || !dtype_ok(dscores_dtype)) return USM_ERR_INVALID_ARG;
    const int c = check_bias(bias, false);
    if (c != USM_OK) return c;
    if (!dtable) return USM_ERR_INVALID_ARG;
    if (!aligned_to(dtable, 4)) return USM_ERR_ALIGNMENT;
    if (M == 0 || nnz == 0)
        return launch_fill_out(dtable, (long long)bias->num_heads * bias->num_buckets, false, as_stream(stream));
    if (K == 0 || !row_offsets || !col_indices || !dscores) return USM_ERR_INVALID_ARG;
    if (!aligned_to(dscores, dtype_size(dscores_dtype)) || !aligned_to(col_indices, 4)) return USM_ERR_ALIGNMENT;
    const size_t need = csr_rel_bias_grad_workspace_bytes(M, nnz, seg_rows, bias->num_heads, bias->num_buckets);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return USM_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return USM_ERR_ALIGNMENT;
    return launch_rel_bias_grad(M, nnz, row_offsets, col_indices, dscores, dscores_dtype == USM_BF16,
                                rel_args(bias, M, seg_rows), dtable, workspace, as_stream(stream));
}

int csr_diff_softmax(int M, int nnz, const int* row_offsets, const float* scores1, const float* scores2,
                     const float* lambda, int num_heads, int seg_rows, void* out, usm_dtype out_dtype, void* stream) {
    if (M < 0 || nnz < 0 || num_heads <= 0 || !dtype_ok(out_dtype)) return USM_ERR_INVALID_ARG;
    if (M == 0 || nnz == 0) return USM_OK;
    if (!row_offsets || !scores1 || !scores2 || !lambda || !out) return USM_ERR_INVALID_ARG;
    if (!aligned_to(scores1, 4) || !aligned_to(scores2, 4) || !aligned_to(lambda, 4) ||
        !aligned_to(out, dtype_size(out_dtype)))
        return USM_ERR_ALIGNMENT;
    const MapArgs a{M,       nnz, row_offsets, scores1, scores2, lambda, num_heads, effective_seg(M, seg_rows),
                    nullptr, 0,   out,         nullptr, out_dtype == USM_BF16, nullptr};
    return launch_diff_softmax(a, as_stream(stream));
}

size_t csr_diff_softmax_grad_workspace_bytes(int M) { return M > 0 ? (size_t)M * 4 : 0; }

int csr_diff_softmax_grad(int M, int nnz, const int* row_offsets, const float* scores1, const float* scores2,
                          const float* lambda, int num_heads, int seg_rows, const void* dout, usm_dtype dout_dtype,
                          void* dscores1, void* dscores2, usm_dtype out_dtype, float* dlambda,
                          void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || nnz < 0 || num_heads <= 0 || !dtype_ok(dout_dtype) || !dtype_ok(out_dtype))
        return USM_ERR_INVALID_ARG;
    if (!aligned_to(dlambda, 4)) return USM_ERR_ALIGNMENT;
    if (M == 0 || nnz == 0)
        return dlambda ? launch_fill_out(dlambda, num_heads, false, as_stream(stream)) : (int)USM_OK;
    if (!row_offsets || !scores1 || !scores2 || !lambda || !dout || !dscores1 || !dscores2)
        return USM_ERR_INVALID_ARG;
    if (!aligned_to(scores1, 4) || !aligned_to(scores2, 4) || !aligned_to(lambda, 4) ||
        !aligned_to(dout, dtype_size(dout_dtype)) || !aligned_to(dscores1, dtype_size(out_dtype)) ||
        !aligned_to(dscores2, dtype_size(out_dtype)))
        return USM_ERR_ALIGNMENT;
    if (dlambda) {
        if (!workspace || workspace_bytes < csr_diff_softmax_grad_workspace_bytes(M)) return USM_ERR_WORKSPACE;
        if (!aligned16(workspace)) return USM_ERR_ALIGNMENT;
    }
    const MapArgs a{M,
                    nnz,
                    row_offsets,
                    scores1,
                    scores2,
                    lambda,
                    num_heads,
                    effective_seg(M, seg_rows),
                    dout,
                    dout_dtype == USM_BF16,
                    dscores1,
                    dscores2,
                    out_dtype == USM_BF16,
                    dlambda ? static_cast<float*>(workspace) : nullptr};
    return launch_diff_softmax_grad(a, dlambda, as_stream(stream));
}

int csr_row_softmax_grad(int M, int nnz, const int* row_offsets, const float* scores, const void* dout,
                         usm_dtype dout_dtype, void* dscores, usm_dtype out_dtype, void* stream) {
    if (M < 0 || nnz < 0 || !dtype_ok(dout_dtype) || !dtype_ok(out_dtype)) return USM_ERR_INVALID_ARG;
    if (M == 0 || nnz == 0) return USM_OK;
    if (!row_offsets || !scores || !dout || !dscores) return USM_ERR_INVALID_ARG;
    if (!aligned_to(scores, 4) || !aligned_to(dout, dtype_size(dout_dtype)) ||
        !aligned_to(dscores, dtype_size(out_dtype)))
        return USM_ERR_ALIGNMENT;
    const MapArgs a{M,    nnz, row_offsets, scores,  nullptr, nullptr, 1, M, dout, dout_dtype == USM_BF16,
                    dscores, nullptr, out_dtype == USM_BF16, nullptr};
    return launch_row_softmax_grad(a, as_stream(stream));
}

size_t csr_attention_workspace_bytes(int M, int K, int D, int N, int nnz, int two_maps, usm_dtype dtype) {
    const int most = dtype == USM_BF16 ? 512 : 256;
    if (M <= 0 || K <= 0 || D < 0 || D > most || N <= 0 || N > most || nnz <= 0) return 0;
    AttnArgs a{};
    a.M = M;
    a.K = K;
    a.D = D;
    a.N = N;
    a.nnz = nnz;
    static const float one = 1.f;
    a.lambda = two_maps ? &one : nullptr;  // only whether there is one
    return attention_workspace_bytes(a, dtype == USM_BF16);
}

int csr_attention(int M, int K, int D, int N, int nnz, const int* row_offsets, const int* col_indices,
                  const void* Q, int ldq, const void* Km, int ldk, const void* Q2, int ldq2, const void* K2, int ldk2,
                  const void* V, int ldv, float scale, const float* lambda, int num_heads, int seg_rows,
                  const usm_rel_bias* bias, float* C, int ldc, usm_dtype dtype, void* workspace,
                  size_t workspace_bytes, void* stream) {
    if (M < 0 || K < 0 || D < 0 || N < 0 || nnz < 0 || num_heads <= 0 || !dtype_ok(dtype))
        return USM_ERR_INVALID_ARG;
    if (bias) {
        const int c = check_bias(bias, true);
        if (c != USM_OK) return c;
        if (bias->num_heads != num_heads) return USM_ERR_INVALID_ARG;
    }
    if (M == 0 || N == 0) return USM_OK;
    const bool two = lambda != nullptr;
    if (D > 0 && (two != (Q2 != nullptr) || two != (K2 != nullptr))) return USM_ERR_INVALID_ARG;
    if (!C || !row_offsets || ldc < N) return USM_ERR_INVALID_ARG;
    if (!aligned16(C) || ldc % 4 != 0) return USM_ERR_ALIGNMENT;
    if (nnz == 0) return launch_fill_f32(C, M, N, ldc, as_stream(stream));
    if (K == 0 || !col_indices || !V || ldv < N) return USM_ERR_INVALID_ARG;
    if (D > 0 && (!Q || !Km || ldq < D || ldk < D || (two && (ldq2 < D || ldk2 < D)))) return USM_ERR_INVALID_ARG;
    const long long es = (long long)dtype_size(dtype);
    const int most = dtype == USM_BF16 ? 512 : 256;
    if (D > most || N > most) return USM_ERR_UNSUPPORTED;
    if (!aligned16(V) || ldv * es % 16 != 0 || !aligned_to(lambda, 4)) return USM_ERR_ALIGNMENT;
    if (D > 0 && (!aligned16(Q) || !aligned16(Km) || ldq * es % 16 != 0 || ldk * es % 16 != 0)) return USM_ERR_ALIGNMENT;
    if (D > 0 && two && (!aligned16(Q2) || !aligned16(K2) || ldq2 * es % 16 != 0 || ldk2 * es % 16 != 0))
        return USM_ERR_ALIGNMENT;
    AttnArgs a{M,    K,   D,   N,    nnz,  row_offsets, col_indices, Q,      Km,        Q2, K2, V,
               ldq,  ldk, ldq2, ldk2, ldv, scale,       lambda,      num_heads, effective_seg(M, seg_rows),
               RelArgs{}, C,   ldc};
    if (bias) a.bias = rel_args(bias, M, seg_rows);
    const size_t need = attention_workspace_bytes(a, dtype == USM_BF16);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return USM_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return USM_ERR_ALIGNMENT;
    return launch_attention(a, dtype == USM_BF16, workspace, as_stream(stream));
}

int rope_table_build(int positions, int rot_dim, double base, float* table, void* stream) {
    if (positions < 0 || rot_dim < 2 || rot_dim % 2 != 0 || !(base > 0.0) || base > 1.7976931348623157e308)
        return USM_ERR_INVALID_ARG;
    if ((long long)positions * rot_dim >= 1LL << 31) return USM_ERR_UNSUPPORTED;
    if (positions == 0) return USM_OK;
    if (!table) return USM_ERR_INVALID_ARG;
    if (!aligned_to(table, 4)) return USM_ERR_ALIGNMENT;
    return launch_rope_table(positions, rot_dim, base, table, as_stream(stream));
}

int paged_append(const usm_paged_cache* cache, int tokens, const usm_tokens* k, const usm_tokens* v, const usm_tokens* q,
                 const usm_tokens* q_out, int q_heads, const float* rope, int rope_positions, int rot_dim,
                 int interleaved, void* stream) {
    if (!cache) return USM_ERR_INVALID_ARG;
    const usm_paged_cache& c = *cache;
    if ((q != nullptr) != (q_out != nullptr) || q_heads < 0 || (q != nullptr) != (q_heads > 0)) return USM_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim % 2 != 0 || (interleaved != 0 && interleaved != 1)) return USM_ERR_INVALID_ARG;
    const int code = check_paged(c, tokens, (long long)q_heads + 2LL * c.kv_heads);
    if (code != USM_OK) return code;
    if (rot_dim > c.head_dim) return USM_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!rope || rope_positions <= 0)) return USM_ERR_INVALID_ARG;
    if (rot_dim > 0 && !aligned16(rope)) return USM_ERR_ALIGNMENT;
    if (tokens == 0 || c.num_seqs == 0) return USM_OK;
    int status = check_tokens(k, c, tokens, c.kv_heads, false);
    if (status == USM_OK) status = check_tokens(v, c, tokens, c.kv_heads, false);
    if (status == USM_OK && q) status = check_tokens(q, c, tokens, q_heads, false);
    if (status == USM_OK && q) status = check_tokens(q_out, c, tokens, q_heads, true);
    if (status != USM_OK) return status;
    AppendArgs a{};
    a.k = k->data, a.k_token = k->token_stride, a.k_head = k->head_stride;
    a.v = v->data, a.v_token = v->token_stride, a.v_head = v->head_stride;
    if (q) {
        a.q = q->data, a.q_token = q->token_stride, a.q_head = q->head_stride;
        a.q_out = q_out->data, a.q_out_token = q_out->token_stride, a.q_out_head = q_out->head_stride;
    }
    a.k_cache = c.k, a.kc_page = c.k_page_stride, a.kc_slot = c.k_slot_stride, a.kc_head = c.k_head_stride;
    a.v_cache = c.v, a.vc_page = c.v_page_stride, a.vc_slot = c.v_slot_stride, a.vc_head = c.v_head_stride;
    a.table = c.page_table, a.lengths = c.lengths, a.q_offsets = c.q_offsets;
    a.table_stride = c.table_stride, a.num_pages = c.num_pages, a.page_size = c.page_size, a.capacity = capacity_of(c);
    a.num_seqs = c.num_seqs, a.tokens = tokens, a.per_seq = tokens / c.num_seqs;
    a.kv_heads = c.kv_heads, a.q_heads = q_heads, a.head_dim = c.head_dim;
    a.rope = rope, a.rope_positions = rope_positions, a.rot = rot_dim, a.interleaved = interleaved;
    return launch_paged_append(a, c.dtype == USM_BF16, as_stream(stream));
}

size_t paged_attention_workspace_bytes(int tokens, int num_seqs, int q_heads, int kv_heads, int head_dim, usm_dtype dtype) {
    if (tokens <= 0 || num_seqs <= 0 || num_seqs > kPagedMaxSeqs || kv_heads <= 0 || q_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0 ||
        head_dim > kPagedMaxHeadDim || !dtype_ok(dtype) || (long long)tokens * q_heads >= 1LL << 31)
        return 0;
    // The caller may or may not bring offsets.
    size_t bytes = paged_attention_workspace(tokens, num_seqs, q_heads, kv_heads, head_dim, dtype == USM_BF16, false);
    if (tokens % num_seqs == 0)
        bytes = std::max(bytes, paged_attention_workspace(tokens, num_seqs, q_heads, kv_heads, head_dim, dtype == USM_BF16, true));
    return bytes;
}

int paged_attention(const usm_paged_cache* cache, int tokens, const usm_tokens* q, int q_heads, float scale, int causal,
                    int window, const usm_tokens* out, void* workspace, size_t workspace_bytes, void* stream) {
    if (!cache) return USM_ERR_INVALID_ARG;
    const usm_paged_cache& c = *cache;
    if (q_heads <= 0 || !(scale >= 0.f) || scale > 3.402823466e38f || (causal != 0 && causal != 1) || window < 0)
        return USM_ERR_INVALID_ARG;
    const int code = check_paged(c, tokens, q_heads);
    if (code != USM_OK) return code;
    if (q_heads % c.kv_heads != 0) return USM_ERR_INVALID_ARG;
    if (tokens == 0 || c.num_seqs == 0) return USM_OK;
    int status = check_tokens(q, c, tokens, q_heads, false);
    if (status == USM_OK) status = check_tokens(out, c, tokens, q_heads, true);
    if (status != USM_OK) return status;
    const bool bf16 = c.dtype == USM_BF16;
    if (!workspace || workspace_bytes < paged_attention_workspace(tokens, c.num_seqs, q_heads, c.kv_heads, c.head_dim, bf16, !c.q_offsets))
        return USM_ERR_WORKSPACE;
    if (!aligned16(workspace)) return USM_ERR_ALIGNMENT;
    PagedArgs a{};
    a.q = q->data, a.q_token = q->token_stride, a.q_head = q->head_stride;
    a.out = out->data, a.out_token = out->token_stride, a.out_head = out->head_stride;
    a.k = c.k, a.k_page = c.k_page_stride, a.k_slot = c.k_slot_stride, a.k_head = c.k_head_stride;
    a.v = c.v, a.v_page = c.v_page_stride, a.v_slot = c.v_slot_stride, a.v_head = c.v_head_stride;
    a.table = c.page_table, a.lengths = c.lengths, a.q_offsets = c.q_offsets;
    a.table_stride = c.table_stride, a.table_pages = c.table_pages;
    a.num_pages = c.num_pages, a.page_size = c.page_size, a.capacity = capacity_of(c);
    a.num_seqs = c.num_seqs, a.tokens = tokens, a.per_seq = tokens / c.num_seqs;
    a.kv_heads = c.kv_heads, a.group = q_heads / c.kv_heads, a.head_dim = c.head_dim;
    // ceil(2^shift / group) with 2^(shift - 31) the next power of two: its error, times
    // any x below 2^31, stays below 2^shift, so the quotients are exact.
    a.group_shift = 31;
    while ((1LL << (a.group_shift - 31)) < a.group) ++a.group_shift;
    a.group_mul = (uint32_t)(((1ULL << a.group_shift) + a.group - 1) / a.group);
    // A scale of 0 weighs all keys alike, as does the smallest normal number; it
    // keeps masked scores at -inf.
    a.scale_log2 = fminf(fmaxf(scale * 1.4426950408889634f, 1.17549435e-38f), 3.402823466e38f);
    a.causal = causal, a.window = window;
    a.status = status_word_for_current_device();
    if (!a.status) return USM_ERR_CUDA;
    return launch_paged_attention(a, bf16, workspace, as_stream(stream));
}

size_t csr_transpose_workspace_bytes(int M, int K, int nnz) {
    if (M < 0 || K < 0 || nnz <= 0) return 0;
    return transpose_workspace_bytes(M, K, nnz);
}

int csr_transpose(int M, int K, int nnz, const int* row_offsets, const int* col_indices, const void* values,
                  usm_dtype dtype, int* row_offsets_t, int* col_indices_t, void* values_t, int* perm_out,
                  void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || K < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    if (dtype != USM_F32 && dtype != USM_BF16) return USM_ERR_INVALID_ARG;
    if (!row_offsets_t) return USM_ERR_INVALID_ARG;
    if (nnz > 0 && (K == 0 || !row_offsets || !col_indices || !col_indices_t)) return USM_ERR_INVALID_ARG;
    if ((values == nullptr) != (values_t == nullptr)) return USM_ERR_INVALID_ARG;
    const size_t need = transpose_workspace_bytes(M, K, nnz);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return USM_ERR_WORKSPACE;
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return USM_ERR_ALIGNMENT;
    return launch_csr_transpose(M, K, nnz, row_offsets, col_indices, values, dtype == USM_BF16, row_offsets_t,
                                col_indices_t, values_t, perm_out, workspace, workspace_bytes, as_stream(stream));
}

int csr_permute_values(int nnz, const int* perm, const void* values, usm_dtype dtype, void* out, void* stream) {
    if (nnz < 0) return USM_ERR_INVALID_ARG;
    if (dtype != USM_F32 && dtype != USM_BF16) return USM_ERR_INVALID_ARG;
    if (nnz == 0) return USM_OK;
    if (!perm || !values || !out) return USM_ERR_INVALID_ARG;
    return launch_permute_values(nnz, perm, values, dtype == USM_BF16, out, as_stream(stream));
}

int csr_validate(int M, int K, int nnz, const int* row_offsets, const int* col_indices, int* result, void* stream) {
    if (M < 0 || K < 0 || nnz < 0) return USM_ERR_INVALID_ARG;
    if (!row_offsets || !result || (nnz > 0 && !col_indices)) return USM_ERR_INVALID_ARG;
    if ((uintptr_t)result % alignof(int) != 0) return USM_ERR_ALIGNMENT;
    return launch_csr_validate(M, K, nnz, row_offsets, col_indices, result, as_stream(stream));
}

int usm_poll_status(void* stream) {
    cudaStream_t st = as_stream(stream);
    if (cudaStreamSynchronize(st) != cudaSuccess) return cuda_failure();
    int* status = status_word_for_current_device();
    if (!status) return USM_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyAsync(&v, status, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return cuda_failure();
    if (cudaMemsetAsync(status, 0, sizeof(int), st) != cudaSuccess) return cuda_failure();
    if (cudaStreamSynchronize(st) != cudaSuccess) return cuda_failure();
    return v;
}

const char* usm_status_string(int status) {
    switch (status) {
        case USM_OK: return "USM_OK";
        case USM_ERR_INVALID_ARG: return "USM_ERR_INVALID_ARG";
        case USM_ERR_ALIGNMENT: return "USM_ERR_ALIGNMENT";
        case USM_ERR_UNSUPPORTED: return "USM_ERR_UNSUPPORTED";
        case USM_ERR_CUDA: return "USM_ERR_CUDA";
        case USM_ERR_TIMEOUT: return "USM_ERR_TIMEOUT";
        case USM_ERR_WORKSPACE: return "USM_ERR_WORKSPACE";
        default: return "USM_UNKNOWN_STATUS";
    }
}

int usm_set_schedule_override(int rows_per_warp, int tiles_per_block, int k_splits) {
    const bool r_ok = rows_per_warp == 0 || (rows_per_warp <= 32 && (rows_per_warp & (rows_per_warp - 1)) == 0);
    if (!r_ok || tiles_per_block < 0 || k_splits < 0 || k_splits > 65535) return USM_ERR_INVALID_ARG;
    g_override_rows.store(rows_per_warp, std::memory_order_relaxed);
    g_override_tiles.store(tiles_per_block, std::memory_order_relaxed);
    g_override_splits.store(k_splits, std::memory_order_relaxed);
    return USM_OK;
}

int usm_selftest_wait_timeout(long long limit_ns, void* stream) {
    if (limit_ns < 1000 || limit_ns > 1000000000LL) return USM_ERR_INVALID_ARG;
    int* status = status_word_for_current_device();
    if (!status) return USM_ERR_CUDA;
    return launch_wait_timeout_selftest(limit_ns, status, as_stream(stream));
}

}  // extern "C"
