// kivi_paged_api.cu - the C ABI of the paged 16-bit cache and of the attention
// over packed rows: validation and launches.  Nothing here allocates.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/kivi.h"
#include "kivi_paged.h"
#include "kivi_status.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool int_array(const void* p) { return p != nullptr && aligned(p, 4); }
bool vec_array(const void* p) { return p != nullptr && aligned(p, 16); }

kivi_status page_shift_of(int32_t page_size, int* shift) {
  if (page_size < 1) return KIVI_ERR_INVALID_ARG;
  if (page_size < kivi::kMinPage || page_size > kivi::kMaxPage ||
      (page_size & (page_size - 1)) != 0)
    return KIVI_ERR_UNSUPPORTED;
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  return KIVI_OK;
}

// Slots and lengths are int32, with room to round up to a page.
bool tokens_ok(int32_t pages, int32_t page_size) {
  return pages >= 1 && (int64_t)pages * page_size < INT32_MAX - kivi::kMaxPage;
}

kivi_status heads_of(int32_t hkv, int32_t hq, int32_t D) {
  if (hkv < 1 || hq < 1) return KIVI_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return KIVI_ERR_UNSUPPORTED;
  if (hq % hkv != 0 || hq / hkv > 128) return KIVI_ERR_UNSUPPORTED;
  return KIVI_OK;
}

// Rows of `heads` x D values, `stride` elements apart: whole 16-byte vectors, no
// overlap, and strides that a tensor map holds (below 2^40 bytes).
bool stride_ok(int64_t stride, int32_t heads, int32_t D) {
  return stride >= (int64_t)heads * D && stride % 8 == 0 && stride < ((int64_t)1 << 38);
}

kivi_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KIVI_OK : KIVI_ERR_CUDA; }

bool device_of(int* device, int* sms) {
  return cudaGetDevice(device) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device) == cudaSuccess;
}

// What both attention forms share; fills `a`.
kivi_status attention_args(kivi::VarlenAttnArgs& a, int32_t dtype, const void* q, int64_t q_stride,
                           void* out, int64_t out_stride, const int32_t* offsets, int32_t batch,
                           int32_t rows, int32_t hkv, int32_t hq, int32_t D, float sm_scale,
                           void* workspace, size_t workspace_bytes) {
  const kivi_status st = heads_of(hkv, hq, D);
  if (st != KIVI_OK) return st;
  if (dtype != KIVI_BF16 && dtype != KIVI_FP16) return KIVI_ERR_UNSUPPORTED;
  if (batch < 1 || rows < 0 || !std::isfinite(sm_scale)) return KIVI_ERR_INVALID_ARG;
  if (batch > kivi::kMaxRequests) return KIVI_ERR_UNSUPPORTED;
  size_t need = 0;
  if (kivi_attention_workspace_bytes(hkv, hq, D, &need) != KIVI_OK) return KIVI_ERR_UNSUPPORTED;
  if (!vec_array(workspace) || !int_array(offsets)) return KIVI_ERR_INVALID_ARG;
  if (workspace_bytes < need) return KIVI_ERR_BUFFER_TOO_SMALL;
  if (rows == 0) return KIVI_OK;
  if (!vec_array(q) || !vec_array(out) || !stride_ok(q_stride, hq, D) ||
      !stride_ok(out_stride, hq, D))
    return KIVI_ERR_INVALID_ARG;
  // (row, head) pairs are counted in int, rounded up to an item
  if ((int64_t)rows * hq > INT32_MAX - 512) return KIVI_ERR_INVALID_ARG;
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.offsets = offsets;
  a.status = static_cast<uint32_t*>(workspace);
  a.tickets = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + 64);
  a.partials = static_cast<uint8_t*>(workspace) + kivi::kPagedHeader;
  a.dtype = dtype;
  a.B = batch;
  a.T = rows;
  a.Hkv = hkv;
  a.Hq = hq;
  a.D = D;
  a.sm_scale = sm_scale;
  return KIVI_OK;
}

}  // namespace

extern "C" {

kivi_status kivi_paged_assign(const int32_t* lengths, const int32_t* new_tokens, int32_t batch,
                              int32_t* block_table, int32_t table_width, int32_t* free_pages,
                              const int32_t* num_free, int32_t num_pages, int32_t page_size,
                              int32_t* kv_lengths, int32_t* num_free_out, int32_t* offsets,
                              int32_t* slots, int32_t* positions, int32_t rows, uint32_t* status,
                              void* stream) {
  kivi::PagedAssignArgs a{};
  const kivi_status st = page_shift_of(page_size, &a.page_shift);
  if (st != KIVI_OK) return st;
  if (batch < 1 || rows < 0 || !tokens_ok(num_pages, page_size) ||
      !tokens_ok(table_width, page_size))
    return KIVI_ERR_INVALID_ARG;
  if (batch > kivi::kMaxRequests) return KIVI_ERR_UNSUPPORTED;
  if (!int_array(lengths) || !int_array(new_tokens) || !int_array(block_table) ||
      !int_array(free_pages) || !int_array(num_free) || !int_array(kv_lengths) ||
      !int_array(num_free_out) || !int_array(offsets) || !int_array(status) ||
      (rows > 0 && (!int_array(slots) || !int_array(positions))))
    return KIVI_ERR_INVALID_ARG;
  if (cudaGetDevice(&a.device) != cudaSuccess) return KIVI_ERR_CUDA;
  a.lengths = lengths;
  a.new_tokens = new_tokens;
  a.table = block_table;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.kv_lengths = kv_lengths;
  a.num_free_out = num_free_out;
  a.offsets = offsets;
  a.slots = slots;
  a.positions = positions;
  a.status = status;
  a.B = batch;
  a.width = table_width;
  a.num_pages = num_pages;
  a.rows = rows;
  return from_cuda(kivi::launch_paged_assign(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_paged_append(const void* k_new, int64_t k_stride, const void* v_new,
                              int64_t v_stride, const int32_t* slots, int32_t rows, void* k_pages,
                              void* v_pages, int32_t num_pages, int32_t page_size,
                              int32_t num_kv_heads, int32_t head_dim, uint32_t* status,
                              void* stream) {
  kivi::PagedAppendArgs a{};
  kivi_status st = page_shift_of(page_size, &a.page_shift);
  if (st != KIVI_OK) return st;
  st = heads_of(num_kv_heads, num_kv_heads, head_dim);
  if (st != KIVI_OK) return st;
  if (rows < 0 || !tokens_ok(num_pages, page_size)) return KIVI_ERR_INVALID_ARG;
  if (rows == 0) return KIVI_OK;
  if (!vec_array(k_new) || !vec_array(v_new) || !vec_array(k_pages) || !vec_array(v_pages) ||
      !int_array(slots) || (status != nullptr && !aligned(status, 4)) ||
      !stride_ok(k_stride, num_kv_heads, head_dim) || !stride_ok(v_stride, num_kv_heads, head_dim))
    return KIVI_ERR_INVALID_ARG;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.status = status;
  a.T = rows;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.num_pages = num_pages;
  if (cudaGetDevice(&a.device) != cudaSuccess) return KIVI_ERR_CUDA;
  return from_cuda(kivi::launch_paged_append(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_attention_workspace_bytes(int32_t num_kv_heads, int32_t num_q_heads,
                                           int32_t head_dim, size_t* bytes) {
  if (!bytes) return KIVI_ERR_INVALID_ARG;
  const kivi_status st = heads_of(num_kv_heads, num_q_heads, head_dim);
  if (st != KIVI_OK) return st;
  *bytes = kivi::kPagedHeader + (size_t)kivi::varlen_partial_bytes(head_dim);
  return KIVI_OK;
}

kivi_status kivi_packed_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, void* out, int64_t out_stride,
                                  int32_t dtype, const int32_t* offsets, int32_t batch,
                                  int32_t rows, int32_t num_kv_heads, int32_t num_q_heads,
                                  int32_t head_dim, float sm_scale, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  kivi::VarlenAttnArgs a{};
  const kivi_status st =
      attention_args(a, dtype, q, q_stride, out, out_stride, offsets, batch, rows, num_kv_heads,
                     num_q_heads, head_dim, sm_scale, workspace, workspace_bytes);
  if (st != KIVI_OK || rows == 0) return st;
  if (!vec_array(k) || !vec_array(v) || !stride_ok(k_stride, num_kv_heads, head_dim) ||
      !stride_ok(v_stride, num_kv_heads, head_dim))
    return KIVI_ERR_INVALID_ARG;
  if (!device_of(&a.device, &a.num_sms)) return KIVI_ERR_CUDA;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.max_new = rows;
  return from_cuda(kivi::launch_varlen_attention(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_paged_attention(const void* q, int64_t q_stride, const void* k_pages,
                                 const void* v_pages, void* out, int64_t out_stride, int32_t dtype,
                                 const int32_t* block_table, int32_t table_width,
                                 const int32_t* kv_lengths, const int32_t* offsets, int32_t batch,
                                 int32_t rows, int32_t max_new, int32_t num_pages,
                                 int32_t page_size, int32_t num_kv_heads, int32_t num_q_heads,
                                 int32_t head_dim, float sm_scale, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  kivi::VarlenAttnArgs a{};
  kivi_status st = page_shift_of(page_size, &a.page_shift);
  if (st != KIVI_OK) return st;
  st = attention_args(a, dtype, q, q_stride, out, out_stride, offsets, batch, rows, num_kv_heads,
                      num_q_heads, head_dim, sm_scale, workspace, workspace_bytes);
  if (st != KIVI_OK) return st;
  if (max_new < (rows > 0 ? 1 : 0) || !tokens_ok(num_pages, page_size) || !tokens_ok(table_width, page_size) ||
      (int64_t)num_pages * page_size * num_kv_heads > INT32_MAX || !int_array(block_table) ||
      !int_array(kv_lengths))
    return KIVI_ERR_INVALID_ARG;
  if (rows == 0) return KIVI_OK;
  if (!vec_array(k_pages) || !vec_array(v_pages)) return KIVI_ERR_INVALID_ARG;
  if (!device_of(&a.device, &a.num_sms)) return KIVI_ERR_CUDA;
  a.k = k_pages;
  a.v = v_pages;
  a.table = block_table;
  a.width = table_width;
  a.kv_lengths = kv_lengths;
  a.num_pages = num_pages;
  a.max_new = max_new < rows ? max_new : rows;
  return from_cuda(kivi::launch_varlen_attention(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_attention_status(void* workspace, void* stream, uint32_t* code_out) {
  if (!workspace) return KIVI_ERR_INVALID_ARG;
  uint32_t code = 0;
  if (!kivi::take_status(workspace, kivi::kPagedHeader, static_cast<cudaStream_t>(stream), &code))
    return KIVI_ERR_CUDA;
  if (code_out) *code_out = code;
  return code ? KIVI_ERR_DEVICE : KIVI_OK;
}

}  // extern "C"
