// kivi_paged.h - launchers of the paged 16-bit cache and of the attention over
// packed rows, called by the C ABI in kivi_paged_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace kivi {

constexpr int kMaxRequests = 4096;   // requests of one call (their prefix sums sit in shared memory)
constexpr int kMinPage = 16, kMaxPage = 256;

// Workspace of the attention calls: the status word, tickets (eight per CTA) from byte 64 on,
// and from kPagedHeader on the partials of at most kMaxGrid CTAs.
constexpr int kMaxGrid = 160;
constexpr int kTickets = 8;
constexpr int kPagedHeader = 8192;
static_assert(64 + 4 * kTickets * kMaxGrid <= kPagedHeader, "tickets");

// Bits of a status word (a call ORs them in; KIVI_PAGED_* in kivi.h).
constexpr uint32_t kPagedTimeout = 1u;     // a bounded wait ran out
constexpr uint32_t kPagedBadPage = 2u;     // a page id or slot outside the pool
constexpr uint32_t kPagedBadLength = 4u;   // offsets or lengths outside their buffers
constexpr uint32_t kPagedNoPages = 8u;     // not enough free pages

struct PagedAssignArgs {
  const int* lengths;     // [B] tokens held
  const int* new_tokens;  // [B] tokens to add, negative: release the request
  int* table;             // [B][width] page ids
  int* free_pages;        // [num_pages] stack of free pages
  const int* num_free;    // [1]
  int* kv_lengths;        // [B], may be `lengths`
  int* num_free_out;      // [1], may be `num_free`
  int* offsets;           // [B + 1]
  int* slots;             // [rows]
  int* positions;         // [rows]
  uint32_t* status;
  int B, width, num_pages, page_shift, rows;
  int device;
};
cudaError_t launch_paged_assign(const PagedAssignArgs& a, cudaStream_t stream);

struct PagedAppendArgs {
  const void* k_new;  // [T][Hkv][D], rows `k_stride` / `v_stride` elements apart
  const void* v_new;
  const int* slots;   // [T]
  void* k_pages;      // [num_pages][Hkv][page][D]
  void* v_pages;
  uint32_t* status;   // or null
  long k_stride, v_stride;
  int T, Hkv, D, num_pages, page_shift;
  int device;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream);

// Attention of packed rows: request b owns rows offsets[b] .. offsets[b+1]-1.
// Packed form (table == null): its keys are the same rows of k and v.  Paged
// form: its kv_lengths[b] keys lie in the pages of its table row, the new rows
// last.
struct VarlenAttnArgs {
  const void* q;       // [T][Hq][D]
  const void* k;       // [T][Hkv][D], or pages [num_pages][Hkv][page][D]
  const void* v;
  void* out;           // [T][Hq][D]
  const int* offsets;  // [B + 1]
  const int* kv_lengths;  // [B], paged only
  const int* table;       // [B][width], paged only
  uint32_t* status;       // workspace header: the status word,
  int* tickets;           // then the tickets, zero between calls
  uint8_t* partials;      // the rest of the workspace
  long q_stride, k_stride, v_stride, out_stride;  // elements between rows (k, v: packed only)
  int dtype;              // 0 bf16, 1 fp16
  int B, T, Hkv, Hq, D;
  int width, num_pages, page_shift;
  int max_new;            // no request has more new rows
  float sm_scale;         // <= 0: 1/sqrt(D)
  int num_sms, device;
};
cudaError_t launch_varlen_attention(const VarlenAttnArgs& a, cudaStream_t stream);
long varlen_partial_bytes(int D);

// Calls whose max_new rows fit one tile (paged form only); scale_log2 = scale * log2 e.
cudaError_t launch_paged_decode(const VarlenAttnArgs& a, float scale_log2, cudaStream_t stream);
long paged_decode_partial_bytes(int D);

#ifdef KIVI_DEBUG_BUILD
// Bytes added to every copy size that the two attention kernels expect (kivi_debug.h).
cudaError_t debug_overstate_varlen(unsigned bytes);
cudaError_t debug_overstate_paged_decode(unsigned bytes);
#endif

}  // namespace kivi
