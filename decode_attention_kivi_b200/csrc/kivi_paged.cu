// kivi_paged.cu - the bookkeeping of a paged 16-bit cache on the GPU: block
// tables, slot map and positions of a step from the requests' lengths, and the
// write of the step's keys and values into the pages.
//
// Step of B requests holding len_b tokens, P tokens to a page, new_b to add
// (negative: the request is done), with a stack F of free pages:
//   back_b = new_b < 0 ? ceil(len_b / P) : 0          pages given back, pushed in order
//   need_b = new_b < 0 ? 0 : ceil((len_b + new_b) / P) - ceil(len_b / P)
//   page j of the step's new ones (request order) = F[top - 1 - j], top = free + sum back
//   row i of request b: position len_b + i, slot = table[b][pos / P] * P + pos mod P.
// All three sums are prefix sums over the requests; every CTA of a cluster forms
// them for itself in shared memory and the rest is independent per element.  The
// read of F and of the table that another CTA would have written is resolved
// from the prefix sums instead, so one cluster barrier is enough: the one
// between the reads of the lengths and the writes of the new lengths, which may
// be the same array.  A cluster of eight is never slower than one CTA (16
// requests, 16 rows: 4.0 for 4.1 us; 1,000 rows: 4.2 for 4.7; 2,000 requests: 8.8
// for 12.2), but too few threads for the rows of a large step: above kRowsHere
// rows a second kernel fills slots and positions from the new tables, four rows
// per thread (measured at the constant).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <climits>

#include "kivi_launch.cuh"
#include "kivi_paged.h"

namespace kivi {
namespace {

namespace cg = cooperative_groups;

constexpr int kAssignThreads = 512;
constexpr int kAssignCluster = 8;
// Rows that the cluster fills itself, for those of the second kernel: 16 requests, 16,000 rows 5.2
// for 6.6 us, 24,000 rows 6.2 for 6.4, 65,000 rows 11.8 for 6.5; 500 requests, 8,000 rows 5.7 for 7.9,
// 16,000 rows 7.4 for 7.7, 24,000 rows 8.4 for 7.8, 65,000 rows 15.7 for 7.8; 4,096 requests, 8,000 rows
// 15.5 for 21.9, 32,000 rows 21.5 for 21.5 (in a graph, back to back).
constexpr int kRowsHere = 16384;

// Exclusive prefix sums of three counts over the block's threads, and the totals.
struct Counts {
  long long tok, need, back;
};
__device__ __forceinline__ Counts operator+(Counts a, Counts b) {
  return {a.tok + b.tok, a.need + b.need, a.back + b.back};
}
__device__ Counts block_exclusive(Counts v, Counts* warp_sums, Counts* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Counts inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Counts o{__shfl_up_sync(0xffffffffu, inc.tok, d), __shfl_up_sync(0xffffffffu, inc.need, d),
                   __shfl_up_sync(0xffffffffu, inc.back, d)};
    if (lane >= d) inc = inc + o;
  }
  __syncthreads();  // warp_sums may still be read from the chunk before
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  Counts before{0, 0, 0}, all{0, 0, 0};
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    if (w < warp) before = before + warp_sums[w];
    all = all + warp_sums[w];
  }
  *total = all;
  return {before.tok + inc.tok - v.tok, before.need + inc.need - v.need,
          before.back + inc.back - v.back};
}

// Largest b with prefix[b] <= x (prefix[0] = 0 <= x < prefix[B]).
__device__ __forceinline__ int find_request(const int* prefix, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The slot of position pos in page id; -1, reported, where the id is negative or its slot no int.
__device__ __forceinline__ int slot_of(const PagedAssignArgs& a, int id, int pos) {
  const long long s = ((long long)id << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  if (id >= 0 && s <= INT_MAX) return (int)s;
  atomicOr(a.status, kPagedBadPage);
  return -1;
}

__global__ void __launch_bounds__(kAssignThreads)
paged_assign_kernel(PagedAssignArgs a, bool rows_here) {
  wait_for_predecessor();
  allow_successor();  // the rows' kernel waits for this one to end
  extern __shared__ int s_mem[];
  __shared__ Counts s_warp[kAssignThreads / 32];
  int* s_len = s_mem;                 // [B]
  int* s_tok = s_len + a.B;           // [B + 1] each
  int* s_need = s_tok + a.B + 1;
  int* s_back = s_need + a.B + 1;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int page = 1 << a.page_shift, rows = rows_here ? a.rows : 0;
  const long long cap = (long long)a.width << a.page_shift;

  Counts base{0, 0, 0};
  int wrong = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    Counts c{0, 0, 0};
    if (b < a.B) {
      const int len = a.lengths[b], add = a.new_tokens[b];
      const bool ok = len >= 0 && len <= cap && (add < 0 || (long long)len + add <= cap);
      wrong |= !ok;
      const int l = ok ? len : 0;
      s_len[b] = l;
      const int have = (int)(((long long)l + page - 1) >> a.page_shift);
      if (ok && add >= 0) {
        c.tok = add;
        c.need = (((long long)l + add + page - 1) >> a.page_shift) - have;
      } else if (ok) {
        c.back = have;
      }
    }
    Counts total;
    const Counts ex = base + block_exclusive(c, s_warp, &total);
    if (b < a.B) {  // sums that do not fit are refused below, before any use
      s_tok[b] = (int)ex.tok;
      s_need[b] = (int)ex.need;
      s_back[b] = (int)ex.back;
    }
    base = base + total;
  }
  const int free0 = *a.num_free;
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0) {
    s_tok[a.B] = (int)base.tok;
    s_need[a.B] = (int)base.need;
    s_back[a.B] = (int)base.back;
  }
  const long long top = free0 + base.back;
  uint32_t status = 0;
  if (wrong || base.tok > a.rows || free0 < 0 || top > a.num_pages) status |= kPagedBadLength;
  else if (base.need > top) status |= kPagedNoPages;
  cluster.sync();  // the lengths and the free count have been read everywhere

  const int tid = rank * blockDim.x + threadIdx.x, step = ranks * blockDim.x;
  if (status != 0) {  // nothing of the step happens; its rows belong to no request
    if (tid == 0) {
      atomicOr(a.status, status);
      *a.num_free_out = free0;
    }
    for (int b = tid; b < a.B; b += step) {
      a.kv_lengths[b] = a.lengths[b];
      a.offsets[b] = 0;
    }
    if (tid == 0) a.offsets[a.B] = 0;
    for (int i = tid; i < rows; i += step) {
      a.slots[i] = -1;
      a.positions[i] = 0;
    }
    return;
  }
  // stack entry x as it stands after the pushes
  auto stack = [&](int x) {
    if (x < free0) return a.free_pages[x];
    const int b = find_request(s_back, a.B, x - free0);
    return a.table[(long)b * a.width + (x - free0 - s_back[b])];
  };
  for (int b = tid; b < a.B; b += step) {
    a.offsets[b] = s_tok[b];
    // a request with new tokens or none keeps its length; one that gave its pages back
    // (or was released without any) holds nothing
    const int n = s_tok[b + 1] - s_tok[b];
    a.kv_lengths[b] = a.new_tokens[b] < 0 ? 0 : s_len[b] + n;
  }
  if (tid == 0) {
    a.offsets[a.B] = (int)base.tok;
    *a.num_free_out = (int)(top - base.need);
  }
  for (int i = tid; i < (int)base.back; i += step) a.free_pages[free0 + i] = stack(free0 + i);
  for (int j = tid; j < (int)base.need; j += step) {
    const int b = find_request(s_need, a.B, j);
    const int have = (s_len[b] + page - 1) >> a.page_shift;
    a.table[(long)b * a.width + have + (j - s_need[b])] = stack((int)top - 1 - j);
  }
  for (int i = tid; i < rows; i += step) {
    int slot = -1, pos = 0;
    if (i < base.tok) {
      const int b = find_request(s_tok, a.B, i);
      pos = s_len[b] + (i - s_tok[b]);
      const int have = (s_len[b] + page - 1) >> a.page_shift, p = pos >> a.page_shift;
      const int id = p < have ? a.table[(long)b * a.width + p]
                              : stack((int)top - 1 - (s_need[b] + p - have));
      slot = slot_of(a, id, pos);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
}

// Slots and positions of a step whose tables, lengths and offsets are made.  The offsets are
// searched in shared memory (from L2 a search is nine dependent reads).
__global__ void __launch_bounds__(256)
paged_rows_kernel(PagedAssignArgs a) {
  extern __shared__ int s_off[];  // [B + 1]
  wait_for_predecessor();
  for (int b = threadIdx.x; b <= a.B; b += blockDim.x) s_off[b] = a.offsets[b];
  __syncthreads();
  const long first = 4 * ((long)blockIdx.x * blockDim.x + threadIdx.x);
  if (first >= a.rows) return;
  const int i0 = (int)first, n = a.rows - i0 < 4 ? a.rows - i0 : 4;
  const int total = s_off[a.B];
  // the request of the first row, and from there on the next ones
  int b = i0 < total ? find_request(s_off, a.B, i0) : a.B;
  for (int x = 0; x < n; ++x) {
    const int i = i0 + x;
    int slot = -1, pos = 0;
    if (i < total) {
      while (s_off[b + 1] <= i) ++b;
      pos = a.kv_lengths[b] - (s_off[b + 1] - i);
      slot = slot_of(a, a.table[(long)b * a.width + (pos >> a.page_shift)], pos);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
}

// ---- append ----

// Bound by HBM: 16,000 rows of 8 heads of 128, 131 MB read and written, in 23.7 us (5.5 TB/s) by
// one wave of blocks that fills the SMs; 5% more by two, 10% by as many as there are vectors.
// One 16-byte vector of K and V per thread and step; a token's row of Hkv * D
// values is contiguous in the input and one run of D values per head in its page.
constexpr int kAppendThreads = 256, kThreadsPerSm = 2048;
__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(PagedAppendArgs a) {
  wait_for_predecessor();
  const int vec_head = a.D / 8, vec_row = a.Hkv * vec_head;
  const long total = (long)a.T * vec_row;
  for (long x = (long)blockIdx.x * blockDim.x + threadIdx.x; x < total;
       x += (long)gridDim.x * blockDim.x) {
    const int t = (int)(x / vec_row), r = (int)(x % vec_row), h = r / vec_head, c = r % vec_head;
    const int slot = a.slots[t];
    if (slot < 0) continue;  // a row of no request
    const int page = slot >> a.page_shift;
    if (page >= a.num_pages) {
      if (a.status != nullptr) atomicOr(a.status, kPagedBadPage);
      continue;
    }
    const long dst = ((((long)page * a.Hkv + h) << a.page_shift) +
                      (slot & ((1 << a.page_shift) - 1))) * vec_head + c;
    const uint4* k = reinterpret_cast<const uint4*>(a.k_new) + t * (a.k_stride / 8) + r;
    const uint4* v = reinterpret_cast<const uint4*>(a.v_new) + t * (a.v_stride / 8) + r;
    static_cast<uint4*>(a.k_pages)[dst] = *k;
    static_cast<uint4*>(a.v_pages)[dst] = *v;
  }
}

}  // namespace

cudaError_t launch_paged_assign(const PagedAssignArgs& a, cudaStream_t stream) {
  const size_t smem = sizeof(int) * (4 * (size_t)a.B + 3);
  int unused = 0;
  cudaError_t e = per_device_setup(a.device, &unused, [](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(paged_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(int) * (4 * (size_t)kMaxRequests + 3)));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kAssignCluster);
  cfg.blockDim = dim3(kAssignThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {kAssignCluster, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const bool rows_here = a.rows <= kRowsHere;
  e = cudaLaunchKernelEx(&cfg, paged_assign_kernel, a, rows_here);
  if (e != cudaSuccess || rows_here) return e;
  return launch_pdl(paged_rows_kernel, dim3((unsigned)((a.rows + 1023L) / 1024)), dim3(256),
                    sizeof(int) * ((size_t)a.B + 1), stream, a);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  int wave = 0;  // blocks that fill the SMs
  const cudaError_t e = per_device_setup(a.device, &wave, [&](int* v) {
    int sms = 0;
    const cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, a.device);
    *v = sms * (kThreadsPerSm / kAppendThreads);
    return e;
  });
  if (e != cudaSuccess) return e;
  const long total = (long)a.T * a.Hkv * (a.D / 8);
  const long blocks = (total + kAppendThreads - 1) / kAppendThreads;
  return launch_pdl(paged_append_kernel, dim3((unsigned)(blocks < wave ? blocks : wave)),
                    dim3(kAppendThreads), 0, stream, a);
}

}  // namespace kivi
