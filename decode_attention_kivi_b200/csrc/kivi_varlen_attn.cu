// kivi_varlen_attn.cu - causal attention of packed rows of different requests,
// over the rows' own keys (whole prompts) or over a paged 16-bit cache (chunks
// of new tokens, single tokens).
//
//   out[t][h] = sum_j softmax_j(sm_scale <q[t][h], k_j[h / g]>) v_j[h / g]
//
// over the keys j that row t of its request sees.  A row without keys is 0.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "kivi_varlen.cuh"

namespace kivi {
namespace {

constexpr float kLog2eV = 1.4426950408889634f;

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
  return __float2half_rn(x);
}

// One warp per (row, query head): lane i holds channels i, i + 32, ...; one pass
// over the keys with the running maximum and sum.
template <typename T, int D>
__global__ void __launch_bounds__(128)
varlen_attention_simple_kernel(VarlenAttnArgs a, bool skip_short) {
  const long w = ((long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= (long)a.T * a.Hq) return;
  const int t = (int)(w / a.Hq), h = (int)(w % a.Hq), kvh = h / (a.Hq / a.Hkv);
  // the request of row t
  Request r{};
  int b = 0;
  for (; b < a.B; ++b) {
    bool bad = false;
    r = load_request(a, b, &bad);
    if (bad && lane == 0) atomicOr(a.status, kPagedBadLength);
    if (t >= r.q0 && t < r.q0 + r.n) break;
  }
  if (b == a.B || (skip_short && is_short(r.n, a.Hq / a.Hkv))) return;
  const T* q = static_cast<const T*>(a.q) + t * a.q_stride + (long)h * D;
  constexpr int E = D / 32;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_float(q[lane + 32 * e]);
    acc[e] = 0.f;
  }
  const float sl2 = (a.sm_scale > 0.f ? a.sm_scale : rsqrtf((float)D)) * kLog2eV;
  float m = -INFINITY, l = 0.f;
  const int last = min(last_key(r, t - r.q0), r.L - 1);
  for (int j = 0; j <= last; ++j) {
    const T *k, *v;
    if (a.table == nullptr) {
      k = static_cast<const T*>(a.k) + (r.q0 + j) * a.k_stride + (long)kvh * D;
      v = static_cast<const T*>(a.v) + (r.q0 + j) * a.v_stride + (long)kvh * D;
    } else {
      const int page = a.table[(long)b * a.width + (j >> a.page_shift)];
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) atomicOr(a.status, kPagedBadPage);
        k = v = nullptr;
      } else {
        const long row = (((long)page * a.Hkv + kvh) << a.page_shift) +
                         (j & ((1 << a.page_shift) - 1));
        k = static_cast<const T*>(a.k) + row * D;
        v = static_cast<const T*>(a.v) + row * D;
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += k ? qv[e] * to_float(k[lane + 32 * e]) : 0.f;
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= sl2;
    const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * al + (v ? p * to_float(v[lane + 32 * e]) : 0.f);
  }
  T* out = static_cast<T*>(a.out) + t * a.out_stride + (long)h * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = from_float<T>(last < 0 ? 0.f : acc[e] / l);
}

template <typename T>
cudaError_t launch_simple(const VarlenAttnArgs& a, bool skip_short, cudaStream_t stream) {
  const long warps = (long)a.T * a.Hq, blocks = (warps + 3) / 4;
  if (a.D == 128)
    varlen_attention_simple_kernel<T, 128><<<(unsigned)blocks, 128, 0, stream>>>(a, skip_short);
  else
    varlen_attention_simple_kernel<T, 64><<<(unsigned)blocks, 128, 0, stream>>>(a, skip_short);
  return cudaGetLastError();
}

}  // namespace

long varlen_partial_bytes(int D) { return paged_decode_partial_bytes(D); }

cudaError_t launch_varlen_attention(const VarlenAttnArgs& a, cudaStream_t stream) {
  const float scale = a.sm_scale > 0.f ? a.sm_scale : 1.f / std::sqrt((float)a.D);
  const bool decode = a.table != nullptr && is_short(1, a.Hq / a.Hkv);
  if (decode) {
    const cudaError_t e = launch_paged_decode(a, scale * kLog2eV, stream);
    if (e != cudaSuccess || is_short(a.max_new, a.Hq / a.Hkv)) return e;
  }
  return a.dtype == 0 ? launch_simple<__nv_bfloat16>(a, decode, stream)
                      : launch_simple<__half>(a, decode, stream);
}

}  // namespace kivi
