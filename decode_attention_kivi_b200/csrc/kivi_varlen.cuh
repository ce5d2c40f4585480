// kivi_varlen.cuh - what the kernels over packed rows share: the two element
// types, and boxes of page or packed rows as tensor copies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kivi_ptx.cuh"
#include "kivi_request.cuh"
#include "kivi_tmap.cuh"

namespace kivi {

// Requests whose n * (query heads per kv head) rows fit one 16-row tensor tile are taken by the
// decode kernel, the others by the chunk kernel.
constexpr int kDecodeRows = 16;
__host__ __device__ __forceinline__ bool is_short(int n, int hpk) { return n <= kDecodeRows / hpk; }

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    mma_bf16(d, a[0], a[1], a[2], a[3], b0, b1);
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_half2(lo, hi); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
  }
};

}  // namespace kivi
