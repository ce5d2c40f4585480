// kivi_request.cuh - a request of a packed batch as the kernels see it: its
// rows, its keys and the causal rule, from device arrays whose values are
// clamped to their buffers (a call with bad lengths sets a status bit and
// touches nothing outside).
#pragma once

#include "kivi_paged.h"

namespace kivi {

struct Request {
  int q0;  // first packed row
  int n;   // new rows
  int L;   // keys, the new rows' last
};

// Row i of the request sees keys 0 .. L - n + i (none where that is negative).
__device__ __forceinline__ int last_key(const Request& r, int i) { return r.L - r.n + i; }

__device__ __forceinline__ Request load_request(const VarlenAttnArgs& a, int b, bool* bad) {
  Request r;
  const int o0 = a.offsets[b], o1 = a.offsets[b + 1];
  r.q0 = min(max(o0, 0), a.T);
  const int q1 = min(max(o1, r.q0), a.T);
  r.n = q1 - r.q0;
  bool wrong = r.q0 != o0 || q1 != o1;
  if (a.table == nullptr) {
    r.L = r.n;
  } else {
    const long cap = (long)a.width << a.page_shift;
    const int l = a.kv_lengths[b];
    r.L = l < 0 ? 0 : l > cap ? (int)cap : l;
    wrong |= r.L != l || r.n > r.L;
  }
  if (r.n > a.max_new) {  // more than the call was told: not computed
    wrong = true;
    r.n = 0;
  }
  *bad = wrong;
  return r;
}

}  // namespace kivi
