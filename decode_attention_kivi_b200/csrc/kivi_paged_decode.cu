// kivi_paged_decode.cu - attention of single tokens (and of a few at once) over
// a paged 16-bit cache.
//
// A request with n new rows and g query heads per kv head, n * g <= 16, gives
// one tensor tile of 16 rows (token i, head h at row i * g + h) per kv head that
// reads the request's keys once: 4 D bytes per key against 4 D g n FLOPs, so the
// bound is HBM.  The tiles of 64 keys of all (request, kv head) items, in order,
// are cut into one contiguous range per CTA, equal to within a tile whatever the
// lengths are; the prefix sums over the requests that this needs are formed by
// every CTA from the device arrays.
//
// Each CTA (one per SM) has a producer warp that streams K and V through a ring
// of stages with tensor copies, one box of min(page, 64) whole rows per lane, the
// page ids read by the lane that needs them.  A box lies in shared memory as
// its 64-channel slabs, one behind the other, so that small pages need no more
// than one copy each (a copy per slab took 10% longer at pages of 16).  Four consumer warps
// take 16 keys of every tile each, on the tensor cores (mma.sync m16n8k16, fp32
// accumulation): S[row][key] = Q K^T with Q in registers, an online softmax in
// base 2 whose weights stay in registers as the operand of O[row][chan] += P V.
// The four states are merged when the item ends.  An item that lies in several
// CTAs leaves a partial (m, l, O in fp32) per CTA; the last CTA to arrive (a
// ticket per CTA that begins such an item) joins them in CTA order, so results
// do not depend on the order of arrival.
// Every wait is bounded; a wait that runs out sets the status word.
//
// 16 requests of up to 8K keys, 32 / 8 heads of 128, pages of 64: 68.6 us, 5.4 TB/s
// (82% of the measured copy rate); 8 requests to 4K, 32 heads, pages of 16: 59.5 us,
// 4.9 TB/s.  Of some 130,000 cycles 1,800 are the prologue, 6,000 the way to the
// first tile (lengths, table, copy, each from DRAM), 6,000 the last item's join.
#include "kivi_launch.cuh"
#include "kivi_varlen.cuh"

namespace kivi {
namespace {

constexpr int kTileD = 64;          // keys per tile
constexpr int kWarpsD = 4;          // consumer warps, 16 keys of each tile
constexpr int kThreadsD = (kWarpsD + 1) * 32;
constexpr int kBoxD = kTileD * 128; // 64 rows of 64 channels, the swizzle span
// Tiles per CTA at least: of an item of t tiles cut into p pieces a CTA works through t / p tiles of
// some 900 cycles, and the last reads p states, for each of its threads' 4-channel groups some 175
// cycles each, so p = sqrt(5 t / groups) is best (16,000 keys of 16 heads: 66 us at two tiles, 26 at
// eight, 25 by this rule); then as many tiles as cut the longest item evenly, since a CTA that ends
// one item and begins the next has two ends to its work (513 keys: 7.4 us at three tiles, some
// 15% more at two).
constexpr int kMinTilesD = 2;
// log2 of a row's largest weight.  A bf16 weight is rounded relative to itself; a fp16 one has steps
// of 2^-24 below 2^-14, so that without the factor (which O / l does not see) a long tail of keys near
// 2^-25 of the row's largest would be lost to P V and still counted in l.  Added behind the
// subtraction, which is exact for the largest scores whatever their size: no weight exceeds 2^15.
template <typename T>
constexpr float kTopD = Elem<T>::kBf16 ? 0.f : 15.f;

template <int D>
struct DCfg {
  static constexpr int kSlabs = D / 64;
  static constexpr int kTileBytes = kSlabs * kBoxD;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = (160 * 1024) / kStageBytes;
  static constexpr int kState = kDecodeRows * (D + 2);  // O[16][D], m[16], l[16]
  static constexpr int kOffMerge = kStages * kStageBytes;
  static constexpr int kOffBars = kOffMerge + kWarpsD * kState * 4;
  static constexpr int kOffPrefix = kOffBars + 2 * kStages * 8 + 80;
  static constexpr int bytes(int B) { return kOffPrefix + 4 * (B + 1) + 1024; }
  static_assert(bytes(kMaxRequests) <= 227 * 1024, "shared-memory plan");
};

// Tiles of one (request, kv head); a request without keys has one, for its zeros.
__device__ __forceinline__ int tiles_of(const Request& r) {
  return r.L > 0 ? (r.L + kTileD - 1) / kTileD : 1;
}

struct Split {
  int n, q, rem;  // CTAs with work; total = n * q + rem
  __device__ __forceinline__ int lo(int c) const { return c * q + min(c, rem); }
  __device__ __forceinline__ int cta_of(int t) const {
    const int big = rem * (q + 1);
    return t < big ? t / (q + 1) : rem + (t - big) / q;
  }
};

// The position of a CTA in its range: request b, kv head, tile j of nt.
struct Cursor {
  int b, kvh, j, nt;
  Request r;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsD, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    VarlenAttnArgs a, float scale_log2) {
  using C = DCfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
  uint64_t* empty = full + C::kStages;
  int* s_flag = reinterpret_cast<int*>(empty + C::kStages);  // the ticket's verdict
  volatile int* s_abort = s_flag + 1;
  volatile int* s_issued = s_flag + 2;
  long long* s_sum = reinterpret_cast<long long*>(s_flag + 4);  // [kWarpsD + 1] sums of the scan,
  int* s_most = reinterpret_cast<int*>(s_sum + kWarpsD + 1);    // and the most tiles of a request
  int* prefix = reinterpret_cast<int*>(smem + C::kOffPrefix);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hpk = a.Hq / a.Hkv;

  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_issued = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarpsD);
    }
    fence_mbar_init();
  }
  wait_for_predecessor();

  // ---- prefix sums of the requests' tiles ----
  long long base = 0;
  int longest = 1;  // tiles of an item
  // up to 32 requests: every warp forms the sums of all of them
  const bool alone = a.B <= 32;
  for (int b0 = 0; b0 < a.B; b0 += kThreadsD) {
    const int b = b0 + (alone ? lane : (int)threadIdx.x);
    long long v = 0;
    int tiles = 0;
    if (b < a.B) {
      bool bad = false;
      const Request r = load_request(a, b, &bad);
      if (bad && blockIdx.x == 0) atomicOr(a.status, kPagedBadLength);
      if (r.n > 0) tiles = tiles_of(r);  // at most max_new rows, which fit the tensor tile
      v = (long long)a.Hkv * tiles;
    }
    long long inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    const int most = __reduce_max_sync(0xffffffffu, tiles);
    if (alone) {
      if (warp == 0 && b < a.B) prefix[b] = (int)(inc - v);  // used where the total fits
      base = __shfl_sync(0xffffffffu, inc, 31);
      longest = max(longest, most);
      break;
    }
    __syncthreads();
    if (lane == 31) {
      s_sum[warp] = inc;
      s_most[warp] = most;
    }
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w <= kWarpsD; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
      longest = max(longest, s_most[w]);
    }
    if (b < a.B) prefix[b] = (int)(base + before + inc - v);  // used where the total fits
    base += all;
  }
  if (threadIdx.x == 0) prefix[a.B] = (int)base;
  __syncthreads();
  if (base > INT32_MAX) {  // more tiles than a call counts: nothing is computed
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, kPagedBadLength);
    return;
  }
  Split sp;
  const int groups = (a.max_new * hpk * (D / 4) + kWarpsD * 32 - 1) / (kWarpsD * 32);
  const int wanted = max(kMinTilesD, (int)ceilf(sqrtf((float)longest * (float)groups * 0.2f)));
  const int pieces = max(1, longest / wanted), least = (longest + pieces - 1) / pieces;
  sp.n = min((int)gridDim.x, (int)((base + least - 1) / least));
  if ((int)blockIdx.x >= sp.n) return;
  sp.q = (int)base / sp.n;
  sp.rem = (int)base - sp.n * sp.q;
  const int cta = blockIdx.x, t_begin = sp.lo(cta), n_tiles = sp.lo(cta + 1) - t_begin;

  auto enter = [&](Cursor& c, int b) {
    bool bad;
    c.b = b;
    c.r = load_request(a, b, &bad);
    c.nt = tiles_of(c.r);
  };
  auto start = [&]() {
    int lo = 0, hi = a.B;  // largest b with prefix[b] <= t_begin
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= t_begin) lo = mid;
      else hi = mid;
    }
    Cursor c;
    enter(c, lo);
    const int t = t_begin - prefix[lo];
    c.kvh = t / c.nt;
    c.j = t - c.kvh * c.nt;
    return c;
  };
  // moves on by a tile; true when that begins another item
  auto next = [&](Cursor& c) {
    if (++c.j < c.nt) return false;
    c.j = 0;
    if (++c.kvh == a.Hkv) {
      int b = c.b + 1;
      // the caller has tiles left (the bound is for lengths that change during the call)
      while (b + 1 < a.B && prefix[b + 1] == prefix[b]) ++b;
      enter(c, min(b, a.B - 1));
      c.kvh = 0;
    }
    return true;
  };

  if (warp == kWarpsD) {
    // ---- producer ----
    const int page = 1 << a.page_shift, rows = page < kTileD ? page : kTileD;
    const int per_tile = kTileD / rows;           // boxes of a slab
    const int boxes = per_tile * 2;               // of a stage, one per lane (at most 8)
    const int is_v = lane & 1, part = lane >> 1;
    const int outside = (a.num_pages * a.Hkv) << a.page_shift;  // a row that reads as zero
    const CUtensorMap* map = is_v ? &tv : &tk;
    Cursor c = start();
    int issued = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int s = i % C::kStages;
      if (i > 0) next(c);
      const int key = c.j * kTileD + part * rows;  // this lane's first key
      const bool mine = lane < boxes && key < c.r.L;
      int y = outside;
      if (mine) {
        const int id = a.table[(long)c.b * a.width + (key >> a.page_shift)];
        if (id >= 0 && id < a.num_pages)
          y = ((id * a.Hkv + c.kvh) << a.page_shift) + (key & (page - 1));
        else
          atomicOr(a.status, kPagedBadPage);
      }
      bool ok = *s_abort == 0;
      if (ok && i >= C::kStages) ok = mbar_wait_bounded(&empty[s], (uint32_t)((i / C::kStages) - 1) & 1u);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) {
          atomicOr(a.status, kPagedTimeout);
          *s_abort = 1;
        }
        break;
      }
      const int n = __popc(__ballot_sync(0xffffffffu, mine));
      unsigned char* st = smem + s * C::kStageBytes;
      if (lane == 0) mbar_expect_tx(&full[s], n * rows * 2 * D + debug_overstate());
      __syncwarp();
      if (mine)
        tma_load_3d(st + is_v * C::kTileBytes + part * rows * 2 * D, map, 0, y, 0, &full[s]);
      issued = i + 1;
    }
    if (lane == 0) *s_issued = issued;
    __syncwarp();
    named_sync(2, kThreadsD);
    return;
  }

  // ---- consumers ----
  const int g = lane >> 2, tig = lane & 3, r0 = 16 * warp;
  // this warp's 16 rows of a tile: where they begin, and the way from slab to slab
  const int box_rows = min(1 << a.page_shift, kTileD), slab_bytes = box_rows * 128;
  const int row_base = r0 / box_rows * box_rows * 2 * D + r0 % box_rows * 128;
  constexpr int kKS = D / 16, kNT = D / 8;
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  uint32_t qf[kKS][4];
  float o[kNT][4];
  float m[2], l[2];  // rows g and g + 8: running maximum (log2 units), sum over this lane's keys
  int last[2];       // the last key each row sees
  bool dead = false;
  int i_dead = n_tiles;

  auto begin_item = [&](const Cursor& c) {
    const int rows = c.r.n * hpk;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = -INFINITY;
      l[e] = 0.f;
      const int row = g + 8 * e, i = row / hpk;
      const bool real = row < rows;
      last[e] = real ? min(last_key(c.r, i), c.r.L - 1) : -1;
      const T* qr = static_cast<const T*>(a.q) + (c.r.q0 + (real ? i : 0)) * a.q_stride +
                    (long)(c.kvh * hpk + (real ? row - i * hpk : 0)) * D;
#pragma unroll
      for (int s = 0; s < kKS; ++s) {
        const uint32_t x0 = *reinterpret_cast<const uint32_t*>(qr + 16 * s + 2 * tig);
        const uint32_t x1 = *reinterpret_cast<const uint32_t*>(qr + 16 * s + 8 + 2 * tig);
        qf[s][e] = real ? x0 : 0u;
        qf[s][2 + e] = real ? x1 : 0u;
      }
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
  };

  // O / l of the item's rows from `count` states at src(x), in order; ld reads a float or float4
  // (other CTAs' states are read past L1).
  auto join = [&](const Cursor& c, int count, auto src, auto ld) {
    const int rows = c.r.n * hpk;
    for (int x = threadIdx.x; x < rows * (D / 4); x += kWarpsD * 32) {
      const int row = x / (D / 4), ch = x % (D / 4);
      // four states at a time: their loads are in flight together
      float M = -INFINITY, L = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int w0 = 0; w0 < count; w0 += 4) {
        float mw[4], lw[4];
        float4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* s = src(min(w0 + i, count - 1));
          mw[i] = ld(s + kDecodeRows * D + row);
          lw[i] = ld(s + kDecodeRows * (D + 1) + row);
          q[i] = ld(reinterpret_cast<const float4*>(s + row * D) + ch);
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < 4; ++i) mn = fmaxf(mn, mw[i]);
        const float mu = mn == -INFINITY ? 0.f : mn, f0 = fast_exp2(M - mu);
        M = mn;
        L *= f0;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= f0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = w0 + i < count ? fast_exp2(mw[i] - mu) : 0.f;
          L += f * lw[i];
          v[0] += f * q[i].x;
          v[1] += f * q[i].y;
          v[2] += f * q[i].z;
          v[3] += f * q[i].w;
        }
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;  // a row without keys is 0
      const int i = row / hpk;
      T* dst = static_cast<T*>(a.out) + (c.r.q0 + i) * a.out_stride +
               (long)(c.kvh * hpk + row - i * hpk) * D + 4 * ch;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(Elem<T>::pack(v[0] * inv, v[1] * inv), Elem<T>::pack(v[2] * inv, v[3] * inv));
    }
  };
  float* partials = reinterpret_cast<float*>(a.partials);
  int* tickets = a.tickets;
  // slot 0: the item a CTA begins in the middle of; slot 1: the one it leaves unfinished
  auto slot = [&](int c, int which) { return partials + ((long)c * 2 + which) * C::kState; };

  auto end_item = [&](const Cursor& c) {
    float* mine = merge + warp * C::kState;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      const int row = g + 8 * e;
      if (tig == 0) {
        mine[kDecodeRows * D + row] = m[e];
        mine[kDecodeRows * (D + 1) + row] = l[e];
      }
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        *reinterpret_cast<float2*>(mine + row * D + 8 * nt + 2 * tig) =
            make_float2(o[nt][2 * e], o[nt][2 * e + 1]);
    }
    named_sync(1, kWarpsD * 32);
    const int first = prefix[c.b] + c.kvh * c.nt, final = first + c.nt - 1;
    const bool head = first < t_begin, tail = final >= t_begin + n_tiles;
    const int rows = c.r.n * hpk;
    if (!head && !tail) {
      join(c, kWarpsD, [&](int w) { return merge + w * C::kState; }, [](auto* x) { return *x; });
      named_sync(1, kWarpsD * 32);  // the merge area is free again
      return;
    }
    // one state out of the four, for the other CTAs of the item
    float* part = slot(cta, head ? 0 : 1);
    for (int x = threadIdx.x; x < rows * (D / 4 + 1); x += kWarpsD * 32) {
      const int row = x / (D / 4 + 1), ch = x % (D / 4 + 1);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarpsD; ++w) M = fmaxf(M, merge[w * C::kState + kDecodeRows * D + row]);
      float L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarpsD; ++w) {
        const float* s = merge + w * C::kState;
        const float mw = s[kDecodeRows * D + row];
        const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
        if (ch == D / 4) {
          L += f * s[kDecodeRows * (D + 1) + row];
        } else {
          const float4 q = *reinterpret_cast<const float4*>(s + row * D + 4 * ch);
          v.x += f * q.x;
          v.y += f * q.y;
          v.z += f * q.z;
          v.w += f * q.w;
        }
      }
      if (ch == D / 4) {
        part[kDecodeRows * D + row] = M;
        part[kDecodeRows * (D + 1) + row] = L;
      } else {
        *reinterpret_cast<float4*>(part + row * D + 4 * ch) = v;
      }
    }
    __threadfence();
    named_sync(1, kWarpsD * 32);
    const int c0 = sp.cta_of(first), c1 = sp.cta_of(final);
    if (threadIdx.x == 0) *s_flag = atomicAdd(&tickets[c0], 1) == c1 - c0;
    named_sync(1, kWarpsD * 32);
    if (*s_flag) {
      __threadfence();
      // c0 leaves the item unfinished (slot 1), the others begin in its middle (slot 0)
      join(c, c1 - c0 + 1, [&](int w) { return slot(c0 + w, w == 0 ? 1 : 0); },
           [](auto* x) { return __ldcg(x); });
      if (threadIdx.x == 0) tickets[c0] = 0;  // ready for the next call
    }
    named_sync(1, kWarpsD * 32);
  };

  Cursor c = start();
  begin_item(c);
  for (int i = 0; i < n_tiles; ++i) {
    if (i > 0) {
      const Cursor before = c;
      if (next(c)) {
        end_item(before);
        begin_item(c);
      }
    }
    const int s = i % C::kStages;
    // after a wait ran out the warps keep to the same items (their merges meet on a named
    // barrier) but consume nothing more
    if (!dead && __any_sync(0xffffffffu, *s_abort != 0)) {
      dead = true;
      i_dead = i;
    }
    if (!dead && !__all_sync(0xffffffffu,
                             mbar_wait_bounded(&full[s], (uint32_t)(i / C::kStages) & 1u))) {
      dead = true;
      i_dead = i;
      if (lane == 0) {
        atomicOr(a.status, kPagedTimeout);
        *s_abort = 1;
      }
    }
    if (dead) continue;
    const int key0 = c.j * kTileD + r0;  // this warp's first key
    const int nv = min(16, c.r.L - key0);
    unsigned char* st = smem + s * C::kStageBytes;
    if (nv > 0) {
      const uint32_t kb = smem_addr(st) + row_base, vb = kb + C::kTileBytes;
      if (nv < 16) {  // keys behind the last: their V rows must be 0 (a weight of 0 times NaN)
        for (int x = lane; x < (16 - nv) * C::kSlabs * 8; x += 32) {
          const int row = nv + x / (C::kSlabs * 8), rest = x % (C::kSlabs * 8);
          *reinterpret_cast<uint4*>(st + C::kTileBytes + row_base + (rest / 8) * slab_bytes +
                                    row * 128 + 16 * (rest % 8)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();  // the stage's next tensor copy comes after these writes
        __syncwarp();
      }
      // ---- scores ----
      float sa[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int krow = (lane & 7) + 8 * (lane >> 4);
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        const int ch = 16 * ks + 8 * ((lane >> 3) & 1);
        uint32_t kf[4];
        ldsm_x4(kf, kb + (ch / 64) * slab_bytes + krow * 128 + ((((ch % 64) >> 3) ^ (krow & 7)) << 4));
        Elem<T>::mma(sa[0], qf[ks], kf[0], kf[1]);
        Elem<T>::mma(sa[1], qf[ks], kf[2], kf[3]);
      }
      // ---- online softmax: rows g, g + 8; keys key0 + 8 nt + 2 tig + x ----
      uint32_t p[4];
      float al[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int key = key0 + 8 * (y >> 1) + 2 * tig + (y & 1);
          x[y] = key <= last[e] ? sa[y >> 1][2 * e + (y & 1)] * scale_log2 : -INFINITY;
        }
        float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[e], mx), mu = mn == -INFINITY ? 0.f : mn;
        al[e] = fast_exp2(m[e] - mu);
        m[e] = mn;
        float w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          w[y] = fast_exp2(Elem<T>::kBf16 ? x[y] - mu : (x[y] - mu) + kTopD<T>);
        l[e] = l[e] * al[e] + ((w[0] + w[1]) + (w[2] + w[3]));
        p[e] = Elem<T>::pack(w[0], w[1]);
        p[2 + e] = Elem<T>::pack(w[2], w[3]);
      }
      if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          o[nt][0] *= al[0];
          o[nt][1] *= al[0];
          o[nt][2] *= al[1];
          o[nt][3] *= al[1];
        }
      }
      // ---- P V ----
      const int vrow = (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
      for (int n2 = 0; n2 < kNT / 2; ++n2) {
        const int ch = 16 * n2 + 8 * (lane >> 4);
        uint32_t vf[4];
        ldsm_x4_trans(vf,
                      vb + (ch / 64) * slab_bytes + vrow * 128 + ((((ch % 64) >> 3) ^ (vrow & 7)) << 4));
        Elem<T>::mma(o[2 * n2], p, vf[0], vf[1]);
        Elem<T>::mma(o[2 * n2 + 1], p, vf[2], vf[3]);
      }
    }
    __syncwarp();
    if (lane == 0) {
      fence_proxy_async();
      mbar_arrive(&empty[s]);
    }
  }
  named_sync(2, kThreadsD);  // the producer is done issuing
  if (dead) {
    const int issued = *s_issued;  // copies that this warp did not see land, at most one per stage
    for (int i = i_dead; i < issued; ++i)
      (void)mbar_wait_bounded(&full[i % C::kStages], (uint32_t)(i / C::kStages) & 1u);
  }
  allow_successor();
  end_item(c);
}

template <typename T, int D>
cudaError_t launch_t(const VarlenAttnArgs& a, float scale_log2, cudaStream_t stream) {
  using C = DCfg<D>;
  int unused = 0;
  cudaError_t e = per_device_setup(a.device, &unused, [](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(paged_decode_kernel<T, D>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::bytes(kMaxRequests));
  });
  if (e != cudaSuccess) return e;
  const long rows = ((long)a.num_pages * a.Hkv) << a.page_shift;
  const int box = a.page_shift < 6 ? 1 << a.page_shift : kTileD;
  CUtensorMap tk, tv;
  if (!encode_bf16_slabs_map(&tk, a.k, rows, D, box) || !encode_bf16_slabs_map(&tv, a.v, rows, D, box))
    return cudaErrorInvalidValue;
  const int grid = a.num_sms < kMaxGrid ? a.num_sms : kMaxGrid;
  e = launch_pdl(paged_decode_kernel<T, D>, dim3(grid), dim3(kThreadsD), C::bytes(a.B), stream, tk,
                 tv, a, scale_log2);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

long paged_decode_partial_bytes(int D) { return (long)kMaxGrid * 2 * kDecodeRows * (D + 2) * 4; }

#ifdef KIVI_DEBUG_BUILD
cudaError_t debug_overstate_paged_decode(unsigned bytes) {
  return cudaMemcpyToSymbol(g_debug_overstate, &bytes, sizeof bytes);
}
#endif

cudaError_t launch_paged_decode(const VarlenAttnArgs& a, float scale_log2, cudaStream_t stream) {
  if (!is_short(a.max_new, a.Hq / a.Hkv)) return cudaErrorInvalidValue;
  if (a.dtype == 0)
    return a.D == 128 ? launch_t<__nv_bfloat16, 128>(a, scale_log2, stream)
                      : launch_t<__nv_bfloat16, 64>(a, scale_log2, stream);
  return a.D == 128 ? launch_t<__half, 128>(a, scale_log2, stream)
                    : launch_t<__half, 64>(a, scale_log2, stream);
}

}  // namespace kivi
