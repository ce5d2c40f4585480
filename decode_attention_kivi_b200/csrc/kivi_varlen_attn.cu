// kivi_varlen_attn.cu - causal attention of packed rows of different requests,
// over the rows' own keys (whole prompts) or over a paged 16-bit cache (chunks
// of new tokens), on the fifth-generation tensor cores.
//
//   out[t][h] = sum_j softmax_j(sm_scale <q[t][h], k_j[h / g]>) v_j[h / g]
//
// over the keys j that row t of its request sees.  A row without keys is 0.
//
// The n new rows and g query heads of a (request, kv head) give n * g tile rows
// (token i, head h at row i * g + h), so that short chunks fill a tile and all
// heads of a group share the keys' copies.  An item is 256 of them, two halves
// of 128 (the TMEM lanes), with the tiles of 128 keys that they see: 4 * 128 *
// 256 * D FLOPs against 2 * 128 * D values copied per tile, 256 FLOPs per byte,
// so long chunks are bound by the tensor cores and, equally, by the 128 * 256
// exponentials of a tile (16 per SM and cycle: 2048 cycles, as long as its
// products take).
// The work of all items, in order, is cut into one contiguous range per CTA,
// equal to within a tile whatever the lengths are, an item counted as kItemCost
// and, for each of its tiles, the units of 64 keys that its halves go through;
// every CTA forms the prefix sums that this needs from the device arrays.
//
// Twelve warps, one CTA per SM:
//   warp 8 (producer)  2D tensor copies of K and V tiles into a ring of four
//                      slots, page by page (a box of min(page, 128) rows x 64
//                      channels per lane) or in one piece;
//   warps 9, 10 (MMA)  one elected lane each, for half i = 0, 1: S_i = Q_i K^T in
//                      units of 64 keys (M = 128, N = 64) into one of the half's
//                      two score buffers and O_i += P_i V, P_i read from TMEM,
//                      where it lies over the first half of S_i.  The scores of
//                      unit n + 2 follow the product of unit n, so that the
//                      softmax of a half has a unit in hand while the tensor
//                      cores work on the other.  Units and 16-key steps without
//                      a key that the half sees are left out;
//   warp 11 (plan)     finds the CTA's range; one lane lists its pieces of items a
//                      few ahead, for the other roles to read;
//   warps 0-7          one row per thread (its TMEM lane): the row of S from
//                      TMEM, the mask where the unit needs one, the online
//                      softmax in base 2, P back to TMEM.  O is rescaled only
//                      when a row's maximum grew by more than kSlack (up to then
//                      the stale maximum is kept; O / l is unchanged).  The next
//                      item's Q rows are fetched during the last unit of this
//                      one.
// An item that lies in several CTAs leaves a partial (m, l, O in fp32) per CTA,
// joined in CTA order, so results do not depend on the order of arrival: by the
// warp that arrives last (a ticket per CTA and warp), or, where few items are
// cut into many pieces, by a second kernel over all SMs.
// TMEM: two buffers of S_0 at columns 0 and 64, of S_1 at 128 and 192, O_0 at 256,
// O_1 behind it.
// Every wait is bounded; a wait that runs out sets the status word, and what was
// issued is drained before TMEM is released.
//
// The weights go into the second product in the element type: the operand in TMEM
// is 16 bits wide, and two of them to a weight would double that product.  In bf16
// the outputs are 0.0023 of their size off the 64-bit values where weights of 32
// bits leave 0.0017, most of it the rounding of the result; fp16 0.00025, 0.00021.
//
// What bounds it (16,384 rows, 32 / 8 heads of 128, bf16): 2.13 ms back to back,
// 1.03 PFLOP/s, where the card lowers the clock to hold its power; single passes
// after a pause take 1.8 to 1.9 ms (1.75 GHz).  A unit of both halves takes 1,780 cycles: its products
// 1,280 (a step of the scores is 48 cycles at N = 64, 6 KB of operands at 128
// bytes a cycle, where its arithmetic takes 32), its exponentials 1,024.  Whole
// tiles of scores (N = 128, 64 cycles a step, no room for a second buffer) take
// 3% less here, but 18% more on 8111 rows of 13 prompts, and 16% more on a step
// of 32 requests.  Taking a quarter of the exponentials
// to the fp32 pipe, fetching the next unit's scores early, warps of their own for
// the items' ends, and one MMA warp for both halves changed nothing or cost time;
// so did a lone half's tiles taken in turn by both (the step: 36% more), whose ring
// then holds too few tiles ahead.
#include <cmath>

#include "kivi_launch.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_varlen.cuh"

namespace kivi {
namespace {

constexpr float kLog2eV = 1.4426950408889634f;
constexpr int kHalf = 128;             // rows of a half = TMEM lanes
constexpr int kTileV = 128;            // keys per tile
constexpr int kUnit = 64;              // keys of a score buffer
constexpr int kSoftWarpsV = 8;
constexpr int kProducerWarpV = kSoftWarpsV, kMmaWarpV = kSoftWarpsV + 1;  // and + 2: by half
constexpr int kPlanWarpV = kMmaWarpV + 2;
constexpr int kThreadsV = (kSoftWarpsV + 4) * 32;  // three warpgroups
// Registers per thread at launch, and after the softmax warpgroups took what the third gave up.
constexpr int kRegsV = 168, kRegsSoft = 208, kRegsRest = 88;
static_assert(2 * kRegsSoft + kRegsRest <= 3 * kRegsV, "a larger sum would wait forever");
constexpr int kPieces = 4;             // pieces planned ahead
constexpr int kPieceReaders = 3 + kSoftWarpsV;
constexpr int kSlabV = 128 * 128;      // 128 rows of 64 channels
constexpr int kSlots = 4;              // K and V tiles in flight
constexpr uint32_t kTmemColsV = 512;
// Half-units per CTA at least (one tile of one item; 4 and 16 took 20% longer on 700 rows of 8
// prompts), and those that an item's start and end take as long as: 5.7 by a fit over the CTAs of 8111
// packed rows of 13 prompts, 32 heads of 128.  Other costs, against 6, over those rows with 32 x 1, 8 x 4,
// 2 x 16 and 1 x 64 kv heads by group: at D = 128 4 takes 17, 8, 8 and 10% longer, 8 within 2% of 6, 11
// up to 4% longer; at D = 64 4 takes 10, 0 and 0% longer, 8 up to 4%, 11 up to 7%.
constexpr int kMinWorkV = 8;
constexpr int kItemCost = 6;
constexpr int kChunk = 32;             // scores turned into weights at a time
// log2 growth of a row maximum before O is rescaled, and the factor 2^kTop of all weights of a row
// (O / l is unchanged): the weights stay below 2^(kTop + kSlack), far inside what the 32-bit sums hold.
// A bf16 weight is rounded relative to itself whatever the slack.  A fp16 one must stay below 2^16
// (two more bits are for the roundings of scores near 2^24) and has steps of 2^-24 below 2^-14: the
// row's largest being 2^kTop at least, each weight is off by at most 2^-(25 + kTop) of it, for 2^20
// keys in all by half a step of the result.  Without the factor a long tail of keys near 2^-25 was
// lost to P V and still counted in l.  8111 rows of 13 prompts, keys with a scale per channel, take
// 142 us at a slack of 8, 139 at 10, 148 at 6, 155 at 4; 137 at 14 without the factor.
template <typename T>
constexpr float kSlack = Elem<T>::kBf16 ? 32.f : 8.f;
template <typename T>
constexpr float kTop = Elem<T>::kBf16 ? 0.f : 6.f;
// one item cut into pieces: what the joining kernel needs
struct Cut {
  int count, q0, kvh, row0, rows, pad[3];
};

template <int D>
struct VCfg {
  static constexpr int kSlabs = D / 64;
  static constexpr int kTileBytes = kSlabs * kSlabV;
  static constexpr int kOffRing = 2 * kTileBytes;  // after the two halves of Q
  static constexpr int kOffBars = kOffRing + kSlots * kTileBytes;
  static constexpr int kOffPieces = kOffBars + 384;
  static constexpr int kOffPrefix = kOffPieces + kPieces * 64;
  static constexpr int kWarpState = 32 * (D + 2);  // O [D/4][32] float4, m [32], l [32]
  static constexpr int kState = kSoftWarpsV * kWarpState;
  static constexpr uint32_t kColO = 2 * kTileV;
  // more than half of the SM's shared memory: one CTA per SM, which holds all of TMEM
  static constexpr int bytes(int B) {
    const int n = kOffPrefix + 4 * (B + 1) + 1024;
    return n > 120 * 1024 ? n : 120 * 1024;
  }
  static_assert(bytes(kMaxRequests) <= 227 * 1024, "shared-memory plan");
  static_assert(kColO + 2 * D <= kTmemColsV, "TMEM plan");
};

// Query heads per kv head, and tile rows to tokens.
struct Heads {
  int n, shift;  // shift: log2 n, or -1
  __device__ __forceinline__ int token(int row) const { return shift >= 0 ? row >> shift : row / n; }
};

__device__ __forceinline__ Heads heads_of(int hpk) {
  return {hpk, (hpk & (hpk - 1)) == 0 ? __popc(hpk - 1) : -1};
}

// Units that the half of rows row0 .. row0 + 127 of an item sees; at least one where it has rows.
__device__ __forceinline__ int half_units(const Request& r, int rows, int row0, const Heads& h) {
  if (row0 >= rows) return 0;
  const int kmax = min(last_key(r, h.token(min(row0 + kHalf, rows) - 1)), r.L - 1);
  return kmax < 0 ? 1 : kmax / kUnit + 1;
}
constexpr int kUnits = kTileV / kUnit;
__device__ __forceinline__ int tiles_of_units(int n) { return (n + kUnits - 1) / kUnits; }
// Tiles of an item: those of its last rows, which see the most keys.
__device__ __forceinline__ int item_tiles(const Request& r, int rows, int tt, const Heads& h) {
  if (tt * 2 * kHalf >= rows) return 0;
  const int kmax = min(last_key(r, h.token(min((tt + 1) * 2 * kHalf, rows) - 1)), r.L - 1);
  return kmax < 0 ? 1 : kmax / kTileV + 1;
}

// Work of a tile of the item, and of an item.  Both halves' units, or the one half's; over pages a
// lone half's tile counts as three: it waits for its copies as long as both would.  Steps of two chunks of
// 509 rows beside 30 single tokens, 32 x 1, 8 x 4, 2 x 16 and 1 x 64 kv heads by group of 128: at two 7, 13,
// 19 and 24% longer, at four 20, 11, 5 and 1% (D = 64: 5 to 19% and 6 to 22%).  Prompts of their own keys,
// which few of the halves are alone in, take 1% longer at three than at two.
template <bool PAGED>
__device__ __forceinline__ int tile_work(int rows, int row0) {
  return rows - row0 > kHalf ? 2 * kUnits : kUnits + (PAGED ? 1 : 0);
}
template <bool PAGED>
__device__ __forceinline__ int item_work(const Request& r, int rows, int tt, const Heads& h) {
  return kItemCost + item_tiles(r, rows, tt, h) * tile_work<PAGED>(rows, tt * 2 * kHalf);
}

struct Ranges {
  int n, q, rem;  // CTAs with work; total = n * q + rem, q at least a tile where n > 1
  __device__ __forceinline__ int lo(int c) const { return c * q + min(c, rem); }
  __device__ __forceinline__ int cta_of(int t) const {
    const int big = rem * (q + 1);
    return t < big ? t / (q + 1) : rem + (t - big) / q;
  }
};

// A CTA's piece of an item: tiles j0 .. j1 - 1 of nt, for half i the units kUnits * j0 .. ei - 1.
// j1 < 0 ends the list.
struct alignas(16) Piece {
  int b, kvh, row0, rows;  // request, kv head, first row and number of rows of the request's heads
  int q0, n, L;            // the request
  int c0, c1;              // the CTAs of the item's first and last tile
  int j0, j1, nt;
  int u;                   // tiles of the pieces before, K and V counted
  int e0, e1, pad;
  __device__ __forceinline__ Request request() const { return {q0, n, L}; }
  __device__ __forceinline__ int end(int half) const { return half ? e1 : e0; }
  __device__ __forceinline__ bool active(int half) const { return end(half) > kUnits * j0; }
};
static_assert(sizeof(Piece) == 64, "a piece is four vectors");

__device__ __forceinline__ float exp2_in_order(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void max_in_order(float& m, float a, float b) {
  asm volatile("max.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(a), "f"(b));
}

// Weights 2^(scale s - mu) of kChunk scores as packed pairs, and their sum.  With kMax the maxima
// mx4 of all kUnit scores are formed between the exponentials, whose unit takes one warp
// instruction in eight cycles: the order is kept by volatile statements.
template <typename T, bool kMax = false>
__device__ __forceinline__ void weights(const float* s, float scale, float mu,
                                        uint32_t (&pk)[kChunk / 2], float2& sum, float (&mx4)[4]) {
  const float2 sc = make_float2(scale, scale), nm = make_float2(-mu, -mu);
  float2 t[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < kChunk / 2; ++c) {
    float2 x = fma2(make_float2(s[2 * c], s[2 * c + 1]), sc, nm);
    if (kMax) {
      x.x = exp2_in_order(x.x);
      max_in_order(mx4[2 * (c & 1)], s[4 * c], s[4 * c + 2]);
      x.y = exp2_in_order(x.y);
      max_in_order(mx4[2 * (c & 1) + 1], s[4 * c + 1], s[4 * c + 3]);
    } else {
      x.x = fast_exp2(x.x);
      x.y = fast_exp2(x.y);
    }
    t[c & 1] = add2(t[c & 1], x);
    pk[c] = Elem<T>::pack(x.x, x.y);
  }
  sum = add2(t[0], t[1]);
}

// The rows' joined output from `count` partials, in order, kTogether of them in flight at a time;
// src(w) is a warp's state.
template <typename T, int D, int C4, int kTogether, typename Src>
__device__ __forceinline__ void join_rows(int count, Src src, int lane, int c4_0, bool real, T* dst) {
  float M = -INFINITY, L = 0.f, acc[4 * C4];
#pragma unroll
  for (int i = 0; i < 4 * C4; ++i) acc[i] = 0.f;
  for (int w0 = 0; w0 < count; w0 += kTogether) {
    float mw[kTogether], lw[kTogether];
    float4 v[kTogether][C4];
#pragma unroll
    for (int x = 0; x < kTogether; ++x) {
      mw[x] = -INFINITY;
      if (w0 + x >= count) continue;
      const float* s = src(w0 + x);
      mw[x] = __ldcg(s + 32 * D + lane);
      lw[x] = __ldcg(s + 32 * (D + 1) + lane);
#pragma unroll
      for (int c = 0; c < C4; ++c)
        v[x][c] = __ldcg(reinterpret_cast<const float4*>(s) + (c4_0 + c) * 32 + lane);
    }
    float mn = M;
#pragma unroll
    for (int x = 0; x < kTogether; ++x) mn = fmaxf(mn, mw[x]);
    if (mn == -INFINITY) continue;
    const float f0 = fast_exp2(M - mn);
    M = mn;
    L *= f0;
#pragma unroll
    for (int i = 0; i < 4 * C4; ++i) acc[i] *= f0;
#pragma unroll
    for (int x = 0; x < kTogether; ++x) {
      if (mw[x] == -INFINITY) continue;  // nothing seen there, its O is not written
      const float f = fast_exp2(mw[x] - mn);
      L += f * lw[x];
#pragma unroll
      for (int c = 0; c < C4; ++c) {
        acc[4 * c] += f * v[x][c].x;
        acc[4 * c + 1] += f * v[x][c].y;
        acc[4 * c + 2] += f * v[x][c].z;
        acc[4 * c + 3] += f * v[x][c].w;
      }
    }
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  if (real)
#pragma unroll
    for (int c = 0; c < C4; c += 2)
      *reinterpret_cast<uint4*>(dst + 4 * (c4_0 + c)) =
          make_uint4(Elem<T>::pack(acc[4 * c] * inv, acc[4 * c + 1] * inv),
                     Elem<T>::pack(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv),
                     Elem<T>::pack(acc[4 * c + 4] * inv, acc[4 * c + 5] * inv),
                     Elem<T>::pack(acc[4 * c + 6] * inv, acc[4 * c + 7] * inv));
}

// The work of a lane's request, for a whole warp: the lanes share the requests of many items.
template <bool PAGED>
__device__ __forceinline__ long long request_work(const Request& r, const Heads& h, int lane) {
  const int rows = r.n * h.n, items = (rows + 2 * kHalf - 1) / (2 * kHalf);
  long long v = 0;
  if (items <= 4)
    for (int tt = 0; tt < items; ++tt) v += item_work<PAGED>(r, rows, tt, h);
  for (uint32_t left = __ballot_sync(0xffffffffu, items > 4); left; left &= left - 1) {
    const int from = __ffs(left) - 1;
    const Request rr{0, __shfl_sync(0xffffffffu, r.n, from), __shfl_sync(0xffffffffu, r.L, from)};
    const int rrows = rr.n * h.n;
    long long sum = 0;
    for (int tt = lane; tt * 2 * kHalf < rrows; tt += 32) sum += item_work<PAGED>(rr, rrows, tt, h);
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == from) v = sum;
  }
  return v;
}
template <typename N>
__device__ __forceinline__ N warp_inclusive(N v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const N o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

template <int D>
__device__ __forceinline__ float* partial_of(const VarlenAttnArgs& a, int cta, int which) {
  return reinterpret_cast<float*>(a.partials + kMaxGrid * sizeof(Cut)) +
         ((long)cta * 2 + which) * VCfg<D>::kState;
}

template <typename T, int D, bool PAGED>
__global__ void __launch_bounds__(kThreadsV, 1)
varlen_attention_kernel(const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, VarlenAttnArgs a, float scale_log2,
                        bool join_here) {
  using C = VCfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);  // [kSlots]
  uint64_t* empty = full + kSlots;
  uint64_t* q_full = empty + kSlots;  // [2] each, by half
  uint64_t* s_full = q_full + 2;      // [4], by half and buffer
  uint64_t* p_full = s_full + 4;      // [4]
  uint64_t* o_done = p_full + 4;      // [4], the product of the buffer's weights
  uint64_t* piece_full = o_done + 4;  // [kPieces]
  uint64_t* piece_empty = piece_full + kPieces;
  uint64_t* drained = piece_empty + kPieces;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
  int* s_sum = reinterpret_cast<int*>(s_tmem + 2);  // [kThreadsV / 32]
  int* prefix = reinterpret_cast<int*>(smem + C::kOffPrefix);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Heads heads = heads_of(a.Hq / a.Hkv);
  const int hpk = heads.n;

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], kHalf);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], kPieceReaders);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_done[i], 1);
      mbar_init(&p_full[i], kHalf);
    }
    mbar_init(drained, 2);
    fence_mbar_init();
  }
  if (warp == kMmaWarpV) {
    tc::alloc(s_tmem, kTmemColsV);
    tc::relinquish();
  }
  wait_for_predecessor();

  // ---- prefix sums of the requests' work: up to 32 requests are left to the plan warp ----
  long long base = 0;
  bool fits = true;
  for (int b0 = 0; a.B > 32 && b0 < a.B; b0 += kThreadsV) {
    const int b = b0 + threadIdx.x;
    Request r{0, 0, 0};
    if (b < a.B) {
      bool bad = false;
      r = load_request(a, b, &bad);
      if (bad && blockIdx.x == 0) atomicOr(a.status, kPagedBadLength);
    }
    const long long v = a.Hkv * request_work<PAGED>(r, heads, lane);
    const long long inc = warp_inclusive(v, lane);
    // a warp's sum that an int does not hold makes the call's total too large
    fits = fits && inc <= INT32_MAX;
    __syncthreads();
    if (lane == 31) s_sum[warp] = (int)inc;
    fits = __syncthreads_and(fits);
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreadsV / 32; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    if (b < a.B) prefix[b] = (int)(base + before + inc - v);
    base += all;
    fits = fits && base <= INT32_MAX;
    if (!fits) break;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *s_tmem;
  const int cta = blockIdx.x;

  Piece* pieces = reinterpret_cast<Piece*>(smem + C::kOffPieces);
  auto fail = [&]() {
    *s_abort = 1;
    atomicOr(a.status, kPagedTimeout);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, s_abort); };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
  };
  // piece k of the CTA, read by a whole warp; false where the wait ran out
  auto read_piece = [&](int k, Piece& p) {
    if (!wait_warp(&piece_full[k % kPieces], (uint32_t)(k / kPieces) & 1u)) return false;
    p = pieces[k % kPieces];
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[k % kPieces]);
    return true;
  };

  if (warp < kSoftWarpsV) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ---- softmax: half `hf`, thread r owns its row r (TMEM lane r) ----
    const int hf = warp >> 2, r = threadIdx.x & (kHalf - 1);
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t col_s = lanes + hf * kTileV, col_o = lanes + C::kColO + hf * D;
    unsigned char* qs = smem + hf * C::kTileBytes;
    // starts the copies of the half's Q rows (a row is 2 D bytes, D / 8 lanes to a row)
    auto fetch_q = [&](const Piece& p) {
      const int row = p.row0 + hf * kHalf + r, i = heads.token(row);
      const bool real = row < p.rows;
      const long off = real ? (p.q0 + i) * a.q_stride + (long)(p.kvh * hpk + row - i * hpk) * D : -1;
      constexpr int kPer = D / 8, kStep = 32 / kPer;  // lanes per row, rows per step
      const int c = lane % kPer, first = (warp & 3) * 32;
#pragma unroll 4
      for (int x = 0; x < 32; x += kStep) {
        const int rr = x + lane / kPer;
        const long o = __shfl_sync(0xffffffffu, off, rr);
        const int row_s = first + rr;
        const uint32_t dst = smem_addr(qs + (c >> 3) * kSlabV + row_s * 128 +
                                       (((c & 7) ^ (row_s & 7)) << 4));
        const T* src = static_cast<const T*>(a.q) + (o < 0 ? 0 : o + 8 * c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                     "r"(o < 0 ? 0 : 16)
                     : "memory");
      }
    };
    auto q_here = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async();  // Q is read by the tensor cores
      mbar_arrive(&q_full[hf]);
    };
    const bool wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride % 16 == 0;
    uint32_t ns = 0;  // phases by buffer: bit b is that of its next scores, its last product had the other
    Cut cut{0, 0, 0, 0, 0, {0, 0, 0}};
    Piece p, nx;  // the next piece is read during the last unit of this one
    int k = 0;
    bool ok = read_piece(k++, p);
    if (ok && p.j1 >= 0 && p.active(hf)) {
      fetch_q(p);
      q_here();
    }
    while (ok && p.j1 >= 0) {
      const int n0 = kUnits * p.j0, e = p.end(hf);
      const bool active = e > n0;
      const Request req = p.request();
      const int row = p.row0 + hf * kHalf + r, qi = heads.token(row);
      const bool real = row < p.rows;
      const int last = real ? min(last_key(req, qi), req.L - 1) : -1;
      // units that end behind this key need the mask
      const int clear = min(last_key(req, heads.token(row - r)), req.L - 1);
      float m = -INFINITY, l = 0.f;  // running maximum (log2 units) and sum
      for (int n = n0; n < e; ++n) {
        const int buf = n % kUnits;
        const uint32_t col = col_s + buf * kUnit;
        if (!(ok = wait_warp(&s_full[2 * hf + buf], ns >> buf & 1u))) break;
        ns ^= 1u << buf;
        tc::fence_after();
        if (n + 1 == e) {  // this item's scores are done with Q
          if (!(ok = read_piece(k++, nx))) break;
          if (nx.j1 >= 0 && nx.active(hf)) fetch_q(nx);
        }
        float s[kUnit];
        tc::ld_x64(col, s);
        const int nv = req.L - n / kUnits * kTileV;  // keys of the tile
        if (buf == 0 && nv > 0 && nv < kTileV && (nv & 15)) {
          // V rows behind the last key up to a whole step: a weight of 0 times NaN (both halves
          // write the zeros)
          const int x = p.u + (n - n0) / kUnits * 2 + 1;
          if (!(ok = wait_warp(&full[x % kSlots], (uint32_t)(x / kSlots) & 1u))) break;
          unsigned char* vs = smem + C::kOffRing + (x % kSlots) * C::kTileBytes;
          for (int y = r; y < (16 - (nv & 15)) * C::kSlabs * 8; y += kHalf) {
            const int row_v = nv + y / (C::kSlabs * 8), rest = y % (C::kSlabs * 8);
            *reinterpret_cast<uint4*>(vs + (rest / 8) * kSlabV + row_v * 128 + 16 * (rest % 8)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        const int key0 = n * kUnit;
        if (key0 + kUnit - 1 > clear) {
          const int lim = last - key0;
#pragma unroll
          for (int c = 0; c < kUnit; ++c) s[c] = c <= lim ? s[c] : -INFINITY;
        }
        // the weights with the maximum so far, while the unit's is formed; they are formed again
        // in the few units where it grew
        float mu = m == -INFINITY ? 0.f : m - kTop<T>;
        float2 sum, sum1;
        uint32_t pk[kChunk / 2], pk1[kChunk / 2];
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        weights<T, true>(s, scale_log2, mu, pk, sum, mx4);
        const float mx = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]) * scale_log2;
        const bool grow = mx > m + kSlack<T>;  // always where m = -inf and a key is seen
        if (__any_sync(0xffffffffu, grow)) {
          const float al = grow ? fast_exp2(m - mx) : 1.f;  // 0 at a row's first keys
          if (grow) {
            m = mx;
            mu = mx - kTop<T>;
          }
          l *= al;
          weights<T>(s, scale_log2, mu, pk, sum, mx4);
          if (n > n0) {  // P V up to the unit before must be in O
            if (!(ok = wait_warp(&o_done[2 * hf + (buf ^ 1)], ~ns >> (buf ^ 1) & 1u))) break;
            tc::fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[32];
              tc::ld_x32(col_o + c0, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= al;
              tc::st_x32(col_o + c0, o);
            }
          }
        }
        tc::st_x16(col, pk);
        weights<T>(s + kChunk, scale_log2, mu, pk1, sum1, mx4);
        tc::st_x16(col + kChunk / 2, pk1);
        sum = add2(sum, sum1);
        l += sum.x + sum.y;
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&p_full[2 * hf + buf]);
      }
      if (!ok) break;
      if (!active) {
        if (!(ok = read_piece(k++, nx))) break;
        if (nx.j1 >= 0 && nx.active(hf)) fetch_q(nx);
      }
      if (nx.j1 >= 0 && nx.active(hf)) q_here();
      if (active) {
        const int buf = (e - 1) % kUnits;
        if (!(ok = wait_warp(&o_done[2 * hf + buf], ~ns >> buf & 1u))) break;
        tc::fence_after();
      }
      T* dst = static_cast<T*>(a.out) + (p.q0 + (real ? qi : 0)) * a.out_stride +
               (long)(p.kvh * hpk + (real ? row - qi * hpk : 0)) * D;
      if (p.j0 == 0 && p.j1 == p.nt) {
        if (active) {
          // a store touches a line per lane whatever its width: 32 bytes of the row where it is aligned
          const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tc::ld_x32(col_o + c0, o);
            if (real)
#pragma unroll
              for (int i = 0; i < 32; i += 16) {
                uint32_t w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)  // no product was made where no key is seen
                  w[x] = l > 0.f ? Elem<T>::pack(o[i + 2 * x] * inv, o[i + 2 * x + 1] * inv) : 0u;
                if (wide_out) {
                  store_32_bytes(dst + c0 + i, w);
                } else {
                  *reinterpret_cast<uint4*>(dst + c0 + i) = make_uint4(w[0], w[1], w[2], w[3]);
                  *reinterpret_cast<uint4*>(dst + c0 + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
              }
          }
        }
      } else {
        const int c0 = p.c0, c1 = p.c1;
        if (p.j0 == 0) cut = Cut{c1 - c0 + 1, p.q0, p.kvh, p.row0, p.rows, {0, 0, 0}};
        if (p.row0 + warp * 32 < p.rows) {
          // slot 0: the item this CTA begins in the middle of; slot 1: the one it leaves unfinished
          float* part = partial_of<D>(a, cta, p.j0 > 0 ? 0 : 1) + warp * C::kWarpState;
          if (active) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tc::ld_x32(col_o + c, o);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4*>(part)[(c / 4 + i) * 32 + lane] =
                    make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
          part[32 * D + lane] = m;
          part[32 * (D + 1) + lane] = l;
          if (join_here) {
            __threadfence();
            __syncwarp();
            int* ticket = a.tickets + c0 * kTickets + warp;
            int arrived = 0;
            if (lane == 0) arrived = atomicAdd(ticket, 1);
            if (__shfl_sync(0xffffffffu, arrived, 0) == c1 - c0) {
              __threadfence();
              join_rows<T, D, D / 4, 1>(
                  c1 - c0 + 1,
                  [&](int x) { return partial_of<D>(a, c0 + x, x == 0 ? 1 : 0) + warp * C::kWarpState; },
                  lane, 0, real, dst);
              if (lane == 0) *ticket = 0;  // ready for the next call
            }
          }
        }
      }
      p = nx;
    }
    if (!ok) {
      asm volatile("cp.async.wait_all;" ::: "memory");  // Q rows on their way
      fail();
    }
    if (!join_here && threadIdx.x == 0) reinterpret_cast<Cut*>(a.partials)[cta] = cut;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kPlanWarpV) {
      // ---- plan: the CTA's range, found by the warp, and its pieces, by one lane ----
      if (a.B <= 32) {
        Request r{0, 0, 0};
        if (lane < a.B) {
          bool bad = false;
          r = load_request(a, lane, &bad);
          if (bad && cta == 0) atomicOr(a.status, kPagedBadLength);
        }
        const long long v = a.Hkv * request_work<PAGED>(r, heads, lane);
        const long long inc = warp_inclusive(v, lane);
        base = __shfl_sync(0xffffffffu, inc, 31);
        fits = base <= INT32_MAX;
        if (lane < a.B) prefix[lane] = (int)(inc - v);  // used where the total fits
      }
      if (lane == 0) {
        prefix[a.B] = (int)base;
        if (!fits && cta == 0) atomicOr(a.status, kPagedBadLength);
      }
      __syncwarp();
      Ranges sp{0, 0, 0};
      int t_begin = 0, t_end = 0;
      if (fits && base > 0) {
        sp.n = min((int)gridDim.x, (int)((base + kMinWorkV - 1) / kMinWorkV));
        sp.q = (int)base / sp.n;
        sp.rem = (int)base - sp.n * sp.q;
        if (cta < sp.n) {
          t_begin = sp.lo(cta);
          t_end = sp.lo(cta + 1);
        }
      }
      bool ok = true, bad;
      int t0 = t_end;
      Piece p{};
      Request r{0, 0, 0};
      if (t_begin < t_end) {
        int lo = 0, hi = a.B;  // largest b with prefix[b] <= t_begin
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (prefix[mid] <= t_begin) lo = mid;
          else hi = mid;
        }
        r = load_request(a, lo, &bad);
        const int rows = r.n * hpk, per_head = (prefix[lo + 1] - prefix[lo]) / a.Hkv;
        p.b = lo;
        p.kvh = (t_begin - prefix[lo]) / per_head;
        int x = t_begin - prefix[lo] - p.kvh * per_head;  // work to pass within the head
        for (int i0 = 0; i0 * 2 * kHalf < rows; i0 += 32) {
          const int tt = i0 + lane;
          const int v = tt * 2 * kHalf < rows ? item_work<PAGED>(r, rows, tt, heads) : 0;
          const int inc = warp_inclusive(v, lane);
          const uint32_t past = __ballot_sync(0xffffffffu, inc > x);
          if (past) {
            const int at = __ffs(past) - 1;
            p.row0 = (i0 + at) * 2 * kHalf;
            t0 = t_begin - (x - __shfl_sync(0xffffffffu, inc - v, at)) + kItemCost;
            break;
          }
          x -= __shfl_sync(0xffffffffu, inc, 31);
        }
      }
      if (lane == 0) {
        int k = 0, u = 0;
        for (;; ++k) {
          ok = k < kPieces || wait(&piece_empty[k % kPieces], (uint32_t)(k / kPieces - 1) & 1u);
          if (!ok) break;
          // tile j belongs to the CTA whose range holds the end of its work
          const int w = tile_work<PAGED>(r.n * hpk, p.row0);
          const bool more = t0 + w <= t_end;
          p.j1 = -1;
          if (more) {
            p.rows = r.n * hpk;
            p.q0 = r.q0;
            p.n = r.n;
            p.L = r.L;
            p.nt = item_tiles(r, p.rows, p.row0 / (2 * kHalf), heads);
            p.j0 = max(0, t_begin - t0) / w;
            p.j1 = min(p.nt, (t_end - t0) / w);
            p.c0 = sp.cta_of(t0 + w - 1);
            p.c1 = sp.cta_of(t0 + p.nt * w - 1);
            p.u = u;
            p.e0 = min(half_units(r, p.rows, p.row0, heads), kUnits * p.j1);
            p.e1 = min(half_units(r, p.rows, p.row0 + kHalf, heads), kUnits * p.j1);
          }
          pieces[k % kPieces] = p;
          mbar_arrive(&piece_full[k % kPieces]);
          if (!more) break;
          u += 2 * (p.j1 - p.j0);
          t0 += p.nt * w + kItemCost;
          if (t0 >= t_end) continue;
          p.row0 += 2 * kHalf;
          if (p.row0 >= p.rows) {
            p.row0 = 0;
            if (++p.kvh == a.Hkv) {
              p.kvh = 0;
              ++p.b;
              while (p.b < a.B && prefix[p.b + 1] == prefix[p.b]) ++p.b;
              if (p.b < a.B)
                r = load_request(a, p.b, &bad);
              else
                t0 = t_end;  // only where the lengths changed during the call
            }
          }
        }
        if (!ok) fail();
      }
    } else if (warp == kProducerWarpV) {
      // ---- producer: tiles u = 2 s (K) and 2 s + 1 (V) of the CTA's step s, slot u mod 4 ----
      const int box = PAGED ? min(1 << a.page_shift, kTileV) : kTileV;
      const int boxes = kTileV / box * C::kSlabs;  // of a tile, one per lane (at most 16)
      const int slab = lane % C::kSlabs, part = lane / C::kSlabs;
      const int outside = PAGED ? (a.num_pages * a.Hkv) << a.page_shift : 0;  // rows of zeros
      int u = 0;
      bool ok = true;
      Piece p;
      for (int k = 0; ok && (ok = read_piece(k, p)) && p.j1 >= 0; ++k) {
        for (int j = p.j0; ok && j < p.j1; ++j) {
          const int key = j * kTileV + part * box;
          const bool mine = lane < boxes && key < p.L;
          int x = 64 * slab, y = 0;
          if (PAGED) {
            y = outside;
            if (mine) {
              const int id = a.table[(long)p.b * a.width + (key >> a.page_shift)];
              if (id >= 0 && id < a.num_pages)
                y = ((id * a.Hkv + p.kvh) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
              else
                atomicOr(a.status, kPagedBadPage);
            }
          } else {
            x += p.kvh * D;
            y = p.q0 + key;
          }
          const int n = __popc(__ballot_sync(0xffffffffu, mine));
          for (int v = 0; v < 2; ++v, ++u) {
            const int s = u % kSlots;
            if (u >= kSlots && !wait_warp(&empty[s], (uint32_t)(u / kSlots - 1) & 1u)) {
              ok = false;
              break;
            }
            unsigned char* dst = smem + C::kOffRing + s * C::kTileBytes;
            if (lane == 0) mbar_expect_tx(&full[s], n * box * 128 + debug_overstate());
            __syncwarp();
            if (mine) tma_load_2d(dst + slab * kSlabV + part * box * 128, v ? &tv : &tk, x, y, &full[s]);
          }
        }
      }
      if (!ok) fail();
      // every copy issued lands before the CTA may exit
      for (int i = max(u - kSlots, 0); i < u; ++i)
        if (!mbar_wait_bounded(&full[i % kSlots], (uint32_t)(i / kSlots) & 1u)) fail();
    } else if (tc::elect_one()) {
      // ---- MMA of half i, by one lane ----
      const int i = warp - kMmaWarpV;
      constexpr uint32_t id_s = tc::idesc_16bit(kHalf, kUnit, false, Elem<T>::kBf16);
      constexpr uint32_t id_o = tc::idesc_16bit(kHalf, D, true, Elem<T>::kBf16);
      constexpr int kTile16 = C::kTileBytes / 16, kUnit16 = kUnit * 128 / 16;
      // descriptors of the half's Q and of ring slot 0; their low words count 16 bytes
      const uint64_t qd = tc::desc_sw128(smem_addr(smem), 16, 1024) + i * kTile16;
      const uint64_t kd = tc::desc_sw128(smem_addr(smem + C::kOffRing), 16, 1024);
      const uint64_t vd = tc::desc_sw128(smem_addr(smem + C::kOffRing), kSlabV, 1024);
      const uint32_t ts = tmem + i * kTileV, to = tmem + C::kColO + i * D;
      uint32_t nq = 0, np = 0;  // phases; bit b of np: of buffer b
      bool ok = true;
      auto wait_tile = [&](int x) { return wait(&full[x % kSlots], (uint32_t)(x / kSlots) & 1u); };
      for (int k = 0; ok; ++k) {
        if (!(ok = wait(&piece_full[k % kPieces], (uint32_t)(k / kPieces) & 1u))) break;
        const Piece p = pieces[k % kPieces];
        mbar_arrive(&piece_empty[k % kPieces]);
        if (p.j1 < 0) break;
        const int n0 = kUnits * p.j0, e = p.end(i), u = p.u;
        // keys that some row of the half sees
        const int seen =
            min(last_key(p.request(), heads.token(min(p.row0 + (i + 1) * kHalf, p.rows) - 1)) + 1, p.L);
        // the scores of unit n from K tile x, released behind the last unit in it
        auto scores = [&](int n, int x) {
          const uint64_t kt = kd + (x % kSlots) * kTile16 + (n % kUnits) * kUnit16;
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const int off = ((s >> 2) * kSlabV + (s & 3) * 32) / 16;
            tc::mma_bf16(ts + (n % kUnits) * kUnit, qd + off, kt + off, id_s, s > 0);
          }
          tc::commit(&s_full[2 * i + n % kUnits]);
          if ((n + 1) % kUnits == 0 || n + 1 == e) tc::commit(&empty[x % kSlots]);
        };
        if (e > n0) {
          if (!(ok = wait(q_full + i, nq++ & 1u) && wait_tile(u))) break;
          tc::fence_after();
          scores(n0, u);
          if (n0 + 1 < e) scores(n0 + 1, u);
        }
        int x = u + 1;  // the V tile of unit n; K of the next tile is x + 1
        for (int n = n0; n < e; ++n) {
          const int half = n % kUnits;
          if (half == 0 && !(ok = wait_tile(x) && (n + 2 >= e || wait_tile(x + 1)))) break;
          const int steps = (min(kUnit, seen - n * kUnit) + 15) >> 4;
          const uint64_t vt = vd + (x % kSlots) * kTile16 + half * kUnit16;
          const uint32_t tp = ts + half * kUnit;
          if (!(ok = wait(p_full + 2 * i + half, np >> half & 1u))) break;
          np ^= 1u << half;
          tc::fence_after();
          if (steps == kUnit / 16) {
#pragma unroll
            for (int s = 0; s < kUnit / 16; ++s)
              tc::mma_16bit_tmem_a(to, tp + s * 8, vt + s * 128, id_o, n > n0 || s > 0);
          } else {
            for (int s = 0; s < steps; ++s)
              tc::mma_16bit_tmem_a(to, tp + s * 8, vt + s * 128, id_o, n > n0 || s > 0);
          }
          tc::commit(o_done + 2 * i + half);
          if (n + 2 < e) scores(n + 2, x + 1);
          if (half == kUnits - 1 || n + 1 == e) tc::commit(&empty[x % kSlots]);
          x += 2 * half;
        }
        // tiles that only the other half sees
        for (int j = max(p.j0, tiles_of_units(e)); ok && j < p.j1; ++j)
          for (int y = u + 2 * (j - p.j0), z = y + 2; ok && y < z; ++y) {
            ok = wait_tile(y);
            if (ok) tc::commit(&empty[y % kSlots]);
          }
      }
      if (!ok) fail();
      // all that was issued has completed before TMEM is released
      tc::commit(drained);
      if (!mbar_wait_bounded(drained, 0)) fail();
    }
    __syncwarp();
  }
  allow_successor();
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarpV) {
    tc::fence_after();
    tc::dealloc(tmem, kTmemColsV);
  }
}

// The join of cut items: block (c, w) takes the 32 rows of warp w of the item that CTA c leaves
// unfinished, D / 32 float4 columns per warp.
template <typename T, int D>
__global__ void __launch_bounds__(256)
varlen_join_kernel(VarlenAttnArgs a) {
  wait_for_predecessor();
  const int c = blockIdx.x / kSoftWarpsV, w8 = blockIdx.x % kSoftWarpsV;
  const Cut cut = reinterpret_cast<const Cut*>(a.partials)[c];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hpk = a.Hq / a.Hkv;
  const int row0 = cut.row0 + 32 * w8;
  if (cut.count == 0 || row0 >= cut.rows) return;
  const int row = min(row0 + lane, cut.rows - 1), qi = row / hpk;
  T* dst = static_cast<T*>(a.out) + (cut.q0 + qi) * a.out_stride +
           (long)(cut.kvh * hpk + row - qi * hpk) * D;
  join_rows<T, D, D / 32, 4>(
      cut.count,
      [&](int x) { return partial_of<D>(a, c + x, x == 0 ? 1 : 0) + w8 * VCfg<D>::kWarpState; },
      lane, warp * (D / 32), row0 + lane < cut.rows, dst);
}

template <typename T, int D, bool PAGED>
cudaError_t launch_t(const VarlenAttnArgs& a, float scale_log2, cudaStream_t stream) {
  using C = VCfg<D>;
  int unused = 0;
  cudaError_t e = per_device_setup(a.device, &unused, [](int* v) {
    *v = 1;
    cudaFuncAttributes at{};
    const cudaError_t e = cudaFuncGetAttributes(&at, varlen_attention_kernel<T, D, PAGED>);
    if (e != cudaSuccess) return e;
    if (at.numRegs < kRegsV) return cudaErrorInvalidConfiguration;  // too few to redistribute
    return cudaFuncSetAttribute(varlen_attention_kernel<T, D, PAGED>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::bytes(kMaxRequests));
  });
  if (e != cudaSuccess) return e;
  CUtensorMap tk, tv;
  if (PAGED) {
    const long rows = ((long)a.num_pages * a.Hkv) << a.page_shift;
    const int box = a.page_shift < 7 ? 1 << a.page_shift : kTileV;
    if (!encode_bf16_map(&tk, a.k, rows, D, box) || !encode_bf16_map(&tv, a.v, rows, D, box))
      return cudaErrorInvalidValue;
  } else if (!encode_bf16_map(&tk, a.k, a.T, a.Hkv * D, kTileV, a.k_stride) ||
             !encode_bf16_map(&tv, a.v, a.T, a.Hkv * D, kTileV, a.v_stride)) {
    return cudaErrorInvalidValue;
  }
  const int grid = a.num_sms < kMaxGrid ? a.num_sms : kMaxGrid;
  // Cut items joined by their last CTA, from four items per CTA on, or by a second kernel over all SMs:
  // 64 rows over 16,000 keys (0.1 items per CTA) take 63 us by the first and 36 by the second, 700 rows
  // of one prompt (0.6) 30 and 23, 1,200 (1) 34 and 33, 2,400 (2) 66.5 and 68, 4,800 (4) 183 and 189,
  // 7,200 (6) and more the same within their spread; 32 / 8 heads of 128.
  const bool join_here = (long)a.T * a.Hq >= 4L * 2 * kHalf * grid;
  e = launch_pdl(varlen_attention_kernel<T, D, PAGED>, dim3(grid), dim3(kThreadsV), C::bytes(a.B),
                 stream, tk, tv, a, scale_log2, join_here);
  // items of one tile are never cut
  const long keys = PAGED ? (long)a.width << a.page_shift : a.T;
  if (e != cudaSuccess || join_here || keys <= kTileV) return e;
  return launch_pdl(varlen_join_kernel<T, D>, dim3(grid * kSoftWarpsV), dim3(256), 0, stream, a);
}

template <typename T>
cudaError_t launch_form(const VarlenAttnArgs& a, float scale_log2, cudaStream_t stream) {
  if (a.table == nullptr)
    return a.D == 128 ? launch_t<T, 128, false>(a, scale_log2, stream)
                      : launch_t<T, 64, false>(a, scale_log2, stream);
  return a.D == 128 ? launch_t<T, 128, true>(a, scale_log2, stream)
                    : launch_t<T, 64, true>(a, scale_log2, stream);
}

}  // namespace

long varlen_partial_bytes(int D) {
  const long here = kMaxGrid * (long)sizeof(Cut) +
                    kMaxGrid * 2L * (D == 128 ? VCfg<128>::kState : VCfg<64>::kState) * 4;
  const long decode = paged_decode_partial_bytes(D);
  return here > decode ? here : decode;
}

#ifdef KIVI_DEBUG_BUILD
cudaError_t debug_overstate_varlen(unsigned bytes) {
  return cudaMemcpyToSymbol(g_debug_overstate, &bytes, sizeof bytes);
}
#endif

cudaError_t launch_varlen_attention(const VarlenAttnArgs& a, cudaStream_t stream) {
  const float scale = (a.sm_scale > 0.f ? a.sm_scale : 1.f / std::sqrt((float)a.D)) * kLog2eV;
  // Single tokens go to the decode kernel.  Where some request may have more rows than its tile,
  // all of them come here: 30 decoding requests beside two chunks of 509 rows, contexts of 4K, take
  // 127 us in one launch, 16% more as the decode kernel and this one in turn.
  if (a.table != nullptr && is_short(a.max_new, a.Hq / a.Hkv))
    return launch_paged_decode(a, scale, stream);
  return a.dtype == 0 ? launch_form<__nv_bfloat16>(a, scale, stream)
                      : launch_form<__half>(a, scale, stream);
}

}  // namespace kivi
