// Dense attention over a paged cache on the tensor cores (bf16): prompts and
// chunks of prompts, and the query heads of a whole batch over a shared prefix.
//
// A CTA owns up to 256 rows (query heads of new tokens) of one KV head, two
// slots of 128, and walks its positions in tiles of 128 tokens:
//   S = Q K^T         tcgen05.mma, bf16 x bf16 -> fp32 in tensor memory
//   P = exp2(S - m)   one thread per row: running maximum m, sum l in fp32, P
//                     rounded to bf16 (one rounding of 2^-9 beside the output's
//                     own) and written over S in tensor memory
//   O += P V          tcgen05.mma with P read from tensor memory, fp32 sums
// The two slots share every K and V tile, so a tile is read once for 256 rows,
// and one slot's softmax runs while the tensor cores work for the other.  O is
// rescaled only when a row's maximum has grown by more than 2^8 (until then
// the old one keeps every exponential within fp32 and bf16 range), which after
// the first tiles is rare, so the softmax threads do it themselves.
// With at most 128 rows both slots take the same rows and every other tile.
//
// What bounds it: the products, 2 x 128 x 128 x 256 flops a tile and slot, and
// beside them as much time of exponentials, which is why a slot weighs scores
// while the other multiplies.  A causal prompt of 8192 tokens (32 query heads, 8
// KV heads) takes 471 us in a burst, 1.17 PFLOP/s or 70% of a large library
// product's rate, and 550 us in a long run under the power cap (1.00); 256
// sequences behind 98304 tokens 382 us (1.08) and 447; the same prompt in eight
// documents 121 us (0.57), whose rows see 1024 tokens at most.  With 256 rows of one
// KV head the tiles' reads (2 x 32 KB for 16.8 MFLOP) stay far below the
// memory's rate.  Where the rows are few or see little (chunks in a window,
// short documents) a CTA's start and end, 7.5 us, and its longest row tile show.
//
// Warps 0-3 and 4-7: softmax of slot 0 and 1; 8: K tiles, 9: V tiles (TMA boxes
// of as many tokens as a page's size allows, or plain loads where a page ends
// inside a swizzle group, at the end of the sequence and at bad pages);
// 10 and 11: the MMAs of slot 0 and 1.
#include <cstdio>
#include <mutex>
#include <type_traits>

#include "attend_paged.cuh"
#include "attend_paged_turns.h"
#include "tc.cuh"

namespace hkv {
namespace {

using pa::Args;
using pa::kKStages;
using pa::kVStages;
using pa::Run;

constexpr int kThreads = 384;
constexpr int kTile = 128;                  // tokens per tile, rows per slot
constexpr uint32_t kHalf = kTile * 128;     // 128 rows x 64 bf16
constexpr uint32_t kBuf = 2 * kHalf;
constexpr int kMaskRing = 8;                // tiles whose valid-token masks are kept
constexpr uint32_t kPolyMask = 0x11;        // of eight pairs of exponentials, the two taken by the polynomial (three: no faster)
constexpr float kGrowth = 8.f;              // rescale when the maximum grows by more than 2^8

struct Layout {
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kBuf;
  static constexpr uint32_t kV = kK + kKStages * kBuf;
  static constexpr uint32_t kMask = kV + kVStages * kBuf;
  static constexpr uint32_t kBars = kMask + kMaskRing * 16;
  static constexpr uint32_t kSeen = kBars + 256;
  static constexpr uint32_t kEnd = kSeen + 64;
};
constexpr size_t kSmem = 1024 + Layout::kEnd;

struct TcArgs {
  Args a;
  int box;       // tokens per TMA box; 0: plain loads only
  int tiles;     // row tiles of 256 (at most), all sequences together
  int splits;
  int part0;     // first partial of this launch; -1: rows are finished here
  int drop;      // testing aid: tiles of keys at the end that are never loaded
};

// ---- instructions beside those of tc.cuh -----------------------------------
// K-major or MN-major 128-byte-swizzled operand with explicit strides: for the
// V tile (tokens x 64-element halves) the fast index is the output column,
// `lbo` leads from one 64-column half to the next, 1024 bytes from 8 tokens to
// the next 8.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D[tmem] (+)= A[tmem] * B[smem], one 128 x 128 x 16 step.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Values from tensor memory are there after the wait only: the empty
// statements make every later use depend on it.
template <int N>
__device__ __forceinline__ void tmem_arrived(uint32_t (&v)[N]) {
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Two fp32 values side by side: one instruction works on both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// NaN if any is: a row that sees a NaN is NaN as a whole.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^x for two x in [-127, 8] without the special-function unit, whose 16
// results a cycle are what a softmax of this shape waits for (128 x 128
// exponentials take it as long as the tensor cores need for the tile's
// products).  x = n + f, n the nearest integer (read off the low bits of
// x + 1.5 * 2^23), 2^f by the degree-4 minimax polynomial on [-1/2, 1/2] with
// constant term 1 (relative error 2.9e-6), n added to the exponent.  At x = -127
// that leaves exactly zero, so scores clamped there count for nothing.
__device__ __forceinline__ float2 exp2_poly(uint64_t x) {
  const float kMagic = 12582912.f;
  const uint64_t r = add2(x, pair(kMagic, kMagic));
  const uint64_t f = fma2(add2(r, pair(-kMagic, -kMagic)), pair(-1.f, -1.f), x);
  uint64_t p = fma2(pair(9.582852945e-03f, 9.582852945e-03f), f, pair(5.590642616e-02f, 5.590642616e-02f));
  p = fma2(p, f, pair(2.402409911e-01f, 2.402409911e-01f));
  p = fma2(p, f, pair(6.931241751e-01f, 6.931241751e-01f));
  p = fma2(p, f, pair(1.f, 1.f));
  const float2 n = unpair(r), v = unpair(p);
  return make_float2(__int_as_float(__float_as_int(v.x) + (__float_as_int(n.x) << 23)),
                     __int_as_float(__float_as_int(v.y) + (__float_as_int(n.y) << 23)));
}
// cap * tanh(f v) for |f v| <= 1/2, as v * (c0 + c1 v^2 + c2 v^4 + c3 v^6): the
// polynomial of pa::capped, with f and cap multiplied into its coefficients once.
struct CapPoly {
  float c[4];
  __device__ __forceinline__ CapPoly(float f, float cap) {
    float power = f * cap;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = pa::kTanh[i] * power, power *= f * f;
  }
  __device__ __forceinline__ uint64_t factor(uint64_t v) const {
    const uint64_t u = mul2(v, v);
    uint64_t p = pair(c[3], c[3]);
#pragma unroll
    for (int i = 2; i >= 0; --i) p = fma2(p, u, pair(c[i], c[i]));
    return p;
  }
};
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Bounded wait as tc::mbar_wait, but the clock (whose read takes longer than
// most waits here) and the abort flag are looked at once in 64 tries.
__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (int i = 1;; ++i) {
    if (tc::mbar_try_wait(b, parity)) return true;
    if (i % 64 == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort) return false;
      if (now - t0 > limit_ns) {
        *abort = 1;
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool all(bool x) { return __all_sync(0xffffffffu, x); }
// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Barrier of the two softmax warpgroups.
__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The tile's rows, found by every warp for itself.
template <bool kPrefix>
__device__ __forceinline__ bool find_tile(const Args& a, int tile, int& b, int64_t& r0, pa::Seq& s) {
  if constexpr (kPrefix) {
    b = 0, s = pa::Seq{0, a.T, 0}, r0 = (int64_t)tile * 2 * kTile;
    return r0 < a.T * a.g;
  } else {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      pa::Seq mine{0, 0, 0};
      if (b0 + lane < a.B) mine = pa::seq_of(a, b0 + lane, false);
      const int n = (int)((mine.n_new * a.g + 2 * kTile - 1) / (2 * kTile));
      int upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, base + upto > tile);
      if (m) {
        const int l = __ffs(m) - 1;
        b = b0 + l;
        s = pa::seq_of(a, b, false);
        const int before = base + __shfl_sync(0xffffffffu, upto - n, l);
        r0 = (int64_t)(tile - before) * 2 * kTile;
        return true;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
  }
}

// The K or the V tiles of a CTA, brought in by one warp: by TMA where a tile is
// whole and its pages are cut into boxes, else row by row with cp.async, whose
// arrival this warp sees to one tile later (the tile before is complete while
// this one is on its way).
struct Loader {
  const TcArgs& t;
  const void* pool;
  const CUtensorMap* map;
  const int32_t* __restrict__ table;
  int n_tok, j;              // tokens behind the table, KV head
  int lo, hi;                // positions that some row sees: the places of others need not exist
  // tiles that start before this position are not read whole.  What lies before
  // the first seen position, in the page that the table names for it, may be
  // NaN; a key's score is masked then, but a weight of zero does not undo a value
  int least;
  int32_t rows[4];           // pool rows of tokens lane, lane + 32, + 64, + 96 of a tile, -1: none
  uint64_t* pending = nullptr;  // the barrier of the tile whose copies have not been waited for

  __device__ __forceinline__ void look(int n) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = n * kTile + 32 * k + (threadIdx.x & 31);
      rows[k] = u >= lo && u < hi ? (int32_t)pa::pool_row(t.a, table, u, j) : -1;
      if (u >= lo && u < hi && rows[k] < 0) report(t.a.status, HKV_ERR_DEVICE_RANGE);
    }
  }
  // Copies of the pending tile have landed, but for the newest `kLater` groups.
  template <int kLater>
  __device__ __forceinline__ void settle() {
    if (pending == nullptr) return;
    asm volatile("cp.async.wait_group %0;" ::"n"(kLater) : "memory");
    async_fence();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(pending);
    pending = nullptr;
  }
  // Tile n into `dst`; `bar` completes when it is there.  `valid` gets the mask
  // of tokens that have a place.
  __device__ __forceinline__ void load(int n, int end, unsigned char* dst, uint64_t* bar, uint4* valid) {
    const int lane = threadIdx.x & 31;
    if (t.box > 0) {
      const int boxes = kTile / t.box;  // at most 16
      int32_t row = 0;
      bool ok = n * kTile >= least && (n + 1) * kTile <= n_tok;
      if (ok && lane < boxes) {
        row = (int32_t)pa::pool_row(t.a, table, n * kTile + lane * t.box, j);
        ok = row >= 0;
      }
      if (__all_sync(0xffffffffu, ok)) {
        settle<0>();
        if (lane == 0) {
          if (valid) *valid = make_uint4(~0u, ~0u, ~0u, ~0u);
          tc::mbar_expect_tx(bar, kBuf);
        }
        __syncwarp();
        if (lane < boxes) {
          tc::tma_load_2d(dst + lane * t.box * 128, map, 0, row, bar);
          tc::tma_load_2d(dst + kHalf + lane * t.box * 128, map, 64, row, bar);
        }
        return;
      }
      look(n);
    }
    uint32_t mask[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) mask[k] = __ballot_sync(0xffffffffu, rows[k] >= 0);
    if (valid && lane == 0) *valid = make_uint4(mask[0], mask[1], mask[2], mask[3]);
    const int c = lane & 15;  // 16-byte piece of a row
    const uint32_t to = tc::smem_u32(dst) + (c >> 3) * kHalf;
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(pool) + c * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll 4
      for (int e = lane >> 4; e < 32; e += 2) {
        const int32_t row = __shfl_sync(0xffffffffu, rows[k], e);
        const int x = 32 * k + e;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + x * 128 + (((c & 7) ^ (x & 7)) << 4)),
                     "l"(from + (row < 0 ? 0 : (int64_t)row * kHeadDim)), "r"(row < 0 ? 0 : 16)
                     : "memory");
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
    settle<1>();
    pending = bar;
    if (t.box == 0 && n + 1 < end) look(n + 1);
  }
};

// How scores are formed: scaled only; capped too; with a bias by distance (and
// a cap or a scale of any sign).
enum { kPlain = 0, kCapped = 1, kBiased = 2 };

// kFineCap: the cap is past pa::kCoarseCap.  An instance each: a choice inside made
// the code of the softmax longer (capped scores behind a prefix: 61 -> 65 us).
template <bool kPrefix, int kMode, bool kFineCap>
__global__ void __launch_bounds__(kThreads, 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ TcArgs t) {
  const Args& a = t.a;
  constexpr uint32_t kIdescS = tc::idesc_bf16_f32(kTile, kTile);
  constexpr uint32_t kIdescO = kIdescS | (1u << 16);  // B (V) with the output column as its fast index
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  uint4* valid_s = reinterpret_cast<uint4*>(smem + Layout::kMask);
  int2* seen_s = reinterpret_cast<int2*>(smem + Layout::kSeen);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Layout::kBars);
  uint64_t* k_full = bars;                    // [kKStages]
  uint64_t* k_empty = k_full + kKStages;
  uint64_t* v_full = k_empty + kKStages;      // [kVStages]
  uint64_t* v_empty = v_full + kVStages;
  uint64_t* s_full = v_empty + kVStages;      // [slot] S in tensor memory
  uint64_t* p_full = s_full + 2;              // [slot] P in tensor memory, O rescaled
  uint64_t* p_half = p_full + 2;              // [slot] the same for the first 64 tokens
  uint64_t* o_done = p_half + 2;              // [slot] O holds the tile
  uint64_t* idle = o_done + 2;                // [slot] every MMA issued has finished
  uint64_t* turn = idle + 2;                  // [slot] the other slot is through with its exponentials
  uint64_t* q_full = turn + 2;                // [slot] queries in shared memory
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv;
  const int split = rest % t.splits, tile = t.tiles - 1 - rest / t.splits;  // long causal tiles first
  int b;
  int64_t r0;
  pa::Seq seq;
  if (!find_tile<kPrefix>(a, tile, b, r0, seq)) return;
  if (threadIdx.x == 0 && r0 == 0 && split == 0 && j == 0 && !kPrefix) pa::seq_of(a, b, true);  // report a cut length
  const int nrows = (int)min((int64_t)2 * kTile, seq.n_new * a.g - r0);
  const bool both = nrows > kTile;  // the slots hold different rows and share every tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKStages; ++i) tc::mbar_init(&k_full[i], 1), tc::mbar_init(&k_empty[i], both ? 2 : 1);
    for (int i = 0; i < kVStages; ++i) tc::mbar_init(&v_full[i], 1), tc::mbar_init(&v_empty[i], both ? 2 : 1);
    for (int i = 0; i < 2; ++i) {
      const int rows = both ? min(kTile, nrows - i * kTile) : nrows;
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&p_full[i], (rows + 31) / 32);  // a warp each; those without a row take no part
      tc::mbar_init(&p_half[i], (rows + 31) / 32);
      tc::mbar_init(&o_done[i], 1);
      tc::mbar_init(&idle[i], 1);
      tc::mbar_init(&turn[1 - i], (rows + 31) / 32);  // a warp of slot i each
      tc::mbar_init(&q_full[i], (rows + 31) / 32);
    }
    *abort = 0;
    tc::mbar_init_fence();
  }
  if (warp == 10) tc::tmem_alloc(tmem_slot, 512);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // what comes next may take the SMs that are free
  // What the softmax threads' rows see, and from the first position to the last
  // what their warps do.
  const int g = a.g, row_base = (int)r0;  // r0 + 255 < T * g < 2^31
  const int row = both ? threadIdx.x : (threadIdx.x & (kTile - 1));
  const bool live = warp < 8 && row < nrows;
  const int tok = (row_base + row) / g;  // new token within its sequence
  pa::Span sp{0, INT32_MAX, 0};  // rows that are only padding see everything: no masks for their sake
  if (live) {
    if constexpr (kPrefix) {
      const int64_t n = min((int64_t)max(a.n_tok[tok], 0), a.n_max);
      sp = pa::Span{0, (int)a.n_prefix, (int)(a.n_prefix + n - 1)};
    } else {
      sp = pa::span_of(a, seq, b, tok);
    }
  }
  if (!kPrefix && warp < 8) {
    const bool sees = live && sp.lo < sp.hi;
    const int lo = __reduce_min_sync(0xffffffffu, sees ? sp.lo : INT32_MAX);
    const int hi = __reduce_max_sync(0xffffffffu, sees ? sp.hi : 0);
    if (lane == 0) seen_s[warp] = make_int2(lo, hi);
  }
  const int n_all = kPrefix ? (int)a.n_prefix : (int)seq.n;
  const int32_t* table = kPrefix ? a.prefix_table : a.pm.table + (int64_t)b * a.pm.max_pages;
  if (warp == 8 && lane < 8) {  // the page ids of the first tiles (about), while the barriers are set up
    const int from = kPrefix ? 0 : pa::span_of(a, seq, b, row_base / g).lo / kTile;
    const int to = ((kPrefix ? n_all : pa::span_of(a, seq, b, (row_base + nrows - 1) / g).hi) + kTile - 1) / kTile;
    const int at = from + split * ((max(to - from, 0) + t.splits - 1) / t.splits) + lane;
    if (at < to) asm volatile("prefetch.global.L2 [%0];" ::"l"(table + (uint32_t)at * kTile / (uint32_t)a.pm.page_size));
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  auto seen_by = [&](int s, int& lo, int& hi) {
    lo = 0, hi = n_all;
    if constexpr (!kPrefix) {
      const int2* w = seen_s + (both ? 4 * s : 0);
      lo = min(min(w[0].x, w[1].x), min(w[2].x, w[3].x)), hi = max(max(w[0].y, w[1].y), max(w[2].y, w[3].y));
      lo = min(lo, hi);
    }
  };
  int lo0, hi0, lo1, hi1;
  seen_by(0, lo0, hi0);
  seen_by(1, lo1, hi1);
  // tiles of the CTA, then this split's run of them
  const int lo = hi0 <= lo0 ? lo1 : hi1 <= lo1 ? lo0 : min(lo0, lo1), hi = max(hi0 > lo0 ? hi0 : 0, hi1 > lo1 ? hi1 : 0);
  const int first = lo < hi ? lo / kTile : 0, last = lo < hi ? (hi + kTile - 1) / kTile : 0;
  const int per = (last - first + t.splits - 1) / t.splits;
  const int t0 = first + split * per, t1 = min(last, t0 + per);
  // the tiles that a slot works on
  auto run_of = [&](int s) -> Run {
    if (!both) return Run{t0 + s, t1, 2};
    const int l = s ? lo1 : lo0, h = s ? hi1 : hi0;
    if (h <= l) return Run{t1, t1, 1};
    return Run{max(t0, l / kTile), min(t1, (h + kTile - 1) / kTile), 1};
  };

  // The softmax threads hold a row's 128 scores: of the launch's 384 x 168
  // registers 2 x 128 x 200 go to them, 128 x 104 stay with the others.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp < 10) {
      // ---------------- K and V tiles ----------------
      const bool is_k = warp == 8;
      const int stages = is_k ? kKStages : kVStages;
      uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
      unsigned char* ring = smem + (is_k ? Layout::kK : Layout::kV);
      const CUtensorMap* map = is_k ? &kmap : &vmap;
      if (t.box > 0 && lane == 0) tc::tma_prefetch_map(map);
      Loader ld{t, is_k ? a.K : a.V, map, table, n_all, j, lo, hi, is_k ? 0 : lo, {-1, -1, -1, -1}};
      if (t.box == 0 && t0 < t1) ld.look(t0);
      int stage = 0, armed = 0;
      uint32_t phase = 0;
      for (int n = t0; n < t1 - (is_k ? t.drop : 0); ++n) {
        if (!all(tc::mbar_try_wait(&empty[stage], phase ^ 1u))) {
          ld.settle<0>();  // what waits for the tile before may be what this one waits for
          if (!all(wait(&empty[stage], phase ^ 1u, abort, a.wait_ns))) break;
        }
        ld.load(n, t1, ring + stage * kBuf, &full[stage], is_k ? &valid_s[(n - t0) % kMaskRing] : nullptr);
        ++armed;
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
      ld.settle<0>();
      // on an abort, let every load already issued land before the CTA leaves
      if (*abort && lane == 0)
        for (int n = max(0, armed - stages); n < armed; ++n) tc::mbar_drain(&full[n % stages], (n / stages) & 1, a.wait_ns);
    } else {
      // ---------------- MMAs ----------------
      // the whole warp goes through the loop and one elected thread issues, so
      // that addresses and descriptors stay in uniform registers (issued from a
      // branch of one lane, eight MMAs took 800 cycles instead of 512)
      const int s = __shfl_sync(0xffffffffu, warp, 0) - 10;
      const uint32_t s_tmem = __shfl_sync(0xffffffffu, tmem, 0) + s * 256, o_tmem = s_tmem + kTile;
      const uint64_t q_desc = tc::sw128_desc(tc::smem_u32(smem + Layout::kQ) + (both ? s : 0) * kBuf);
      const uint64_t k_desc0 = tc::sw128_desc(tc::smem_u32(smem + Layout::kK));
      const uint64_t v_desc0 = sw128_desc_mn(tc::smem_u32(smem + Layout::kV), kHalf);
      const Run run = run_of(s);
      int done = 0, ks = 0, vs = 0;
      uint32_t kph = 0, vph = 0;
      auto advance = [&](int by) {
        if ((ks += by) >= kKStages) ks -= kKStages, kph ^= 1u;
        if ((vs += by) >= kVStages) vs -= kVStages, vph ^= 1u;
      };
      // tiles that only the other slot needs are given back as they come
      auto pass = [&](int from, int to) -> bool {
        for (int n = from; n < to; ++n) {
          if (!all(wait(&k_full[ks], kph, abort, a.wait_ns))) return false;
          if (lane == 0) tc::mbar_arrive(&k_empty[ks]);
          if (!all(wait(&v_full[vs], vph, abort, a.wait_ns))) return false;
          if (lane == 0) tc::mbar_arrive(&v_empty[vs]);
          advance(1);
        }
        return true;
      };
      bool ok = true;
      if (both)
        ok = pass(t0, min(t1, run.first));
      else if (s == 1)
        advance(1);
      auto issue_s = [&](int stage) {
        const uint64_t k_desc = k_desc0 + stage * (kBuf >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t at = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          tc::mma_bf16(s_tmem, q_desc + at, k_desc + at, kIdescS, kk != 0);
        }
        tc::mma_commit(&s_full[s]);
        tc::mma_commit(&k_empty[stage]);
      };
      if (ok && run.first < run.last) {
        ok = all(wait(&q_full[both ? s : 0], 0, abort, a.wait_ns)) && all(wait(&k_full[ks], kph, abort, a.wait_ns));
        tc::fence_after_sync();
        if (ok && elected()) issue_s(ks);
        __syncwarp();
      }
      for (int n = run.first; ok && n < run.last; n += run.step) {
        const int v_at = vs;
        if (!(ok = all(wait(&v_full[vs], vph, abort, a.wait_ns)))) break;
        advance(run.step);
        const bool more = n + run.step < run.last;
        if (more && !(ok = all(wait(&k_full[ks], kph, abort, a.wait_ns)))) break;
        const uint64_t v_desc = v_desc0 + v_at * (kBuf >> 4);
        if (!(ok = all(wait(&p_half[s], done & 1, abort, a.wait_ns)))) break;
        tc::fence_after_sync();
        if (elected()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(o_tmem, s_tmem + kk * 8, v_desc + kk * (16 * 128 >> 4), kIdescO, (done | kk) != 0);
        }
        __syncwarp();
        if (!(ok = all(wait(&p_full[s], done & 1, abort, a.wait_ns)))) break;
        tc::fence_after_sync();
        if (elected()) {
#pragma unroll
          for (int kk = 4; kk < 8; ++kk)
            mma_bf16_ts(o_tmem, s_tmem + kk * 8, v_desc + kk * (16 * 128 >> 4), kIdescO, 1u);
          tc::mma_commit(&v_empty[v_at]);
          tc::mma_commit(&o_done[s]);
          // the next tile's S overwrites this one's P: MMAs of one thread run in order
          if (more) issue_s(ks);
        }
        __syncwarp();
        ++done;
      }
      if (ok && both) pass(max(run.last, run.first), t1);
      if (elected()) {
        tc::mma_commit(&idle[s]);
        tc::mbar_drain(&idle[s], 0, a.wait_ns);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---------------- softmax: one row per thread ----------------
    const int slot = warp >> 2, head = (row_base + row) % g;
    const bool active = (both ? warp : warp & 3) * 32 < nrows;
    const int64_t my_out = (seq.first + tok) * a.Hq + j * g + head;     // row of out
    if (active && (both || slot == 0)) {
      // queries to shared memory, two rows at a time
      const int64_t my_q = (seq.first + tok) * a.q_stride + (int64_t)(j * g + head) * kHeadDim;
      const int c = lane & 15, x0 = row & (kTile - 32);
      const uint32_t dst = tc::smem_u32(smem + Layout::kQ) + slot * kBuf + (c >> 3) * kHalf;
#pragma unroll 1
      for (int x = lane >> 4; x < 32; x += 2) {
        const int64_t at = __shfl_sync(0xffffffffu, my_q, x);
        const bool in = row - lane + x < nrows;  // rows behind the last one are zeros
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (in ? at + c * 8 : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (x0 + x) * 128 + (((c & 7) ^ (x & 7)) << 4)),
                     "l"(src), "r"(in ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      async_fence();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&q_full[slot]);
    }
    // tiles within [all_lo, all_hi) are seen whole by every row of the warp
    const int all_lo = __reduce_max_sync(0xffffffffu, sp.lo), all_hi = __reduce_min_sync(0xffffffffu, sp.hi);
    const uint32_t s_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16) + slot * 256, o_tmem = s_tmem + kTile;
    float m = -INFINITY, l = 0.f;
    int done = 0;  // tiles that this slot has been through
    const Run run = run_of(slot);
    const pa::Turns turns = pa::turns_of(run, run_of(1 - slot), both);
    int at_turn = -turns.from;
    // a score in units of log2(e) is value * c: value is q.k, or its tanh, or
    // (biased) the score itself
    const float to_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f, cap = a.softcap * pa::kLog2e;
    const float c = kMode == kPlain ? a.scale * pa::kLog2e : kMode == kCapped ? cap : 1.f;
    const CapPoly poly(to_cap, cap);
    const float slope = kMode == kBiased && a.slopes && live ? a.slopes[j * a.g + head] * pa::kLog2e : 0.f;
    for (int n = run.first; active && n < run.last; n += run.step) {
      const bool ok = wait(&s_full[slot], done & 1, abort, a.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::fence_after_sync();
      const int u0 = n * kTile;
      const uint4 there = valid_s[(n - t0) % kMaskRing];
      const bool masked = all_lo > u0 || all_hi < u0 + kTile || (there.x & there.y & there.z & there.w) != ~0u;
      // Scores that are more than a multiple of the products are formed first
      // and go back to tensor memory.  Loops over 32 columns stay rolled: a
      // row's 128 scores in registers meant spills and code that the
      // instruction cache could not hold, and reading them again is cheap.
      auto form = [&] {
        const float d0 = (float)(sp.pos - u0);
        const uint32_t w[4] = {there.x, there.y, there.z, there.w};
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t v[32];
          tc::tmem_ld32(s_tmem + 32 * k, v);
          tmem_arrived(v);
          const uint32_t in = k == 0 ? w[0] : k == 1 ? w[1] : k == 2 ? w[2] : w[3];
          const int lo = min(max(sp.lo - u0 - 32 * k, 0), 32), hi = min(max(sp.hi - u0 - 32 * k, 0), 32);
          // bit i: token i is seen
          const uint32_t see = masked ? in & (uint32_t)((1ull << hi) - 1) & ~(uint32_t)((1ull << lo) - 1) : ~0u;
          const float d = d0 - (float)(32 * k);
          if (kMode != kPlain && cap > 0.f) {
            const float size = kMode == kBiased ? cap : 1.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = __uint_as_float(v[i]) * to_cap;
              v[i] = __float_as_uint(kFineCap ? pa::capped_fine(x, size) : pa::capped(x, size));
            }
          }
          const float by = cap > 0.f ? 1.f : a.scale * pa::kLog2e;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float z = __uint_as_float(v[i]);
            if (kMode == kBiased) z = fmaf(-slope, fabsf(d - (float)i), z * by);
            v[i] = see >> i & 1u ? __float_as_uint(z) : 0xff800000u;  // -inf
          }
          tmem_st32(s_tmem + 32 * k, v);
        }
        tmem_wait_st();
      };
      bool formed = kMode == kBiased || masked;
      if (formed) form();
      float top, low;
      auto extremes = [&] {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, mn[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          uint32_t v[2][32];
          tc::tmem_ld32(s_tmem + 32 * k, v[0]);
          tc::tmem_ld32(s_tmem + 32 * k + 32, v[1]);
          tmem_arrived(v[0]);
          tmem_arrived(v[1]);
#pragma unroll
          for (int i = 0; i < 32; i += 2)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int q = h * 2 + (i >> 1 & 1);
              mx[q] = max3(mx[q], __uint_as_float(v[h][i]), __uint_as_float(v[h][i + 1]));
              if (kMode == kCapped) mn[q] = min3(mn[q], __uint_as_float(v[h][i]), __uint_as_float(v[h][i + 1]));
            }
        }
        top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]), low = min3(min3(mn[0], mn[1], mn[2]), mn[3], mn[3]);
      };
      extremes();
      if constexpr (kMode == kCapped) {
        // the polynomial serves while the warp's scores are below half the cap
        if (!formed && !all(fmaxf(top, -low) * fabsf(to_cap) <= 0.5f)) {
          form(), formed = true;
          extremes();
        }
        if (!formed) {
          const float x = to_cap > 0.f ? top : low;
          top = x * unpair(poly.factor(pair(x, x))).x / c;
        }
      }
      top *= c;  // c is positive: the largest value is the largest score
      const bool grown = !(top <= m + kGrowth);  // from nothing to something, and to NaN, too
      if (__any_sync(0xffffffffu, grown)) {
        float f = 1.f;
        if (grown) f = pa::ex2(m - top), l *= f, m = top;  // m = -inf: 0
        if (done > 0) {
          const bool ok2 = wait(&o_done[slot], (done - 1) & 1, abort, a.wait_ns);
          if (!__all_sync(0xffffffffu, ok2)) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tc::tmem_ld32(o_tmem + 32 * k, o);
            tmem_arrived(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(o_tmem + 32 * k, o);
          }
        }
      }
      // One slot's exponentials at a time: together they would take as long, and
      // the tensor cores would wait for both instead of working for the other.
      const bool in_turn = (unsigned)at_turn < (unsigned)turns.n;
      if (in_turn && (slot == 1 || at_turn > 0)) {
        const bool ok3 = wait(&turn[slot], (slot == 1 ? at_turn : at_turn - 1) & 1, abort, a.wait_ns);
        if (!__all_sync(0xffffffffu, ok3)) break;
      }
      const float off = m == -INFINITY ? 0.f : m;
      uint64_t sum[2] = {0, 0};
      const uint64_t c2 = pair(c, c), off2 = pair(-off, -off);
      // 32 scores to weights
      auto weigh = [&](const uint32_t(&v)[32], int k, auto raw) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint64_t z = pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          float2 x = unpair(fma2(z, decltype(raw)::value ? poly.factor(z) : c2, off2));
          if (kPolyMask >> (i % 8) & 1)
            x = exp2_poly(pair(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f)));
          else
            x = make_float2(pa::ex2(x.x), pa::ex2(x.y));
          sum[i & 1] = add2(sum[i & 1], pair(x.x, x.y));
          p[i] = pack_bf16(x.x, x.y);
        }
        tmem_st16(s_tmem + 16 * k, p);  // behind the columns still to be read
      };
      auto weigh_all = [&](auto raw) {
        // the next 32 columns are on their way while these are weighed
        uint32_t va[32], vb[32], vc[32], vd[32];
        tc::tmem_ld32(s_tmem, va);
        tmem_arrived(va);
        tc::tmem_ld32(s_tmem + 32, vb);
        weigh(va, 0, raw);
        tmem_arrived(vb);
        tc::tmem_ld32(s_tmem + 64, vc);
        weigh(vb, 1, raw);
        tmem_arrived(vc);
        // P V may start on these 64 tokens
        tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_half[slot]);
        tc::tmem_ld32(s_tmem + 96, vd);
        weigh(vc, 2, raw);
        tmem_arrived(vd);
        weigh(vd, 3, raw);
      };
      if (kMode == kCapped && !formed)
        weigh_all(std::true_type{});
      else
        weigh_all(std::false_type{});
      const float2 both_sums = unpair(add2(sum[0], sum[1]));
      l += both_sums.x + both_sums.y;
      __syncwarp();
      if (in_turn && lane == 0) tc::mbar_arrive(&turn[1 - slot]);
      tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&p_full[slot]);
      ++done, ++at_turn;
    }
    tmem_wait_st();  // a loop left on an abort may have stores on their way
    if (done > 0) {
      const bool ok = wait(&o_done[slot], (done - 1) & 1, abort, a.wait_ns);
      __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
    }
    // ---- results ----
    float scale1 = 0.f;  // weight of the other slot's O, when it has the same rows
    float* const other = reinterpret_cast<float*>(smem + Layout::kK);  // [128 columns][128 rows], then m, l
    if (!both) {
      softmax_barrier();  // every MMA has finished: the tiles' memory is free
      if (slot == 1 && active) {
        other[kTile * kTile + row] = m, other[kTile * kTile + kTile + row] = l;
        if (done > 0) {
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tc::tmem_ld32(o_tmem + 32 * k, o);
            tmem_arrived(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) other[(32 * k + i) * kTile + row] = __uint_as_float(o[i]);
          }
        }
      }
      softmax_barrier();
    }
    if (active && (both || slot == 0) && all(*abort == 0)) {
      float scale0 = 1.f;
      if (!both) {
        const float m1 = other[kTile * kTile + row], l1 = other[kTile * kTile + kTile + row];
        const float top = max3(m, m1, m1);
        scale0 = m == -INFINITY ? 0.f : pa::ex2(m - top);
        scale1 = m1 == -INFINITY ? 0.f : pa::ex2(m1 - top);
        l = l * scale0 + l1 * scale1, m = top;
      }
      const bool partial = t.part0 >= 0;
      const bool none = m == -INFINITY;  // nothing seen: O was never written, or is zero
      const float inv = partial ? 1.f : none ? 0.f : 1.f / l;
      const int64_t out_row = (partial ? (t.part0 + split) * a.T * a.Hq : 0) + my_out;
      if (live && partial) a.part_ml[out_row] = make_float2(m, none ? 0.f : l);
      if (live && !partial && a.lse) a.lse[out_row] = none ? -INFINITY : (m + log2f(l)) * pa::kLn2;
      // one weight for the row's values: the sum, and in the other slot's favour
      const float w0 = none ? 0.f : scale0 * inv, w1 = none ? 0.f : scale1 * inv;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t o[32];
        tc::tmem_ld32(o_tmem + 32 * k, o);
        tmem_arrived(o);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = w0 != 0.f ? __uint_as_float(o[i]) * w0 : 0.f;
        if (w1 != 0.f)
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = fmaf(other[(32 * k + i) * kTile + row], w1, x[i]);
        // a thread writes its own row, 64 or 128 bytes a step: whole lines by
        // way of shared memory took as long
        if (live && partial) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + out_row * kHeadDim + 32 * k);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        } else if (live) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + out_row * kHeadDim + 32 * k);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                                pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *abort) report(a.status, HKV_ERR_TIMEOUT);
  if (warp == 10) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_free(tmem, 512);
  }
  // launched while the own tokens' kernel may still run: whatever waits for
  // this grid waits for that one too
  if constexpr (kPrefix) asm volatile("griddepcontrol.wait;" ::: "memory");
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const TcArgs);
template <int kMode, bool kFineCap>
Kernel pick(bool prefix) {
  return prefix ? attend_tc_kernel<true, kMode, kFineCap> : attend_tc_kernel<false, kMode, kFineCap>;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// The pool as rows of 128 bf16, read in boxes of `box` rows x 64 columns.
int pool_map(CUtensorMap* map, const void* pool, int64_t rows, int box) {
  EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return fail(HKV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kHeadDim * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, ones[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, boxes, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? HKV_OK : fail(HKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

}  // namespace

// Row tiles of all sequences together, at most: a sequence's last tile may be
// partly filled.
int64_t tc_tiles(const PagedAttend& p, bool prefix) {
  const int64_t rows = p.T * (p.Hq / p.Hkv);
  return prefix ? ceil_div(rows, 2 * kTile) : rows / (2 * kTile) + (p.B < p.T ? p.B : p.T);
}

// Runs that the positions are cut into.  A prefix is cut to take the least time
// on `sms` SMs: whole waves of CTAs, each 7.5 us and 1.75 us for a tile of 128
// tokens (half of it where a CTA's two slots take turns), and the joining of
// parts at 4 TB/s.  Prompts, whose rows mostly see different lengths, are cut
// only where they leave SMs idle, down to two tiles.
int tc_splits(const PagedAttend& p, bool prefix, int sms) {
  if (sms < 1) sms = 1;  // no device (sizes only), or one whose SMs are all spoken for
  const int64_t ctas = tc_tiles(p, prefix) * p.Hkv;
  if (!prefix) {
    const int64_t most = ceil_div(p.n_max, 2 * kTile);
    int64_t s = sms / (ctas < 1 ? 1 : ctas);
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s);
  }
  const int64_t tiles = ceil_div(p.n_prefix, kTile);
  const double tile_us = p.T * (p.Hq / p.Hkv) > kTile ? 1.75 : 0.9, part_us = (double)p.T * p.Hq * 512 / 4e6;
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= 64 && s <= tiles; ++s) {
    const double t = (double)ceil_div(ctas * s, sms) * ((double)ceil_div(tiles, s) * tile_us + 7.5) + s * part_us;
    if (t < least) least = t, best = s;
  }
  return best;
}

int launch_attend_tc(const PagedAttend& p, const pa::Args& a, bool prefix, int splits, int part0, cudaStream_t st) {
  TcArgs t{a, 0, (int)tc_tiles(p, prefix), splits, part0, debug_flags() & kDebugDropTile ? 1 : 0};
  // the largest power of two that divides the page: a box never leaves its
  // page, and whole swizzle groups of 8 rows keep the tile's layout
  int box = p.pm.page_size & -p.pm.page_size;
  box = box < kTile ? box : kTile;
  const int64_t rows = p.pm.num_pages * p.Hkv * p.pm.page_size;
  alignas(64) CUtensorMap kmap{}, vmap{};
  if (box >= 8 && rows <= INT32_MAX) {
    int rc = pool_map(&kmap, p.K_pool, rows, box);
    if (rc == HKV_OK) rc = pool_map(&vmap, p.V_pool, rows, box);
    if (rc != HKV_OK) return rc;
    t.box = box;
  }
  const int mode = a.slopes != nullptr || (!(a.scale > 0.f) && a.softcap == 0.f) ? kBiased : a.softcap > 0.f ? kCapped : kPlain;
  const bool fine = a.softcap > pa::kCoarseCap;
  auto kernel = mode == kPlain ? pick<kPlain, false>(prefix)
                : mode == kCapped ? (fine ? pick<kCapped, true>(prefix) : pick<kCapped, false>(prefix))
                                  : (fine ? pick<kBiased, true>(prefix) : pick<kBiased, false>(prefix));
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return cuda_check(e, "attention smem attribute");
  const int64_t grid = (int64_t)t.tiles * splits * p.Hkv;
  if (grid > INT32_MAX) return fail(HKV_ERR_UNSUPPORTED, "too many row tiles (%lld)", (long long)grid);
  if (prefix) e = launch_after(kernel, dim3((unsigned)grid), kThreads, kSmem, st, kmap, vmap, t);  // beside the own tokens' kernel
  else kernel<<<(unsigned)grid, kThreads, kSmem, st>>>(kmap, vmap, t), e = cudaGetLastError();
  return cuda_check(e, "attention launch");
}

}  // namespace hkv
