// What the kernels of the dense attention over a paged cache share: the
// arguments, which cache positions a query sees, and how a score is formed.
//
// A row is one query head of one new token.  Token t of sequence b sits at
// position p = tokens of b before it + its place among b's new tokens; it sees
// the positions [lo, hi) of its sequence,
//   lo = max(0, q_first[t], p + 1 - window),   hi = min(n, max(p + 1, prefix_len[b]))
// (an interval, whatever the masks), and its scores are
//   z(u) = cap tanh(scale q.k_u / cap) - slope_h |p - u|.
// Scores are kept times log2(e), so that every exponential is one exp2.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"

namespace hkv {
namespace pa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
  int B, Hq, Hkv, g;
  int64_t T;                  // rows of q, out and lse
  int max_q;                  // new tokens of a sequence, at most
  const void* q;
  int64_t q_stride;
  const void *K, *V;
  PageMap pm;
  const int32_t* cu;          // [B + 1] first new token of each sequence; null: token b is sequence b's only one
  const int32_t* n_tok;       // [B] tokens in each sequence's own pages
  int64_t n_max;
  const int32_t* prefix_table;  // pages of the shared prefix, null without one
  int64_t n_prefix;             // tokens of the shared prefix
  float scale, softcap;
  int window;
  const float* slopes;
  const int32_t *prefix_len, *q_first;
  void* out;
  float* lse;
  // partials of rows whose positions are split: [part][T * Hq] rows
  float* part_o;
  float2* part_ml;            // running maximum (log2 units) and sum
  int prefix_parts, own_parts;
  int prefix_items;           // items of the prefix that the row kernel takes
  int32_t* status;
  uint64_t wait_ns;
};

// One sequence's new tokens and cache length.
struct Seq {
  int64_t first, n_new, n;  // first row of q, number of them, tokens in the sequence's own pages
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b, bool tell) {
  Seq s;
  s.first = a.cu ? a.cu[b] : b;
  s.n_new = a.cu ? a.cu[b + 1] - s.first : 1;
  s.n = a.n_tok[b];
  bool bad = false;
  if (s.first < 0 || s.n_new < 0 || s.first + s.n_new > a.T) bad = true, s.first = 0, s.n_new = 0;
  if (s.n_new > a.max_q) bad = true, s.n_new = a.max_q;
  if (s.n < 0) bad = true, s.n = 0;
  if (s.n > a.n_max) bad = true, s.n = a.n_max;
  if (bad && tell) report(a.status, HKV_ERR_DEVICE_RANGE);
  return s;
}

struct Span {
  int lo, hi, pos;
};
// Positions seen by new token i of sequence b, whose pages hold all of it.
__device__ __forceinline__ Span span_of(const Args& a, const Seq& s, int b, int64_t i) {
  Span r;
  // more new tokens than the sequence has: positions below zero see nothing but
  // a prefix
  const int64_t p = s.n - s.n_new + i;
  int64_t lo = 0, hi = p + 1;
  if (a.window > 0 && p + 1 - a.window > lo) lo = p + 1 - a.window;
  if (a.q_first) {
    const int64_t f = a.q_first[s.first + i];
    lo = f > lo ? f : lo;
  }
  if (a.prefix_len) {
    const int64_t f = a.prefix_len[b];
    hi = f > hi ? f : hi;
  }
  hi = hi < s.n ? hi : s.n;
  hi = hi > 0 ? hi : 0;
  lo = lo < hi ? lo : hi;
  r.lo = (int)lo, r.hi = (int)hi, r.pos = (int)p;
  return r;
}

// Pool row (of KV head j) that holds token u behind `table`, -1 for a page
// outside the pool.
__device__ __forceinline__ int64_t pool_row(const Args& a, const int32_t* __restrict__ table, uint32_t u, int j) {
  const uint32_t P = a.pm.page_size, at = u / P;
  const int64_t page = table[at];
  if (page < 0 || page >= a.pm.num_pages) return -1;
  return (page * a.Hkv + j) * P + (u - at * P);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The odd minimax polynomial of degree 7 of tanh on [-1/2, 1/2]: absolute error
// 1.6e-7, 2.4e-6 of a small argument.
__device__ constexpr float kTanh[4] = {9.999976754e-01f, -3.332065642e-01f, 1.314514428e-01f, -4.337245598e-02f};
// cap tanh x as cap (1 - 2 / (1 + e^(2x))): off by at most 2^-21 of the cap, up to
// caps of kCoarseCap less than a 30th of the weights' rounding to bf16.
constexpr float kCoarseCap = 64.f;
__device__ __forceinline__ float capped(float x, float cap) {
  return cap - __fdividef(2.f * cap, 1.f + ex2(x * (2.f * kLog2e)));
}
// The same within 2.4e-6 of the result: where x is small the difference above
// would lose what a large cap multiplies (a hundredth of a score at 1e5), so
// the polynomial serves.
__device__ __forceinline__ float capped_fine(float x, float cap) {
  const float u = x * x, small = x * cap * fmaf(u, fmaf(u, fmaf(u, kTanh[3], kTanh[2]), kTanh[1]), kTanh[0]);
  return fabsf(x) <= 0.5f ? small : capped(x, cap);
}

// Sequence of row t: the largest b in [0, B) with cu[b] <= t, found by the
// whole warp, 32 candidates a round.
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, int B, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool le = lane * step < n && (lane == 0 || (int64_t)__ldg(cu + b) <= t);
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int last = 31 - __clz(m);  // bit 0 is always set
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

}  // namespace pa

// Launches a kernel that may be scheduled while the one before it on the stream
// still runs (it waits for that one itself).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid, c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at, c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// The tensor-core kernel (attend_paged_tc.cu): row tiles, splits, launch.
int64_t tc_tiles(const PagedAttend& p, bool prefix);
int tc_splits(const PagedAttend& p, bool prefix, int sms);
int launch_attend_tc(const PagedAttend& p, const pa::Args& a, bool prefix, int splits, int part0, cudaStream_t st);

}  // namespace hkv
