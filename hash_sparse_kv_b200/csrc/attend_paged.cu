// Dense attention over a paged cache for few rows at a time: the single-token
// (decode) form of the prompt attention, the own tokens of sequences behind a
// shared prefix, a short prefix itself, and everything in fp32.
//
// An item is up to 16 rows of one KV head (the g query heads of 16 / g new
// tokens) and one run of their cache positions.  A warp goes through items on
// its own, reads each run once and keeps the softmax's running maximum and sum
// and the weighted values in registers (fp32).  Where few items would be left,
// the positions are cut into more runs and a second launch joins their partial
// results.
//
// K and V arrive by cp.async in steps of 8 KB (16 tokens in bf16, 8 in fp32),
// two steps ahead, and the loads run on into the warp's next item while this
// one is finished, so that the eight warps of an SM keep 128 KB on their way
// without ever waiting for each other.  The work is bound by reading K and V: a
// 128-row tcgen05 tile would be seven eighths padding, so scores and products
// are mma.sync with the 16 rows as M.  64 sequences of 4259 to 8172 tokens
// (bf16, capped scores) take 284 to 288 us, 5.7 TB/s.  fp32 is bound by the
// latency of its three dependent products instead: chunks of 47, 41 and 35
// tokens behind 520 to 893 take 25 us, 16 single tokens over 4344 to 8088 tokens
// 234 us, 3.5 TB/s.
//   bf16: m16n8k16; P is rounded to bf16 for the product, sums stay fp32.
//   fp32: m16n8k8 tf32 in three products.  x = hi + lo, both of tf32's 11 bits;
//         hi hi + hi lo + lo hi leaves out lo lo (2^-22 of a product at most)
//         and the rounding of both lo (2^-21.5 each), without a sign of their own.
#include <cstdio>

#include "attend_paged.cuh"

namespace hkv {
namespace {

using pa::Args;

constexpr int kRows = 16;

__device__ __forceinline__ void put4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// NaN if either is: a row that sees a NaN is NaN as a whole.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t sm32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {  // bytes 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kStepBytes = 4096;             // of K, and again of V
template <typename T>
constexpr int kStep = kStepBytes / (kHeadDim * (int)sizeof(T));  // tokens: 16 or 8
constexpr size_t kRingBytes = (size_t)kWarps * kStages * 2 * kStepBytes;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// hi is x rounded to the nearest tf32 (half a step is added, the bits below are
// dropped): dropping bits alone would leave errors of one sign.  The bits of lo
// below tf32 are dropped by the instruction, so it is taken a third of a step
// per unit of its mantissa larger first, half a step on average.  That addition
// is a multiplication: where x is a NaN (or infinite) hi may be anything, its
// bits having carried into the sign, but x - hi is a NaN, and has to stay one.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint((x - __uint_as_float(hi)) * (1.f + 0x1p-10f / 3.f));
}
// d += a b for fp32 a (16 x 8) and b (8 x 8).
__device__ __forceinline__ void mma_fp32(float (&d)[4], const float (&a)[4], float b0, float b1) {
  uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_tf32(a[i], ah[i], al[i]);
  split_tf32(b0, bh[0], bl[0]);
  split_tf32(b1, bh[1], bl[1]);
  mma_tf32(d, al, bh[0], bh[1]);
  mma_tf32(d, ah, bl[0], bl[1]);
  mma_tf32(d, ah, bh[0], bh[1]);
}
__device__ __forceinline__ float lds32(uint32_t p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds128(uint32_t p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// An item as every lane of its warp sees it; `mine` is what row `lane` sees.
struct Item {
  int j, part, nrows;      // KV head, partial result, rows
  int64_t row0;            // first new token among all
  const int32_t* table;
  int lo, hi;              // positions that the rows see together
  int first, last;         // the steps of this run
  pa::Span mine;
};
// Items are the runs of the shared prefix first (rows of all sequences side by
// side), then those of the sequences' own tokens.
template <typename T>
__device__ __forceinline__ Item open_item(const Args& a, int w, bool tell) {
  const int lane = threadIdx.x & 31, tpt = kRows / a.g;
  Item it;
  const bool prefix = w < a.prefix_items;
  if (!prefix) w -= a.prefix_items;
  const int parts = prefix ? a.prefix_parts : a.own_parts, run = w % parts, rest = w / parts;
  it.j = rest % a.Hkv;
  it.part = prefix ? run : a.prefix_parts + run;
  const int at = rest / a.Hkv;
  it.mine = pa::Span{0, INT32_MAX, 0};  // padding rows see everything: no masks for their sake
  int lo = INT32_MAX, hi = 0;
  if (prefix) {
    it.row0 = (int64_t)at * tpt;
    it.nrows = (int)min((int64_t)tpt, a.T - it.row0) * a.g;
    it.table = a.prefix_table;
    if (lane < it.nrows) {
      const int64_t n = min((int64_t)max(a.n_tok[it.row0 + lane / a.g], 0), a.n_max);
      it.mine = pa::Span{0, (int)a.n_prefix, (int)(a.n_prefix + n - 1)};
    }
  } else {
    const int tiles = sizeof(T) == 4 ? (a.max_q + tpt - 1) / tpt : 1, b = at / tiles, i0 = at % tiles * tpt;
    const pa::Seq s = pa::seq_of(a, b, tell && lane == 0 && run == 0 && it.j == 0 && i0 == 0);
    it.row0 = s.first + i0;
    it.nrows = (int)min((int64_t)tpt, max(s.n_new - i0, (int64_t)0)) * a.g;
    it.table = a.pm.table + (int64_t)b * a.pm.max_pages;
    if (lane < it.nrows) it.mine = pa::span_of(a, s, b, i0 + lane / a.g);
  }
  if (lane < it.nrows && it.mine.lo < it.mine.hi) lo = it.mine.lo, hi = it.mine.hi;
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = min(__reduce_min_sync(0xffffffffu, lo), hi);
  it.lo = lo, it.hi = hi;
  constexpr int S = kStep<T>;
  const int s0 = lo / S, s1 = (hi + S - 1) / S, per = (s1 - s0 + parts - 1) / parts;
  it.first = s0 + run * per;
  it.last = hi > lo ? min(s1, it.first + per) : it.first;
  return it;
}

// How scores are formed: scaled only; capped or with a bias by distance; the
// same with a cap past pa::kCoarseCap (bf16).  A kernel each: a choice per call
// inside took 2% of a decode step's time.
enum { kPlain = 0, kGeneral = 1, kFineCap = 2 };

template <typename T, int kForm>
__global__ void __launch_bounds__(kWarps * 32, 1)
rows_kernel(const __grid_constant__ Args a, int items) {
  constexpr int D = kHeadDim, S = kStep<T>, NT = S / 8;  // tiles of 8 tokens in a step
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr uint32_t kAll = (1u << S) - 1;
  extern __shared__ __align__(1024) unsigned char ring[];  // [warp][stage][K step, V step]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c4 = lane & 3, r8 = lane >> 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the prefix's kernel may take the other SMs
  const int worker = warp * gridDim.x + blockIdx.x, workers = gridDim.x * kWarps;
  const uint32_t P = a.pm.page_size, pages = (uint32_t)a.pm.num_pages;
  const uint32_t my_ring = sm32(ring) + warp * kStages * 2 * kStepBytes;

  // ---- where the loads are: item, step, and the page of this lane's token ----
  // A step's rows are brought whole, 512 bytes an instruction (64 bytes of
  // eight rows at a time took longer).  Their 16-byte pieces are permuted by
  // the row so that the fragments' reads meet no bank twice: in bf16 piece c of
  // token x lies at c ^ (x % 8); in fp32 at c ^ 4 (x % 2) for K, whose readers
  // take four pieces of eight tokens, and at c ^ 2 (x / 2) for V, whose readers
  // take two pieces of every other token.
  int p_w = worker, p_step = 0, p_last = 0, p_lo = 0, p_hi = 0, p_j = 0, p_page = -1;
  const int32_t* __restrict__ p_table = nullptr;
  auto page_of = [&]() -> int {
    const uint32_t u = (uint32_t)p_step * S + (lane & (S - 1));
    return p_step < p_last && (int)u >= p_lo && (int)u < p_hi ? p_table[u / P] : -1;
  };
  auto open_loads = [&] {
    const Item it = open_item<T>(a, p_w, true);
    p_step = it.first, p_last = it.nrows > 0 ? it.last : it.first, p_lo = it.lo, p_hi = it.hi, p_j = it.j;
    p_table = it.table;
    p_page = page_of();
  };
  // Bits 16 s ..: which tokens of the step loaded s steps ago have a place in
  // the pool.
  uint64_t there_of = 0;
  int slot = 0;
  auto load_next = [&] {
    while (p_step >= p_last && p_w < items) {
      p_w += workers;
      if (p_w < items) open_loads();
    }
    bool ok = false;
    if (p_w < items) {
      const uint32_t u = (uint32_t)p_step * S + (lane & (S - 1));
      const bool in = (int)u >= p_lo && (int)u < p_hi;
      ok = in && (uint32_t)p_page < pages;
      if (in && !ok && lane < S) report(a.status, HKV_ERR_DEVICE_RANGE);
      const uint32_t row = ok ? ((uint32_t)p_page * a.Hkv + p_j) * P + u % P : 0xffffffffu;
      const uint32_t base = my_ring + slot * 2 * kStepBytes;
      constexpr int kPieces = kStepBytes / S / 16, kRowsAt = 32 / kPieces;  // 16-byte pieces of a row; rows an instruction
      const int c = lane & (kPieces - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = kRowsAt * i + lane / kPieces;
        const uint32_t rx = __shfl_sync(0xffffffffu, row, x);
        const uint32_t k_to = base + x * (kStepBytes / S) + ((kBf16 ? c ^ (x & 7) : c ^ ((x & 1) << 2)) << 4);
        const uint32_t v_to = base + kStepBytes + x * (kStepBytes / S) + ((kBf16 ? c ^ (x & 7) : c ^ ((x >> 1) << 1)) << 4);
        const int64_t off = rx == 0xffffffffu ? 0 : (int64_t)rx * D + c * (16 / (int)sizeof(T));
        const int bytes = rx == 0xffffffffu ? 0 : 16;
        cp16(k_to, static_cast<const T*>(a.K) + off, bytes);
        cp16(v_to, static_cast<const T*>(a.V) + off, bytes);
      }
      ++p_step;
      p_page = page_of();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    there_of = there_of << 16 | (__ballot_sync(0xffffffffu, ok) & kAll);
    if (++slot == kStages) slot = 0;
  };
  // The first lines that an own item needs, the start of its page table and its
  // queries, are called into L2 while the warp's items before it are worked on.
  auto call_in = [&](int w) {
    if (w >= items || w < a.prefix_items) return;
    const int rest = (w - a.prefix_items) / a.own_parts, j = rest % a.Hkv, tpt = kRows / a.g;
    const int tiles = kBf16 ? 1 : (a.max_q + tpt - 1) / tpt, b = rest / a.Hkv / tiles;
    const int64_t tok = (a.cu ? a.cu[b] : b) + rest / a.Hkv % tiles * tpt;
    constexpr int kLine = 128 / (int)sizeof(T);
    const void* at = lane == 0 ? static_cast<const void*>(a.pm.table + (int64_t)b * a.pm.max_pages)
                               : static_cast<const T*>(a.q) + tok * a.q_stride + (int64_t)j * a.g * D + (lane - 1) * kLine;
    if (lane == 0 ? a.pm.max_pages > 0 : lane <= a.g * D / kLine && tok >= 0 && tok < a.T) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
  };
  call_in(worker);
  call_in(worker + workers);
  if (p_w < items) open_loads();
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) load_next();

  const float zs = kForm != kPlain && a.softcap > 0.f ? a.scale / a.softcap : a.scale * pa::kLog2e;
  const float cap = a.softcap * pa::kLog2e;
  const bool whole_rows = a.prefix_parts + a.own_parts == 1;  // rows are finished here
#pragma unroll 1
  for (int w = worker; w < items; w += workers) {
    call_in(w + 2 * workers);
    const Item it = open_item<T>(a, w, false);
    if (it.nrows == 0) continue;
    // this thread's two rows of every fragment, and their queries as A fragments
    pa::Span sp[2];
    float slope[2];
    uint32_t qf[kBf16 ? 8 : 1][4];    // bf16: k = kk * 16 ..
    float4 qv[kBf16 ? 1 : 8][2];      // fp32: elements 16 kk + 4 c4 .. of both rows, two k steps of four
    int64_t row_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r8 + 8 * h;
      sp[h] = pa::Span{__shfl_sync(0xffffffffu, it.mine.lo, r), __shfl_sync(0xffffffffu, it.mine.hi, r),
                       __shfl_sync(0xffffffffu, it.mine.pos, r)};
      const int head = it.j * a.g + r % a.g;
      slope[h] = kForm != kPlain && a.slopes && r < it.nrows ? a.slopes[head] * pa::kLog2e : 0.f;
      row_at[h] = (it.row0 + r / a.g) * a.Hq + head;
      const T* q = static_cast<const T*>(a.q) + (it.row0 + r / a.g) * a.q_stride + (int64_t)head * D;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        if constexpr (kBf16) {
          const uint32_t* p = reinterpret_cast<const uint32_t*>(q) + kk * 8 + c4;
          qf[kk][h] = r < it.nrows ? __ldg(p) : 0u;
          qf[kk][2 + h] = r < it.nrows ? __ldg(p + 4) : 0u;
        } else {
          qv[kk][h] = r < it.nrows ? __ldg(reinterpret_cast<const float4*>(q) + kk * 4 + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
    float acc[16][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
    for (int step = it.first; step < it.last; ++step) {
      const uint32_t there = (uint32_t)(there_of >> (16 * (kStages - 2))) & kAll;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      // `slot` is the next one to fill, which the last step left: this step's is one on
      const uint32_t kb = my_ring + (slot + 1 == kStages ? 0 : slot + 1) * 2 * kStepBytes, vb = kb + kStepBytes;
      float z[NT][4] = {}, y[NT][4] = {};  // even and odd kk: half as long a chain of MMAs
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        if constexpr (kBf16) {
          // tokens 0-7 and 8-15 of the step, elements kk * 16 + 0-7 and 8-15
          uint32_t b[4];
          const int x = (lane & 7) + (lane >> 4) * 8, ch = kk * 2 + ((lane >> 3) & 1);
          ldsm4(b, kb + x * 256 + ((ch ^ (x & 7)) << 4));
          mma16816(kk & 1 ? y[0] : z[0], qf[kk], b[0], b[1]);
          mma16816(kk & 1 ? y[NT - 1] : z[NT - 1], qf[kk], b[2], b[3]);
        } else {
          // token r8, elements 16 kk + 4 c4 ..: the order of the sum's terms is free
          const float4 b = lds128(kb + r8 * 512 + (((kk * 4 + c4) ^ ((r8 & 1) << 2)) << 4));
          const float4 u = qv[kk][0], v = qv[kk][1];
          const float a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
          mma_fp32(z[0], a0, b.x, b.y);
          mma_fp32(y[0], a1, b.z, b.w);
        }
      }
      load_next();  // here, where the scores are not there yet
      const int u0 = step * S + c4 * 2;  // this thread's tokens: u0, u0 + 1 (and u0 + 8, u0 + 9)
      float top[2] = {-INFINITY, -INFINITY};
      const bool whole = there == kAll && sp[0].lo <= step * S && sp[1].lo <= step * S && sp[0].hi >= (step + 1) * S &&
                         sp[1].hi >= (step + 1) * S;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1, u = u0 + n * 8 + (e & 1);
          float x = (z[n][e] + y[n][e]) * zs;
          if (kForm != kPlain) {
            if (cap > 0.f) x = !kBf16 ? cap * tanhf(x) : kForm == kFineCap ? pa::capped_fine(x, cap) : pa::capped(x, cap);
            x = fmaf(-slope[h], fabsf((float)(sp[h].pos - u)), x);
          }
          if (!whole && (u < sp[h].lo || u >= sp[h].hi || !(there >> (u & (S - 1)) & 1u))) x = -INFINITY;
          z[n][e] = x;
          top[h] = max_nan(top[h], x);
        }
      bool grown = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = max_nan(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = max_nan(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        grown |= !(top[h] <= m[h] + 8.f);  // from nothing to something, and to NaN, too
      }
      if (__any_sync(0xffffffffu, grown)) {  // rare after the first steps
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = max_nan(m[h], top[h]), f = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn);
          m[h] = mn, l[h] *= f;
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[i][2 * h] *= f, acc[i][2 * h + 1] *= f;
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1;
          const float x = z[n][e] - (m[h] == -INFINITY ? 0.f : m[h]);
          z[n][e] = kBf16 ? pa::ex2(x) : exp2f(x);
          l[h] += z[n][e];
        }
      if constexpr (kBf16) {
        const uint32_t pf[4] = {pack2(z[0][0], z[0][1]), pack2(z[0][2], z[0][3]), pack2(z[NT - 1][0], z[NT - 1][1]),
                                pack2(z[NT - 1][2], z[NT - 1][3])};
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          uint32_t b[4];
          const int x = lane & 15, ch = d * 2 + (lane >> 4);
          ldsm4t(b, vb + x * 256 + ((ch ^ (x & 7)) << 4));
          mma16816(acc[2 * d], pf, b[0], b[1]);
          mma16816(acc[2 * d + 1], pf, b[2], b[3]);
        }
      } else {
        // k = c4 is token 2 c4 and k = c4 + 4 token 2 c4 + 1, as the weights lie
        const float pf[4] = {z[0][0], z[0][2], z[0][1], z[0][3]};
#pragma unroll
        for (int d = 0; d < 16; ++d) {
          const uint32_t at = vb + c4 * 1024 + (((2 * d + (lane >> 4)) ^ (c4 << 1)) << 4) + (r8 & 3) * 4;
          mma_fp32(acc[d], pf, lds32(at), lds32(at + 512));
        }
      }
      __syncwarp();
    }
    // this run's part, or the finished rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (r8 + 8 * h >= it.nrows) continue;
      const bool any = l[h] != 0.f;  // NaN is something
      const float by = !whole_rows ? 1.f : any ? 1.f / l[h] : 0.f;
      const int64_t row = row_at[h] + (whole_rows ? 0 : it.part * a.T * a.Hq);
      if (c4 == 0) {
        if (!whole_rows) a.part_ml[row] = make_float2(m[h], l[h]);
        else if (a.lse) a.lse[row] = any ? (m[h] + log2f(l[h])) * pa::kLn2 : -INFINITY;
      }
      if (kBf16 && whole_rows) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row * D) + c4;
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[i * 4] = pack2(acc[i][2 * h] * by, acc[i][2 * h + 1] * by);
      } else {
        float2* dst = reinterpret_cast<float2*>((whole_rows ? static_cast<float*>(a.out) : a.part_o) + row * D) + c4;
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[i * 4] = make_float2(acc[i][2 * h] * by, acc[i][2 * h + 1] * by);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Joins the parts of every row: out = sum_p 2^(m_p - M) o_p / L, with M the
// largest m_p and L = sum_p 2^(m_p - M) l_p.  One warp per row, four columns a
// lane; kAhead parts' loads are on their way together (four are enough for a few
// parts; eight take 2.5 us from 64).
template <typename T, int kAhead>
__global__ void __launch_bounds__(128)
join_parts_kernel(const __grid_constant__ Args a) {
  constexpr int Q = kHeadDim / 4;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), n_rows = a.T * a.Hq;
  const int lane = threadIdx.x & 31, parts = a.prefix_parts + a.own_parts;
  bool mine = row < n_rows;
  if (mine && a.cu) {
    const int64_t t = row / a.Hq;
    const pa::Seq s = pa::seq_of(a, pa::find_seq(a.cu, a.B, t), false);
    mine = t >= s.first && t < s.first + s.n_new;  // not behind the last sequence
  }
  // by every block: a call must not be over before the kernel whose parts these are
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const float2* ml = a.part_ml + row;
  const float4* part = reinterpret_cast<const float4*>(a.part_o) + row * Q + lane;
  float M = -INFINITY;
  for (int p = lane; p < parts; p += 32) M = fmaxf(M, ml[p * n_rows].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < parts; p0 += 32) {
    // lane p holds the weight of part p0 + p; an empty part's values need not
    // have been written
    const float2 one = p0 + lane < parts ? ml[(p0 + lane) * n_rows] : make_float2(-INFINITY, 0.f);
    const float w = one.x == -INFINITY ? 0.f : exp2f(one.x - M);
    L = fmaf(w, one.y, L);
    const int n = min(32, parts - p0);
    for (int p = 0; p < n; p += kAhead) {
      float4 x[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        x[e] = p + e < n ? part[(p0 + p + e) * n_rows * Q] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const float v = __shfl_sync(0xffffffffu, w, (p + e) & 31);
        if (v > 0.f && p + e < n)
          o.x = fmaf(v, x[e].x, o.x), o.y = fmaf(v, x[e].y, o.y), o.z = fmaf(v, x[e].z, o.z), o.w = fmaf(v, x[e].w, o.w);
      }
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
  const float inv = L != 0.f ? 1.f / L : 0.f;
  put4(static_cast<T*>(a.out) + row * kHeadDim + lane * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (lane == 0 && a.lse) a.lse[row] = L != 0.f ? (M + log2f(L)) * pa::kLn2 : -INFINITY;
}

// Items of one kind: `n` of them, each over `steps` steps of positions.
struct Kind {
  int64_t n, steps;
  int64_t runs(int64_t length) const { return n > 0 ? ceil_div(steps, length) : 0; }
};

// Steps of a run: items are cut into runs until every worker has one, down to
// sqrt(steps / 10): a step alone on its SM takes 0.5 us, joining one more part
// 0.05 us (single tokens of 8 sequences of 300 tokens: 15.7 us with eight steps a
// run at least, 10.1 with two; of 1000 tokens: 14.4 us in one wave of 16 runs,
// 17.9 in a wave and a bit).  Longer work is cut only into runs of at least 32
// steps, six for every worker, so that the last ones to run are short.
int64_t run_steps(const Kind& a, const Kind& b, int64_t workers) {
  const int64_t longest = a.steps > b.steps ? a.steps : b.steps;
  auto fits = [&](int64_t length, int64_t most) {
    while (length < longest && a.n * a.runs(length) + b.n * b.runs(length) > most) length += length / 8 + 1;
    return length;
  };
  int64_t least = 2;
  while (10 * least * least < longest) ++least;
  const int64_t few = fits(least, workers), many = fits(32, 6 * workers), most_runs = ceil_div(longest, 64);
  const int64_t r = few < many ? few : many;
  return r > most_runs ? r : most_runs;
}

// How a call is cut up; from its shape and the device alone, so that the
// workspace can be sized before the call.
struct Plan {
  bool tc = false;         // prompts: the tensor-core kernel takes all rows
  int64_t own_items = 0;   // rows of one sequence (16 at most), all KV heads together
  int prefix_parts = 0, own_parts = 1;
  int prefix_items = 0;    // runs of the prefix that this file's kernel takes
  int row_ctas = 0;        // blocks of this file's kernel, one per SM
  int parts = 0;           // a row's partial results, 0 when its block finishes it
  size_t o = 0, total = 0;  // byte offset of part_o behind part_ml, and the size
};

Plan plan(const PagedAttend& p) {
  Plan r;
  const int g = p.Hq / p.Hkv, tpt = kRows / g, sms = sm_count();
  const bool bf16 = p.dtype == HKV_BF16;
  // a sequence's new tokens fill more than the 16 rows of one block: 128-row tiles
  r.tc = bf16 && p.cu_q_rows && (int64_t)p.max_q * g > kRows;
  if (r.tc) {
    r.own_parts = tc_splits(p, false, sms);
  } else {
    r.own_items = (int64_t)p.B * ceil_div(p.max_q, tpt) * p.Hkv;
    const int step = bf16 ? kStep<__nv_bfloat16> : kStep<float>;
    const int64_t workers = (int64_t)kWarps * sms;
    const Kind own{r.own_items, p.n_max > 0 ? ceil_div(p.n_max, step) : 1};
    Kind prefix{p.n_prefix > 0 ? ceil_div(p.B, tpt) * p.Hkv : 0, ceil_div(p.n_prefix, step)};
    // A short prefix goes the way of the own tokens, in bf16 too: one launch
    // less, and no CTA's start and end (8 sequences behind 400 tokens 9.6 us
    // instead of 11.9, 32 behind 256 11.3 instead of 15.2; 32 behind 2000, which
    // are read for every 16 rows again, 27 instead of 19).
    const bool tc_prefix = prefix.n > 0 && bf16 && (p.n_prefix > 1024 || prefix.n * prefix.steps > 4 * workers);
    if (tc_prefix) prefix = Kind{0, 0};
    // beside the prefix's kernel, on fewer SMs, twice as many runs keep the
    // warps busy to the end (16 sequences of up to 2000 tokens behind 32768:
    // 68 us, 56 with twice as many)
    const int64_t length = run_steps(own, prefix, tc_prefix ? 2 * workers : workers);
    r.own_parts = (int)own.runs(length);
    r.prefix_parts = (int)prefix.runs(length);
    r.prefix_items = (int)(prefix.n * r.prefix_parts);
    const int64_t items = r.own_items * r.own_parts + r.prefix_items;
    r.row_ctas = (int)(items < sms ? items : sms);
    if (tc_prefix) {
      // The prefix (bound by the tensor cores) and the sequences' own tokens
      // (bound by memory) run side by side on SMs of their own, shared out by
      // the time that each would take of one SM: 1.75 us for a tile of 128
      // tokens and 256 rows, 45 GB/s and 0.5 us an item for the own tokens,
      // taken to be half as long as they may be.  (64 sequences of up to 512
      // tokens behind 32768: one after the other 73 us, side by side 63 to 66;
      // 256 of up to 128 behind 98304: 409 and 375 us.)
      const double prefix_us = 1.75 * (double)tc_tiles(p, true) * p.Hkv * (double)ceil_div(p.n_prefix, 128);
      const double own_us = (double)p.B * p.Hkv * (double)p.n_max * 0.5 * 512 / 45e3 + 0.5 * (double)items;
      const int share = (int)(sms * own_us / (own_us + prefix_us) + 0.5);
      r.row_ctas = share < 1 ? 1 : share > sms - sms / 8 ? sms - sms / 8 : share;
      if (r.row_ctas > items) r.row_ctas = (int)items;
      r.prefix_parts = tc_splits(p, true, sms - r.row_ctas);
    }
  }
  r.parts = r.prefix_parts > 0 || r.own_parts > 1 ? r.prefix_parts + r.own_parts : 0;
  r.o = align_up(sizeof(float2) * r.parts * p.T * p.Hq, 256);
  r.total = r.parts ? r.o + sizeof(float) * kHeadDim * r.parts * p.T * p.Hq : 0;
  return r;
}

template <typename T>
int run(const PagedAttend& p, const Plan& pl, const Args& a, cudaStream_t st) {
  int rc = HKV_OK;
  if (pl.tc) {
    rc = launch_attend_tc(p, a, false, pl.own_parts, pl.parts ? 0 : -1, st);
  } else {
    const int64_t items = pl.prefix_items + pl.own_items * pl.own_parts;
    if (items > INT32_MAX / 2) return fail(HKV_ERR_UNSUPPORTED, "too many sequences and heads");
    auto kernel = a.softcap > 0.f || a.slopes ? rows_kernel<T, kGeneral> : rows_kernel<T, kPlain>;
    if constexpr (sizeof(T) == 2)
      if (a.softcap > pa::kCoarseCap) kernel = rows_kernel<T, kFineCap>;
    rc = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes),
                    "paged attention smem attribute");
    if (rc != HKV_OK) return rc;
    kernel<<<pl.row_ctas, kWarps * 32, kRingBytes, st>>>(a, (int)items);
    rc = cuda_check(cudaGetLastError(), "paged attention launch");
    if (rc == HKV_OK && pl.prefix_parts > 0 && pl.prefix_items == 0) rc = launch_attend_tc(p, a, true, pl.prefix_parts, 0, st);
  }
  if (rc != HKV_OK || pl.parts == 0) return rc;
  auto join = pl.parts > 4 ? join_parts_kernel<T, 8> : join_parts_kernel<T, 4>;
  return cuda_check(launch_after(join, dim3((unsigned)ceil_div(a.T * a.Hq, 4)), 128, 0, st, a),
                    "attention join launch");
}

}  // namespace

size_t attend_paged_ws_bytes(const PagedAttend& p) { return plan(p).total; }

int launch_attend_paged(const PagedAttend& p, void* ws, size_t ws_bytes, cudaStream_t st) {
  const Plan pl = plan(p);
  if (pl.total > 0 && (ws == nullptr || ws_bytes < pl.total))
    return fail(HKV_ERR_CAPACITY, "workspace of %zu bytes, %zu needed", ws_bytes, pl.total);
  Args a{};
  a.B = p.B, a.Hq = p.Hq, a.Hkv = p.Hkv, a.g = p.Hq / p.Hkv, a.T = p.T, a.max_q = p.max_q;
  a.q = p.q, a.q_stride = p.q_stride, a.K = p.K_pool, a.V = p.V_pool, a.pm = p.pm, a.cu = p.cu_q, a.n_tok = p.n_tok;
  a.n_max = p.n_max, a.prefix_table = p.prefix_table, a.n_prefix = p.n_prefix;
  a.scale = p.scale, a.softcap = p.softcap, a.window = p.window, a.slopes = p.slopes;
  a.prefix_len = p.prefix_len, a.q_first = p.q_first, a.out = p.out, a.lse = p.lse, a.status = p.status;
  a.wait_ns = wait_limit_ns();
  a.prefix_parts = pl.prefix_parts, a.own_parts = pl.own_parts, a.prefix_items = pl.prefix_items;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.part_ml = reinterpret_cast<float2*>(w);
  a.part_o = reinterpret_cast<float*>(w + pl.o);
  return p.dtype == HKV_BF16 ? run<__nv_bfloat16>(p, pl, a, st) : run<float>(p, pl, a, st);
}

}  // namespace hkv
