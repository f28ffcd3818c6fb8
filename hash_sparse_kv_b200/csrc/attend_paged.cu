// Dense attention over a paged cache for few rows at a time: the single-token
// (decode) form of the prompt attention, the own tokens of sequences behind a
// shared prefix, and fp32 caches.
//
// A block takes the rows of up to 16 / g new tokens of one KV head (g query
// heads a token share its keys) and one run of their cache positions, reads
// that run once, and keeps the softmax's running maximum and sum and the
// weighted values in registers (fp32).  Where few blocks would be left, the
// positions are split over several blocks and a second launch joins their
// partial results.
#include <cstdio>

#include "attend_paged.cuh"

namespace hkv {
namespace {

using pa::Args;

constexpr int kThreads = 256;
constexpr int kRows = 16;
constexpr int kTile = 32;

__device__ __forceinline__ void put4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Which rows a block has and which positions of which table they see.
struct Item {
  int b, j, nrows;
  int64_t i0, row0;  // first new token within its sequence, and among all
  pa::Seq s;
};

template <bool kPrefix>
__device__ __forceinline__ bool item_of(const Args& a, Item& it) {
  const int tpt = kRows / a.g;  // tokens per block
  it.j = blockIdx.y;
  if constexpr (kPrefix) {  // rows of all sequences side by side
    it.b = 0, it.i0 = (int64_t)blockIdx.x * tpt, it.row0 = it.i0;
    it.s = pa::Seq{0, a.T, 0};
  } else {
    const int tiles = (a.max_q + tpt - 1) / tpt;
    it.b = blockIdx.x / tiles, it.i0 = (int64_t)(blockIdx.x % tiles) * tpt;
    it.s = pa::seq_of(a, it.b, it.i0 == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0);
    it.row0 = it.s.first + it.i0;
  }
  if (it.i0 >= it.s.n_new) return false;
  it.nrows = (int)min((int64_t)tpt, it.s.n_new - it.i0) * a.g;
  return true;
}

// What row r of the item sees; positions count from the start of its table.
template <bool kPrefix>
__device__ __forceinline__ pa::Span row_span(const Args& a, const Item& it, int r) {
  const int64_t i = it.i0 + r / a.g;
  if constexpr (kPrefix) {
    const int64_t n = min((int64_t)max(a.n_tok[i], 0), a.n_max);
    return pa::Span{0, (int)a.n_prefix, (int)(a.n_prefix + n - 1)};
  } else {
    return pa::span_of(a, it.s, it.b, i);
  }
}

__device__ __forceinline__ int64_t out_row(const Args& a, const Item& it, int r) {
  return (it.row0 + r / a.g) * a.Hq + it.j * a.g + r % a.g;
}

// The block's result: maximum, sum and weighted values of its rows, in shared
// memory (o_s [kRows][kHeadDim], m_s and l_s [kRows]).  Every thread of the block
// comes here after a barrier.
template <typename T, bool kPrefix>
__device__ void finish(const Args& a, const Item& it, const float* o_s, const float* m_s, const float* l_s) {
  constexpr int Q = kHeadDim / 4;  // float4 pieces of a row
  const int parts = a.prefix_parts + a.own_parts;
  for (int i = threadIdx.x; i < it.nrows * Q; i += blockDim.x) {
    const int r = i / Q;
    int64_t row = out_row(a, it, r);
    float4 x = reinterpret_cast<const float4*>(o_s)[i];
    if (parts > 1) {
      row += (kPrefix ? blockIdx.z : a.prefix_parts + blockIdx.z) * a.T * a.Hq;
      reinterpret_cast<float4*>(a.part_o)[row * Q + i % Q] = x;
      if (i % Q == 0) a.part_ml[row] = make_float2(m_s[r], l_s[r]);
    } else {
      const float inv = l_s[r] > 0.f ? 1.f / l_s[r] : 0.f;
      x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
      put4(static_cast<T*>(a.out) + row * kHeadDim + i % Q * 4, x);
      if (i % Q == 0 && a.lse) a.lse[row] = l_s[r] > 0.f ? (m_s[r] + log2f(l_s[r])) * pa::kLn2 : -INFINITY;
    }
  }
}

__device__ __forceinline__ uint32_t sm32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {  // bytes 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
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

// fp32: eight warps, tiles of 32 tokens staged in shared memory (cp.async, two
// tiles ahead, their places looked up one tile before that).  A warp has two rows to itself: lane u scores
// them against token u, then holds four output columns of each, so that only
// the staging makes warps wait for each other.  Bound by the shared memory
// reads of the two products; two rows a warp and 16-byte reads keep them at
// three for 16 multiply-adds, which go two to an instruction.
constexpr int kSimtStages = 3, kSimtKPitch = kHeadDim + 4;
struct SimtStage {
  float k[kTile][kSimtKPitch];
  float v[kTile][kHeadDim];
  bool there[kTile];
};

template <bool kPrefix>
__global__ void __launch_bounds__(kThreads, 2)
rows_simt_kernel(const __grid_constant__ Args a) {
  constexpr int D = kHeadDim;
  static_assert(kRows == 2 * (kThreads / 32) && kTile == 32, "two rows a warp, a token a lane");
  __shared__ __align__(16) float q_s[kRows][D];  // the block's result in the end
  __shared__ __align__(16) float p_s[kRows][kTile];
  __shared__ float m_s[kRows], l_s[kRows];
  extern __shared__ __align__(16) unsigned char simt_smem[];
  SimtStage* const stages = reinterpret_cast<SimtStage*>(simt_smem);
  __shared__ int lo_s, hi_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Item it;
  if (!item_of<kPrefix>(a, it)) return;
  if (tid == 0) lo_s = INT32_MAX, hi_s = 0;
  pa::Span sp[2];
  float slope[2];
  const int r0 = warp * 2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + h;
    const float* q = static_cast<const float*>(a.q) + (it.row0 + r / a.g) * a.q_stride + (int64_t)(it.j * a.g + r % a.g) * D;
    *reinterpret_cast<float4*>(&q_s[r][lane * 4]) =
        r < it.nrows ? __ldg(reinterpret_cast<const float4*>(q) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    sp[h] = r < it.nrows ? row_span<kPrefix>(a, it, r) : pa::Span{0, 0, 0};
    slope[h] = a.slopes && r < it.nrows ? a.slopes[it.j * a.g + r % a.g] * pa::kLog2e : 0.f;
  }
  __syncthreads();
  if (lane < 2) {
    const pa::Span x = lane ? sp[1] : sp[0];
    if (x.lo < x.hi) {
      atomicMin(&lo_s, x.lo);
      atomicMax(&hi_s, x.hi);
    }
  }
  __syncthreads();
  const int lo = min(lo_s, hi_s), hi = hi_s;
  const int tiles = (hi - lo + kTile - 1) / kTile, per = (tiles + gridDim.z - 1) / gridDim.z;
  const int t0 = blockIdx.z * per, t1 = min(tiles, t0 + per);
  const int32_t* table = kPrefix ? a.prefix_table : a.pm.table + (int64_t)it.b * a.pm.max_pages;
  // this thread moves piece tid % 32 of tokens tid / 32 + 8 k
  const int x0 = tid / 32, piece = tid % 32 * 4;
  // lane u looks up token u of a tile
  auto row_at = [&](int t) -> int64_t {
    const int at = lo + t * kTile + lane;
    if (t >= t1 || at >= hi) return -1;
    const int64_t row = pa::pool_row(a, table, at, it.j);
    if (row < 0) report(a.status, HKV_ERR_DEVICE_RANGE);
    return row;
  };
  int64_t row = row_at(t0);
  int ahead = t0, to = 0;
  auto fetch_next = [&] {
    if (ahead < t1) {
      SimtStage& st = stages[to];
      if (warp == 0) st.there[lane] = row >= 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t from = __shfl_sync(0xffffffffu, row, x0 + 8 * k);
        const int64_t off = from >= 0 ? from * D + piece : 0;
        cp16(sm32(&st.k[x0 + 8 * k][piece]), static_cast<const float*>(a.K) + off, from >= 0 ? 16 : 0);
        cp16(sm32(&st.v[x0 + 8 * k][piece]), static_cast<const float*>(a.V) + off, from >= 0 ? 16 : 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    row = row_at(++ahead);
    if (++to == kSimtStages) to = 0;
  };
  uint64_t acc[2][2] = {};  // rows r0 and r0 + 1, columns 4 lane .. 4 lane + 3
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
  for (int k = 0; k < kSimtStages - 1; ++k) fetch_next();
  int at = 0;
  for (int t = t0; t < t1; ++t) {
    const int pos = lo + t * kTile + lane;
    const SimtStage& st = stages[at];
    if (++at == kSimtStages) at = 0;
    asm volatile("cp.async.wait_group %0;" ::"n"(kSimtStages - 2) : "memory");
    __syncthreads();  // this tile is there; the one before it has been used
    fetch_next();
    uint64_t z2[2][2] = {};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&st.k[lane][d]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&q_s[r0 + h][d]);
        z2[h][0] = fma2(q.x, k.x, z2[h][0]);
        z2[h][1] = fma2(q.y, k.y, z2[h][1]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = unpair(z2[h][0]), y = unpair(z2[h][1]);
      float s = ((x.x + x.y) + (y.x + y.y)) * a.scale;
      if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
      s = s * pa::kLog2e - slope[h] * (float)abs(sp[h].pos - pos);
      if (pos < sp[h].lo || pos >= sp[h].hi || !st.there[lane]) s = -INFINITY;
      float top = s;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(m[h], top), use = mn == -INFINITY ? 0.f : mn;
      const float p = exp2f(s - use), f = exp2f(m[h] - use);
      p_s[r0 + h][lane] = p;
      l[h] = l[h] * f + p;  // this lane's tokens; the lanes' sums meet in the end
      m[h] = mn;
      const uint64_t f2 = pair(f, f);
      acc[h][0] = fma2(acc[h][0], f2, 0), acc[h][1] = fma2(acc[h][1], f2, 0);
    }
    __syncwarp();
#pragma unroll 1
    for (int x = 0; x < kTile; x += 4) {
      const float4 pa4 = *reinterpret_cast<const float4*>(&p_s[r0][x]), pb4 = *reinterpret_cast<const float4*>(&p_s[r0 + 1][x]);
      const float pr[2][4] = {{pa4.x, pa4.y, pa4.z, pa4.w}, {pb4.x, pb4.y, pb4.z, pb4.w}};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&st.v[x + e][lane * 4]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t p2 = pair(pr[h][e], pr[h][e]);
          acc[h][0] = fma2(p2, v.x, acc[h][0]);
          acc[h][1] = fma2(p2, v.y, acc[h][1]);
        }
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int o = 16; o; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
    *reinterpret_cast<ulonglong2*>(&q_s[r0 + h][lane * 4]) = make_ulonglong2(acc[h][0], acc[h][1]);  // this warp's own rows
    if (lane == 0) m_s[r0 + h] = m[h], l_s[r0 + h] = l[h];
  }
  __syncthreads();
  finish<float, kPrefix>(a, it, q_s[0], m_s, l_s);
}

// ---- bf16: a warp per item ---------------------------------------------------
// An item is the up to 16 rows of one sequence and KV head and one run of
// their positions.  A warp goes through items on its own: K and V arrive by
// cp.async in steps of 16 tokens, three steps (24 KB) ahead, and the loads run
// on into the warp's next item while this one is finished, so that the eight
// warps of an SM keep 192 KB on their way without ever waiting for each other.
// Scores and products are mma.sync m16n8k16 with the 16 rows as M: the work is
// bound by reading K and V, and a 128-row tcgen05 tile would be seven eighths
// padding.  P is rounded to bf16 for the product, sums stay fp32.
constexpr int kWarps = 8;
constexpr int kStep = 16;                    // tokens
constexpr int kStages = 3;
constexpr int kStepBytes = kStep * 256;      // of K, and again of V
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
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// An item as every lane of its warp sees it; `mine` is what row `lane` sees.
struct WarpItem {
  int b, j, part, nrows;
  int64_t row0;       // first new token among all
  int lo, hi;         // positions that the rows see together
  int first, last;    // the steps of this run
  pa::Span mine;
};
__device__ __forceinline__ WarpItem open_item(const Args& a, int w, bool tell) {
  const int lane = threadIdx.x & 31;
  WarpItem it;
  it.part = w % a.own_parts;
  const int rest = w / a.own_parts;
  it.j = rest % a.Hkv, it.b = rest / a.Hkv;
  const pa::Seq s = pa::seq_of(a, it.b, tell && lane == 0 && it.part == 0 && it.j == 0);
  it.row0 = s.first;
  it.nrows = (int)s.n_new * a.g;
  it.mine = pa::Span{0, INT32_MAX, 0};  // padding rows see everything: no masks for their sake
  int lo = INT32_MAX, hi = 0;
  if (lane < it.nrows) {
    it.mine = pa::span_of(a, s, it.b, lane / a.g);
    if (it.mine.lo < it.mine.hi) lo = it.mine.lo, hi = it.mine.hi;
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = min(__reduce_min_sync(0xffffffffu, lo), hi);
  it.lo = lo, it.hi = hi;
  const int s0 = lo / kStep, s1 = (hi + kStep - 1) / kStep, per = (s1 - s0 + a.own_parts - 1) / a.own_parts;
  it.first = s0 + it.part * per;
  it.last = hi > lo ? min(s1, it.first + per) : it.first;
  return it;
}

template <bool kGeneral>
__global__ void __launch_bounds__(kWarps * 32, 1)
rows_mma_kernel(const __grid_constant__ Args a, int items) {
  constexpr int D = kHeadDim;
  extern __shared__ __align__(1024) unsigned char ring[];  // [warp][stage][K step, V step]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the prefix's kernel may take the other SMs
  const int worker = warp * gridDim.x + blockIdx.x, workers = gridDim.x * kWarps;
  const uint32_t P = a.pm.page_size, pages = (uint32_t)a.pm.num_pages;
  const uint32_t my_ring = sm32(ring) + warp * kStages * 2 * kStepBytes;

  // ---- where the loads are: item, step, and the page of this lane's token ----
  // A step's tokens are brought two whole rows at a time (64 bytes of eight rows
  // at a time took longer); piece c of token x lies at c ^ (x % 8).
  int p_w = worker, p_step = 0, p_last = 0, p_lo = 0, p_hi = 0, p_j = 0, p_page = -1;
  const int32_t* __restrict__ p_table = nullptr;
  auto page_of = [&]() -> int {
    const uint32_t u = (uint32_t)p_step * kStep + (lane & 15);
    return p_step < p_last && (int)u >= p_lo && (int)u < p_hi ? p_table[u / P] : -1;
  };
  auto open_loads = [&] {
    const WarpItem it = open_item(a, p_w, true);
    p_step = it.first, p_last = it.nrows > 0 ? it.last : it.first, p_lo = it.lo, p_hi = it.hi, p_j = it.j;
    p_table = a.pm.table + (int64_t)it.b * a.pm.max_pages;
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
      const uint32_t u = (uint32_t)p_step * kStep + (lane & 15);
      const bool in = (int)u >= p_lo && (int)u < p_hi;
      ok = in && (uint32_t)p_page < pages;
      if (in && !ok && lane < 16) report(a.status, HKV_ERR_DEVICE_RANGE);
      const uint32_t row = ok ? ((uint32_t)p_page * a.Hkv + p_j) * P + u % P : 0xffffffffu;
      const uint32_t base = my_ring + slot * 2 * kStepBytes;
      const int c = lane & 15;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = 2 * i + (lane >> 4);
        const uint32_t rx = __shfl_sync(0xffffffffu, row, x);
        const uint32_t dst = base + x * 256 + ((c ^ (x & 7)) << 4);
        const int64_t off = rx == 0xffffffffu ? 0 : (int64_t)rx * D + c * 8;
        const int bytes = rx == 0xffffffffu ? 0 : 16;
        cp16(dst, static_cast<const __nv_bfloat16*>(a.K) + off, bytes);
        cp16(dst + kStepBytes, static_cast<const __nv_bfloat16*>(a.V) + off, bytes);
      }
      ++p_step;
      p_page = page_of();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    there_of = there_of << 16 | (__ballot_sync(0xffffffffu, ok) & 0xffffu);
    if (++slot == kStages) slot = 0;
  };
  // The first lines that an item needs, the start of its page table and its
  // queries, are called into L2 while the warp's item before it is worked on.
  auto call_in = [&](int w) {
    if (w >= items) return;
    const int rest = w / a.own_parts, j = rest % a.Hkv, b = rest / a.Hkv;
    const int64_t tok = a.cu ? a.cu[b] : b;
    const void* at = lane == 0 ? static_cast<const void*>(a.pm.table + (int64_t)b * a.pm.max_pages)
                               : static_cast<const __nv_bfloat16*>(a.q) + tok * a.q_stride + (int64_t)j * a.g * D + (lane - 1) * 64;
    if (lane <= 2 * a.g && (lane == 0 || tok < a.T)) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
  };
  call_in(worker);
  call_in(worker + workers);
  if (p_w < items) open_loads();
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) load_next();

  const float zs = kGeneral && a.softcap > 0.f ? a.scale / a.softcap : a.scale * pa::kLog2e;
  const float cap = a.softcap * pa::kLog2e;
  const int parts = a.prefix_parts + a.own_parts;
#pragma unroll 1
  for (int w = worker; w < items; w += workers) {
    call_in(w + 2 * workers);
    const WarpItem it = open_item(a, w, false);
    if (it.nrows == 0) continue;
    // this thread's two rows of every fragment, and the queries of them: A
    // fragments straight from memory
    pa::Span sp[2];
    float slope[2];
    uint32_t qf[8][4];
    int64_t row_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane / 4 + 8 * h;
      sp[h] = pa::Span{__shfl_sync(0xffffffffu, it.mine.lo, r), __shfl_sync(0xffffffffu, it.mine.hi, r),
                       __shfl_sync(0xffffffffu, it.mine.pos, r)};
      const int head = it.j * a.g + r % a.g;
      slope[h] = kGeneral && a.slopes && r < it.nrows ? a.slopes[head] * pa::kLog2e : 0.f;
      row_at[h] = (it.row0 + r / a.g) * a.Hq + head;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + (it.row0 + r / a.g) * a.q_stride +
                                                            (int64_t)head * D) + lane % 4;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qf[kk][h] = r < it.nrows ? __ldg(q + kk * 8) : 0u;
        qf[kk][2 + h] = r < it.nrows ? __ldg(q + kk * 8 + 4) : 0u;
      }
    }
    float acc[16][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
    for (int step = it.first; step < it.last; ++step) {
      const uint32_t there = (uint32_t)(there_of >> (16 * (kStages - 2))) & 0xffffu;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      // `slot` is the next one to fill, which the last step left: this step's is one on
      const uint32_t kb = my_ring + (slot + 1 == kStages ? 0 : slot + 1) * 2 * kStepBytes, vb = kb + kStepBytes;
      float z[2][4] = {}, y[2][4] = {};  // even and odd kk: half as long a chain of MMAs
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        // tokens 0-7 and 8-15 of the step, elements kk * 16 + 0-7 and 8-15
        uint32_t b[4];
        const int x = (lane & 7) + (lane >> 4) * 8, ch = kk * 2 + ((lane >> 3) & 1);
        ldsm4(b, kb + x * 256 + ((ch ^ (x & 7)) << 4));
        mma16816(kk & 1 ? y[0] : z[0], qf[kk], b[0], b[1]);
        mma16816(kk & 1 ? y[1] : z[1], qf[kk], b[2], b[3]);
      }
      load_next();  // here, where the scores are not there yet
      const int u0 = step * kStep + (lane & 3) * 2;  // this thread's tokens: u0, u0 + 1, u0 + 8, u0 + 9
      float top[2] = {-INFINITY, -INFINITY};
      const bool whole = there == 0xffffu && sp[0].lo <= step * kStep && sp[1].lo <= step * kStep &&
                         sp[0].hi >= (step + 1) * kStep && sp[1].hi >= (step + 1) * kStep;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1, u = u0 + n * 8 + (e & 1);
          float x = (z[n][e] + y[n][e]) * zs;
          if (kGeneral) {
            if (cap > 0.f) x = pa::capped(x, cap);
            x = fmaf(-slope[h], fabsf((float)(sp[h].pos - u)), x);
          }
          if (!whole && (u < sp[h].lo || u >= sp[h].hi || !(there >> (u & 15) & 1u))) x = -INFINITY;
          z[n][e] = x;
          top[h] = fmaxf(top[h], x);
        }
      bool grown = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        grown |= top[h] > m[h] + 8.f || (m[h] == -INFINITY && top[h] > -INFINITY);
      }
      if (__any_sync(0xffffffffu, grown)) {  // rare after the first steps
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m[h], top[h]), f = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn);
          m[h] = mn, l[h] *= f;
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[i][2 * h] *= f, acc[i][2 * h + 1] *= f;
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1;
          z[n][e] = pa::ex2(z[n][e] - (m[h] == -INFINITY ? 0.f : m[h]));
          l[h] += z[n][e];
        }
      const uint32_t pf[4] = {pack2(z[0][0], z[0][1]), pack2(z[0][2], z[0][3]), pack2(z[1][0], z[1][1]),
                              pack2(z[1][2], z[1][3])};
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        uint32_t b[4];
        const int x = lane & 15, ch = d * 2 + (lane >> 4);
        ldsm4t(b, vb + x * 256 + ((ch ^ (x & 7)) << 4));
        mma16816(acc[2 * d], pf, b[0], b[1]);
        mma16816(acc[2 * d + 1], pf, b[2], b[3]);
      }
      __syncwarp();
    }
    // this run's part, or the finished rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (lane / 4 + 8 * h >= it.nrows) continue;
      if (parts > 1) {
        const int64_t row = (a.prefix_parts + it.part) * a.T * a.Hq + row_at[h];
        if ((lane & 3) == 0) a.part_ml[row] = make_float2(m[h], l[h]);
        float2* dst = reinterpret_cast<float2*>(a.part_o + row * D) + (lane & 3);
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[i * 4] = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
      } else {
        const float inv = l[h] > 0.f ? 1.f / l[h] : 0.f;
        if ((lane & 3) == 0 && a.lse) a.lse[row_at[h]] = l[h] > 0.f ? (m[h] + log2f(l[h])) * pa::kLn2 : -INFINITY;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row_at[h] * D) + (lane & 3);
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[i * 4] = pack2(acc[i][2 * h] * inv, acc[i][2 * h + 1] * inv);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Joins the parts of every row: out = sum_p 2^(m_p - M) o_p / L, with M the
// largest m_p and L = sum_p 2^(m_p - M) l_p.  One warp per row, four columns a
// lane; the parts' loads are independent of one another.
template <typename T>
__global__ void __launch_bounds__(128)
join_parts_kernel(const __grid_constant__ Args a) {
  constexpr int Q = kHeadDim / 4, kAhead = 4;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), n_rows = a.T * a.Hq;
  const int lane = threadIdx.x & 31, parts = a.prefix_parts + a.own_parts;
  if (row >= n_rows) return;
  if (a.cu) {
    const int64_t t = row / a.Hq;
    const pa::Seq s = pa::seq_of(a, pa::find_seq(a.cu, a.B, t), false);
    if (t < s.first || t >= s.first + s.n_new) return;  // behind the last sequence
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
    const float2 mine = p0 + lane < parts ? ml[(p0 + lane) * n_rows] : make_float2(-INFINITY, 0.f);
    const float w = mine.x == -INFINITY ? 0.f : exp2f(mine.x - M);
    L = fmaf(w, mine.y, L);
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
  const float inv = L > 0.f ? 1.f / L : 0.f;
  put4(static_cast<T*>(a.out) + row * kHeadDim + lane * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (lane == 0 && a.lse) a.lse[row] = L > 0.f ? (M + log2f(L)) * pa::kLn2 : -INFINITY;
}

// Runs of positions that an item is cut into.  Few items are cut until every
// worker has one, down to 128 tokens; many items only into runs of at least
// 512 tokens, six for every worker, so that the last ones to run are short.
int splits_for(int64_t items, int64_t tokens, int64_t workers) {
  auto cut = [&](int64_t want, int64_t least) {
    want = ceil_div(want, items < 1 ? 1 : items);
    const int64_t most = ceil_div(tokens, least);
    return want < most ? want : most;
  };
  const int64_t few = cut(workers, 128), many = cut(6 * workers, 512), s = few > many ? few : many;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

// How a call is cut up; from its shape and the device alone, so that the
// workspace can be sized before the call.
struct Plan {
  bool tc = false;         // prompts: the tensor-core kernel takes all rows
  int64_t own_items = 0;   // rows of one sequence (16 at most), all KV heads together
  int prefix_parts = 0, own_parts = 1;
  int row_ctas = 0;        // bf16: blocks of the single-token kernel, one per SM
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
    // two fp32 blocks, or eight bf16 warps, per SM
    r.own_parts = splits_for(r.own_items, p.n_max, (bf16 ? kWarps : 2) * sms);
    const int64_t items = r.own_items * r.own_parts;
    r.row_ctas = (int)(items < sms ? items : sms);
    if (p.n_prefix > 0 && bf16) {
      // The prefix (bound by the tensor cores) and the sequences' own tokens
      // (bound by memory) run side by side on SMs of their own, shared out by
      // the time that each would take of one SM: 1.75 us for a tile of 128
      // tokens and 256 rows, 45 GB/s and 0.5 us an item for the own tokens,
      // taken to be half as long as they may be.  (64 sequences of up to 512
      // tokens behind 32768: one after the other 73 us, side by side 63 us; 256
      // of up to 128 behind 98304: 409 and 375 us.)
      const double prefix_us = 1.75 * (double)tc_tiles(p, true) * p.Hkv * (double)ceil_div(p.n_prefix, 128);
      const double own_us = (double)p.B * p.Hkv * (double)p.n_max * 0.5 * 512 / 45e3 + 0.5 * (double)items;
      const int share = (int)(sms * own_us / (own_us + prefix_us) + 0.5);
      r.row_ctas = share < 1 ? 1 : share > sms - sms / 8 ? sms - sms / 8 : share;
      if (r.row_ctas > items) r.row_ctas = (int)items;
      r.prefix_parts = tc_splits(p, true, sms - r.row_ctas);
    } else if (p.n_prefix > 0) {
      r.prefix_parts = splits_for(ceil_div(p.B, tpt) * p.Hkv, p.n_prefix, 2 * sms);
    }
  }
  r.parts = r.prefix_parts > 0 || r.own_parts > 1 ? r.prefix_parts + r.own_parts : 0;
  r.o = align_up(sizeof(float2) * r.parts * p.T * p.Hq, 256);
  r.total = r.parts ? r.o + sizeof(float) * kHeadDim * r.parts * p.T * p.Hq : 0;
  return r;
}

int run_fp32(const PagedAttend& p, const Plan& pl, const Args& a, cudaStream_t st) {
  constexpr size_t smem = kSimtStages * sizeof(SimtStage);
  for (int prefix = pl.prefix_parts > 0; prefix >= 0; --prefix) {
    auto kernel = prefix ? rows_simt_kernel<true> : rows_simt_kernel<false>;
    const int rc = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem),
                              "paged attention smem attribute");
    if (rc != HKV_OK) return rc;
    const int64_t blocks = prefix ? ceil_div(p.B, kRows / a.g) : pl.own_items / p.Hkv;
    kernel<<<dim3((unsigned)blocks, p.Hkv, prefix ? pl.prefix_parts : pl.own_parts), kThreads, smem, st>>>(a);
    const int rc2 = cuda_check(cudaGetLastError(), "paged attention launch");
    if (rc2 != HKV_OK) return rc2;
  }
  return HKV_OK;
}

int run_bf16(const PagedAttend& p, const Plan& pl, const Args& a, cudaStream_t st) {
  if (pl.tc) return launch_attend_tc(p, a, false, pl.own_parts, pl.parts ? 0 : -1, st);
  const int64_t items = pl.own_items * pl.own_parts;
  if (items > INT32_MAX / 2) return fail(HKV_ERR_UNSUPPORTED, "too many sequences and heads");
  auto kernel = a.softcap > 0.f || a.slopes ? rows_mma_kernel<true> : rows_mma_kernel<false>;
  int rc = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes),
                      "paged attention smem attribute");
  if (rc != HKV_OK) return rc;
  kernel<<<pl.row_ctas, kWarps * 32, kRingBytes, st>>>(a, (int)items);
  rc = cuda_check(cudaGetLastError(), "paged attention launch");
  return rc == HKV_OK && pl.prefix_parts > 0 ? launch_attend_tc(p, a, true, pl.prefix_parts, 0, st) : rc;
}

template <typename T>
int run(const PagedAttend& p, const Plan& pl, const Args& a, cudaStream_t st) {
  const int rc = sizeof(T) == 2 ? run_bf16(p, pl, a, st) : run_fp32(p, pl, a, st);
  if (rc != HKV_OK || pl.parts == 0) return rc;
  return cuda_check(launch_after(join_parts_kernel<T>, dim3((unsigned)ceil_div(a.T * a.Hq, 4)), 128, 0, st, a),
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
  a.prefix_pages = p.n_prefix > 0 ? ceil_div(p.n_prefix, p.pm.page_size) : 0;
  a.scale = p.scale, a.softcap = p.softcap, a.window = p.window, a.slopes = p.slopes;
  a.prefix_len = p.prefix_len, a.q_first = p.q_first, a.out = p.out, a.lse = p.lse, a.status = p.status;
  a.wait_ns = wait_limit_ns();
  a.prefix_parts = pl.prefix_parts, a.own_parts = pl.own_parts;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.part_ml = reinterpret_cast<float2*>(w);
  a.part_o = reinterpret_cast<float*>(w + pl.o);
  return p.dtype == HKV_BF16 ? run<__nv_bfloat16>(p, pl, a, st) : run<float>(p, pl, a, st);
}

}  // namespace hkv
