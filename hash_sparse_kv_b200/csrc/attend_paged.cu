// Dense attention over a paged cache for few rows at a time: the single-token
// (decode) form of the prompt attention, the own tokens of sequences behind a
// shared prefix, and fp32 caches.
//
// A block takes the rows of up to 16 / g new tokens of one KV head (g query
// heads a token share its keys) and one run of their cache positions, reads
// that run once, and keeps the softmax's running maximum and sum and the
// weighted values in registers (fp32).  Where few blocks would be left, the
// positions are split over several blocks; each stores its partial and the
// last to finish (a ticket per item) joins them.
#include <cstdio>

#include "attend_paged.cuh"

namespace hkv {
namespace {

using pa::Args;

constexpr int kThreads = 256;
constexpr int kRows = 16;
constexpr int kTile = 32;

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

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

// The block's partial result: `m_s`, `l_s` of its rows (shared memory) and
// acc[k], the weighted values of row (tid / 128) * 8 + k, column tid % 128.
template <typename T, bool kPrefix>
__device__ void finish(const Args& a, const Item& it, const float (&acc)[8], const float* m_s, const float* l_s,
                       int* last_s) {
  const int tid = threadIdx.x, col = tid % kHeadDim, r0 = tid / kHeadDim * 8;
  const int64_t n_rows = a.T * a.Hq;
  const int parts = a.prefix_parts + a.own_parts;
  const int mine = kPrefix ? blockIdx.z : a.prefix_parts + blockIdx.z;
  const bool alone = !kPrefix && a.own_parts == 1;  // this block's partial need not go through memory
  if (!alone) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (r0 + k < it.nrows) {
        const int64_t row = mine * n_rows + out_row(a, it, r0 + k);
        a.part_o[row * kHeadDim + col] = acc[k];
        if (col == 0) a.part_ml[row] = make_float2(m_s[r0 + k], l_s[r0 + k]);
      }
    if constexpr (kPrefix) return;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      uint32_t* t = a.tickets + (int64_t)blockIdx.x * a.Hkv + it.j;
      *last_s = atomicAdd(t, 1u) == (uint32_t)a.own_parts - 1;
      if (*last_s) *t = 0;  // ready for the next call
    }
    __syncthreads();
    if (!*last_s) return;
    __threadfence();
  }
  const int from_memory = alone ? a.prefix_parts : parts;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (r0 + k >= it.nrows) continue;
    const int64_t row = out_row(a, it, r0 + k);
    float M = alone ? m_s[r0 + k] : -INFINITY;
    for (int p = 0; p < from_memory; ++p) M = fmaxf(M, __ldcg(&a.part_ml[p * n_rows + row].x));
    float L = 0.f, o = 0.f;
    if (M != -INFINITY) {
      if (alone) {
        const float w = exp2f(m_s[r0 + k] - M);
        L = w * l_s[r0 + k], o = w * acc[k];
      }
      for (int p = 0; p < from_memory; ++p) {
        const float2 ml = __ldcg(&a.part_ml[p * n_rows + row]);
        if (ml.x == -INFINITY) continue;  // an empty part's values need not be written
        const float w = exp2f(ml.x - M);
        L = fmaf(w, ml.y, L);
        o = fmaf(w, __ldcg(&a.part_o[(p * n_rows + row) * kHeadDim + col]), o);
      }
    }
    put(static_cast<T*>(a.out) + row * kHeadDim + col, L > 0.f ? o / L : 0.f);
    if (col == 0 && a.lse) a.lse[row] = L > 0.f ? (M + log2f(L)) * pa::kLn2 : -INFINITY;
  }
}

template <typename T, bool kPrefix>
__global__ void __launch_bounds__(kThreads)
rows_simt_kernel(const __grid_constant__ Args a) {
  constexpr int D = kHeadDim, KP = D + 1;
  __shared__ float q_s[kRows][D];
  __shared__ float k_s[kTile][KP];
  __shared__ float v_s[kTile][D];
  __shared__ float p_s[kRows][kTile];
  __shared__ float m_s[kRows], l_s[kRows], f_s[kRows];
  __shared__ int64_t row_s[kTile];
  __shared__ int last_s;
  const int tid = threadIdx.x;
  Item it;
  if (!item_of<kPrefix>(a, it)) return;
  for (int i = tid; i < kRows * D; i += kThreads) {
    const int r = i / D, d = i % D;
    const T* q = static_cast<const T*>(a.q) + (it.row0 + r / a.g) * a.q_stride + (int64_t)(it.j * a.g + r % a.g) * D;
    q_s[r][d] = r < it.nrows ? to_f32(q[d]) : 0.f;
  }
  // thread (r, u) scores row r against tokens u and u + 16 of a tile
  const int r = tid / 16, u = tid % 16;
  pa::Span sp{0, 0, 0};
  if (r < it.nrows) sp = row_span<kPrefix>(a, it, r);
  const float slope = a.slopes && r < it.nrows ? a.slopes[it.j * a.g + r % a.g] * pa::kLog2e : 0.f;
  __shared__ int lo_s, hi_s;
  if (tid == 0) lo_s = INT32_MAX, hi_s = 0;
  if (u == 0) m_s[r] = -INFINITY, l_s[r] = 0.f;
  __syncthreads();
  if (u == 0 && sp.lo < sp.hi) {
    atomicMin(&lo_s, sp.lo);
    atomicMax(&hi_s, sp.hi);
  }
  __syncthreads();
  const int lo = min(lo_s, hi_s), hi = hi_s;
  const int tiles = (hi - lo + kTile - 1) / kTile, per = (tiles + gridDim.z - 1) / gridDim.z;
  const int t_end = min(tiles, ((int)blockIdx.z + 1) * per);
  const int32_t* table = kPrefix ? a.prefix_table : a.pm.table + (int64_t)it.b * a.pm.max_pages;
  float acc[8] = {};
  const int col = tid % D, ar0 = tid / D * 8;
  for (int t = blockIdx.z * per; t < t_end; ++t) {
    const int u0 = lo + t * kTile;
    __syncthreads();
    if (tid < kTile) {
      row_s[tid] = u0 + tid < hi ? pa::pool_row(a, table, u0 + tid, it.j) : -1;
      if (u0 + tid < hi && row_s[tid] < 0) report(a.status, HKV_ERR_DEVICE_RANGE);
    }
    __syncthreads();
    for (int i = tid; i < kTile * (D / 4); i += kThreads) {
      const int x = i / (D / 4), d = i % (D / 4) * 4;
      float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f), v4 = k4;
      if (row_s[x] >= 0) {
        k4 = load4_f32(static_cast<const T*>(a.K) + row_s[x] * D + d);
        v4 = load4_f32(static_cast<const T*>(a.V) + row_s[x] * D + d);
      }
      k_s[x][d] = k4.x, k_s[x][d + 1] = k4.y, k_s[x][d + 2] = k4.z, k_s[x][d + 3] = k4.w;
      *reinterpret_cast<float4*>(&v_s[x][d]) = v4;
    }
    __syncthreads();
    float z[2] = {0.f, 0.f};
#pragma unroll 8
    for (int d = 0; d < D; ++d) {
      const float q = q_s[r][d];
      z[0] = fmaf(q, k_s[u][d], z[0]);
      z[1] = fmaf(q, k_s[u + 16][d], z[1]);
    }
    float mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = u + 16 * e, pos = u0 + x;
      float s = z[e] * a.scale;
      if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
      s = s * pa::kLog2e - slope * (float)abs(sp.pos - pos);
      z[e] = pos >= sp.lo && pos < sp.hi && row_s[x] >= 0 ? s : -INFINITY;
      mx = fmaxf(mx, z[e]);
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m_old = m_s[r], m_new = fmaxf(m_old, mx), m_use = m_new == -INFINITY ? 0.f : m_new;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float p = exp2f(z[e] - m_use);
      p_s[r][u + 16 * e] = p;
      sum += p;
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    if (u == 0) {
      const float f = exp2f(m_old - m_use);
      f_s[r] = f, m_s[r] = m_new, l_s[r] = l_s[r] * f + sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= f_s[ar0 + k];
#pragma unroll 4
    for (int x = 0; x < kTile; ++x) {
      const float v = v_s[x][col];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(p_s[ar0 + k][x], v, acc[k]);
    }
  }
  __syncthreads();
  finish<T, kPrefix>(a, it, acc, m_s, l_s, &last_s);
}

// Splits that fill the GPU about twice over, each with at least four tiles.
int splits_for(int64_t items, int64_t tokens, int tile) {
  const int64_t want = ceil_div(2 * (int64_t)sm_count(), items < 1 ? 1 : items);
  const int64_t most = ceil_div(tokens, 4 * (int64_t)tile);
  const int64_t s = want < most ? want : most;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

// How a call is cut up; from its shape and the device alone, so that the
// workspace can be sized before the call.
struct Plan {
  bool tc = false;         // prompts: the tensor-core kernel takes all rows
  bool tc_prefix = false;  // it takes the shared prefix
  int64_t own_items = 0;
  int prefix_parts = 0, own_parts = 1;
  size_t ml = 0, o = 0, total = 0;  // byte offsets of part_ml and part_o, and the size
};

Plan plan(const PagedAttend& p) {
  Plan r;
  const int g = p.Hq / p.Hkv, tpt = kRows / g;
  const bool bf16 = p.dtype == HKV_BF16;
  int64_t parts = 0;
  // a sequence's new tokens fill more than the 16 rows of one block: 128-row tiles
  r.tc = bf16 && p.cu_q_rows && (int64_t)p.max_q * g > kRows;
  if (r.tc) {
    r.own_parts = tc_splits(p, false);
  } else {
    r.own_items = (int64_t)p.B * ceil_div(p.max_q, tpt);
    r.own_parts = splits_for(r.own_items * p.Hkv, p.n_max, kTile);
    r.tc_prefix = bf16 && p.n_prefix > 0;
    if (r.tc_prefix)
      r.prefix_parts = tc_splits(p, true);
    else if (p.n_prefix > 0)
      r.prefix_parts = splits_for(ceil_div(p.B, tpt) * p.Hkv, p.n_prefix, kTile);
  }
  parts = r.prefix_parts + (r.own_parts > 1 ? r.own_parts : 0);
  r.ml = align_up(sizeof(uint32_t) * r.own_items * p.Hkv, 256);
  r.o = r.ml + align_up(sizeof(float2) * parts * p.T * p.Hq, 256);
  r.total = parts ? r.o + sizeof(float) * kHeadDim * parts * p.T * p.Hq : 0;
  return r;
}

template <typename T>
int run(const PagedAttend& p, const Plan& pl, Args& a, cudaStream_t st) {
  if (pl.tc) return launch_attend_tc(p, a, false, pl.own_parts, pl.own_parts > 1 ? 0 : -1, st);
  if (pl.tc_prefix) {
    const int rc = launch_attend_tc(p, a, true, pl.prefix_parts, 0, st);
    if (rc != HKV_OK) return rc;
  } else if (pl.prefix_parts > 0) {
    const dim3 grid((unsigned)ceil_div(p.B, kRows / a.g), p.Hkv, pl.prefix_parts);
    rows_simt_kernel<T, true><<<grid, kThreads, 0, st>>>(a);
    const int rc = cuda_check(cudaGetLastError(), "prefix attention launch");
    if (rc != HKV_OK) return rc;
  }
  const dim3 grid((unsigned)pl.own_items, p.Hkv, pl.own_parts);
  rows_simt_kernel<T, false><<<grid, kThreads, 0, st>>>(a);
  return cuda_check(cudaGetLastError(), "paged attention launch");
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
  a.tickets = reinterpret_cast<uint32_t*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + pl.ml);
  a.part_o = reinterpret_cast<float*>(w + pl.o);
  return p.dtype == HKV_BF16 ? run<__nv_bfloat16>(p, pl, a, st) : run<float>(p, pl, a, st);
}

}  // namespace hkv
