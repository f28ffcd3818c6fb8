// Appending new keys and values to a paged cache, with the rotary positions
// applied on the way and the hash codes of the stored keys beside them.
//
// Pair i of a head (elements i and i + pairs, or 2 i and 2 i + 1 when
// interleaved) turns by the angle a = position * inv_freq[i]:
//   y_lo = x_lo cos a - x_hi sin a,   y_hi = x_hi cos a + x_lo sin a
// The angle is taken in fp64 (a position of 2^19 times an fp32 frequency has
// up to 43 significant bits), reduced to one turn by two fused steps, and its
// sine and cosine are rounded once to fp32; products and sums are separate
// fp32 operations, so the stored key does not depend on how the compiler
// contracts them, and the codes are those of the stored (rounded) key.
//
// Every byte is read once and written once: 8 lanes own one row of 128
// elements, each lane two chunks of 8 that hold both members of its pairs, so
// a row is turned in registers and moves as 16-byte accesses.  A block takes a
// group of tokens at a time; its angles are computed once and serve all of
// the tokens' heads.  The bf16 projection hash runs on the block's keys while
// they are still in shared memory (mma.sync m16n8k16: the 2 * 128 * bits flops
// per key are far below what the key's own traffic allows).
#include <cstdio>

#include "attend_paged.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowLanes = 8;                          // lanes of one row
constexpr int kSlots = kThreads / kRowLanes;          // rows in flight per block and pass
constexpr int kMaxGroup = 8;                          // tokens per block and step
constexpr int kKeyPitch = kHeadDim + 8;               // shared key rows: 272 bytes, conflict-free for ldmatrix
enum { kHashNone = 0, kHashSign = 1, kHashLsh = 2, kHashStage = 3 };

struct AppendArgs {
  int B, Hq, Hkv, group, pairs, interleaved, words;
  int64_t T;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, qo_stride;
  void* q_out;
  const int32_t *cu, *n_past, *positions;
  const float* inv_freq;
  void *K, *V;
  uint32_t* codes;
  uint16_t* norms;
  const void* R;
  void* staged;  // kHashStage: the stored keys again, [T, Hkv, 128]
  PageMap pm;
  int32_t* status;
  uint8_t axis[64];
};

struct Chunk {
  float x[8];
};
__device__ __forceinline__ Chunk load_chunk(const __nv_bfloat16* p) {
  Chunk c;
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c.x[2 * i] = __uint_as_float(w[i] << 16);
    c.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return c;
}
__device__ __forceinline__ Chunk load_chunk(const float* p) {
  Chunk c;
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  c.x[0] = a.x, c.x[1] = a.y, c.x[2] = a.z, c.x[3] = a.w;
  c.x[4] = b.x, c.x[5] = b.y, c.x[6] = b.z, c.x[7] = b.w;
  return c;
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const Chunk& c) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(c.x[2 * i], c.x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_chunk(float* p, const Chunk& c) {
  *reinterpret_cast<float4*>(p) = make_float4(c.x[0], c.x[1], c.x[2], c.x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(c.x[4], c.x[5], c.x[6], c.x[7]);
}
// the value that the cache holds for x
__device__ __forceinline__ float stored(float x, const __nv_bfloat16*) { return __bfloat162float(__float2bfloat16_rn(x)); }
__device__ __forceinline__ float stored(float x, const float*) { return x; }

__device__ __forceinline__ void turn(float& lo, float& hi, float2 cs) {
  const float a = __fsub_rn(__fmul_rn(lo, cs.x), __fmul_rn(hi, cs.y));
  hi = __fadd_rn(__fmul_rn(hi, cs.x), __fmul_rn(lo, cs.y));
  lo = a;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T, int HASH>
__global__ void __launch_bounds__(kThreads)
append_paged_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int D = kHeadDim;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 cs[kMaxGroup][64];   // (cos, sin) of each token's angles
  __shared__ int64_t row0[kMaxGroup];    // pool row of (token, KV head 0); -1: nothing is written
  __shared__ int32_t at[kMaxGroup];      // position in the cache
  __nv_bfloat16* keys = reinterpret_cast<__nv_bfloat16*>(smem);  // kHashLsh: [group * Hkv, rounded up to 16][kKeyPitch]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = tid % kRowLanes, slot = tid / kRowLanes;
  const int rows_tok = a.Hq + 2 * a.Hkv;  // rows of one token (Hq is 0 when no queries are given)
  const T* const xq = static_cast<const T*>(a.q);
  const T* const xk = static_cast<const T*>(a.k);
  const T* const xv = static_cast<const T*>(a.v);
  // this lane's two chunks: both members of its pairs, or two untouched chunks behind the turned part
  const int pc = a.pairs / 8;
  const bool split = !a.interleaved && c < pc;
  const int c0 = split ? c : 2 * c, c1 = split ? c + pc : 2 * c + 1;

  // kHashLsh: warp w computes bits [16 w, 16 w + 16) (bits [8 w, 8 w + 8) of a 64-bit code)
  const int ntile = HASH == kHashLsh ? a.words / 2 : 0;  // n8 tiles per warp: 2 or 1
  uint32_t rb[2][8][2];
  if constexpr (HASH == kHashLsh) {
    const __nv_bfloat16* R = static_cast<const __nv_bfloat16*>(a.R);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int bit = (warp * ntile + n) * 8 + lane / 4;
        const uint32_t* p = reinterpret_cast<const uint32_t*>(R + (int64_t)bit * D + kk * 16) + lane % 4;
        rb[n][kk][0] = n < ntile ? __ldg(p) : 0u;
        rb[n][kk][1] = n < ntile ? __ldg(p + 4) : 0u;
      }
    // rows behind the group's last key are multiplied too: give them a value
    for (int i = tid; i < (a.group * a.Hkv + 15) / 16 * 16 * kKeyPitch; i += kThreads) keys[i] = __nv_bfloat16(0.f);
  }

  for (int64_t t0 = (int64_t)blockIdx.x * a.group; t0 < a.T; t0 += (int64_t)gridDim.x * a.group) {
    const int nt = (int)min((int64_t)a.group, a.T - t0);
    __syncthreads();  // the last step's angles, slots and keys have been used
    if (warp < nt) {
      const int64_t t = t0 + warp;
      const int b = pa::find_seq(a.cu, a.B, t);
      if (lane == 0) {
        const int64_t first = a.cu[b], end = a.cu[b + 1];
        int64_t row = -1;
        int64_t pos = (int64_t)a.n_past[b] + t - first;
        const bool live = t >= first && t < end;  // else behind the last sequence: left alone
        if (live) {
          if (pos < 0 || pos >= a.pm.max_pages * a.pm.page_size) {
            report(a.status, HKV_ERR_DEVICE_RANGE);
          } else {
            const int64_t page = a.pm.table[(int64_t)b * a.pm.max_pages + pos / a.pm.page_size];
            if (page < 0 || page >= a.pm.num_pages)
              report(a.status, HKV_ERR_DEVICE_RANGE);
            else
              row = page * a.Hkv * a.pm.page_size + pos % a.pm.page_size;
          }
        }
        row0[warp] = live ? (row < 0 ? -2 : row) : -1;  // -2: no slot, the queries are still turned
        at[warp] = (int32_t)pos;
      }
    }
    __syncthreads();
    for (int i = tid; i < nt * a.pairs; i += kThreads) {
      const int tok = i / a.pairs, p = i % a.pairs;
      if (row0[tok] == -1) continue;
      const int pos = a.positions ? __ldg(a.positions + (int64_t)a.axis[p] * a.T + t0 + tok) : at[tok];
      const double ang = (double)pos * (double)__ldg(a.inv_freq + p);
      const double n = rint(ang * 0.15915494309189535);
      double r = fma(-n, 6.283185307179586, ang);
      r = fma(-n, 2.4492935982947064e-16, r);
      double s, co;
      sincos(r, &s, &co);
      cs[tok][p] = make_float2((float)co, (float)s);
    }
    __syncthreads();
    for (int i = slot; i < nt * rows_tok; i += kSlots) {
      const int tok = i / rows_tok, r = i % rows_tok;
      const int64_t base = row0[tok];
      const int64_t t = t0 + tok;
      const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv;
      const int j = is_q ? r : is_v ? r - a.Hq - a.Hkv : r - a.Hq;
      const bool skip = base == -1 || (base == -2 && !is_q);
      const T* src = is_q ? xq + t * a.q_stride : is_v ? xv + t * a.v_stride : xk + t * a.k_stride;
      src += (int64_t)j * D;
      Chunk u, w;
      if (!skip) {
        u = load_chunk(src + c0 * 8);
        w = load_chunk(src + c1 * 8);
        if (!is_v) {
          if (split) {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn(u.x[e], w.x[e], cs[tok][c * 8 + e]);
          } else if (a.interleaved && c < pc) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              turn(u.x[2 * e], u.x[2 * e + 1], cs[tok][c * 8 + e]);
              turn(w.x[2 * e], w.x[2 * e + 1], cs[tok][c * 8 + 4 + e]);
            }
          }
        }
        T* dst;
        if (is_q)
          dst = static_cast<T*>(a.q_out) + t * a.qo_stride + (int64_t)j * D;
        else
          dst = static_cast<T*>(is_v ? a.V : a.K) + (base + (int64_t)j * a.pm.page_size) * D;
        store_chunk(dst + c0 * 8, u);
        store_chunk(dst + c1 * 8, w);
        if (!is_q && !is_v) {
          if constexpr (HASH == kHashLsh) {
            T* kd = reinterpret_cast<T*>(keys + (tok * a.Hkv + j) * kKeyPitch);
            store_chunk(kd + c0 * 8, u);
            store_chunk(kd + c1 * 8, w);
          }
          if constexpr (HASH == kHashStage) {
            T* kd = static_cast<T*>(a.staged) + (t * a.Hkv + j) * D;
            store_chunk(kd + c0 * 8, u);
            store_chunk(kd + c1 * 8, w);
          }
        }
      }
      if constexpr (HASH == kHashSign) {
        // signs and fp16 norm of the stored key; the eight lanes of a row are
        // all here or all not, so the shuffles stay within the row's lanes
        if (!skip && !is_q && !is_v) {
          const uint32_t mask = 0xffu << (lane & 24);
          uint32_t word[4] = {0u, 0u, 0u, 0u};
          double ss = 0.0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int ch = h ? c1 : c0;
            uint32_t byte = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = stored(h ? w.x[e] : u.x[e], src);
              byte |= (uint32_t)(x > 0.f) << e;
              ss = fma((double)x, (double)x, ss);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z)
              if (ch / 4 == z) word[z] |= byte << (8 * (ch % 4));
          }
#pragma unroll
          for (int o = 1; o < kRowLanes; o <<= 1) {
#pragma unroll
            for (int z = 0; z < 4; ++z) word[z] |= __shfl_xor_sync(mask, word[z], o);
            ss += __shfl_xor_sync(mask, ss, o);
          }
          if (c == 0) {
            const int64_t row = base + (int64_t)j * a.pm.page_size;
            *reinterpret_cast<uint4*>(a.codes + row * 4) = make_uint4(word[0], word[1], word[2], word[3]);
            if (a.norms) a.norms[row] = __half_as_ushort(__double2half(sqrt(ss)));
          }
        }
      }
    }
    if constexpr (HASH == kHashLsh) {
      __syncthreads();
      const int rows = nt * a.Hkv;
      for (int m0 = 0; m0 < rows; m0 += 16) {
        float y[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t af[4];
          ldsm4(af, keys + (m0 + lane % 16) * kKeyPitch + kk * 16 + (lane / 16) * 8);
          mma16816(y[0], af, rb[0][kk][0], rb[0][kk][1]);
          if (ntile == 2) mma16816(y[1], af, rb[1][kk][0], rb[1][kk][1]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // rows lane / 4 and lane / 4 + 8
          uint32_t bits = 0;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) bits |= (uint32_t)(y[n][2 * h + e] > 0.f) << (n * 8 + (lane % 4) * 2 + e);
          bits |= __shfl_xor_sync(0xffffffffu, bits, 1);
          bits |= __shfl_xor_sync(0xffffffffu, bits, 2);
          const int i = m0 + lane / 4 + 8 * h;
          if (lane % 4 == 0 && i < rows && row0[i / a.Hkv] >= 0) {
            const int64_t row = row0[i / a.Hkv] + (int64_t)(i % a.Hkv) * a.pm.page_size;
            if (ntile == 2)
              reinterpret_cast<uint16_t*>(a.codes + row * 4)[warp] = (uint16_t)bits;
            else
              reinterpret_cast<uint8_t*>(a.codes + row * 2)[warp] = (uint8_t)bits;
          }
        }
      }
    }
  }
}

// Codes of the staged keys to their places in the pool: one thread per
// (token, KV head).
__global__ void __launch_bounds__(kThreads)
scatter_codes_kernel(const __grid_constant__ AppendArgs a, const uint32_t* __restrict__ staged_codes) {
  const int64_t n = a.T * a.Hkv;
  const int lane = threadIdx.x & 31;
  for (int64_t w0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * 32; w0 < n; w0 += (int64_t)gridDim.x * kThreads) {
    const int64_t i = w0 + lane;
    // a warp's rows belong to few tokens: find each one's sequence together
    const int64_t t_lo = w0 / a.Hkv, t_hi = min(n - 1, w0 + 31) / a.Hkv;
    for (int64_t t = t_lo; t <= t_hi; ++t) {
      const int b = pa::find_seq(a.cu, a.B, t);
      if (i >= n || i / a.Hkv != t) continue;
      const int64_t first = a.cu[b], end = a.cu[b + 1], pos = (int64_t)a.n_past[b] + t - first;
      if (t < first || t >= end || pos < 0 || pos >= a.pm.max_pages * a.pm.page_size) continue;
      const int64_t page = a.pm.table[(int64_t)b * a.pm.max_pages + pos / a.pm.page_size];
      if (page < 0 || page >= a.pm.num_pages) continue;
      const int64_t row = (page * a.Hkv + i % a.Hkv) * a.pm.page_size + pos % a.pm.page_size;
      for (int w = 0; w < a.words; ++w) a.codes[row * a.words + w] = staged_codes[i * a.words + w];
    }
  }
}

template <typename T>
int run_append(const AppendArgs& a, int hash, cudaStream_t st) {
  auto kernel = hash == kHashSign ? append_paged_kernel<T, kHashSign>
                : hash == kHashStage ? append_paged_kernel<T, kHashStage> : append_paged_kernel<T, kHashNone>;
  size_t smem = 0;
  if constexpr (sizeof(T) == 2) {
    if (hash == kHashLsh) {
      kernel = append_paged_kernel<T, kHashLsh>;
      smem = align_up((size_t)a.group * a.Hkv, 16) * kKeyPitch * sizeof(T);
      if (smem + 8192 > (size_t)max_smem_optin()) return fail(HKV_ERR_UNSUPPORTED, "Hkv %d too large", a.Hkv);
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return cuda_check(e, "append smem attribute");
    }
  }
  const int64_t steps = ceil_div(a.T, a.group), most = (int64_t)sm_count() * 4;
  kernel<<<(unsigned)(steps < most ? steps : most), kThreads, smem, st>>>(a);
  return cuda_check(cudaGetLastError(), "append launch");
}

}  // namespace

size_t append_ws_bytes(const hkv_hash* h, int64_t T, int Hkv) {
  if (h == nullptr || h->kind == HKV_HASH_SIGN || (h->kind == HKV_HASH_LSH && h->dtype == HKV_BF16)) return 0;
  const size_t elt = h->dtype == HKV_BF16 ? 2 : 4;
  return align_up((size_t)T * Hkv * kHeadDim * elt, 256) + align_up((size_t)T * Hkv * (h->code_bits / 8), 256);
}

int launch_append_paged(const AppendPaged& p, const PageMap& pm, void* ws, cudaStream_t st) {
  AppendArgs a{};
  a.B = p.B, a.Hq = p.q ? p.Hq : 0, a.Hkv = p.Hkv, a.T = p.T;
  a.q = p.q, a.k = p.k_new, a.v = p.v_new, a.q_out = p.q_out;
  a.q_stride = p.q_stride, a.qo_stride = p.qo_stride, a.k_stride = p.k_stride, a.v_stride = p.v_stride;
  a.cu = p.cu_new, a.n_past = p.n_past, a.positions = p.positions;
  a.K = p.K_pool, a.V = p.V_pool, a.codes = p.codes_pool, a.norms = p.norms_pool;
  a.pm = pm, a.status = p.status;
  if (p.rope) {
    a.pairs = p.rope->pairs, a.interleaved = p.rope->interleaved, a.inv_freq = p.rope->inv_freq;
    for (int i = 0; i < 64; ++i) a.axis[i] = p.rope->axis[i];
  }
  int hash = kHashNone;
  if (p.hash) {
    a.words = p.hash->code_bits / 32, a.R = p.hash->R;
    hash = p.hash->kind == HKV_HASH_SIGN ? kHashSign
           : p.hash->kind == HKV_HASH_LSH && p.hash->dtype == HKV_BF16 ? kHashLsh : kHashStage;
  }
  // One token per step while that leaves SMs idle (latency); else groups that
  // share the angles' and slots' latency over up to 8 tokens, with at most 64
  // keys (four 16-row tiles) in shared memory for the projection.
  int group = (int)(p.T / (2 * sm_count()));
  const int most = p.Hkv <= 8 ? kMaxGroup : p.Hkv >= 64 ? 1 : 64 / p.Hkv;
  a.group = group < 1 ? 1 : group > most ? most : group;
  a.staged = ws;
  int rc = p.dtype == HKV_BF16 ? run_append<__nv_bfloat16>(a, hash, st) : run_append<float>(a, hash, st);
  if (rc != HKV_OK || hash != kHashStage) return rc;
  // other hashes: their encoders read the stored keys' copy, then the codes move to the pool
  const size_t elt = p.dtype == HKV_BF16 ? 2 : 4;
  const int64_t rows = p.T * p.Hkv;
  uint32_t* codes = reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(ws) + align_up((size_t)rows * kHeadDim * elt, 256));
  RowMap m{rows, rows, 0, kHeadDim, 0, a.words, 0, 1};
  rc = launch_encode(*p.hash, ws, m, codes, nullptr, st, p.status);
  if (rc != HKV_OK) return rc;
  const int64_t blocks = ceil_div(rows, kThreads), cap = (int64_t)sm_count() * 8;
  scatter_codes_kernel<<<(unsigned)(blocks < cap ? blocks : cap), kThreads, 0, st>>>(a, codes);
  return cuda_check(cudaGetLastError(), "append scatter launch");
}

}  // namespace hkv
