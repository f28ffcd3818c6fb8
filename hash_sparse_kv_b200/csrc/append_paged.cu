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
// a row is turned in registers and moves as 16-byte accesses.  A warp takes one
// token (or, when there are few, a part of its rows): it finds the token's
// place, takes the angles, keeps each lane's eight in registers for all of the
// token's heads, and goes through the rows four at a time with the next four
// on their way.  Warps need no one else, but for the bf16 projection hash,
// which runs on the keys of a block's tokens while they are still in shared
// memory (mma.sync m16n8k16: the 2 * 128 * bits flops per key are far below
// what the key's own traffic allows).
#include <cstdio>

#include "attend_paged.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowLanes = 8;                     // lanes of one row
constexpr int kKeyPitch = kHeadDim + 8;          // shared key rows: 272 bytes, conflict-free for ldmatrix
constexpr int kMaxKeys = 64;                     // keys of a step in shared memory, unless one token has more
enum { kHashNone = 0, kHashSign = 1, kHashLsh = 2, kHashStage = 3 };

struct AppendArgs {
  int B, Hq, Hkv, parts, pairs, interleaved, words;  // parts: warps of one token
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

// Eight consecutive elements as they lie in memory, and widened to fp32.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
struct Chunk {
  float x[8];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ Chunk widen(const Raw<__nv_bfloat16>& r) {
  Chunk c;
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c.x[2 * i] = __uint_as_float(w[i] << 16);
    c.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return c;
}
__device__ __forceinline__ Chunk widen(const Raw<float>& r) {
  return Chunk{{__uint_as_float(r.v[0].x), __uint_as_float(r.v[0].y), __uint_as_float(r.v[0].z), __uint_as_float(r.v[0].w),
                __uint_as_float(r.v[1].x), __uint_as_float(r.v[1].y), __uint_as_float(r.v[1].z), __uint_as_float(r.v[1].w)}};
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

// Where new token t goes: the pool row of its KV head 0, -1 for a token behind
// the last sequence, -2 for one without a place (its queries are still
// turned).  The whole warp takes part and gets the same answer.
struct Place {
  int64_t row;
  int32_t pos;
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int64_t t) {
  const int b = pa::find_seq(a.cu, a.B, t);
  const int64_t first = a.cu[b], end = a.cu[b + 1];
  if (t < first || t >= end) return Place{-1, 0};
  const int64_t pos = (int64_t)a.n_past[b] + t - first;
  if (pos < 0 || pos >= a.pm.max_pages * a.pm.page_size) return Place{-2, (int32_t)pos};
  const uint32_t P = a.pm.page_size, at = (uint32_t)pos / P;
  const int64_t page = a.pm.table[(int64_t)b * a.pm.max_pages + at];
  if (page < 0 || page >= a.pm.num_pages) return Place{-2, (int32_t)pos};
  return Place{page * a.Hkv * P + ((uint32_t)pos - at * P), (int32_t)pos};
}

// fp16 norm of a row from its squares' sum, as the sign encoder's: the fp32
// sum of bf16 squares is off by less than 8e-6, which matters only next to a
// rounding border; there, and for fp32 rows, the fp64 sum decides.
template <typename T>
__device__ __forceinline__ uint16_t row_norm(const Chunk& u, const Chunk& w) {
  float ss = 0.f;
#pragma unroll
  for (int z = 0; z < 8; ++z) ss = fmaf(u.x[z], u.x[z], fmaf(w.x[z], w.x[z], ss));
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float n = sqrtf(ss);
  const uint16_t lo = __half_as_ushort(__float2half_rn(n * (1.f - 8e-6f))), hi = __half_as_ushort(__float2half_rn(n * (1.f + 8e-6f)));
  uint16_t out = hi;
  if (__any_sync(0xffffffffu, sizeof(T) == 4 || lo != hi)) {
    double d = 0.0;
#pragma unroll
    for (int z = 0; z < 8; ++z) d = fma((double)u.x[z], (double)u.x[z], fma((double)w.x[z], (double)w.x[z], d));
#pragma unroll
    for (int o = 1; o < kRowLanes; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    out = __half_as_ushort(__double2half(sqrt(d)));
  }
  return out;
}

template <typename T, int HASH>
__global__ void __launch_bounds__(kThreads, HASH == kHashLsh ? 2 : 3)
append_paged_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int D = kHeadDim;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float2 cs_s[kWarps][64];  // (cos, sin) of a warp's token
  __shared__ int64_t row_s[2][kWarps];               // kHashLsh: pool rows of a step's tokens
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane % kRowLanes, sub = lane / kRowLanes;
  const int tokens = kWarps / a.parts, part = warp % a.parts;  // tokens of the block per step
  // this lane's two chunks: both members of its pairs, or two untouched chunks behind the turned part
  const int pc = a.pairs / 8;
  const bool turned = c < pc, split = !a.interleaved && turned;
  const int c0 = (split ? c : 2 * c) * 8, c1 = (split ? c + pc : 2 * c + 1) * 8;
  // a token's rows four at a time: queries, keys, values
  const int q4 = (a.Hq + 3) / 4, k4 = (a.Hkv + 3) / 4, all4 = q4 + 2 * k4;

  // kHashLsh: warp w computes bits [16 w, 16 w + 16) (bits [8 w, 8 w + 8) of a 64-bit code)
  const int key_rows = (tokens * a.Hkv + 15) / 16 * 16;
  __nv_bfloat16* keys = reinterpret_cast<__nv_bfloat16*>(smem);  // kHashLsh: [2][key_rows][kKeyPitch]
  const int ntile = HASH == kHashLsh ? a.words / 2 : 0;          // n8 tiles per warp: 2 or 1
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
    // rows behind a step's last key are multiplied too: give them a value
    for (int i = tid; i < 2 * key_rows * kKeyPitch; i += kThreads) keys[i] = __nv_bfloat16(0.f);
    __syncthreads();
  }

  int buf = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.T; t0 += (int64_t)gridDim.x * tokens) {
    const int64_t t = t0 + warp / a.parts;
    if (t < a.T) {
      const T* const xq = static_cast<const T*>(a.q) + t * a.q_stride;
      const T* const xk = static_cast<const T*>(a.k) + t * a.k_stride;
      const T* const xv = static_cast<const T*>(a.v) + t * a.v_stride;
      // row `sub` of group i: which head, and where it comes from
      auto row_of = [&](int i, int& head, int& heads) -> const T* {
        const bool is_q = i < q4, is_k = i < q4 + k4;
        head = (is_q ? i : is_k ? i - q4 : i - q4 - k4) * 4 + sub;
        heads = is_q ? a.Hq : a.Hkv;
        return (is_q ? xq : is_k ? xk : xv) + head * D;
      };
      int head, heads;
      Raw<T> ra{}, rw{};
      {
        const T* src = row_of(part, head, heads);
        if (part < all4 && head < heads) ra = load_raw(src + c0), rw = load_raw(src + c1);
      }
      const Place at = place_of(a, t);
      if (lane == 0 && part == 0) {
        if (at.row == -2) report(a.status, HKV_ERR_DEVICE_RANGE);
        if (HASH == kHashLsh) row_s[buf][warp / a.parts] = at.row;
      }
      if (at.row != -1) {
        for (int p = lane; p < a.pairs; p += 32) {
          const int pos = a.positions ? __ldg(a.positions + (int64_t)a.axis[p] * a.T + t) : at.pos;
          const double ang = (double)pos * (double)__ldg(a.inv_freq + p);
          const double n = rint(ang * 0.15915494309189535);
          double r = fma(-n, 6.283185307179586, ang);
          r = fma(-n, 2.4492935982947064e-16, r);
          double s, co;
          sincos(r, &s, &co);
          cs_s[warp][p] = make_float2((float)co, (float)s);
        }
        __syncwarp();
        float2 cs[8];
        if (turned) {
#pragma unroll
          for (int z = 0; z < 8; z += 2) {
            const float4 x = *reinterpret_cast<const float4*>(&cs_s[warp][c * 8 + z]);
            cs[z] = make_float2(x.x, x.y), cs[z + 1] = make_float2(x.z, x.w);
          }
        }
        __syncwarp();
        T* const oq = static_cast<T*>(a.q_out) + t * a.qo_stride;
#pragma unroll 1
        for (int i = part; i < all4; i += a.parts) {
          const Raw<T> xa = ra, xw = rw;
          const int h = head;
          const bool is_q = i < q4, is_k = !is_q && i < q4 + k4, in = h < heads && (is_q || at.row >= 0);
          if (i + a.parts < all4) {
            const T* src = row_of(i + a.parts, head, heads);
            if (head < heads) ra = load_raw(src + c0), rw = load_raw(src + c1);
          }
          T* dst = is_q ? oq + h * D : static_cast<T*>(is_k ? a.K : a.V) + (at.row + (int64_t)h * a.pm.page_size) * D;
          Chunk u = widen(xa), w = widen(xw);
          if (turned && (is_q || is_k)) {
            if (split) {
#pragma unroll
              for (int z = 0; z < 8; ++z) turn(u.x[z], w.x[z], cs[z]);
            } else {
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                turn(u.x[2 * z], u.x[2 * z + 1], cs[z]);
                turn(w.x[2 * z], w.x[2 * z + 1], cs[4 + z]);
              }
            }
          }
          if (in) {
            store_chunk(dst + c0, u);
            store_chunk(dst + c1, w);
          }
          if constexpr (HASH == kHashLsh) {
            if (is_k && in) {
              T* kd = reinterpret_cast<T*>(keys + (buf * key_rows + warp / a.parts * a.Hkv + h) * kKeyPitch);
              store_chunk(kd + c0, u);
              store_chunk(kd + c1, w);
            }
          }
          if constexpr (HASH == kHashStage) {
            if (is_k && in) {
              T* kd = static_cast<T*>(a.staged) + (t * a.Hkv + h) * D;
              store_chunk(kd + c0, u);
              store_chunk(kd + c1, w);
            }
          }
          if constexpr (HASH == kHashSign) {
            if (is_k) {  // the whole warp: signs and norms of the stored keys
              uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                Chunk& x = half ? w : u;
                const int ch = (half ? c1 : c0) / 8;
                uint32_t byte = 0;
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                  x.x[z] = stored(x.x[z], static_cast<const T*>(nullptr));
                  byte |= (uint32_t)(x.x[z] > 0.f) << z;
                }
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  if (ch / 4 == z) word[z] |= byte << (8 * (ch % 4));
              }
#pragma unroll
              for (int o = 1; o < kRowLanes; o <<= 1)
#pragma unroll
                for (int z = 0; z < 4; ++z) word[z] |= __shfl_xor_sync(0xffffffffu, word[z], o);
              const int64_t row = at.row + (int64_t)h * a.pm.page_size;
              if (in && c == 0) *reinterpret_cast<uint4*>(a.codes + row * 4) = make_uint4(word[0], word[1], word[2], word[3]);
              if (a.norms) {
                const uint16_t norm = row_norm<T>(u, w);
                if (in && c == 0) a.norms[row] = norm;
              }
            }
          }
        }
      }
    }
    if constexpr (HASH == kHashLsh) {
      __syncthreads();  // a step's keys are there; the other buffer has been used
      const int rows = (int)min((int64_t)tokens, a.T - t0) * a.Hkv;
      for (int m0 = 0; m0 < rows; m0 += 16) {
        float y[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t af[4];
          ldsm4(af, keys + (buf * key_rows + m0 + lane % 16) * kKeyPitch + kk * 16 + (lane / 16) * 8);
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
          const int tok = i / a.Hkv;
          if (lane % 4 == 0 && i < rows && row_s[buf][tok] >= 0) {
            const int64_t row = row_s[buf][tok] + (int64_t)(i - tok * a.Hkv) * a.pm.page_size;
            if (ntile == 2)
              reinterpret_cast<uint16_t*>(a.codes + row * 4)[warp] = (uint16_t)bits;
            else
              reinterpret_cast<uint8_t*>(a.codes + row * 2)[warp] = (uint8_t)bits;
          }
        }
      }
      buf ^= 1;
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
      smem = 2 * align_up((size_t)(kWarps / a.parts) * a.Hkv, 16) * kKeyPitch * sizeof(T);
      if (smem + 8192 > (size_t)max_smem_optin()) return fail(HKV_ERR_UNSUPPORTED, "Hkv %d too large", a.Hkv);
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return cuda_check(e, "append smem attribute");
    }
  }
  const int64_t steps = ceil_div(a.T, kWarps / a.parts), most = (int64_t)sm_count() * (hash == kHashLsh ? 2 : 3);
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
  // A warp per token once there are enough of them to fill the SMs; before
  // that, up to eight warps share a token's rows.
  a.parts = 1;
  while (a.parts < kWarps && p.T * a.parts * 2 <= (int64_t)sm_count() * 24) a.parts *= 2;
  if (hash == kHashLsh)
    while (a.parts < kWarps && kWarps / a.parts * p.Hkv > kMaxKeys) a.parts *= 2;
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
