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
//
// Bound by memory, with the arithmetic of the turn close behind (15396 prompt
// tokens of 32 / 8 heads with sign codes: 71 us, 5.4 TB/s, the ALU busy 55% of
// the time); with the projection (9725 tokens, 64 bits: 61.5 us, 3.9 TB/s, 49
// without a hash) by the loads that 24 warps an SM can keep on their way, none
// of them while a step is hashed.  One token takes 5 us, a chain of latencies:
// the sequence and its page, the angles, the rows.  (Device times of a captured
// graph; among other calls 75, 63.5 and 14.)  Hashes by way of the workspace, for
// the same 9725 tokens: MLP of 128 units and bits 74 us, fp32 LSH 177.
#include <cstdio>

#include "attend_paged.cuh"

namespace hkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowLanes = 8;                     // lanes of one row
constexpr int kKeyPitch = kHeadDim + 8;          // shared key rows: 272 bytes, conflict-free for ldmatrix
constexpr int kMaxKeys = 64;                     // keys of a step in shared memory, unless one token has more
// Blocks per SM.  More warps hide the memory's latency best (15396 prompt tokens
// with the sign hash: 84, 76 and 72 us with two, three and four).  The
// projection's blocks are three, since with 128 bits and 64 keys a step they take
// 70 KB each, and 76 registers a thread: their warps have two groups of rows on
// their way instead of one.
enum { kHashNone = 0, kHashSign = 1, kHashLsh = 2, kHashStage = 3 };
constexpr int blocks_per_sm(int hash) { return hash == kHashLsh ? 3 : 4; }

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
  uint64_t most;  // positions that have a place: those of the page table, as far as int32 goes
  int32_t* status;
  uint8_t axis[64];
};

// Eight consecutive elements as they lie in memory, and widened to fp32.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
// Eight values as four pairs: one instruction works on two.
struct Chunk {
  uint64_t x[4];
};
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
// Pair k is elements (2 k, 2 k + 1); with kZip, chunk `u` gets the even elements
// of both chunks and `w` the odd ones, so that a pair of neighbours is one
// element of each.
template <bool kZip>
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& a, const Raw<__nv_bfloat16>& b, Chunk& u, Chunk& w) {
  const uint32_t p[8] = {a.v[0].x, a.v[0].y, a.v[0].z, a.v[0].w, b.v[0].x, b.v[0].y, b.v[0].z, b.v[0].w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (kZip) {
      u.x[k] = pair(p[2 * k] << 16, p[2 * k + 1] << 16);
      w.x[k] = pair(p[2 * k] & 0xffff0000u, p[2 * k + 1] & 0xffff0000u);
    } else {
      u.x[k] = pair(p[k] << 16, p[k] & 0xffff0000u);
      w.x[k] = pair(p[4 + k] << 16, p[4 + k] & 0xffff0000u);
    }
  }
}
template <bool kZip>
__device__ __forceinline__ void widen(const Raw<float>& a, const Raw<float>& b, Chunk& u, Chunk& w) {
  const uint4 q[4] = {a.v[0], a.v[1], b.v[0], b.v[1]};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (kZip) {
      u.x[k] = pair(q[k].x, q[k].z), w.x[k] = pair(q[k].y, q[k].w);
      u.x[2 + k] = pair(q[2 + k].x, q[2 + k].z), w.x[2 + k] = pair(q[2 + k].y, q[2 + k].w);
    } else {
      u.x[2 * k] = pair(q[k].x, q[k].y), u.x[2 * k + 1] = pair(q[k].z, q[k].w);
      w.x[2 * k] = pair(q[2 + k].x, q[2 + k].y), w.x[2 * k + 1] = pair(q[2 + k].z, q[2 + k].w);
    }
  }
}
// Back to memory order, rounded to the type.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool kZip>
__device__ __forceinline__ void narrow(const Chunk& u, const Chunk& w, Raw<__nv_bfloat16>& a, Raw<__nv_bfloat16>& b) {
  uint32_t p[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = unpair(u.x[k]), y = unpair(w.x[k]);
    if constexpr (kZip)
      p[2 * k] = bf16_pair(x.x, y.x), p[2 * k + 1] = bf16_pair(x.y, y.y);
    else
      p[k] = bf16_pair(x.x, x.y), p[4 + k] = bf16_pair(y.x, y.y);
  }
  a.v[0] = make_uint4(p[0], p[1], p[2], p[3]), b.v[0] = make_uint4(p[4], p[5], p[6], p[7]);
}
template <bool kZip>
__device__ __forceinline__ void narrow(const Chunk& u, const Chunk& w, Raw<float>& a, Raw<float>& b) {
  float p[16];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = unpair(u.x[k]), y = unpair(w.x[k]);
    if constexpr (kZip)
      p[4 * k] = x.x, p[4 * k + 1] = y.x, p[4 * k + 2] = x.y, p[4 * k + 3] = y.y;
    else
      p[2 * k] = x.x, p[2 * k + 1] = x.y, p[8 + 2 * k] = y.x, p[8 + 2 * k + 1] = y.y;
  }
  const uint4* q = reinterpret_cast<const uint4*>(p);
  a.v[0] = q[0], a.v[1] = q[1], b.v[0] = q[2], b.v[1] = q[3];
}
template <typename T>
__device__ __forceinline__ void store_raw(T* p, const Raw<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}
// element k of a stored chunk
__device__ __forceinline__ float element(const Raw<__nv_bfloat16>& r, int k) {
  const uint32_t p[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
  return __uint_as_float(k & 1 ? p[k / 2] & 0xffff0000u : p[k / 2] << 16);
}
__device__ __forceinline__ float element(const Raw<float>& r, int k) {
  const uint32_t p[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
  return __uint_as_float(p[k]);
}

// Products and sums rounded one by one (as packed f32x2 operations the products
// came out fused with the sums).
__device__ __forceinline__ void turn(uint64_t& lo, uint64_t& hi, uint64_t c, uint64_t s) {
  const float2 a = unpair(lo), b = unpair(hi), co = unpair(c), si = unpair(s);
  const float x = __fsub_rn(__fmul_rn(a.x, co.x), __fmul_rn(b.x, si.x)), y = __fsub_rn(__fmul_rn(a.y, co.y), __fmul_rn(b.y, si.y));
  const float z = __fadd_rn(__fmul_rn(b.x, co.x), __fmul_rn(a.x, si.x)), w = __fadd_rn(__fmul_rn(b.y, co.y), __fmul_rn(a.y, si.y));
  lo = pair(__float_as_uint(x), __float_as_uint(y));
  hi = pair(__float_as_uint(z), __float_as_uint(w));
}

// Sine and cosine in fp64 of any angle below 2^31 turns: the nearest multiple n
// of pi / 2 is taken off in two fused steps (the second constant is what the
// first one lacks), and the Taylor series on [-pi / 4, pi / 4] up to r^13 and
// r^14 are off by less than 2^-45, far below the fp32 results' own rounding.
__device__ __forceinline__ float2 cos_sin(double angle) {
  const double n = rint(angle * 0.63661977236758134);
  double r = fma(-n, 1.5707963267948966, angle);
  r = fma(-n, 6.123233995736766e-17, r);
  const double z = r * r;
  double s = fma(z, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  s = fma(z, s, 1.0 / 362880.0);
  s = fma(z, s, -1.0 / 5040.0);
  s = fma(z, s, 1.0 / 120.0);
  s = fma(z, s, -1.0 / 6.0);
  s = fma(r * z, s, r);
  double c = fma(z, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  c = fma(z, c, -1.0 / 3628800.0);
  c = fma(z, c, 1.0 / 40320.0);
  c = fma(z, c, -1.0 / 720.0);
  c = fma(z, c, 1.0 / 24.0);
  c = fma(z, c, -0.5);
  c = fma(z, c, 1.0);
  const float fs = (float)s, fc = (float)c;
  const uint32_t q = (uint32_t)(int64_t)n & 3u;
  const float x = q & 1u ? fs : fc, y = q & 1u ? fc : fs;
  return make_float2(q == 1u || q == 2u ? -x : x, q & 2u ? -y : y);
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
  if ((uint64_t)pos >= a.most) return Place{-2, (int32_t)pos};
  const uint32_t P = a.pm.page_size, at = (uint32_t)pos / P;
  const int64_t page = a.pm.table[(int64_t)b * a.pm.max_pages + at];
  if (page < 0 || page >= a.pm.num_pages) return Place{-2, (int32_t)pos};
  return Place{page * a.Hkv * P + ((uint32_t)pos - at * P), (int32_t)pos};
}

// fp16 norm of a row from its squares' sum, as the sign encoder's: the fp32
// sum of bf16 squares is off by less than 8e-6, which matters only next to a
// rounding border; there, and for fp32 rows, the fp64 sum decides.
template <typename T>
__device__ __forceinline__ uint16_t row_norm(const Raw<T>& a, const Raw<T>& b) {
  float ss = 0.f;
#pragma unroll
  for (int z = 0; z < 8; ++z) ss = fmaf(element(a, z), element(a, z), fmaf(element(b, z), element(b, z), ss));
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float n = sqrtf(ss);
  const uint16_t lo = __half_as_ushort(__float2half_rn(n * (1.f - 8e-6f))), hi = __half_as_ushort(__float2half_rn(n * (1.f + 8e-6f)));
  uint16_t out = hi;
  if (__any_sync(0xffffffffu, sizeof(T) == 4 || lo != hi)) {
    double d = 0.0;
#pragma unroll 1
    for (int z = 0; z < 8; ++z) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k == z) x = element(a, k), y = element(b, k);
      d = fma((double)x, (double)x, fma((double)y, (double)y, d));
    }
#pragma unroll
    for (int o = 1; o < kRowLanes; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    out = __half_as_ushort(__double2half(sqrt(d)));
  }
  return out;
}

template <typename T, int HASH>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(HASH))
append_paged_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int D = kHeadDim, kAhead = HASH == kHashLsh ? 2 : 1;  // groups of four rows that a warp has on their way
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float cos_s[kWarps][64], sin_s[kWarps][64];  // of a warp's token
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
  __nv_bfloat16* R_s = keys + 2 * key_rows * kKeyPitch;           // kHashLsh: [bits][kKeyPitch]
  if constexpr (HASH == kHashLsh) {
    for (int i = tid; i < a.words * 32 * (D / 8); i += kThreads)
      *reinterpret_cast<uint4*>(R_s + i / (D / 8) * kKeyPitch + i % (D / 8) * 8) = __ldg(static_cast<const uint4*>(a.R) + i);
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
      Raw<T> ra[kAhead], rw[kAhead];  // the next groups, on their way
      int head[kAhead], heads[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const T* src = row_of(part + e * a.parts, head[e], heads[e]);
        if (part + e * a.parts < all4 && head[e] < heads[e]) ra[e] = load_raw(src + c0), rw[e] = load_raw(src + c1);
      }
      const Place at = place_of(a, t);
      if (lane == 0 && part == 0) {
        if (at.row == -2) report(a.status, HKV_ERR_DEVICE_RANGE);
        if (HASH == kHashLsh) row_s[buf][warp / a.parts] = at.row;
      }
      if (at.row != -1) {
        for (int p = lane; p < a.pairs; p += 32) {
          const int pos = a.positions ? __ldg(a.positions + (int64_t)a.axis[p] * a.T + t) : at.pos;
          const float2 cs = cos_sin((double)pos * (double)__ldg(a.inv_freq + p));
          cos_s[warp][p] = cs.x, sin_s[warp][p] = cs.y;
        }
        __syncwarp();
        uint64_t cs[4], sn[4];
        if (turned) {
          // pairs 8 c .. 8 c + 7 (neighbours: those of both chunks in order)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            cs[z] = *reinterpret_cast<const uint64_t*>(&cos_s[warp][c * 8 + 2 * z]);
            sn[z] = *reinterpret_cast<const uint64_t*>(&sin_s[warp][c * 8 + 2 * z]);
          }
        }
        __syncwarp();
        T* const oq = static_cast<T*>(a.q_out) + t * a.qo_stride;
        for (int i0 = part; i0 < all4; i0 += kAhead * a.parts) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int i = i0 + e * a.parts;
          if (i >= all4) break;
          Raw<T> xa = ra[e], xw = rw[e];
          const int h = head[e];
          const bool is_q = i < q4, is_k = !is_q && i < q4 + k4, in = h < heads[e] && (is_q || at.row >= 0);
          {
            const int next = i + kAhead * a.parts;
            const T* src = row_of(next, head[e], heads[e]);
            if (next < all4 && head[e] < heads[e]) ra[e] = load_raw(src + c0), rw[e] = load_raw(src + c1);
          }
          T* dst = is_q ? oq + h * D : static_cast<T*>(is_k ? a.K : a.V) + (at.row + (int64_t)h * a.pm.page_size) * D;
          if (turned && (is_q || is_k)) {
            Chunk u, w;
            if (split) {
              widen<false>(xa, xw, u, w);
#pragma unroll
              for (int z = 0; z < 4; ++z) turn(u.x[z], w.x[z], cs[z], sn[z]);
              narrow<false>(u, w, xa, xw);
            } else {
              widen<true>(xa, xw, u, w);
#pragma unroll
              for (int z = 0; z < 4; ++z) turn(u.x[z], w.x[z], cs[z], sn[z]);
              narrow<true>(u, w, xa, xw);
            }
          }
          if (in) store_raw(dst + c0, xa), store_raw(dst + c1, xw);
          if constexpr (HASH == kHashLsh) {
            if (is_k && in) {
              T* kd = reinterpret_cast<T*>(keys + (buf * key_rows + warp / a.parts * a.Hkv + h) * kKeyPitch);
              store_raw(kd + c0, xa), store_raw(kd + c1, xw);
            }
          }
          if constexpr (HASH == kHashStage) {
            if (is_k && in) {
              T* kd = static_cast<T*>(a.staged) + (t * a.Hkv + h) * D;
              store_raw(kd + c0, xa), store_raw(kd + c1, xw);
            }
          }
          if constexpr (HASH == kHashSign) {
            if (is_k) {  // the whole warp: signs and norms of the stored keys
              uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const int ch = (half ? c1 : c0) / 8;
                uint32_t byte = 0;
#pragma unroll
                for (int z = 0; z < 8; ++z) byte |= (uint32_t)(element(half ? xw : xa, z) > 0.f) << z;
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
                const uint16_t norm = row_norm<T>(xa, xw);
                if (in && c == 0) a.norms[row] = norm;
              }
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
          uint32_t bf[4];  // both tiles of 8 bits, k halves next to each other
          const int bit = (warp * ntile + (ntile == 2 ? lane >> 4 : 0)) * 8 + (lane & 7);
          ldsm4(bf, R_s + bit * kKeyPitch + kk * 16 + ((lane >> 3) & 1) * 8);
          mma16816(y[0], af, bf[0], bf[1]);
          if (ntile == 2) mma16816(y[1], af, bf[2], bf[3]);
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
      if (t < first || t >= end || (uint64_t)pos >= a.most) continue;
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
      smem = (2 * align_up((size_t)(kWarps / a.parts) * a.Hkv, 16) + a.words * 32) * kKeyPitch * sizeof(T);
      if (smem + 8192 > (size_t)max_smem_optin()) return fail(HKV_ERR_UNSUPPORTED, "Hkv %d too large", a.Hkv);
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return cuda_check(e, "append smem attribute");
    }
  }
  const int64_t steps = ceil_div(a.T, kWarps / a.parts), most = (int64_t)sm_count() * blocks_per_sm(hash);
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
  a.most = pm.max_pages <= INT32_MAX / pm.page_size ? pm.max_pages * pm.page_size : 1ull << 31;
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
