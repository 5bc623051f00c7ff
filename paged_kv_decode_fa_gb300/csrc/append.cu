// Appending keys and values to a paged KV cache, with the position rotation
// on the way: the calls fa_append_* (declared in include/fa_decode.h).
//
// The mathematics.  A token at position t rotates each pair (x1, x2) of its
// first rotary_dim dims by the angle a_i = t * inv_freq[i]:
//     y1 = x1 cos a_i - x2 sin a_i,   y2 = x2 cos a_i + x1 sin a_i,
// pairs (i, i + rotary_dim/2), or (2i, 2i+1) when interleaved; V and the
// other dims stay.  K (rotated), V and, on request, rotated q are rounded once
// from fp32.  An angle only matters modulo a turn, and fp32 (24 bits) loses
// it at far positions (t = 10^6 at inv_freq 1: 0.06 radians).  So the plan
// stores inv_freq[i] / 2 pi modulo 1 as a 64-bit fraction f_i; t * f_i modulo
// 2^64 is then the exact fraction of a turn, whatever t, in integer
// multiplies.  Its cosine and sine are rounded once, and so is each product and
// sum of the rotation: the values that elementary operations give.
//
// E4M3 caches: code = rn(x / s) saturated at 448, with s per tensor, per kv
// head, per token (amax over the row / 448, written here) or per block, a
// page's tokens of one kv head: the smallest power of two with amax <= 448 s.
// A power of two costs a code no relative precision (E4M3 is floating point),
// and a page that goes on filling keeps max(old, needed): when that grows, the
// codes it holds are divided by a power of two, exactly but for subnormals,
// so a page filled a token at a time reads as one filled at once.
//
// Work: one CTA per (page run, a few kv heads: heads_of_cta); a run is the new
// tokens of one request in one page, at most 16.  A thread serves one token and
// both halves of eight of its pairs (or 16 dims in a row), so that a pair never
// leaves its registers, and goes over its heads with the same eight angles.  The
// angles of a run are computed once, into shared memory.  All K and V loads of
// a thread are issued before that.  A block's amax needs all its tokens, which
// the CTA holds: one reduction in shared memory, no second pass over the
// inputs.
//
// What bounds it (us per launch in a CUDA graph).  Long appends are bound by HBM:
// 779 MB of prompts (32 / 8 heads, head_dim 128, bf16, q included) in 120.0 us =
// 6.5 TB/s, 0.97 of the copy rate; 910 MB into a block-scaled cache (64 / 8 heads) in
// 152.3 us = 6.0 TB/s, 0.90, where a run passes two more barriers around the
// conversions.  Single tokens are bound by the launch and one chain of loads
// (unit, rows and page id, the page's scale): 4 tokens 2.6 us, 450 tokens 3.3 us,
// 128 tokens into a block-scaled cache 4.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>
#include <new>
#include <type_traits>
#include <vector>

#include "fa_decode.h"
#include "kernels.h"
#include "staging.h"

namespace fadecode {
namespace {

// Measured at the sizes above (prompts / block-scaled prompts, us): 2 heads, 4 q rows
// and 80 registers 122.4 / 150.4; 1 head 137.7 / 167.4 (256 threads); 2 q rows 124.5 /
// 176.4 (256 threads), 8 q rows at 96 registers 141.2 / 182.4, at 128 123.3 / 155.7; 4
// heads at 128 registers 127.5 / 175.3.
constexpr int kHeads = 2;      // kv heads a thread holds K and V of
constexpr int kMaxHeads = 16;  // kv heads of one CTA at most
constexpr int kQRows = 4;      // q rows a thread loads at a time
constexpr int kCtasPerSm = 6;  // CTAs per SM the registers are held to (80 each)
constexpr int kMaxPairs = 64;  // rotary_dim / 2 at most

// How an E4M3 cache is scaled (kNative: q's type, no scale).
enum Mode { kNative = 0, kStatic = 1, kToken = 2, kBlock = 3 };

struct AppendUnit {
  int32_t row;       // first of its rows of k, v and q
  int32_t entry;     // its page's entry in the index table
  int32_t slots;     // first slot | tokens << 8
  int32_t position;  // rotation position of the first token
};
static_assert(sizeof(AppendUnit) == 16, "read as int4");

// Element strides of one input [rows, heads, D].
struct Rows {
  const void* p;
  int64_t token, head;
};

struct AppendParams {
  Rows k, v, q;
  void* q_out;  // [rows, Hq, D] or nullptr
  void* kv;
  float* k_scales;  // kToken [pages, Hkv, 16], kBlock [pages, Hkv]: read and written
  float* v_scales;
  const float* head_k_scales;  // kStatic: [Hkv], or nullptr for the scalars
  const float* head_v_scales;
  float k_scale, v_scale;
  const int32_t* indices;
  const AppendUnit* units;
  const unsigned long long* turns;  // [pairs] turns a position, 2^-64 units
  int* err;
  int64_t num_pages;
  int hq, hkv;
  int heads;  // kv heads of one CTA, kHeads per thread at most
  int pairs;  // rotary_dim / 2
};

__device__ __forceinline__ float2 unpack(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack(uint32_t w, __half) {
  __half2 h;
  memcpy(&h, &w, sizeof h);
  return __half22float2(h);
}
__device__ __forceinline__ uint32_t pack(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  uint32_t w;
  memcpy(&w, &v, sizeof w);
  return w;
}
__device__ __forceinline__ uint32_t pack(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  uint32_t w;
  memcpy(&w, &v, sizeof w);
  return w;
}

// Eight consecutive elements: as stored, and widened.
template <typename T>
struct Group {
  uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void widen(const Group<T>& g, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {g.w[0].x, g.w[0].y, g.w[0].z, g.w[0].w,
                           g.w[1].x, g.w[1].y, g.w[1].z, g.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {g.w[0].x, g.w[0].y, g.w[0].z, g.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack(w[i], T{});
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ Group<T> narrow(const float (&x)[8]) {
  Group<T> g;
  if constexpr (sizeof(T) == 4) {
    g.w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                        __float_as_uint(x[3]));
    g.w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                        __float_as_uint(x[7]));
  } else {
    g.w[0] = make_uint4(pack(x[0], x[1], T{}), pack(x[2], x[3], T{}), pack(x[4], x[5], T{}),
                        pack(x[6], x[7], T{}));
  }
  return g;
}

// Plain loads, not through the read-only path: q_out may be q itself.
template <typename T>
__device__ __forceinline__ Group<T> load_group(const T* p, bool ok) {
  Group<T> g;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    g.w[i] = ok ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
  return g;
}

template <typename T>
__device__ __forceinline__ void store_group(T* p, const Group<T>& g) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = g.w[i];
}

// Two fp32 operations at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "  mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 w, x, y, z; mov.b64 w, {%2, %3}; mov.b64 x, {%4, %5}; mov.b64 y, {%6, %7};\n"
      "  fma.rn.f32x2 z, w, x, y; mov.b64 {%0, %1}, z; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float c) {
  return fma2(a, b, make_float2(c, c));
}
__device__ __forceinline__ float2 fma2(float2 a, float b, float2 c) {
  return fma2(a, make_float2(b, b), c);
}
__device__ __forceinline__ float2 minus(float2 a) { return make_float2(-a.x, -a.y); }

// A thread's 16 elements of a row: dims da .. da+7 and db .. db+7.
struct Piece {
  float a[8], b[8];
};

// Its rotation: eight pairs, (a[j], b[j]), or interleaved within a and b.
struct Turn {
  float c[8], s[8];
  bool on;
};

// Products and sums are rounded one by one, as elementary operations round
// them: an element fused into one rounding would differ from theirs in fp32's last
// bit, and now and then in the type it is stored in.  (Scalar, since the assembler
// fuses add.rn.f32x2 with a product of mul.rn.f32x2.  The products' order was
// timed: block-scaled prompts of 27476 tokens 177.7 us for 179.6, interleaved
// ones 172.6 for 180.6, the others the same or 2 us less.)
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(const Turn& r, Piece* x) {
  if (!r.on) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (INTERLEAVED) {
      float* y = j < 4 ? x->a : x->b;
      const int e = 2 * (j % 4);
      const float u = y[e], v = y[e + 1];
      const float us = __fmul_rn(u, r.s[j]);
      y[e] = __fsub_rn(__fmul_rn(u, r.c[j]), __fmul_rn(v, r.s[j]));
      y[e + 1] = __fadd_rn(__fmul_rn(v, r.c[j]), us);
    } else {
      const float u = x->a[j], v = x->b[j];
      const float vs = __fmul_rn(v, r.s[j]), us = __fmul_rn(u, r.s[j]);
      const float uc = __fmul_rn(u, r.c[j]), vc = __fmul_rn(v, r.c[j]);
      x->a[j] = __fsub_rn(uc, vs);
      x->b[j] = __fadd_rn(vc, us);
    }
  }
}

// The largest magnitude of the piece's finite elements.  E4M3 cannot tell an
// infinity from a large value: infinities become NaN here, which fmaxf passes
// over and the conversion keeps, and *infinite is set.
__device__ __forceinline__ float finite_amax(Piece* x, bool* infinite) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(x->a[j]), fabsf(x->b[j])));
  if (m == INFINITY) {
    m = 0.f;
    *infinite = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (fabsf(x->a[j]) == INFINITY) x->a[j] = NAN;
      if (fabsf(x->b[j]) == INFINITY) x->b[j] = NAN;
      m = fmaxf(m, fmaxf(fabsf(x->a[j]), fabsf(x->b[j])));
    }
  }
  return m;
}

// Two numbers, each a sum of two floats.
struct Sum2 {
  float2 hi, lo;
};

// c + z * p, |c| above |z p|: the product's and the sum's rounding errors are
// kept (fma), to about 2^-47 of c.
__device__ __forceinline__ Sum2 horner(const Sum2& z, float2 p, float c, float2 low) {
  Sum2 r;
  r.hi = fma2(z.hi, p, c);
  const float2 err = fma2(z.hi, p, make_float2(c - r.hi.x, c - r.hi.y));
  low = fma2(z.lo, p, low);
  r.lo = make_float2(err.x + low.x, err.y + low.y);
  return r;
}

// A whole number below 2^23, exactly (its bits under 2^23's).
__device__ __forceinline__ float small_float(unsigned n) {
  return __uint_as_float(0x4b000000u | n) - 8388608.f;
}

// (cos, sin) of two fractions of a turn, in 2^-64 turns, rounded to nearest but for
// one angle in 10^5 (2^-37 of a cosine and 2^-40 of a sine before the last
// rounding; the elementary operations on a float64 angle give the same).
// The nearest quarter turn is taken off in integers.  The rest, at most an eighth
// of a turn, becomes radians in a sum of two floats, and the series of sine and
// cosine keep two floats in the terms that need them.  (sincospif, an ulp off
// in one angle in six, put elements of q and codes of K on the other side of
// a rounding border.)
__device__ __forceinline__ float4 cos_sin(unsigned long long turn0, unsigned long long turn1) {
  const unsigned long long turn[2] = {turn0, turn1};
  unsigned quarter[2];
  float ra[2], rb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    quarter[i] = (unsigned)((turn[i] + (1ull << 61)) >> 62);
    const long long rest = (long long)(turn[i] - ((unsigned long long)quarter[i] << 62));
    // its bits from 39 (signed: under 1.5 * 2^23), 16 and 0
    const float top = __uint_as_float(0x4b400000u + (unsigned)(int)(rest >> 39)) - 12582912.f;
    const float mid = small_float((unsigned)(rest >> 16) & 0x7fffffu);
    ra[i] = fmaf(top, 8388608.f, mid);
    rb[i] = fmaf(fmaf(top, 8388608.f, -ra[i]) + mid, 65536.f, small_float((unsigned)rest & 0xffffu));
  }
  const float2 a = make_float2(ra[0], ra[1]), b = make_float2(rb[0], rb[1]);
  // (a * 2^16 + b) * 2 pi / 2^64, 2 pi in two floats
  constexpr float two_pi = 6.2831855f, two_pi_low = -1.7484555e-7f;
  constexpr float k16 = 3.5527137e-15f, k0 = 5.4210109e-20f;  // 2^-48, 2^-64
  const float2 h = mul2(a, make_float2(two_pi * k16, two_pi * k16));
  const float2 e = fma2(b, two_pi * k0, fma2(a, two_pi_low * k16, fma2(a, two_pi * k16, minus(h))));
  Sum2 z;  // the angle's square
  z.hi = mul2(h, h);
  z.lo = fma2(mul2(h, make_float2(2.f, 2.f)), e, fma2(h, h, minus(z.hi)));
  auto next = [&](const Sum2& p, float c) {
    return horner(z, p.hi, c, mul2(z.hi, p.lo));
  };
  // sin: coefficients 1 / n!, in two floats from 1 / 5!
  float2 p = fma2(z.hi, 1.6059044e-10f, make_float2(-2.5052108e-8f, -2.5052108e-8f));
  p = fma2(z.hi, fma2(z.hi, p, 2.7557319e-6f), -1.9841270e-4f);
  Sum2 r = horner(z, p, 8.3333337e-3f, make_float2(-4.3461720e-10f, -4.3461720e-10f));
  r = horner(z, r.hi, -1.6666667e-1f, fma2(z.hi, r.lo, 4.9670534e-9f));
  r = next(r, 1.f);
  const float2 v = mul2(h, r.hi);
  const float2 vl = fma2(e, r.hi, fma2(h, r.lo, fma2(h, r.hi, minus(v))));
  const float s[2] = {__fadd_rn(v.x, vl.x), __fadd_rn(v.y, vl.y)};
  // cos, in two floats from 1 / 4!
  p = fma2(z.hi, -1.1470746e-11f, make_float2(2.0876757e-9f, 2.0876757e-9f));
  p = fma2(z.hi, fma2(z.hi, p, -2.7557319e-7f), 2.4801587e-5f);
  p = fma2(z.hi, p, -1.3888889e-3f);
  r = horner(z, p, 4.1666668e-2f, make_float2(-1.2417634e-9f, -1.2417634e-9f));
  r = next(next(r, -0.5f), 1.f);
  const float c[2] = {__fadd_rn(r.hi.x, r.lo.x), __fadd_rn(r.hi.y, r.lo.y)};
  float x[2], y[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool odd = quarter[i] & 1;
    x[i] = odd ? s[i] : c[i];
    y[i] = odd ? c[i] : s[i];
    // the signs: cos is negative in quarters 1 and 2, sin in 2 and 3
    x[i] = __uint_as_float(__float_as_uint(x[i]) ^ ((quarter[i] ^ (quarter[i] << 1)) & 2) << 30);
    y[i] = __uint_as_float(__float_as_uint(y[i]) ^ (quarter[i] & 2) << 30);
  }
  return make_float4(x[0], y[0], x[1], y[1]);
}

template <int LPR>
__device__ __forceinline__ float row_max(float m) {
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// Codes of x * inv, saturated at 448.
__device__ __forceinline__ uint32_t code2(float a, float b, float inv) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[8], float inv) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(code2(x[0], x[1], inv) | (code2(x[2], x[3], inv) << 16),
                 code2(x[4], x[5], inv) | (code2(x[6], x[7], inv) << 16));
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8: the
// carry out of the mantissa marks one above .75); 0 for 0.
__device__ __forceinline__ float block_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;  // biased exponent
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// 1 / scale, 0 for a scale of 0 (or below the normal numbers, whose inverse
// may overflow).
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126
__device__ __forceinline__ float inverse(float scale) {
  return scale >= kMinScale ? 1.f / scale : 0.f;
}

template <int D>
struct Cfg {
  static constexpr int THREADS = 128;
  static constexpr int LPR = D / 16;          // threads of a row
  static constexpr int ROWS = THREADS / LPR;  // rows in step
  static_assert(ROWS >= kPageSize && 2 * kMaxHeads <= THREADS, "a run's tokens; a thread a scale");
};

// INTERLEAVED as a constant: with both orders in one kernel, its code outgrew the
// instruction cache (block-scaled prompts 155.9 us for 160.5, others 121.4 for 123.2).
template <typename T, int D, int MODE, bool INTERLEAVED>
__global__ void __launch_bounds__(Cfg<D>::THREADS, kCtasPerSm)
    fa_append_kernel(const __grid_constant__ AppendParams p) {
  using C = Cfg<D>;
  constexpr int LPR = C::LPR;
  __shared__ __align__(16) float2 angle[kPageSize * kMaxPairs];
  __shared__ int amax_bits[2 * kMaxHeads];                 // K heads, then V heads
  __shared__ float item_scale[2 * kMaxHeads], item_ratio[2 * kMaxHeads];

  const AppendUnit u = p.units[blockIdx.x];
  const int slot0 = u.slots & 0xff, n = u.slots >> 8;
  const int h0 = blockIdx.y * p.heads, heads = min(p.heads, p.hkv - h0);
  const int tid = threadIdx.x;
  // this thread: 16 elements of rows of token `tok`, of heads hg, hg + HG, ...
  const int c = tid % LPR, r = tid / LPR;
  const int lg = n > 8 ? 4 : n > 4 ? 3 : n > 2 ? 2 : n > 1 ? 1 : 0;
  const int tok = r & ((1 << lg) - 1), hg = r >> lg, HG = C::ROWS >> lg;
  const bool live = tok < n;
  const int64_t row = u.row + tok;
  // its dims: the two halves of eight pairs, or 16 in a row
  const bool split = !INTERLEAVED && 8 * c < p.pairs;
  const int da = split ? 8 * c : 16 * c, db = split ? p.pairs + 8 * c : 16 * c + 8;
  // the page id first: a block's scale hangs on it
  const int page = __ldg(p.indices + u.entry);
  Group<T> kr[kHeads][2], vr[kHeads][2];
  {
    const T* k = static_cast<const T*>(p.k.p) + row * p.k.token + h0 * p.k.head;
    const T* v = static_cast<const T*>(p.v.p) + row * p.v.token + h0 * p.v.head;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = i * HG + hg;
      const bool ok = live && h < heads;
      kr[i][0] = load_group(k + h * p.k.head + da, ok);
      kr[i][1] = load_group(k + h * p.k.head + db, ok);
      vr[i][0] = load_group(v + h * p.v.head + da, ok);
      vr[i][1] = load_group(v + h * p.v.head + db, ok);
    }
  }
  const bool page_ok = page >= 0 && (int64_t)page < p.num_pages;
  if (!page_ok && tid == 0) atomicOr(p.err, 1);

  // two pairs of a token at a time (their number is a multiple of eight)
  for (int i = 2 * tid; i < n * p.pairs; i += 2 * C::THREADS) {
    const int t = i / p.pairs, j = i - t * p.pairs;
    const ulonglong2 turns = *reinterpret_cast<const ulonglong2*>(p.turns + j);
    const unsigned long long at = (unsigned)(u.position + t);
    *reinterpret_cast<float4*>(angle + t * kMaxPairs + j) = cos_sin(at * turns.x, at * turns.y);
  }
  const int64_t scale_at = (int64_t)page * p.hkv + h0 + (tid < heads ? tid : tid - heads);
  float old_scale = 0.f;
  if (MODE == kBlock && tid < 2 * heads) {
    amax_bits[tid] = 0;
    if (page_ok && slot0 > 0) old_scale = (tid < heads ? p.k_scales : p.v_scales)[scale_at];
  }
  __syncthreads();

  Turn turn;
  turn.on = live && 8 * c < p.pairs;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 cs = turn.on ? angle[tok * kMaxPairs + 8 * c + j] : make_float2(1.f, 0.f);
    turn.c[j] = cs.x;
    turn.s[j] = cs.y;
  }
  auto piece = [&](const Group<T>(&g)[2]) {
    Piece x;
    widen<T>(g[0], x.a);
    widen<T>(g[1], x.b);
    return x;
  };

  bool infinite = false;  // among this thread's K and V
  if constexpr (MODE == kBlock) {
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (i * HG >= heads) break;
      Piece k = piece(kr[i]), v = piece(vr[i]);
      rotate<INTERLEAVED>(turn, &k);
      const float km = row_max<LPR>(finite_amax(&k, &infinite));
      const float vm = row_max<LPR>(finite_amax(&v, &infinite));
      if (c == 0 && live && i * HG + hg < heads) {
        atomicMax(&amax_bits[i * HG + hg], __float_as_int(km));
        atomicMax(&amax_bits[heads + i * HG + hg], __float_as_int(vm));
      }
    }
    __syncthreads();
    if (tid < 2 * heads) {
      const float now = fmaxf(old_scale, block_scale(__int_as_float(amax_bits[tid])));
      if (page_ok && (slot0 == 0 || !(now == old_scale)))
        (tid < heads ? p.k_scales : p.v_scales)[scale_at] = now;
      item_scale[tid] = now;
      item_ratio[tid] = now > old_scale ? old_scale * inverse(now) : 1.f;
    }
    __syncthreads();
    if (slot0 > 0 && page_ok) {
      // codes the page already holds, under the scales that grew
      for (int it = 0; it < 2 * heads; ++it) {
        const float ratio = item_ratio[it];
        if (ratio == 1.f) continue;
        const bool is_k = it < heads;
        uint8_t* base = static_cast<uint8_t*>(p.kv) +
                        (((int64_t)page * 2 + (is_k ? 0 : 1)) * kPageSize * p.hkv + h0 +
                         (is_k ? it : it - heads)) * D;
        for (int e = tid; e < slot0 * (D / 4); e += C::THREADS) {
          uint32_t* w = reinterpret_cast<uint32_t*>(base + (int64_t)(e / (D / 4)) * p.hkv * D) +
                        e % (D / 4);
          const uint32_t old4 = *w;
          const float2 lo = __half22float2(
              __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(old4 & 0xffffu), __NV_E4M3)));
          const float2 hi = __half22float2(
              __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(old4 >> 16), __NV_E4M3)));
          *w = code2(lo.x, lo.y, ratio) | (code2(hi.x, hi.y, ratio) << 16);
        }
      }
    }
  }

  // K rows, then V rows
  auto write = [&](Piece x, bool is_k, const Group<T>(&raw)[2], int h, bool ok) {
    float inv = 1.f, scale = 1.f;
    if constexpr (MODE != kNative) {
      // the block form has its amax already: 155.3 us for 155.9 without the second look
      const float m = MODE != kBlock || infinite ? finite_amax(&x, &infinite) : 0.f;
      if constexpr (MODE == kStatic) {
        const float* hs = is_k ? p.head_k_scales : p.head_v_scales;
        inv = inverse(!hs ? (is_k ? p.k_scale : p.v_scale) : ok ? __ldg(hs + h0 + h) : 1.f);
      } else if constexpr (MODE == kToken) {
        const float rm = row_max<LPR>(m);
        scale = rm > 0.f ? fmaxf(rm / 448.f, kMinScale) : 0.f;
        inv = inverse(scale);
      } else {
        inv = ok ? inverse(item_scale[is_k ? h : heads + h]) : 0.f;
      }
    }
    if (!ok || !page_ok) return;
    const int64_t at =
        ((((int64_t)page * 2 + (is_k ? 0 : 1)) * kPageSize + slot0 + tok) * p.hkv + h0 + h) * D;
    if constexpr (MODE == kNative) {
      T* out = static_cast<T*>(p.kv) + at;
      store_group(out + da, is_k ? narrow<T>(x.a) : raw[0]);
      store_group(out + db, is_k ? narrow<T>(x.b) : raw[1]);
    } else {
      if (MODE == kToken && c == 0)
        (is_k ? p.k_scales : p.v_scales)[((int64_t)page * p.hkv + h0 + h) * kPageSize + slot0 +
                                         tok] = scale;
      uint8_t* out = static_cast<uint8_t*>(p.kv) + at;
      store_codes(out + da, x.a, inv);
      store_codes(out + db, x.b, inv);
    }
  };
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i * HG >= heads) break;
    const int h = i * HG + hg;
    const bool ok = live && h < heads;
    Piece k = piece(kr[i]);
    rotate<INTERLEAVED>(turn, &k);
    write(k, true, kr[i], h, ok);
    write(piece(vr[i]), false, vr[i], h, ok);
  }

  if (p.q.p == nullptr) return;
  // q rows, kQRows at a time so that as many loads are in flight; q_out may be
  // q itself: a row's elements are read and written by one thread
  const int group = p.hq / p.hkv, rows_q = heads * group;
  const T* q = static_cast<const T*>(p.q.p) + row * p.q.token + (int64_t)h0 * group * p.q.head;
  T* out = static_cast<T*>(p.q_out) + (row * p.hq + h0 * group) * D;
  for (int i0 = hg; i0 - hg < rows_q; i0 += kQRows * HG) {
    Group<T> in[kQRows][2];
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
      const int h = i0 + i * HG;
      in[i][0] = load_group(q + h * p.q.head + da, live && h < rows_q);
      in[i][1] = load_group(q + h * p.q.head + db, live && h < rows_q);
    }
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
      const int h = i0 + i * HG;
      if (!live || h >= rows_q) break;
      Piece x = piece(in[i]);
      rotate<INTERLEAVED>(turn, &x);
      store_group(out + h * D + da, narrow<T>(x.a));
      store_group(out + h * D + db, narrow<T>(x.b));
    }
  }
}

struct AppendKernel {
  const void* func = nullptr;
  int threads = 0, rows = 0;
};

template <typename T, int MODE>
AppendKernel kernel_of(int head_dim, bool interleaved) {
  auto of = [&](auto d) {
    constexpr int D = decltype(d)::value;
    const void* f = interleaved ? reinterpret_cast<const void*>(&fa_append_kernel<T, D, MODE, true>)
                                : reinterpret_cast<const void*>(&fa_append_kernel<T, D, MODE, false>);
    return AppendKernel{f, Cfg<D>::THREADS, Cfg<D>::ROWS};
  };
  return head_dim == 64 ? of(std::integral_constant<int, 64>{})
                        : of(std::integral_constant<int, 128>{});
}

// A kernel for q's type, the cache being E4M3 unless mode is kNative.
AppendKernel find_append_kernel(fa_dtype q, int head_dim, Mode mode, bool interleaved) {
  if (q == FA_DTYPE_F32) return kernel_of<float, kNative>(head_dim, interleaved);
  if (q == FA_DTYPE_BF16) {
    if (mode == kStatic) return kernel_of<__nv_bfloat16, kStatic>(head_dim, interleaved);
    if (mode == kToken) return kernel_of<__nv_bfloat16, kToken>(head_dim, interleaved);
    if (mode == kBlock) return kernel_of<__nv_bfloat16, kBlock>(head_dim, interleaved);
    return kernel_of<__nv_bfloat16, kNative>(head_dim, interleaved);
  }
  if (mode == kStatic) return kernel_of<__half, kStatic>(head_dim, interleaved);
  if (mode == kToken) return kernel_of<__half, kToken>(head_dim, interleaved);
  if (mode == kBlock) return kernel_of<__half, kBlock>(head_dim, interleaved);
  return kernel_of<__half, kNative>(head_dim, interleaved);
}

// kv heads of one CTA, for runs of `longest` tokens at most, `tokens` in all:
// as many (a power of two) as keep a thread's rows of K, V and q to kMaxRows,
// and its kv heads to kHeads.  More rows share a CTA's fixed cost, the angles
// first (block-scaled prompts at 12 / 24 rows: 160.6 / 150.5 us, with 256 threads);
// single tokens, many rows in step, then take all their heads in one CTA
// (450 tokens: 6.1 us at 4 of 8 heads, 4.1 at 8; filling every SM with CTAs instead
// cost the 128-token batches 5.8 us for 3.8).
constexpr int kMaxRows = 24;
int heads_of_cta(const AppendKernel& k, int64_t tokens, int64_t units, int longest, int hkv,
                 int group) {
  auto step = [&](int64_t n) {  // rows of one token in step, for runs of n
    int t = 1;
    while (t < n) t *= 2;
    return k.rows / t;
  };
  const int64_t mean = (tokens + units - 1) / units;
  int heads = 1;
  while (2 * heads <= kMaxHeads && heads < hkv && 2 * heads <= kHeads * step(longest) &&
         2 * heads * (2 + group) <= kMaxRows * step(mean))
    heads *= 2;
  return heads;
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Device-check word, then the units, then the turns.
struct AppendLayout {
  size_t units, turns, total;
};
AppendLayout append_layout(int64_t n_units, int pairs) {
  AppendLayout L;
  L.units = kAlign;
  L.turns = align_up(L.units + sizeof(AppendUnit) * (size_t)n_units);
  L.total = align_up(L.turns + 8 * (size_t)pairs);
  return L;
}

// Radians a position at most (models use at most 1): the turns below then keep
// 64 bits of their fraction, the rounding of freq / 2 pi included.
constexpr double kMaxFrequency = 4294967296.0;

// freq / 2 pi modulo 1 in units of 2^-64, rounded down in magnitude: the
// product with 1 / 2 pi in two doubles (its rounding error recovered by fma),
// so that the 64 bits carry the double's own precision.
unsigned long long turns_of(double freq) {
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;  // 1 / 2 pi = hi + lo
  const double x = std::fabs(freq);
  const double a = x * hi, b = std::fma(x, hi, -a) + x * lo;
  const double f = (a - std::floor(a)) * 4294967296.0;  // exact, in 2^-32 units
  const double top = std::floor(f);
  const double low = (f - top + b * 4294967296.0) * 4294967296.0;  // may reach over its 32 bits
  const unsigned long long t = ((unsigned long long)top << 32) +
                               (unsigned long long)(long long)std::floor(low);
  return freq < 0 ? 0ull - t : t;
}

}  // namespace
}  // namespace fadecode

using namespace fadecode;

struct fa_append_plan_s {
  int device = 0;
  int hq = 0, hkv = 0, d = 0;
  fa_dtype q_dtype = FA_DTYPE_F32, kv_dtype = FA_DTYPE_F32;
  const int32_t* indices = nullptr;
  uint8_t* ws = nullptr;
  AppendLayout layout{};
  int64_t num_units = 0, num_rows = 0;
  int longest = 0;  // tokens of the longest run
  int pairs = 0;
  bool interleaved = false;
};

namespace {

bool append_pair_built(fa_dtype q, fa_dtype kv) {
  if (kv == FA_DTYPE_E4M3) return q == FA_DTYPE_BF16 || q == FA_DTYPE_F16;
  return q == kv && (q == FA_DTYPE_F32 || q == FA_DTYPE_BF16 || q == FA_DTYPE_F16);
}

bool rows_ok(const fa_append_plan_s* plan, const fa_rows* in) {
  const int64_t es = plan->q_dtype == FA_DTYPE_F32 ? 4 : 2;
  return in && in->data && reinterpret_cast<uintptr_t>(in->data) % 16 == 0 &&
         in->token_stride >= 0 && in->head_stride >= 0 && in->token_stride * es % 16 == 0 &&
         in->head_stride * es % 16 == 0;
}

int append_run(fa_append_plan_s* plan, Mode mode, const fa_rows* k, const fa_rows* v,
               const fa_rows* q, void* q_out, void* paged_kv, int64_t num_pages, float k_scale,
               float v_scale, const float* head_k, const float* head_v, float* k_scales,
               float* v_scales, void* cuda_stream) {
  if (plan->num_rows == 0) return FA_OK;
  if (!rows_ok(plan, k) || !rows_ok(plan, v) || !paged_kv || num_pages <= 0 ||
      reinterpret_cast<uintptr_t>(paged_kv) % 16)
    return FA_ERR_INVALID_ARG;
  if (q && (!rows_ok(plan, q) || !q_out || reinterpret_cast<uintptr_t>(q_out) % 16))
    return FA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev != plan->device) return FA_ERR_INVALID_ARG;
  AppendParams p;
  std::memset(&p, 0, sizeof p);
  p.k = Rows{k->data, k->token_stride, k->head_stride};
  p.v = Rows{v->data, v->token_stride, v->head_stride};
  if (q) p.q = Rows{q->data, q->token_stride, q->head_stride};
  p.q_out = q_out;
  p.kv = paged_kv;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.head_k_scales = head_k;
  p.head_v_scales = head_v;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.indices = plan->indices;
  p.units = reinterpret_cast<const AppendUnit*>(plan->ws + plan->layout.units);
  p.turns = reinterpret_cast<const unsigned long long*>(plan->ws + plan->layout.turns);
  p.err = reinterpret_cast<int*>(plan->ws);
  p.num_pages = num_pages;
  p.hq = plan->hq;
  p.hkv = plan->hkv;
  p.pairs = plan->pairs;
  const AppendKernel kern = find_append_kernel(plan->q_dtype, plan->d, mode, plan->interleaved);
  void* args[1] = {&p};
  p.heads = heads_of_cta(kern, plan->num_rows, plan->num_units, plan->longest, plan->hkv,
                         plan->hq / plan->hkv);
  const dim3 grid((unsigned)plan->num_units, (unsigned)((plan->hkv + p.heads - 1) / p.heads));
  // An ordinary launch.  As a programmatic dependent it saved 0.4-0.5 us of a
  // small append in a chain of appends, but placed its CTAs among those of a
  // decode kernel before it (a step of append and decode: 60.5 to 61.6 us, 78.8
  // where it let the decode kernel behind it in early as well).
  return cudaLaunchKernel(kern.func, grid, dim3(kern.threads), args, 0,
                          static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t fa_append_workspace_size(int batch, int64_t num_tokens) {
  if (batch < 0 || num_tokens < 0 || num_tokens > std::numeric_limits<int32_t>::max()) return 0;
  // a request's n tokens lie in at most n / 16 + 2 pages, and in at most n
  const int64_t units = std::min(num_tokens, num_tokens / kPageSize + 2 * (int64_t)batch);
  return append_layout(units, kMaxPairs).total;
}

int fa_append_plan(const int32_t* indptr_host, const int32_t* indices_dev,
                   const int32_t* last_page_len_host, const int32_t* append_indptr_host,
                   const int32_t* position_offset_host, int batch, int num_qo_heads,
                   int num_kv_heads, int head_dim, int page_size, fa_dtype q_dtype,
                   fa_dtype kv_dtype, const double* inv_freq_host, int rotary_dim,
                   int interleaved, void* workspace_dev, size_t workspace_bytes,
                   void* cuda_stream, fa_append_plan_t* out_plan) {
  if (!out_plan) return FA_ERR_INVALID_ARG;
  *out_plan = nullptr;
  if (!indptr_host || !append_indptr_host || batch < 0 || num_qo_heads <= 0 ||
      num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || num_qo_heads % num_kv_heads ||
      !workspace_dev || reinterpret_cast<uintptr_t>(workspace_dev) % kAlign)
    return FA_ERR_INVALID_ARG;
  if (batch > 0 && !last_page_len_host) return FA_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > head_dim || (rotary_dim > 0 && !inv_freq_host))
    return FA_ERR_INVALID_ARG;
  for (int i = 0; i < rotary_dim / 2; ++i)  // NaN fails the comparison
    if (!(std::fabs(inv_freq_host[i]) <= kMaxFrequency)) return FA_ERR_INVALID_ARG;
  if (page_size != kPageSize || (head_dim != 64 && head_dim != 128) ||
      !append_pair_built(q_dtype, kv_dtype) || rotary_dim % 16 ||
      num_kv_heads > 65535)
    return FA_ERR_UNSUPPORTED;
  if (indptr_host[0] != 0 || append_indptr_host[0] != 0) return FA_ERR_INVALID_ARG;

  std::vector<uint8_t> meta;
  fa_append_plan_s* plan = nullptr;
  int64_t units = 0;
  int longest = 0;
  AppendLayout L{};
  for (int pass = 0; pass < 2; ++pass) {  // count the units, then write them
    AppendUnit* out =
        pass ? reinterpret_cast<AppendUnit*>(meta.data() + L.units) : nullptr;
    units = 0;
    for (int i = 0; i < batch; ++i) {
      const int64_t n = (int64_t)append_indptr_host[i + 1] - append_indptr_host[i];
      const int64_t np = (int64_t)indptr_host[i + 1] - indptr_host[i];
      if (n < 0 || np < 0) return FA_ERR_INVALID_ARG;
      if (np > 0 && (last_page_len_host[i] < 1 || last_page_len_host[i] > page_size))
        return FA_ERR_INVALID_ARG;
      const int64_t len = np > 0 ? (np - 1) * page_size + last_page_len_host[i] : 0;
      const int64_t off = position_offset_host ? position_offset_host[i] : 0;
      if (n > len || off < 0 || off + len > std::numeric_limits<int32_t>::max())
        return FA_ERR_INVALID_ARG;
      for (int64_t t = len - n; t < len;) {
        const int64_t page = t / page_size, end = std::min(len, (page + 1) * page_size);
        if (out)
          out[units] = AppendUnit{(int32_t)(append_indptr_host[i] + (t - (len - n))),
                                  (int32_t)(indptr_host[i] + page),
                                  (int32_t)(t - page * page_size) | (int32_t)((end - t) << 8),
                                  (int32_t)(off + t)};
        longest = std::max(longest, (int)(end - t));
        ++units;
        t = end;
      }
    }
    if (pass == 0) {
      if (append_indptr_host[batch] > 0 && !indices_dev) return FA_ERR_INVALID_ARG;
      L = append_layout(units, rotary_dim / 2);
      if (L.total > workspace_bytes) return FA_ERR_WORKSPACE_TOO_SMALL;
      try {
        meta.assign(L.total, 0);
      } catch (const std::bad_alloc&) {
        return FA_ERR_INVALID_ARG;
      }
    }
  }
  unsigned long long* turns = reinterpret_cast<unsigned long long*>(meta.data() + L.turns);
  for (int i = 0; i < rotary_dim / 2; ++i) turns[i] = turns_of(inv_freq_host[i]);

  plan = new (std::nothrow) fa_append_plan_s();
  if (!plan) return FA_ERR_INVALID_ARG;
  plan->hq = num_qo_heads;
  plan->hkv = num_kv_heads;
  plan->d = head_dim;
  plan->q_dtype = q_dtype;
  plan->kv_dtype = kv_dtype;
  plan->indices = indices_dev;
  plan->ws = static_cast<uint8_t*>(workspace_dev);
  plan->layout = L;
  plan->num_units = units;
  plan->num_rows = append_indptr_host[batch];
  plan->longest = longest;
  plan->pairs = rotary_dim / 2;
  plan->interleaved = interleaved != 0;
  if (cudaGetDevice(&plan->device) != cudaSuccess ||
      upload_async(plan->ws, meta.data(), meta.size(), static_cast<cudaStream_t>(cuda_stream)) !=
          cudaSuccess) {
    delete plan;
    return FA_ERR_CUDA;
  }
  *out_plan = plan;
  return FA_OK;
}

int fa_append_run(fa_append_plan_t plan, const fa_rows* k, const fa_rows* v, const fa_rows* q,
                  void* q_out, void* paged_kv, int64_t num_pages, float k_scale, float v_scale,
                  void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  const bool e4m3 = plan->kv_dtype == FA_DTYPE_E4M3;
  // per-tensor scales belong to an E4M3 cache; another one is written as it is
  if (!e4m3 && (k_scale != 1.f || v_scale != 1.f)) return FA_ERR_INVALID_ARG;
  if (!(k_scale >= kMinScale && k_scale < INFINITY && v_scale >= kMinScale && v_scale < INFINITY))
    return FA_ERR_INVALID_ARG;
  return append_run(plan, e4m3 ? kStatic : kNative, k, v, q, q_out, paged_kv, num_pages, k_scale,
                    v_scale, nullptr, nullptr, nullptr, nullptr, cuda_stream);
}

int fa_append_run_head_scales(fa_append_plan_t plan, const fa_rows* k, const fa_rows* v,
                              const fa_rows* q, void* q_out, void* paged_kv, int64_t num_pages,
                              const float* k_head_scales, const float* v_head_scales,
                              void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->kv_dtype != FA_DTYPE_E4M3) return FA_ERR_UNSUPPORTED;
  if (!k_head_scales || !v_head_scales || reinterpret_cast<uintptr_t>(k_head_scales) % 4 ||
      reinterpret_cast<uintptr_t>(v_head_scales) % 4)
    return FA_ERR_INVALID_ARG;
  return append_run(plan, kStatic, k, v, q, q_out, paged_kv, num_pages, 1.f, 1.f, k_head_scales,
                    v_head_scales, nullptr, nullptr, cuda_stream);
}

static int append_run_dynamic(fa_append_plan_t plan, Mode mode, const fa_rows* k,
                              const fa_rows* v, const fa_rows* q, void* q_out, void* paged_kv,
                              int64_t num_pages, float* k_scales, float* v_scales,
                              void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->kv_dtype != FA_DTYPE_E4M3) return FA_ERR_UNSUPPORTED;
  if (!k_scales || !v_scales || reinterpret_cast<uintptr_t>(k_scales) % 4 ||
      reinterpret_cast<uintptr_t>(v_scales) % 4)
    return FA_ERR_INVALID_ARG;
  return append_run(plan, mode, k, v, q, q_out, paged_kv, num_pages, 1.f, 1.f, nullptr, nullptr,
                    k_scales, v_scales, cuda_stream);
}

int fa_append_run_token_scales(fa_append_plan_t plan, const fa_rows* k, const fa_rows* v,
                               const fa_rows* q, void* q_out, void* paged_kv, int64_t num_pages,
                               float* k_scales, float* v_scales, void* cuda_stream) {
  return append_run_dynamic(plan, kToken, k, v, q, q_out, paged_kv, num_pages, k_scales,
                            v_scales, cuda_stream);
}

int fa_append_run_block_scales(fa_append_plan_t plan, const fa_rows* k, const fa_rows* v,
                               const fa_rows* q, void* q_out, void* paged_kv, int64_t num_pages,
                               float* k_scales, float* v_scales, void* cuda_stream) {
  return append_run_dynamic(plan, kBlock, k, v, q, q_out, paged_kv, num_pages, k_scales,
                            v_scales, cuda_stream);
}

int fa_append_check(fa_append_plan_t plan, void* cuda_stream, int* flags) {
  if (!plan || !flags) return FA_ERR_INVALID_ARG;
  int word = 0;
  if (take_word(reinterpret_cast<int*>(plan->ws), &word,
                static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess)
    return FA_ERR_CUDA;
  *flags = word;
  return word ? FA_ERR_DEVICE_CHECK : FA_OK;
}

int fa_append_plan_destroy(fa_append_plan_t plan) {
  delete plan;
  return FA_OK;
}

}  // extern "C"
