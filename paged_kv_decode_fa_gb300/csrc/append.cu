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
// multiplies, and its top 32 bits go to sincospi as half-turns in [-1, 1).
//
// E4M3 caches: code = rn(x / s) saturated at 448, with s per tensor, per kv
// head, per token (amax over the row / 448, written here) or per block, a
// page's tokens of one kv head: the smallest power of two with amax <= 448 s.
// A power of two costs a code no relative precision (E4M3 is floating point),
// and a page that goes on filling keeps max(old, needed): when that grows, the
// codes it holds are divided by a power of two, exactly but for subnormals,
// so a page filled a token at a time reads as one filled at once.
//
// Work: one CTA per (page run, up to 4 kv heads); a run is the new tokens of
// one request in one page, at most 16.  The angles of a run are computed once
// into shared memory (they depend on the token and the pair only) and kept in
// registers by a thread, which serves one token and 16 bytes of a row and
// goes over its heads.  All K and V loads of a thread are issued before the
// angles are computed.  A block's amax needs all its tokens, which the CTA
// holds: one reduction in shared memory, no second pass over the inputs.
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

constexpr int kHeads = 4;        // kv heads of one CTA
constexpr int kItems = 2 * kHeads;  // K rows, then V rows, of a token in one CTA
constexpr int kMaxPairs = 64;    // rotary_dim / 2 at most

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
  int pairs;  // rotary_dim / 2
  int interleaved;
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

template <typename T, int E>
__device__ __forceinline__ void widen(const uint4& r, float (&x)[E]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = unpack(w[i], T{});
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <typename T, int E>
__device__ __forceinline__ uint4 narrow(const float (&x)[E]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E == 4)
      w[i] = __float_as_uint(x[i]);
    else
      w[i] = pack(x[2 * i], x[2 * i + 1], T{});
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// x * inv as an E4M3 code: finite values saturate at 448; a non-finite x,
// which E4M3 cannot tell from a large one, becomes NaN (x - x is 0 or NaN).
__device__ __forceinline__ uint32_t code2(float a, float b, float inv) {
  const float2 y = make_float2(fmaf(a, inv, a - a), fmaf(b, inv, b - b));
  return __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8: the
// carry out of the mantissa marks one above .75); 0 for 0.
__device__ __forceinline__ float block_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;  // biased exponent
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

__device__ __forceinline__ float inverse(float scale) { return scale > 0.f ? 1.f / scale : 0.f; }

template <typename T, int D>
struct Cfg {
  static constexpr int E = 16 / (int)sizeof(T);  // elements of a thread's 16 bytes
  static constexpr int LPR = D / E;              // threads of a row
  static constexpr int THREADS = LPR * 16 < 256 ? 256 : LPR * 16;
  static constexpr int ROWS = THREADS / LPR;  // rows in step, at least a page's tokens
};

// A thread's rotation: cos and sin of its E elements (interleaved: E / 2
// pairs), and the lane that holds the other halves of its pairs.
template <int E>
struct Turn {
  float c[E], s[E];
  int partner;
  bool on, first, interleaved;
};

template <typename T, int E>
__device__ __forceinline__ void rotate(const uint4& raw, const Turn<E>& r, float (&x)[E]) {
  widen<T, E>(raw, x);
  if (r.interleaved) {
    if (!r.on) return;
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      const float a = x[j], b = x[j + 1];
      x[j] = a * r.c[j / 2] - b * r.s[j / 2];
      x[j + 1] = b * r.c[j / 2] + a * r.s[j / 2];
    }
    return;
  }
  uint4 other;
  other.x = __shfl_sync(0xffffffffu, raw.x, r.partner);
  other.y = __shfl_sync(0xffffffffu, raw.y, r.partner);
  other.z = __shfl_sync(0xffffffffu, raw.z, r.partner);
  other.w = __shfl_sync(0xffffffffu, raw.w, r.partner);
  if (!r.on) return;
  float y[E];
  widen<T, E>(other, y);
#pragma unroll
  for (int j = 0; j < E; ++j)
    x[j] = r.first ? x[j] * r.c[j] - y[j] * r.s[j] : x[j] * r.c[j] + y[j] * r.s[j];
}

template <int E, int LPR>
__device__ __forceinline__ float row_amax(const float (&x)[E]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const float a = fabsf(x[j]);
    m = fmaxf(m, a < INFINITY ? a : 0.f);
  }
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(Cfg<T, D>::THREADS)
    fa_append_kernel(const AppendParams p) {
  using C = Cfg<T, D>;
  constexpr int E = C::E, LPR = C::LPR;
  __shared__ float2 angle[kPageSize * kMaxPairs];
  __shared__ int amax_bits[kItems];
  __shared__ float item_scale[kItems], item_ratio[kItems];

  const AppendUnit u = p.units[blockIdx.x];
  const int slot0 = u.slots & 0xff, n = u.slots >> 8;
  const int h0 = blockIdx.y * kHeads, heads = min(kHeads, p.hkv - h0), items = 2 * heads;
  const int tid = threadIdx.x, lane = tid & 31;
  // this thread: 16 bytes of a row from dim d0, of token `tok`, and of rows
  // hg, hg + HG, ... of the CTA's K and V rows, and then of its q rows
  const int c = tid % LPR, r = tid / LPR, d0 = c * E;
  const int lg = n > 8 ? 4 : n > 4 ? 3 : n > 2 ? 2 : n > 1 ? 1 : 0;
  const int tok = r & ((1 << lg) - 1), hg = r >> lg, HG = C::ROWS >> lg;
  const bool live = tok < n;
  const int64_t row = u.row + tok;

  uint4 raw[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (i * HG >= items) break;
    const int it = i * HG + hg;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live && it < items) {
      const Rows& in = it < heads ? p.k : p.v;
      const int h = h0 + (it < heads ? it : it - heads);
      raw[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(in.p) +
                                                    row * in.token + h * in.head + d0));
    }
  }
  const int page = __ldg(p.indices + u.entry);
  const bool page_ok = page >= 0 && (int64_t)page < p.num_pages;
  if (!page_ok && tid == 0) atomicOr(p.err, 1);

  for (int i = tid; i < n * p.pairs; i += C::THREADS) {
    const int t = i / p.pairs;
    const unsigned long long turn =
        (unsigned long long)(unsigned)(u.position + t) * p.turns[i - t * p.pairs];
    const int half_turns = (int)(turn >> 32);  // 2^-31 half-turns
    float2 cs;
    sincospif((float)half_turns * 4.656612873077393e-10f, &cs.y, &cs.x);
    angle[t * kMaxPairs + (i - t * p.pairs)] = cs;
  }
  if (MODE == kBlock && tid < kItems) amax_bits[tid] = 0;
  __syncthreads();

  Turn<E> turn;
  turn.interleaved = p.interleaved != 0;
  turn.on = live && d0 < 2 * p.pairs;
  turn.first = d0 < p.pairs;
  turn.partner = lane;
  if (!turn.interleaved && d0 < 2 * p.pairs)
    turn.partner = turn.first ? lane + p.pairs / E : lane - p.pairs / E;
#pragma unroll
  for (int j = 0; j < E; ++j) turn.c[j] = turn.s[j] = 0.f;
  if (turn.on) {
    const int at = tok * kMaxPairs + (turn.interleaved ? d0 / 2 : turn.first ? d0 : d0 - p.pairs);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (j < E / 2 || !turn.interleaved) {
        const float2 cs = angle[at + j];
        turn.c[j] = cs.x;
        turn.s[j] = cs.y;
      }
    }
  }

  if constexpr (MODE == kBlock) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (i * HG >= items) break;
      const int it = i * HG + hg;
      Turn<E> t = turn;
      // K and V rows may share a warp: V rows take part in the exchange only
      t.on = turn.on && it < heads;
      float x[E];
      rotate<T, E>(raw[i], t, x);
      const float m = row_amax<E, LPR>(x);
      if (c == 0 && live && it < items) atomicMax(&amax_bits[it], __float_as_int(m));
    }
    __syncthreads();
    if (tid < items) {
      const bool is_k = tid < heads;
      float* scales = is_k ? p.k_scales : p.v_scales;
      const float need = block_scale(__int_as_float(amax_bits[tid]));
      float old = 0.f, now = need;
      if (page_ok) {
        const int64_t at = (int64_t)page * p.hkv + h0 + (is_k ? tid : tid - heads);
        if (slot0 > 0) old = scales[at];
        now = fmaxf(old, need);
        if (slot0 == 0 || now > old) scales[at] = now;
      }
      item_scale[tid] = now;
      item_ratio[tid] = now > old ? old * inverse(now) : 1.f;
    }
    __syncthreads();
    if (slot0 > 0 && page_ok) {
      // codes the page already holds, under the scales that grew
      for (int it = 0; it < items; ++it) {
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

#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (i * HG >= items) break;
    const int it = i * HG + hg;
    const bool is_k = it < heads;
    const int h = h0 + (is_k ? it : it - heads);
    Turn<E> t = turn;
    t.on = turn.on && is_k;
    float x[E];
    rotate<T, E>(raw[i], t, x);
    float inv = 1.f, scale = 1.f;
    if constexpr (MODE == kStatic) {
      const float* hs = is_k ? p.head_k_scales : p.head_v_scales;
      inv = inverse(!hs ? (is_k ? p.k_scale : p.v_scale) : it < items ? __ldg(hs + h) : 1.f);
    } else if constexpr (MODE == kToken) {
      const float m = row_amax<E, LPR>(x);
      scale = m > 0.f ? fmaxf(m / 448.f, 1.17549435e-38f) : 0.f;
      inv = inverse(scale);
    } else if constexpr (MODE == kBlock) {
      inv = it < items ? inverse(item_scale[it]) : 0.f;
    }
    if (!live || it >= items || !page_ok) continue;
    const int64_t at =
        ((((int64_t)page * 2 + (is_k ? 0 : 1)) * kPageSize + slot0 + tok) * p.hkv + h) * D + d0;
    if constexpr (MODE == kNative) {
      *reinterpret_cast<uint4*>(static_cast<T*>(p.kv) + at) = narrow<T, E>(x);
    } else {
      if constexpr (MODE == kToken) {
        if (c == 0)
          (is_k ? p.k_scales : p.v_scales)[((int64_t)page * p.hkv + h) * kPageSize + slot0 + tok] =
              scale;
      }
      static_assert(MODE == kNative || E == 8, "E4M3 caches take 16-bit inputs");
      uint2 w;
      w.x = code2(x[0], x[1], inv) | (code2(x[2], x[3], inv) << 16);
      w.y = code2(x[E - 4], x[E - 3], inv) | (code2(x[E - 2], x[E - 1], inv) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.kv) + at) = w;
    }
  }

  if (p.q.p == nullptr) return;
  const int group = p.hq / p.hkv, rows_q = heads * group;
  for (int i0 = 0; i0 < rows_q; i0 += HG) {
    const int h = h0 * group + i0 + hg;
    const bool ok = live && i0 + hg < rows_q;
    uint4 in = make_uint4(0u, 0u, 0u, 0u);
    // not through the read-only path: q_out may be q itself
    if (ok)
      in = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q.p) + row * p.q.token +
                                           h * p.q.head + d0);
    float x[E];
    rotate<T, E>(in, turn, x);
    if (ok)
      *reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + (row * p.hq + h) * D + d0) =
          narrow<T, E>(x);
  }
}

struct AppendKernel {
  const void* func = nullptr;
  int threads = 0;
};

template <typename T, int MODE>
AppendKernel kernel_of(int head_dim) {
  if (head_dim == 64)
    return {reinterpret_cast<const void*>(&fa_append_kernel<T, 64, MODE>), Cfg<T, 64>::THREADS};
  return {reinterpret_cast<const void*>(&fa_append_kernel<T, 128, MODE>), Cfg<T, 128>::THREADS};
}

// A kernel for q's type, the cache being E4M3 unless mode is kNative.
AppendKernel find_append_kernel(fa_dtype q, int head_dim, Mode mode) {
  if (q == FA_DTYPE_F32) return kernel_of<float, kNative>(head_dim);
  if (q == FA_DTYPE_BF16) {
    if (mode == kStatic) return kernel_of<__nv_bfloat16, kStatic>(head_dim);
    if (mode == kToken) return kernel_of<__nv_bfloat16, kToken>(head_dim);
    if (mode == kBlock) return kernel_of<__nv_bfloat16, kBlock>(head_dim);
    return kernel_of<__nv_bfloat16, kNative>(head_dim);
  }
  if (mode == kStatic) return kernel_of<__half, kStatic>(head_dim);
  if (mode == kToken) return kernel_of<__half, kToken>(head_dim);
  if (mode == kBlock) return kernel_of<__half, kBlock>(head_dim);
  return kernel_of<__half, kNative>(head_dim);
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
  int pairs = 0, interleaved = 0;
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
  p.interleaved = plan->interleaved;
  const AppendKernel kern = find_append_kernel(plan->q_dtype, plan->d, mode);
  void* args[1] = {&p};
  const dim3 grid((unsigned)plan->num_units, (unsigned)((plan->hkv + kHeads - 1) / kHeads));
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
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!std::isfinite(inv_freq_host[i])) return FA_ERR_INVALID_ARG;
  if (page_size != kPageSize || (head_dim != 64 && head_dim != 128) ||
      !append_pair_built(q_dtype, kv_dtype) || rotary_dim % 16 ||
      num_kv_heads > 65535 * kHeads)
    return FA_ERR_UNSUPPORTED;
  if (indptr_host[0] != 0 || append_indptr_host[0] != 0) return FA_ERR_INVALID_ARG;

  std::vector<uint8_t> meta;
  fa_append_plan_s* plan = nullptr;
  int64_t units = 0;
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
  plan->pairs = rotary_dim / 2;
  plan->interleaved = interleaved ? 1 : 0;
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
  if (!(k_scale > 0.f && k_scale < INFINITY && v_scale > 0.f && v_scale < INFINITY))
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
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess ||
      cudaMemcpy(&word, plan->ws, sizeof word, cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(plan->ws, 0, sizeof word) != cudaSuccess)
    return FA_ERR_CUDA;
  *flags = word;
  return word ? FA_ERR_DEVICE_CHECK : FA_OK;
}

int fa_append_plan_destroy(fa_append_plan_t plan) {
  delete plan;
  return FA_OK;
}

}  // extern "C"
