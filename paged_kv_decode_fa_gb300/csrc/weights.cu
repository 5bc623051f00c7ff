// Attention weights accumulated per cached token: the calls fa_weights_* (declared
// in include/fa_decode.h).
//
// The mathematics.  A cached token t of a request gains, in its kv head,
//     w_t += sum over query rows r that see t and the group's heads g of
//            2^(c q_rg . k_t - lse_rg log2 e),   c = sm_scale log2 e,
// the weight that the softmax of those rows gave it; lse is what the attention
// of the same rows returned.  One pass over K, none over V.
//
// Work.  Requests of more than eight columns (query row x head of the group) go
// through weights_tc.cuh.  Of the others a CTA takes a kv head and a run of pages, a
// warp one page at a time: its 16 tokens are the MMA's M side (m16n8k16, mma.sync), the
// columns its N side.  The dot product does not mind the order of dims, so a lane's
// fragments are whole 16-byte pieces of a K row and of a q row: lane c of a row's four
// holds dims 8c .. 8c+7 of every 32 (16 of every 64 codes of an E4M3 cache), straight
// from global memory into registers.  Every token's weight is one addition to
// memory a call, so the result does not depend on the schedule.  (Pages that two
// requests share receive two.)
//
// What bounds it: HBM.  128 requests of 1024-8192 tokens, 64 / 8 heads, bf16, 1.28 GB:
// 209 us = 6.1 TB/s, 0.91 of the copy rate (246 us with each page's id loaded in front
// of its rows).  Over an E4M3 cache (618 MB, scales per block) 172 us = 3.6 TB/s: a warp
// has one page on its way, of half the bytes.  Few short requests: the launch and one
// chain of loads, 8 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <new>
#include <type_traits>
#include <vector>

#include "decode_mma.cuh"
#include "fa_decode.h"
#include "staging.h"
#include "tensor_map.h"

namespace fadecode {

// A run of a request's pages.
struct WeightsUnit {
  int32_t row0, rows;    // query rows of the request
  int32_t entry, pages;  // table entries of the run
  int32_t pos0;          // position of its first token
  int32_t before;        // length - rows: row r sees positions up to before + r
  int32_t pad[2];
};
static_assert(sizeof(WeightsUnit) == 32, "read as two int4");

struct WeightsParams {
  const void* q;  // [rows, Hq, D], by strides in elements
  int64_t q_token, q_head;
  const void* kv;
  const float* lse;           // [rows, Hq]
  float* weights;             // [pages, Hkv, 16]
  const float* k_scales;      // kScalePerToken [pages, Hkv, 16], kScalePerBlock [pages, Hkv]
  const float* head_k_scales; // [Hkv] times scale, or nullptr
  const int32_t* indices;
  const WeightsUnit* units;
  int* err;
  int64_t num_pages;
  int hq, hkv;
  int group_log2;
  float scale;  // sm_scale * k_scale * log2(e)
};

// Two E4M3 codes as a pair of T (exact in both 16-bit types).
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  if constexpr (std::is_same<T, __half>::value) {
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
  } else {
    // four significant bits at most: the upper halves of the floats are exact
    const float2 f = __half22float2(__half2(h));
    return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
  }
}

}  // namespace fadecode

#include "weights_tc.cuh"

namespace fadecode {
namespace {

constexpr int kWarps = 8;
constexpr int kMostPages = 64;  // of a run
constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1, bool bf16) {
  if (bf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragments of a page's K: two MMAs' A operands (rows n and n + 8, 16 dims each) for each
// 16-byte piece of a q row.
template <int D>
struct Fragments {
  uint32_t a[D / 32][2][4];
};

template <typename T, typename KVT, int D>
__device__ __forceinline__ void widen_page(const uint4 (&k)[2][D * sizeof(KVT) / 64],
                                           Fragments<D>* f) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    if constexpr (!std::is_same<T, KVT>::value) {
      const uint4 lo = k[0][j / 2], hi = k[1][j / 2];
      const uint32_t l[2] = {j % 2 ? lo.z : lo.x, j % 2 ? lo.w : lo.y};
      const uint32_t h[2] = {j % 2 ? hi.z : hi.x, j % 2 ? hi.w : hi.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f->a[j][i][0] = widen2<T>(l[i] & 0xffffu);
        f->a[j][i][1] = widen2<T>(h[i] & 0xffffu);
        f->a[j][i][2] = widen2<T>(l[i] >> 16);
        f->a[j][i][3] = widen2<T>(h[i] >> 16);
      }
    } else {
      const uint4 lo = k[0][j], hi = k[1][j];
      const uint32_t w[2][4] = {{lo.x, hi.x, lo.y, hi.y}, {lo.z, hi.z, lo.w, hi.w}};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) f->a[j][i][e] = w[i][e];
    }
  }
}

// What a CTA works on, and its loads.
template <typename T, typename KVT, int D, int SC>
struct Worker {
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr bool kE4m3 = !std::is_same<T, KVT>::value;
  static constexpr int kPiece = 16 / sizeof(KVT);  // elements of a lane's 16 bytes of K
  static constexpr int kPieces = D / (4 * kPiece);  // of them in a row
  static constexpr int kQPieces = D / 32;
  const WeightsParams& p;
  int row0, rows, entry, pages, pos0, before;  // see WeightsUnit
  int h, lane, c, n;  // c: piece of a row; n: token and column of the fragments
  int columns;
  int ids[2];  // of the run's pages lane and lane + 32, -1 for none
  float head_scale;

  __device__ __forceinline__ explicit Worker(const WeightsParams& params) : p(params) {
    const int4* up = reinterpret_cast<const int4*>(p.units + blockIdx.x / p.hkv);
    const int4 a = __ldg(up), b = __ldg(up + 1);
    row0 = a.x;
    rows = a.y;
    entry = a.z;
    pages = a.w;
    pos0 = b.x;
    before = b.y;
    h = blockIdx.x % p.hkv;
    lane = threadIdx.x & 31;
    c = lane % 4;
    n = lane / 4;
    columns = rows << p.group_log2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = lane + 32 * i;
      ids[i] = at < pages ? __ldg(p.indices + entry + at) : -1;
      if (ids[i] < 0 || (int64_t)ids[i] >= p.num_pages) {
        if (at < pages) atomicOr(p.err, 1);
        ids[i] = -1;
      }
    }
    head_scale = p.head_k_scales ? p.scale * __ldg(p.head_k_scales + h) : p.scale;
  }
  // K of the run's page i; -1 if there is none
  __device__ __forceinline__ int load_page(int i, uint4 (&k)[2][kPieces]) const {
    static_assert(kMostPages <= 64, "the run's page ids are held two a lane");
    const int lo = __shfl_sync(0xffffffffu, ids[0], i % 32);
    const int hi = __shfl_sync(0xffffffffu, ids[1], i % 32);
    const int page = i < 32 ? lo : i < 64 ? hi : -1;
    const int64_t token_stride = (int64_t)p.hkv * D;
    const KVT* base = static_cast<const KVT*>(p.kv) +
                      (int64_t)max(page, 0) * 2 * kPageSize * token_stride + (int64_t)h * D;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        k[t][j] = page < 0 ? make_uint4(0u, 0u, 0u, 0u)
                           : __ldg(reinterpret_cast<const uint4*>(
                                 base + (n + 8 * t) * token_stride + (4 * j + c) * kPiece));
    return page;
  }
  // column x = (row, head of the group): its q row as B fragments
  __device__ __forceinline__ void load_column(int x, uint4 (&b)[kQPieces]) const {
    const T* q = static_cast<const T*>(p.q) + (row0 + (x >> p.group_log2)) * p.q_token +
                 (int64_t)((h << p.group_log2) + (x & ((1 << p.group_log2) - 1))) * p.q_head;
#pragma unroll
    for (int j = 0; j < kQPieces; ++j) {
      // the dims that this lane's piece of K holds
      const int d = kE4m3 ? (j / 2) * 64 + c * 16 + (j % 2) * 8 : (4 * j + c) * 8;
      b[j] = x < columns ? __ldg(reinterpret_cast<const uint4*>(q + d))
                         : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // its lse in log2 units; +inf (weight 0) behind the last column and where the row
  // saw nothing
  __device__ __forceinline__ float load_lse(int x) const {
    const int row = x >> p.group_log2, g = x & ((1 << p.group_log2) - 1);
    const float lse = x < columns ? __ldg(p.lse + (int64_t)(row0 + row) * p.hq +
                                          (h << p.group_log2) + g) * 1.4426950408889634f
                                  : INFINITY;
    return lse == -INFINITY ? INFINITY : lse;
  }
  // the logit scales of tokens n and n + 8 of a page
  __device__ __forceinline__ void load_scales(int page, float (&scale)[2]) const {
    const int64_t at = ((int64_t)page * p.hkv + h) * kPageSize;
    scale[0] = scale[1] = head_scale;
    if constexpr (SC == kScalePerToken) {
      scale[0] *= __ldg(p.k_scales + at + n);
      scale[1] *= __ldg(p.k_scales + at + n + 8);
    } else if constexpr (SC == kScalePerBlock) {
      scale[0] = scale[1] = head_scale * __ldg(p.k_scales + at / kPageSize);
    }
  }
  // The columns against a page whose token n is at position pos: their weights' sums
  // for tokens n and n + 8, this lane's two columns
  __device__ __forceinline__ void add_columns(const Fragments<D>& k, const uint4 (&b)[kQPieces],
                                              const float (&lse)[2], const float (&scale)[2],
                                              int pos, float (&sum)[2]) const {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kQPieces; ++j) {
      mma_16816(s, k.a[j][0], b[j].x, b[j].y, kBf16);
      mma_16816(s, k.a[j][1], b[j].z, b[j].w, kBf16);
    }
    // s[0], s[1]: token n, columns 2c, + 1; s[2], s[3]: token n + 8
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // a column behind the last, or whose row has an lse of -inf, adds nothing, whatever
      // its score is (zeros times an infinite K are NaN, as may be a padded row's q)
      const int last = lse[e] != INFINITY ? before + ((2 * c + e) >> p.group_log2) : -1;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (pos + 8 * t <= last) sum[t] += dev::fast_exp2(fmaf(s[2 * t + e], scale[t], -lse[e]));
    }
  }
  // A page's sums over its columns, added to the weights; tokens that no row sees
  // (slots behind the request's last) stay
  __device__ __forceinline__ void store(int page, int pos, float (&sum)[2]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], 1);
      sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], 2);
    }
    if (page >= 0 && c < 2 && pos + 8 * c <= before + rows - 1)
      atomicAdd(p.weights + ((int64_t)page * p.hkv + h) * kPageSize + n + 8 * c, sum[c]);
  }
};

// Eight columns at most (a decode step): they stay in registers while the pages
// pass, each loaded while the one before is worked on.
template <typename T, typename KVT, int D, int SC>
__global__ void __launch_bounds__(kWarps * 32, 2) fa_weights_kernel(const WeightsParams p) {
  using W = Worker<T, KVT, D, SC>;
  const W w(p);
  uint4 q[W::kQPieces];
  w.load_column(w.n, q);
  const float lse[2] = {w.load_lse(2 * w.c), w.load_lse(2 * w.c + 1)};
  uint4 raw[2][W::kPieces];
  const int warp = threadIdx.x >> 5;
  int page = w.load_page(warp, raw);
  for (int i = warp; i < w.pages; i += kWarps) {
    Fragments<D> k;
    widen_page<T, KVT, D>(raw, &k);
    const int this_page = page;
    page = w.load_page(i + kWarps, raw);
    if (this_page < 0) continue;
    float scale[2], sum[2] = {0.f, 0.f};
    w.load_scales(this_page, scale);
    const int pos = w.pos0 + i * kPageSize + w.n;
    w.add_columns(k, q, lse, scale, pos, sum);
    w.store(this_page, pos, sum);
  }
}

using WeightsFn = void (*)(const WeightsParams);

template <typename T, typename KVT, int D>
WeightsFn weights_kernel(int sc) {
  if constexpr (std::is_same<T, KVT>::value) {
    return &fa_weights_kernel<T, KVT, D, kScaleNone>;
  } else {
    return sc == kScalePerToken   ? &fa_weights_kernel<T, KVT, D, kScalePerToken>
           : sc == kScalePerBlock ? &fa_weights_kernel<T, KVT, D, kScalePerBlock>
                                  : &fa_weights_kernel<T, KVT, D, kScaleNone>;
  }
}

template <int D>
WeightsFn find_weights_kernel(fa_dtype q, bool e4m3, int sc) {
  if (q == FA_DTYPE_BF16)
    return e4m3 ? weights_kernel<__nv_bfloat16, uint8_t, D>(sc)
                : weights_kernel<__nv_bfloat16, __nv_bfloat16, D>(sc);
  return e4m3 ? weights_kernel<__half, uint8_t, D>(sc) : weights_kernel<__half, __half, D>(sc);
}

template <typename T, typename KVT, int D>
const void* weights_tc_kernel(int sc) {
  const auto f = [](auto k) { return reinterpret_cast<const void*>(k); };
  if constexpr (std::is_same<T, KVT>::value) {
    return f(&fa_weights_tc_kernel<T, KVT, D, kScaleNone>);
  } else {
    return sc == kScalePerToken   ? f(&fa_weights_tc_kernel<T, KVT, D, kScalePerToken>)
           : sc == kScalePerBlock ? f(&fa_weights_tc_kernel<T, KVT, D, kScalePerBlock>)
                                  : f(&fa_weights_tc_kernel<T, KVT, D, kScaleNone>);
  }
}

template <int D>
const void* find_weights_tc_kernel(fa_dtype q, bool e4m3, int sc) {
  if (q == FA_DTYPE_BF16)
    return e4m3 ? weights_tc_kernel<__nv_bfloat16, uint8_t, D>(sc)
                : weights_tc_kernel<__nv_bfloat16, __nv_bfloat16, D>(sc);
  return e4m3 ? weights_tc_kernel<__half, uint8_t, D>(sc)
              : weights_tc_kernel<__half, __half, D>(sc);
}

bool weights_pair_built(fa_dtype q, fa_dtype kv) {
  return (q == FA_DTYPE_BF16 || q == FA_DTYPE_F16) && (kv == q || kv == FA_DTYPE_E4M3);
}

// Pages of a run: 64 (eight a warp), halved while that leaves under four CTAs an SM.
int run_pages(int64_t total_pages, int heads, int sms) {
  int n = kMostPages;
  while (n > kWarps && total_pages * heads < (int64_t)n * 4 * sms) n /= 2;
  return n;
}

// Requests of more columns than this go through the tcgen05 kernel, in runs of
// kTcPages.  (16 requests of 4096 tokens, 32 / 8 heads, us there and with the columns
// eight at a time on mma.sync: 12 columns 31 and 38, 32 columns 31 and 52, 64
// columns 33 and 83; over an E4M3 cache 29 and 29, 30 and 42, 35 and 70.)
constexpr int kFewColumns = 8;
constexpr int kTcPages = 2 * wt::kPages;
// Columns of one request.  A job passes through them all, 128 a tile of at most 1.7 us
// (2460 cycles with masks, at 1.5 GHz), and the kernel's other warps wait for it 2 s.
constexpr int64_t kMostColumns = (int64_t)1 << 26;

// Runs of a batch's requests of many columns (`many`) or of the others; -1 for
// malformed arguments.
int64_t make_units(const int32_t* indptr, const int32_t* last_page_len, const int32_t* qo_indptr,
                   int batch, int group, bool many, int run, WeightsUnit* out) {
  int64_t units = 0;
  for (int i = 0; i < batch; ++i) {
    const int64_t n = (int64_t)qo_indptr[i + 1] - qo_indptr[i];
    const int64_t pages = (int64_t)indptr[i + 1] - indptr[i];
    if (n < 0 || pages < 0) return -1;
    if (pages > 0 && (last_page_len[i] < 1 || last_page_len[i] > kPageSize)) return -1;
    const int64_t len = pages > 0 ? (pages - 1) * kPageSize + last_page_len[i] : 0;
    if (len > std::numeric_limits<int32_t>::max() - 2 * wt::kTok ||
        n * group > std::numeric_limits<int32_t>::max() - wt::kTok)
      return -1;
    if (n == 0 || (n * group > kFewColumns) != many) continue;
    for (int64_t e = 0; e < pages; e += run, ++units)
      if (out)
        out[units] = WeightsUnit{qo_indptr[i],
                                 (int32_t)n,
                                 (int32_t)(indptr[i] + e),
                                 (int32_t)std::min<int64_t>(run, pages - e),
                                 (int32_t)(e * kPageSize),
                                 (int32_t)(len - n),
                                 {0, 0}};
  }
  return units;
}

}  // namespace
}  // namespace fadecode

using namespace fadecode;

struct fa_weights_plan_s {
  int device = 0;
  int hq = 0, hkv = 0, d = 0;
  fa_dtype q_dtype = FA_DTYPE_BF16, kv_dtype = FA_DTYPE_BF16;
  const int32_t* indices = nullptr;
  uint8_t* ws = nullptr;
  int64_t few = 0, many = 0;  // units of few columns, then of many
  int64_t rows = 0;
  int sms = 0;
  bool ready[3] = {false, false, false};  // the tcgen05 kernel, by kScale...
};

namespace {

int weights_run(fa_weights_plan_s* plan, int sc, const fa_rows* q, const void* paged_kv,
                int64_t num_pages, float sm_scale, const float* lse, float k_scale,
                const float* head_k, const float* k_scales, float* weights, void* cuda_stream) {
  if (plan->few + plan->many == 0) return FA_OK;
  if (!q || !q->data || !paged_kv || !lse || !weights || num_pages <= 0 ||
      num_pages >= (1 << 30) || reinterpret_cast<uintptr_t>(paged_kv) % 16 ||
      reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(weights) % 4 ||
      !q_rows_fit(*q, plan->rows, plan->hq))
    return FA_ERR_INVALID_ARG;
  if (!std::isfinite(k_scale)) return FA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev != plan->device) return FA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f)) sm_scale = 1.0f / std::sqrt((float)plan->d);
  WeightsParams p;
  std::memset(&p, 0, sizeof p);
  p.q = q->data;
  p.q_token = q->token_stride;
  p.q_head = q->head_stride;
  p.kv = paged_kv;
  p.lse = lse;
  p.weights = weights;
  p.k_scales = k_scales;
  p.head_k_scales = head_k;
  p.indices = plan->indices;
  p.units = reinterpret_cast<const WeightsUnit*>(plan->ws + kAlign);
  p.err = reinterpret_cast<int*>(plan->ws);
  p.num_pages = num_pages;
  p.hq = plan->hq;
  p.hkv = plan->hkv;
  while ((plan->hkv << p.group_log2) < plan->hq) ++p.group_log2;
  p.scale = sm_scale * k_scale * 1.4426950408889634f;
  const bool e4m3 = plan->kv_dtype == FA_DTYPE_E4M3;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  // all that can be refused comes before the first launch
  CUtensorMap maps[2];
  const void* tc = nullptr;
  const int smem = plan->d == 128 ? wt::Smem<128>::kBytes : wt::Smem<64>::kBytes;
  if (plan->many > 0) {
    std::memset(maps, 0, sizeof maps);
    if (!encode_q_rows(&maps[0], plan->q_dtype, *q, plan->rows, plan->hq, plan->d,
                       plan->hq / plan->hkv) ||
        !(e4m3 ? encode_codes(&maps[1], paged_kv, num_pages, plan->hkv, plan->d)
               : encode_pages(&maps[1], plan->q_dtype, paged_kv, num_pages, plan->hkv, plan->d)))
      return FA_ERR_CUDA;
    tc = plan->d == 128 ? find_weights_tc_kernel<128>(plan->q_dtype, e4m3, sc)
                        : find_weights_tc_kernel<64>(plan->q_dtype, e4m3, sc);
    if (!plan->ready[sc]) {
      // the kernel's warpgroups share out the registers it is launched with
      cudaFuncAttributes attr;
      if (cudaFuncGetAttributes(&attr, tc) != cudaSuccess ||
          (e4m3 && attr.numRegs < wt::kLaunchRegs) ||
          cudaFuncSetAttribute(tc, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
              cudaSuccess)
        return FA_ERR_CUDA;
      plan->ready[sc] = true;
    }
  }
  if (plan->few > 0) {
    const WeightsFn f = plan->d == 128 ? find_weights_kernel<128>(plan->q_dtype, e4m3, sc)
                                       : find_weights_kernel<64>(plan->q_dtype, e4m3, sc);
    void* args[1] = {&p};
    if (cudaLaunchKernel(reinterpret_cast<const void*>(f),
                         dim3((unsigned)(plan->few * plan->hkv)), dim3(kWarps * 32), args, 0,
                         st) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  if (plan->many > 0) {
    p.units += plan->few;
    int jobs = (int)(plan->many * plan->hkv);
    void* args[4] = {&maps[0], &maps[1], &p, &jobs};
    if (cudaLaunchKernel(tc, dim3((unsigned)std::min(jobs, plan->sms)), dim3(wt::threads(e4m3)),
                         args, (size_t)smem, st) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_weights_workspace_size(int batch, int64_t total_pages) {
  if (batch < 0 || total_pages < 0 || total_pages > std::numeric_limits<int32_t>::max()) return 0;
  // runs of eight pages at least
  return kAlign + align_up(sizeof(WeightsUnit) * (size_t)(total_pages / kWarps + batch));
}

int fa_weights_plan(const int32_t* indptr_host, const int32_t* indices_dev,
                    const int32_t* last_page_len_host, const int32_t* qo_indptr_host, int batch,
                    int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                    fa_dtype q_dtype, fa_dtype kv_dtype, void* workspace_dev,
                    size_t workspace_bytes, void* cuda_stream, fa_weights_plan_t* out_plan) {
  if (!out_plan) return FA_ERR_INVALID_ARG;
  *out_plan = nullptr;
  if (!indptr_host || !qo_indptr_host || batch < 0 || num_qo_heads <= 0 || num_kv_heads <= 0 ||
      head_dim <= 0 || page_size <= 0 || num_qo_heads % num_kv_heads ||
      (batch > 0 && !last_page_len_host) || !workspace_dev ||
      reinterpret_cast<uintptr_t>(workspace_dev) % kAlign)
    return FA_ERR_INVALID_ARG;
  const int G = num_qo_heads / num_kv_heads;
  if (page_size != kPageSize || (head_dim != 64 && head_dim != 128) ||
      (G != 1 && G != 2 && G != 4 && G != 8) || !weights_pair_built(q_dtype, kv_dtype))
    return FA_ERR_UNSUPPORTED;
  if (indptr_host[0] != 0 || qo_indptr_host[0] != 0) return FA_ERR_INVALID_ARG;
  if (indptr_host[batch] > 0 && !indices_dev) return FA_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  auto units = [&](bool many, int run, WeightsUnit* out) {
    return make_units(indptr_host, last_page_len_host, qo_indptr_host, batch, G, many, run, out);
  };
  // the arguments are checked before any CUDA call
  const int64_t many = units(true, kTcPages, nullptr);
  if (many < 0) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < batch; ++i)
    if (((int64_t)qo_indptr_host[i + 1] - qo_indptr_host[i]) * G > kMostColumns)
      return FA_ERR_UNSUPPORTED;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  const int run = run_pages(indptr_host[batch], num_kv_heads, sms);
  const int64_t few = units(false, run, nullptr);
  const size_t bytes = kAlign + sizeof(WeightsUnit) * (size_t)(few + many);
  if (bytes > workspace_bytes) return FA_ERR_WORKSPACE_TOO_SMALL;
  if (std::max(few, many) * num_kv_heads > std::numeric_limits<int32_t>::max() - 1024)
    return FA_ERR_UNSUPPORTED;
  try {
    std::vector<uint8_t> meta(bytes, 0);
    WeightsUnit* out = reinterpret_cast<WeightsUnit*>(meta.data() + kAlign);
    units(false, run, out);
    units(true, kTcPages, out + few);
    fa_weights_plan_s* plan = new fa_weights_plan_s();
    plan->device = dev;
    plan->hq = num_qo_heads;
    plan->hkv = num_kv_heads;
    plan->d = head_dim;
    plan->q_dtype = q_dtype;
    plan->kv_dtype = kv_dtype;
    plan->indices = indices_dev;
    plan->ws = static_cast<uint8_t*>(workspace_dev);
    plan->few = few;
    plan->many = many;
    plan->sms = sms;
    plan->rows = qo_indptr_host[batch];
    if (upload_async(plan->ws, meta.data(), bytes, static_cast<cudaStream_t>(cuda_stream)) !=
        cudaSuccess) {
      delete plan;
      return FA_ERR_CUDA;
    }
    *out_plan = plan;
  } catch (const std::bad_alloc&) {
    return FA_ERR_INVALID_ARG;
  }
  return FA_OK;
}

int fa_weights_run(fa_weights_plan_t plan, const fa_rows* q, const void* paged_kv,
                   int64_t num_pages, float sm_scale, float k_scale, const float* lse,
                   float* weights, void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->kv_dtype != FA_DTYPE_E4M3 && k_scale != 1.f) return FA_ERR_INVALID_ARG;
  return weights_run(plan, kScaleNone, q, paged_kv, num_pages, sm_scale, lse, k_scale, nullptr,
                     nullptr, weights, cuda_stream);
}

static int weights_run_scales(fa_weights_plan_t plan, int sc, bool heads, const fa_rows* q,
                              const void* paged_kv, int64_t num_pages, float sm_scale,
                              const float* k_scales, const float* lse, float* weights,
                              void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->kv_dtype != FA_DTYPE_E4M3) return FA_ERR_UNSUPPORTED;
  if (!k_scales || reinterpret_cast<uintptr_t>(k_scales) % 4) return FA_ERR_INVALID_ARG;
  return weights_run(plan, sc, q, paged_kv, num_pages, sm_scale, lse, 1.f,
                     heads ? k_scales : nullptr, heads ? nullptr : k_scales, weights, cuda_stream);
}

int fa_weights_run_head_scales(fa_weights_plan_t plan, const fa_rows* q, const void* paged_kv,
                               int64_t num_pages, float sm_scale, const float* k_head_scales,
                               const float* lse, float* weights, void* cuda_stream) {
  return weights_run_scales(plan, kScaleNone, true, q, paged_kv, num_pages, sm_scale,
                            k_head_scales, lse, weights, cuda_stream);
}

int fa_weights_run_token_scales(fa_weights_plan_t plan, const fa_rows* q, const void* paged_kv,
                                int64_t num_pages, float sm_scale, const float* k_scales,
                                const float* lse, float* weights, void* cuda_stream) {
  return weights_run_scales(plan, kScalePerToken, false, q, paged_kv, num_pages, sm_scale,
                            k_scales, lse, weights, cuda_stream);
}

int fa_weights_run_block_scales(fa_weights_plan_t plan, const fa_rows* q, const void* paged_kv,
                                int64_t num_pages, float sm_scale, const float* k_scales,
                                const float* lse, float* weights, void* cuda_stream) {
  return weights_run_scales(plan, kScalePerBlock, false, q, paged_kv, num_pages, sm_scale,
                            k_scales, lse, weights, cuda_stream);
}

int fa_weights_check(fa_weights_plan_t plan, void* cuda_stream, int* flags) {
  if (!plan || !flags) return FA_ERR_INVALID_ARG;
  int word = 0;
  if (take_word(reinterpret_cast<int*>(plan->ws), &word, static_cast<cudaStream_t>(cuda_stream)) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  *flags = word;
  return word ? FA_ERR_DEVICE_CHECK : FA_OK;
}

int fa_weights_plan_destroy(fa_weights_plan_t plan) {
  delete plan;
  return FA_OK;
}

}  // extern "C"
