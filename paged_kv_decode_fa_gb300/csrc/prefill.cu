// Attention of packed query rows (whole prompts, chunks, single tokens) over the
// paged KV cache: the calls fa_prefill_* (declared in include/fa_decode.h), their
// planner, and the kernels around fa_prefill_kernel (prefill.cuh).
#include "prefill.cuh"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <new>
#include <queue>
#include <vector>

#include "fa_decode.h"
#include "staging.h"
#include "tensor_map.h"

namespace fadecode {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// ------------------------------------------------------------ the plan

// What an item costs beside its tiles, in tiles: its first scores and its
// output; and a piece of a split item, its fp32 state.
constexpr int kItemCost = 2, kPieceCost = 1, kMergeCost = 3;
constexpr int kLeastTiles = 4;  // tiles of a split item's pieces at least

struct Block {  // up to 256 rows of one kv head, the same for every kv head
  int row0, tokens, pos0, entry, tiles;
};

struct PrefillWork {
  std::vector<int32_t> cta_offsets, items, merge;  // merge: see MergeUnit
  int slots = 0;
};

// The blocks of a batch; false for malformed arguments.
bool make_blocks(const int32_t* indptr, const int32_t* last_page_len, const int32_t* qo_indptr,
                 int batch, int group, std::vector<Block>* out) {
  if (indptr[0] != 0 || qo_indptr[0] != 0) return false;
  const int step = 2 * pf::kRows / group;
  for (int i = 0; i < batch; ++i) {
    const int64_t n = (int64_t)qo_indptr[i + 1] - qo_indptr[i];
    const int64_t pages = (int64_t)indptr[i + 1] - indptr[i];
    if (n < 0 || pages < 0) return false;
    if (pages > 0 && (last_page_len[i] < 1 || last_page_len[i] > kPageSize)) return false;
    const int64_t len = pages > 0 ? (pages - 1) * kPageSize + last_page_len[i] : 0;
    if (n > len || len > std::numeric_limits<int32_t>::max() - pf::kTok) return false;
    for (int64_t t = 0; t < n; t += step) {
      const int64_t tokens = std::min<int64_t>(step, n - t), keys = len - n + t + tokens;
      out->push_back(Block{(int)(qo_indptr[i] + t), (int)tokens, (int)(len - n + t), indptr[i],
                           (int)((keys + pf::kTok - 1) / pf::kTok)});
    }
  }
  return true;
}

// Pieces of a block of `tiles` tiles where none has more than `longest`.
int pieces_of(int tiles, int longest) { return (tiles + longest - 1) / longest; }

struct Piece {
  int block, t0, t1, cost;
};

std::vector<Piece> cut(const std::vector<Block>& blocks, int longest) {
  std::vector<Piece> out;
  out.reserve(blocks.size());
  for (size_t b = 0; b < blocks.size(); ++b) {
    const int n = pieces_of(blocks[b].tiles, longest);
    for (int i = 0; i < n; ++i) {
      const int t0 = (int)((int64_t)blocks[b].tiles * i / n);
      const int t1 = (int)((int64_t)blocks[b].tiles * (i + 1) / n);
      out.push_back(Piece{(int)b, t0, t1, t1 - t0 + kItemCost + (n > 1 ? kPieceCost : 0)});
    }
  }
  // the costliest first; blocks of equal cost in order
  std::stable_sort(out.begin(), out.end(),
                   [](const Piece& a, const Piece& b) { return a.cost > b.cost; });
  return out;
}

// Each piece of each kv head to the CTA with the least so far; returns the
// largest CTA's cost.  `owner`, if asked for: [pieces * heads].
int64_t assign(const std::vector<Piece>& pieces, int heads, int ctas, std::vector<int>* owner) {
  using Load = std::pair<int64_t, int>;
  std::vector<Load> heap;
  heap.reserve(ctas);
  for (int c = 0; c < ctas; ++c) heap.emplace_back(0, c);
  const auto after = std::greater<Load>();
  int64_t most = 0;
  for (const Piece& p : pieces)
    for (int h = 0; h < heads; ++h) {
      std::pop_heap(heap.begin(), heap.end(), after);
      Load& l = heap.back();
      l.first += p.cost;
      most = std::max(most, l.first);
      if (owner) owner->push_back(l.second);
      std::push_heap(heap.begin(), heap.end(), after);
    }
  return most;
}

// The work list for at most max_ctas CTAs.  Blocks stay whole where that
// leaves no CTA much more than its share; else they are cut into pieces of a
// share, a half or a third of one, whichever ends first by the costs above.
// (A serving step of few rows over long contexts has fewer blocks than SMs.)
void make_work(const std::vector<Block>& blocks, int heads, int max_ctas, PrefillWork* w) {
  int64_t total = 0;
  int longest = 1;
  for (const Block& b : blocks) {
    total += (int64_t)(b.tiles + kItemCost) * heads;
    longest = std::max(longest, b.tiles);
  }
  const int64_t share = (total + max_ctas - 1) / max_ctas;
  std::vector<Piece> best = cut(blocks, longest);
  int64_t least = assign(best, heads, max_ctas, nullptr);
  int chosen = longest;
  if (least > share + share / 8 + kMergeCost) {
    for (int part = 1; part <= 3; ++part) {
      const int l = (int)std::max<int64_t>(kLeastTiles, (share + part - 1) / part);
      if (l >= longest) continue;
      std::vector<Piece> pieces = cut(blocks, l);
      const int64_t m = assign(pieces, heads, max_ctas, nullptr) + kMergeCost;
      if (m < least) {
        least = m;
        chosen = l;
        best.swap(pieces);
      }
    }
  }
  const int64_t n = (int64_t)best.size() * heads;
  const int ctas = (int)std::min<int64_t>(n, max_ctas);
  std::vector<int> owner;
  owner.reserve(n);
  assign(best, heads, std::max(ctas, 1), &owner);
  // partial slots: a split block's pieces side by side, head by head
  std::vector<int> slot(blocks.size(), -1);
  w->slots = 0;
  for (size_t b = 0; b < blocks.size(); ++b) {
    const int k = pieces_of(blocks[b].tiles, chosen);
    if (k < 2) continue;
    slot[b] = w->slots;
    for (int h = 0; h < heads; ++h) {
      const int32_t unit[8] = {blocks[b].row0, blocks[b].tokens, w->slots, k, h, 0, 0, 0};
      w->merge.insert(w->merge.end(), unit, unit + 8);
      w->slots += k;
    }
  }
  w->cta_offsets.assign(ctas + 1, 0);
  for (int c : owner) ++w->cta_offsets[c + 1];
  for (int c = 0; c < ctas; ++c) w->cta_offsets[c + 1] += w->cta_offsets[c];
  std::vector<int> at(w->cta_offsets.begin(), w->cta_offsets.end());
  w->items.resize((size_t)n * pf::kItemInts);
  size_t i = 0;
  for (const Piece& p : best) {
    const Block& b = blocks[p.block];
    const int k = pieces_of(b.tiles, chosen);
    // the piece's number among its block's
    int index = (int)((int64_t)p.t0 * k / b.tiles);
    while ((int64_t)b.tiles * index / k < p.t0) ++index;
    for (int h = 0; h < heads; ++h, ++i) {
      int32_t* o = w->items.data() + (size_t)at[owner[i]]++ * pf::kItemInts;
      o[0] = b.row0;
      o[1] = b.tokens;
      o[2] = b.pos0;
      o[3] = b.entry;
      o[4] = p.t0;
      o[5] = p.t1;
      o[6] = slot[p.block] < 0 ? -1 : slot[p.block] + h * k + index;
      o[7] = h;
    }
  }
}

// Device-check word, the work list, the table entries to widen, then the partial
// states and, for an E4M3 cache, its scales by table entry and its pages in q's type.
struct PrefillLayout {
  size_t offsets, items, merge, entries, meta, part_o, part_lse, scales, rests, wide, total;
};

// scale_bytes, wide_bytes: of an E4M3 cache's scales by token (K's, and the rests of
// V's), and its pages.
PrefillLayout layout_of(const PrefillWork& w, size_t entries, size_t scale_bytes,
                        size_t wide_bytes, int D) {
  PrefillLayout L;
  L.offsets = kAlign;
  L.items = align_up(L.offsets + 4 * w.cta_offsets.size());
  L.merge = align_up(L.items + 4 * w.items.size());
  L.entries = align_up(L.merge + 4 * w.merge.size());
  L.meta = align_up(L.entries + 4 * entries);
  L.part_o = L.meta;
  L.part_lse = align_up(L.part_o + 4 * (size_t)w.slots * 256 * D);
  L.scales = align_up(L.part_lse + 4 * (size_t)w.slots * 256);
  L.rests = align_up(L.scales + scale_bytes);
  L.wide = align_up(L.rests + scale_bytes);
  L.total = align_up(L.wide + wide_bytes);
  return L;
}

// ------------------------------------------------------------ around the kernel

// One split block of a kv head.
struct MergeUnit {
  int row0, tokens, slot, pieces, head;
};

struct PrefillMergeParams {
  const int32_t* units;
  const float* part_o;
  const float* part_lse;
  void* o;
  float* lse;
  int num_qo_heads;
  int group;
};

// The rows of split blocks from their pieces' states: o = sum_c u_c o_c / sum_c u_c,
// u_c = 2^(lse_c - max), a warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) fa_prefill_merge_kernel(const PrefillMergeParams p) {
  constexpr int V = D / 32;  // dims of a lane
  const int32_t* u = p.units + (size_t)(blockIdx.x / 32) * 8;
  const int r = (blockIdx.x % 32) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const MergeUnit w{u[0], u[1], u[2], u[3], u[4]};
  if (r >= w.tokens * p.group) return;
  const size_t at = (size_t)w.slot * 256 + r;
  float top = -INFINITY;
  for (int c = lane; c < w.pieces; c += 32) top = fmaxf(top, p.part_lse[at + (size_t)c * 256]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float o[V] = {}, d = 0.f;
  for (int c = 0; c < w.pieces; ++c) {
    const float l = p.part_lse[at + (size_t)c * 256];
    if (l == -INFINITY) continue;  // the piece holds nothing this row sees
    const float f = dev::fast_exp2(l - top);
    d += f;
    const float* x = p.part_o + (at + (size_t)c * 256) * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(f, x[i], o[i]);
  }
  const float inv = d > 0.f || d != d ? 1.f / d : 0.f;
  const size_t row =
      (size_t)(w.row0 + r / p.group) * p.num_qo_heads + (size_t)w.head * p.group + r % p.group;
  T* out = static_cast<T*>(p.o) + row * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(out + i) =
        mma::pack2(o[i] * inv, o[i + 1] * inv, std::is_same<T, __nv_bfloat16>::value);
  if (p.lse && lane == 0)
    p.lse[row] = d > 0.f || d != d ? (top + log2f(d)) * dev::kLn2 : -INFINITY;
}

struct WidenParams {
  const uint8_t* kv;
  uint4* out;               // [entries, 2, 16, Hkv, D] bf16
  const int32_t* indices;
  const int32_t* entries;   // table entries to widen
  const float* k_scales;    // kScalePerToken [pages, Hkv, 16], kScalePerBlock [pages, Hkv]
  const float* v_scales;
  float* out_scales;        // the K scales by table entry: [entries, Hkv(, 16)]
  float* out_rests;         // per token: the rests of V's likewise (pf::scale_rest)
  int* err;
  int64_t num_pages;
  int hkv;
};

// One page of an E4M3 cache in bf16: the codes as they are (4 significant bits:
// exact).  Scales per block: V's multiply its elements (exact for powers of two, which
// append writes; otherwise one rounding, as the weights' own); per token the power of
// two in V's, exactly, and the rests are laid out by table entry for the weights.  K's
// are laid out so for the scores, whose precision lse has.  A streaming pass over the cache, read
// once here and as bf16 by every block of rows: bound by HBM, 97 us for the 202 MB of
// 6155 pages of 8 heads of 128 (6.2 TB/s, read and written).
template <int D, int SC>
__global__ void __launch_bounds__(256) fa_prefill_widen_kernel(const WidenParams p) {
  const int entry = p.entries[blockIdx.x];
  const int page = __ldg(p.indices + entry);
  const bool ok = page >= 0 && (int64_t)page < p.num_pages;
  if (!ok && threadIdx.x == 0) atomicOr(p.err, 1);
  const int groups = 2 * kPageSize * p.hkv * (D / 16);  // of 16 codes
  const uint4* src = reinterpret_cast<const uint4*>(p.kv) + (ok ? (int64_t)page * groups : 0);
  uint4* dst = p.out + (int64_t)entry * groups * 2;
  if constexpr (SC != kScaleNone) {
    const int n = p.hkv * (SC == kScalePerToken ? kPageSize : 1);
    for (int i = threadIdx.x; i < n; i += 256) {
      const int64_t from = (int64_t)page * n + i, to = (int64_t)entry * n + i;
      p.out_scales[to] = ok ? __ldg(p.k_scales + from) : 0.f;
      if constexpr (SC == kScalePerToken)
        p.out_rests[to] = ok ? pf::scale_rest(__ldg(p.v_scales + from)) : 1.f;
    }
  }
  for (int i = threadIdx.x; i < groups; i += 256) {
    const uint4 c = ok ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
    float scale = 1.f;
    if constexpr (SC != kScaleNone) {
      const int row = i / (D / 16), head = row % p.hkv, slot = row / p.hkv % kPageSize;
      const int64_t at = (int64_t)page * p.hkv + head;
      if (ok && row >= kPageSize * p.hkv)
        scale = SC == kScalePerToken ? pf::scale_power(__ldg(p.v_scales + at * kPageSize + slot))
                                     : __ldg(p.v_scales + at);
    }
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = dev::e4m3x2_to_float2((uint16_t)(in[j] & 0xffffu));
      const float2 b = dev::e4m3x2_to_float2((uint16_t)(in[j] >> 16));
      out[2 * j] = mma::pack2(a.x * scale, a.y * scale, true);
      out[2 * j + 1] = mma::pack2(b.x * scale, b.y * scale, true);
    }
    dst[2 * i] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[2 * i + 1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

struct PrefillKernel {
  const void* attend[3] = {nullptr, nullptr, nullptr};  // by kScale... (E4M3: bf16 only)
  const void* merge = nullptr;
  int smem = 0;
};

template <typename T, int D>
PrefillKernel kernel_for() {
  PrefillKernel k;
  const auto f = [](auto kernel) { return reinterpret_cast<const void*>(kernel); };
  k.attend[kScaleNone] = f(&fa_prefill_kernel<T, D, kScaleNone>);
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    k.attend[kScalePerToken] = f(&fa_prefill_kernel<T, D, kScalePerToken>);
    k.attend[kScalePerBlock] = f(&fa_prefill_kernel<T, D, kScalePerBlock>);
  }
  k.merge = reinterpret_cast<const void*>(&fa_prefill_merge_kernel<T, D>);
  k.smem = pf::Smem<D>::kBytes;
  return k;
}

PrefillKernel find_prefill_kernel(fa_dtype q, int D) {
  if (q == FA_DTYPE_BF16)
    return D == 128 ? kernel_for<__nv_bfloat16, 128>() : kernel_for<__nv_bfloat16, 64>();
  return D == 128 ? kernel_for<__half, 128>() : kernel_for<__half, 64>();
}

const void* find_widen_kernel(int D, int sc) {
  const auto of = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    return sc == kScalePerToken
               ? reinterpret_cast<const void*>(&fa_prefill_widen_kernel<kD, kScalePerToken>)
           : sc == kScalePerBlock
               ? reinterpret_cast<const void*>(&fa_prefill_widen_kernel<kD, kScalePerBlock>)
               : reinterpret_cast<const void*>(&fa_prefill_widen_kernel<kD, kScaleNone>);
  };
  return D == 128 ? of(std::integral_constant<int, 128>{}) : of(std::integral_constant<int, 64>{});
}

bool prefill_pair_built(fa_dtype q, fa_dtype kv) {
  return (q == FA_DTYPE_BF16 && (kv == FA_DTYPE_BF16 || kv == FA_DTYPE_E4M3)) ||
         (q == FA_DTYPE_F16 && kv == FA_DTYPE_F16);
}

// Shared checks of the plan and of its size; FA_OK or an error.
int check_prefill(const int32_t* indptr, const int32_t* last_page_len, const int32_t* qo_indptr,
                  int batch, int hq, int hkv, int D, int page_size, fa_dtype q, fa_dtype kv) {
  if (!indptr || !qo_indptr || batch < 0 || hq <= 0 || hkv <= 0 || D <= 0 || page_size <= 0 ||
      hq % hkv || (batch > 0 && !last_page_len))
    return FA_ERR_INVALID_ARG;
  const int G = hq / hkv;
  if (page_size != kPageSize || (D != 64 && D != 128) || (G != 1 && G != 2 && G != 4 && G != 8) ||
      !prefill_pair_built(q, kv))
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Entries of the page table that an E4M3 run widens: those of requests with rows.
size_t wide_entries(const int32_t* indptr, const int32_t* qo_indptr, int batch,
                    std::vector<int32_t>* out) {
  size_t n = 0;
  for (int i = 0; i < batch; ++i) {
    if (qo_indptr[i + 1] == qo_indptr[i]) continue;
    n += indptr[i + 1] - indptr[i];
    if (out)
      for (int e = indptr[i]; e < indptr[i + 1]; ++e) out->push_back(e);
  }
  return n;
}

int device_sms(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
    return FA_ERR_CUDA;
  return FA_OK;
}

}  // namespace
}  // namespace fadecode

using namespace fadecode;

struct fa_prefill_plan_s {
  int device = 0;
  int hq = 0, hkv = 0, d = 0;
  fa_dtype q_dtype = FA_DTYPE_BF16, kv_dtype = FA_DTYPE_BF16;
  const int32_t* indices = nullptr;
  uint8_t* ws = nullptr;
  PrefillLayout layout{};
  int64_t rows = 0, table = 0, entries = 0;
  int ctas = 0, merge_units = 0;
  PrefillKernel kernel;
};

namespace {

int prefill_run(fa_prefill_plan_s* plan, int sc, const fa_rows* q, const void* paged_kv,
                int64_t num_pages, float sm_scale, float k_scale, float v_scale,
                const float* head_k, const float* head_v, const float* k_scales,
                const float* v_scales, void* o, float* lse, void* cuda_stream) {
  if (plan->rows == 0) return FA_OK;
  if (!q || !q->data || !paged_kv || !o || num_pages <= 0 || num_pages >= (1 << 30) ||
      reinterpret_cast<uintptr_t>(paged_kv) % 16 || reinterpret_cast<uintptr_t>(o) % 32 ||
      reinterpret_cast<uintptr_t>(lse) % 4 || !q_rows_fit(*q, plan->rows, plan->hq))
    return FA_ERR_INVALID_ARG;
  if (!(k_scale >= 0.f && k_scale < INFINITY && v_scale >= 0.f && v_scale < INFINITY))
    return FA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev != plan->device) return FA_ERR_INVALID_ARG;
  const int D = plan->d, hkv = plan->hkv, G = plan->hq / plan->hkv;
  if (!(sm_scale > 0.f)) sm_scale = 1.0f / std::sqrt((float)D);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const bool wide = plan->kv_dtype == FA_DTYPE_E4M3;
  const void* kv = wide ? plan->ws + plan->layout.wide : paged_kv;
  const int64_t pages = wide ? plan->table : num_pages;

  CUtensorMap maps[2];
  if (!encode_q_rows(&maps[0], plan->q_dtype, *q, plan->rows, plan->hq, D, G) ||
      !encode_pages(&maps[1], plan->q_dtype, kv, pages, hkv, D))
    return FA_ERR_CUDA;
  pf::Params p;
  std::memset(&p, 0, sizeof p);
  p.cta_offsets = reinterpret_cast<const int32_t*>(plan->ws + plan->layout.offsets);
  p.items = reinterpret_cast<const int32_t*>(plan->ws + plan->layout.items);
  p.indices = wide ? nullptr : plan->indices;
  p.q = q->data;
  p.q_token = q->token_stride;
  p.q_head = q->head_stride;
  p.kv = kv;
  p.num_kv_heads = hkv;
  p.k_scales = reinterpret_cast<const float*>(plan->ws + plan->layout.scales);
  p.v_rests = reinterpret_cast<const float*>(plan->ws + plan->layout.rests);
  p.o = o;
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(plan->ws + plan->layout.part_o);
  p.part_lse = reinterpret_cast<float*>(plan->ws + plan->layout.part_lse);
  p.err = reinterpret_cast<int*>(plan->ws);
  p.num_pages = pages;
  p.num_qo_heads = plan->hq;
  p.group = G;
  p.scale = sm_scale * k_scale * 1.4426950408889634f;
  p.v_scale = v_scale;
  p.head_k_scales = head_k;
  p.head_v_scales = head_v;
  if (wide) {
    WidenParams w;
    std::memset(&w, 0, sizeof w);
    w.kv = static_cast<const uint8_t*>(paged_kv);
    w.out = reinterpret_cast<uint4*>(plan->ws + plan->layout.wide);
    w.indices = plan->indices;
    w.entries = reinterpret_cast<const int32_t*>(plan->ws + plan->layout.entries);
    w.k_scales = k_scales;
    w.v_scales = v_scales;
    w.out_scales = reinterpret_cast<float*>(plan->ws + plan->layout.scales);
    w.out_rests = reinterpret_cast<float*>(plan->ws + plan->layout.rests);
    w.err = p.err;
    w.num_pages = num_pages;
    w.hkv = hkv;
    void* args[1] = {&w};
    if (cudaLaunchKernel(find_widen_kernel(D, sc), dim3((unsigned)plan->entries), dim3(256), args,
                         0, st) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  void* args[3] = {&maps[0], &maps[1], &p};
  if (cudaLaunchKernel(plan->kernel.attend[sc], dim3((unsigned)plan->ctas), dim3(pf::kThreads),
                       args, (size_t)plan->kernel.smem, st) != cudaSuccess)
    return FA_ERR_CUDA;
  if (plan->merge_units > 0) {
    PrefillMergeParams m;
    m.units = reinterpret_cast<const int32_t*>(plan->ws + plan->layout.merge);
    m.part_o = p.part_o;
    m.part_lse = p.part_lse;
    m.o = o;
    m.lse = lse;
    m.num_qo_heads = plan->hq;
    m.group = G;
    void* margs[1] = {&m};
    if (cudaLaunchKernel(plan->kernel.merge, dim3((unsigned)plan->merge_units * 32), dim3(256),
                         margs, 0, st) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_prefill_workspace_size(const int32_t* indptr_host, const int32_t* last_page_len_host,
                                 const int32_t* qo_indptr_host, int batch, int num_qo_heads,
                                 int num_kv_heads, int head_dim, fa_dtype q_dtype,
                                 fa_dtype kv_dtype) {
  if (check_prefill(indptr_host, last_page_len_host, qo_indptr_host, batch, num_qo_heads,
                    num_kv_heads, head_dim, kPageSize, q_dtype, kv_dtype) != FA_OK)
    return 0;
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != FA_OK) return 0;
  try {
    std::vector<Block> blocks;
    if (!make_blocks(indptr_host, last_page_len_host, qo_indptr_host, batch,
                     num_qo_heads / num_kv_heads, &blocks))
      return 0;
    PrefillWork w;
    make_work(blocks, num_kv_heads, sms, &w);
    size_t entries = 0, scales = 0, wide = 0;
    if (kv_dtype == FA_DTYPE_E4M3) {
      entries = wide_entries(indptr_host, qo_indptr_host, batch, nullptr);
      scales = (size_t)indptr_host[batch] * kPageSize * num_kv_heads * 4;
      wide = scales * head_dim;  // K and V, two bytes each
    }
    return layout_of(w, entries, scales, wide, head_dim).total;
  } catch (const std::bad_alloc&) {
    return 0;
  }
}

int fa_plan_prefill_host(const int32_t* indptr_host, const int32_t* last_page_len_host,
                         const int32_t* qo_indptr_host, int batch, int group, int num_kv_heads,
                         int max_ctas, int32_t* cta_offsets, int32_t* items, int items_room,
                         int32_t* merge, int merge_room, int* num_ctas, int* num_items,
                         int* num_merge, int* num_slots) {
  if (max_ctas < 1 || !cta_offsets || !items || !merge || !num_ctas || !num_items || !num_merge ||
      !num_slots || group < 1)
    return FA_ERR_INVALID_ARG;
  const int rc = check_prefill(indptr_host, last_page_len_host, qo_indptr_host, batch,
                               group * num_kv_heads, num_kv_heads, 128, kPageSize, FA_DTYPE_BF16,
                               FA_DTYPE_BF16);
  if (rc != FA_OK) return rc;
  try {
    std::vector<Block> blocks;
    if (!make_blocks(indptr_host, last_page_len_host, qo_indptr_host, batch, group, &blocks))
      return FA_ERR_INVALID_ARG;
    PrefillWork w;
    make_work(blocks, num_kv_heads, max_ctas, &w);
    *num_ctas = (int)w.cta_offsets.size() - 1;
    *num_items = (int)(w.items.size() / pf::kItemInts);
    *num_merge = (int)(w.merge.size() / 8);
    *num_slots = w.slots;
    if (*num_items > items_room || *num_merge > merge_room) return FA_ERR_WORKSPACE_TOO_SMALL;
    std::memcpy(cta_offsets, w.cta_offsets.data(), 4 * w.cta_offsets.size());
    if (!w.items.empty()) std::memcpy(items, w.items.data(), 4 * w.items.size());
    if (!w.merge.empty()) std::memcpy(merge, w.merge.data(), 4 * w.merge.size());
  } catch (const std::bad_alloc&) {
    return FA_ERR_INVALID_ARG;
  }
  return FA_OK;
}

int fa_prefill_plan(const int32_t* indptr_host, const int32_t* indices_dev,
                    const int32_t* last_page_len_host, const int32_t* qo_indptr_host, int batch,
                    int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                    fa_dtype q_dtype, fa_dtype kv_dtype, void* workspace_dev,
                    size_t workspace_bytes, void* cuda_stream, fa_prefill_plan_t* out_plan) {
  if (!out_plan) return FA_ERR_INVALID_ARG;
  *out_plan = nullptr;
  const int rc = check_prefill(indptr_host, last_page_len_host, qo_indptr_host, batch,
                               num_qo_heads, num_kv_heads, head_dim, page_size, q_dtype, kv_dtype);
  if (rc != FA_OK) return rc;
  if (!workspace_dev || reinterpret_cast<uintptr_t>(workspace_dev) % kAlign ||
      (indptr_host[batch] > 0 && !indices_dev))
    return FA_ERR_INVALID_ARG;
  try {
    std::vector<Block> blocks;
    if (!make_blocks(indptr_host, last_page_len_host, qo_indptr_host, batch,
                     num_qo_heads / num_kv_heads, &blocks))
      return FA_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (device_sms(&dev, &sms) != FA_OK) return FA_ERR_CUDA;
    PrefillWork w;
    make_work(blocks, num_kv_heads, sms, &w);
    std::vector<int32_t> entries;
    size_t scales = 0, wide = 0;
    if (kv_dtype == FA_DTYPE_E4M3) {
      wide_entries(indptr_host, qo_indptr_host, batch, &entries);
      scales = (size_t)indptr_host[batch] * kPageSize * num_kv_heads * 4;
      wide = scales * head_dim;  // K and V, two bytes each
    }
    const PrefillLayout L = layout_of(w, entries.size(), scales, wide, head_dim);
    if (L.total > workspace_bytes) return FA_ERR_WORKSPACE_TOO_SMALL;
    std::vector<uint8_t> meta(L.meta, 0);
    auto put = [&](size_t at, const std::vector<int32_t>& v) {
      if (!v.empty()) std::memcpy(meta.data() + at, v.data(), 4 * v.size());
    };
    put(L.offsets, w.cta_offsets);
    put(L.items, w.items);
    put(L.merge, w.merge);
    put(L.entries, entries);
    fa_prefill_plan_s* plan = new fa_prefill_plan_s();
    plan->device = dev;
    plan->hq = num_qo_heads;
    plan->hkv = num_kv_heads;
    plan->d = head_dim;
    plan->q_dtype = q_dtype;
    plan->kv_dtype = kv_dtype;
    plan->indices = indices_dev;
    plan->ws = static_cast<uint8_t*>(workspace_dev);
    plan->layout = L;
    plan->rows = qo_indptr_host[batch];
    plan->table = indptr_host[batch];
    plan->entries = (int64_t)entries.size();
    plan->ctas = (int)w.cta_offsets.size() - 1;
    plan->merge_units = (int)(w.merge.size() / 8);
    plan->kernel = find_prefill_kernel(q_dtype, head_dim);
    // the kernels' warpgroups share out the registers they are launched with
    cudaError_t e = cudaSuccess;
    for (int sc = 0; sc < (kv_dtype == FA_DTYPE_E4M3 ? 3 : 1); ++sc) {
      const void* f = plan->kernel.attend[sc];
      cudaFuncAttributes attr;
      if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, f);
      if (e == cudaSuccess && attr.numRegs < pf::kLaunchRegs) e = cudaErrorInvalidDeviceFunction;
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 plan->kernel.smem);
    }
    if (e != cudaSuccess || upload_async(plan->ws, meta.data(), meta.size(),
                                         static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) {
      delete plan;
      return FA_ERR_CUDA;
    }
    *out_plan = plan;
  } catch (const std::bad_alloc&) {
    return FA_ERR_INVALID_ARG;
  }
  return FA_OK;
}

int fa_prefill_run(fa_prefill_plan_t plan, const fa_rows* q, const void* paged_kv,
                   int64_t num_pages, float sm_scale, float k_scale, float v_scale, void* o,
                   float* lse, void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->kv_dtype != FA_DTYPE_E4M3 && (k_scale != 1.f || v_scale != 1.f))
    return FA_ERR_INVALID_ARG;
  return prefill_run(plan, kScaleNone, q, paged_kv, num_pages, sm_scale, k_scale, v_scale,
                     nullptr, nullptr, nullptr, nullptr, o, lse, cuda_stream);
}

int fa_prefill_run_head_scales(fa_prefill_plan_t plan, const fa_rows* q, const void* paged_kv,
                               int64_t num_pages, float sm_scale, const float* k_head_scales,
                               const float* v_head_scales, void* o, float* lse,
                               void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->kv_dtype != FA_DTYPE_E4M3) return FA_ERR_UNSUPPORTED;
  if (!k_head_scales || !v_head_scales || reinterpret_cast<uintptr_t>(k_head_scales) % 4 ||
      reinterpret_cast<uintptr_t>(v_head_scales) % 4)
    return FA_ERR_INVALID_ARG;
  return prefill_run(plan, kScaleNone, q, paged_kv, num_pages, sm_scale, 1.f, 1.f, k_head_scales,
                     v_head_scales, nullptr, nullptr, o, lse, cuda_stream);
}

static int prefill_run_scales(fa_prefill_plan_t plan, int sc, const fa_rows* q,
                              const void* paged_kv, int64_t num_pages, float sm_scale,
                              const float* k_scales, const float* v_scales, void* o, float* lse,
                              void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->kv_dtype != FA_DTYPE_E4M3) return FA_ERR_UNSUPPORTED;
  if (!k_scales || !v_scales || reinterpret_cast<uintptr_t>(k_scales) % 4 ||
      reinterpret_cast<uintptr_t>(v_scales) % 4)
    return FA_ERR_INVALID_ARG;
  return prefill_run(plan, sc, q, paged_kv, num_pages, sm_scale, 1.f, 1.f, nullptr, nullptr,
                     k_scales, v_scales, o, lse, cuda_stream);
}

int fa_prefill_run_token_scales(fa_prefill_plan_t plan, const fa_rows* q, const void* paged_kv,
                                int64_t num_pages, float sm_scale, const float* k_scales,
                                const float* v_scales, void* o, float* lse, void* cuda_stream) {
  return prefill_run_scales(plan, kScalePerToken, q, paged_kv, num_pages, sm_scale, k_scales,
                            v_scales, o, lse, cuda_stream);
}

int fa_prefill_run_block_scales(fa_prefill_plan_t plan, const fa_rows* q, const void* paged_kv,
                                int64_t num_pages, float sm_scale, const float* k_scales,
                                const float* v_scales, void* o, float* lse, void* cuda_stream) {
  return prefill_run_scales(plan, kScalePerBlock, q, paged_kv, num_pages, sm_scale, k_scales,
                            v_scales, o, lse, cuda_stream);
}

int fa_prefill_check(fa_prefill_plan_t plan, void* cuda_stream, int* flags) {
  if (!plan || !flags) return FA_ERR_INVALID_ARG;
  int word = 0;
  if (take_word(reinterpret_cast<int*>(plan->ws), &word, static_cast<cudaStream_t>(cuda_stream)) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  *flags = word;
  return word ? FA_ERR_DEVICE_CHECK : FA_OK;
}

int fa_prefill_plan_destroy(fa_prefill_plan_t plan) {
  delete plan;
  return FA_OK;
}

}  // extern "C"
