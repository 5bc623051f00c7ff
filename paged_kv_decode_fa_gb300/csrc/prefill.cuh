// Causal attention of packed query rows over the paged KV cache, on the
// fifth-generation tensor cores (tcgen05).
//
// The mathematics.  Row r of a request (its last n tokens are the query rows) at
// position p = len - n + r sees the keys t <= p:
//     o_r = sum_t w_t v_t / sum_t w_t,   w_t = 2^(c q_r . k_t - m),
// c = sm_scale log2 e, with a running reference m: the largest score so far, moved
// only when a tile's maximum passes it by more than 2^8 (an exact rescale of o and
// of the sum), so that weights stay within 2^8 and the division at the end
// removes m.  (In f16 the reference stands 2^7 below that score: weights within 2^15.)
// lse = (m + log2 sum) ln 2.
//
// Work.  An item is one kv head, up to 256 rows of one request and a range of
// its 128-token tiles.  Rows are (token, query head of the group), a token's heads
// together, so that a K/V tile serves the whole group and a tile of 128 rows
// spans 128 / group tokens: two blocks A and B of 128 rows share every tile, and
// while one block's softmax runs the tensor cores work for the other.  The grid
// is persistent, one CTA per SM, with the plan's list of items for each CTA:
//  - warp 9 loads K and V tiles into one ring, K(0) V(0) K(1) V(1) ..., by tensor
//    copies of 16 tokens x 64 dims (one half of a page's rows of the head, 128-byte
//    swizzled); its lanes issue a tile's copies side by side.  Pages behind the
//    item's last visible token come from an out-of-range index: zeros.
//  - warp 11 loads the blocks' Q (rows of a token's group adjacent in the tensor,
//    so a block is one box of tokens x heads x 64 dims).
//  - warp 8, one lane, issues the MMAs: S = Q K^T (M 128, N 128) into the block's
//    score columns of TMEM, O += P V with P from TMEM and V MN-major from its slot.
//    Order: S_A(0) S_B(0), then per tile P V_A(j) S_A(j+1) P V_B(j) S_B(j+1), which
//    holds the blocks half a period apart.  MMAs complete in order, so a block's
//    scores of tile j+1 being there also means that its O holds the tiles up to j.
//  - warps 0-3 and 4-7, the softmax of A and B: a thread per row = TMEM lane.  It
//    reads its 128 scores, writes its weights as packed pairs over the first 64 of
//    the score columns, in two halves, each handed to the MMAs as it is there;
//    rescales its row of O when its reference moves; and at the item's end writes
//    the row: o and lse, or an fp32 partial state where the plan split the item's keys
//    (folded by fa_prefill_merge_kernel).
//  - warp 10 clears the V rows behind an item's last visible token.
// Items follow each other without a barrier across the CTA: the loads and the first
// scores of an item run under the softmax and the output of the one before.
//
// Slots behind the item's last visible token may hold anything: their scores are
// replaced (select, not add), and their V rows are cleared in shared memory before
// the tile's P V (0 * NaN would be NaN).  For tokens that only some of the rows see
// there is fix_row.
//
// Roundings.  Scores, sums, O and partial states are fp32; the weights are rounded to
// q's 16 bits, the operand type that P V takes, while their sum takes them unrounded
// (lse has fp32's precision).  Half a step a weight, independent: over 9000 keys the
// output is 2.9e-4 off in f16 (rms; 2.1e-4 by its own rounding alone), 2.3e-3 in bf16
// (1.7e-3).  Weights in two terms would halve the rate of P V.  f16 has no weights
// below its smallest subnormal, 2^-24: next to a reference 2^7 below the largest score
// a weight is held to 2^-32 of the largest, and one below that is lost to the output,
// however large its v - 2^-32 sum |v| in all (2^-25 with the reference at the score).
//
// What bounds it.  Long prompts: the tensor cores under the power limit.  8192 rows on a
// context of 24576 (32 / 8 heads, head_dim 128, bf16): 2.44-2.62 ms = 1.47-1.58
// PFLOP/s, 0.84-0.90 of what cuBLAS holds for seconds (0.78 of its burst).  A
// tile of both blocks takes 2100-2600 cycles: 2048 of MMAs at head_dim 128 (1024 at
// 64, where the two softmaxes, 1250 cycles each and half overlapped, set it).  Whole
// prompts of 2048-6144 tokens 1.06-1.24 ms (1.30-1.52): an item's output and the next
// one's first scores cost about two tiles, of 17 on average.
// On the way (8192 rows on 24576): 4.52 ms with the MMAs issued by a whole warp and
// 514 bytes of spills in the softmax; 2.65 with the registers split by warpgroup; 2.58
// with four MMAs an election; 2.53 with one lane and the waits behind issued MMAs.
// Slower and not kept: a warp for each block's MMAs (the blocks fall in step, 3.11 ms);
// the first half's weights against the old reference while the maximum is found (3 %);
// the next item's first scores before the other block's last tile (1 %, the issuing
// lane waits for its Q); K and V loaded by a warp each, boxes of 4 KB, half the
// bytes (no change: the copies are not what it waits for).
//
// Every wait is bounded: it runs out where for 2 s no softmax warp has got on (each
// counts its tiles, and the tokens of a row that it computes again, in shared memory),
// sets bit 1 of the device-check word and the CTA drains.  (A bound on the time alone
// would also end waits that are merely long: 32 rows computed again over 150000 tokens
// each, or a block or the ragged-end warp without work through millions of tokens of
// other items.)
#pragma once

#include <cuda.h>

#include <cstdint>
#include <type_traits>

#include "decode_mma.cuh"
#include "tcgen05.cuh"

namespace fadecode {
namespace pf {

constexpr int kRows = 128;                       // rows of a block
constexpr int kTok = 128;                        // tokens of a tile
constexpr int kPages = kTok / kPageSize;         // 8
constexpr int kThreads = 384;
// Registers a thread: as launched, and as the warpgroups split them (the softmax's
// two take what the third, which loads and issues, gives back).
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 200, kIssueRegs = 104;
static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs <= kThreads * kLaunchRegs,
              "a larger share would be waited for without end");
constexpr uint32_t kTmemCols = 512;
// Log2 units: how far a maximum may pass the reference's score before that moves, and
// how far the reference stands below its score (f16: 2^(8 + 7) and its rounding are in
// range, and the smallest weights are as far from the subnormals' end as they can be).
constexpr float kRescaleAbove = 8.f;
template <typename T>
constexpr float kBelowScore = std::is_same<T, __half>::value ? 7.f : 0.f;
constexpr int kItemInts = 8;

struct Params {
  const int32_t* cta_offsets;  // [CTAs + 1]
  const int32_t* items;        // [n * 8], see Item
  const int32_t* indices;      // page ids, or nullptr: entry i of the table is page i
  const void* q;               // [rows, Hq, D], by strides in elements
  int64_t q_token, q_head;
  const void* kv;
  const float* k_scales;       // SC: times scores; [table entries, Hkv, 16] by token or
                               // [table entries, Hkv] by block
  const float* v_rests;        // SC per token: V's rests, times weights, [entries, Hkv, 16]
  int num_kv_heads;
  void* o;                     // [rows, Hq, D]
  float* lse;                  // [rows, Hq] or nullptr
  float* part_o;               // [slots][256][D] normalised
  float* part_lse;             // [slots][256] log2 units
  int* err;
  int64_t num_pages;
  int num_qo_heads;
  int group;
  float scale;    // sm_scale * k_scale * log2(e) (> 0)
  float v_scale;  // times o
  const float* head_k_scales;  // [Hkv] times scale, or nullptr
  const float* head_v_scales;  // [Hkv] times v_scale, or nullptr
};

// One item of a CTA's list.
struct Item {
  int row0;    // first query token (row of q)
  int tokens;  // query tokens, 256 / group at most
  int pos0;    // position of the first
  int entry;   // the request's first entry of the page table
  int t0, t1;  // its tiles
  int slot;    // partial state, or -1: the whole range of keys is here
  int head;    // kv head
  __device__ __forceinline__ static Item load(const int32_t* items, int i) {
    const int4 a = __ldg(reinterpret_cast<const int4*>(items) + 2 * i);
    const int4 b = __ldg(reinterpret_cast<const int4*>(items) + 2 * i + 1);
    return Item{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
  // keys the block's last row sees, and the item's tiles that hold any
  __device__ __forceinline__ int keys(int block, int block_tokens) const {
    return pos0 + min(tokens, (block + 1) * block_tokens);
  }
  __device__ __forceinline__ int tiles(int block, int block_tokens) const {
    if (block * block_tokens >= tokens) return 0;
    return max(0, min(t1, (keys(block, block_tokens) + kTok - 1) / kTok) - t0);
  }
  // the last of its `all` tiles ends inside a page
  __device__ __forceinline__ bool ragged(int keys, int all) const {
    return keys < (t0 + all) * kTok && keys % kPageSize;
  }
};

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = kTok * 128;              // [128 tokens][64 dims]
  static constexpr int kSlotBytes = kHalves * kHalf;    // one tile of K or V
  static constexpr int kSlots = D == 128 ? 5 : 10;
  static constexpr int kQBytes = kHalves * kRows * 128;  // one block's Q
  static constexpr int kOffRing = 2 * kQBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
  // kv_full[n], kv_empty[n]; q_full, q_empty, s_full [2], p_full [2][2], o_full, o_empty [2],
  // v_there, v_clean; sc_full, sc_empty [kScaleSlots]
  static constexpr int kScaleSlots = D == 128 ? 2 : 3;
  static constexpr int kScaleBytes = kTok * 8;           // of a slot: K's scales, V's rests
  static constexpr int kNumBars = 2 * kSlots + 16 + 2 * kScaleSlots;
  static constexpr int kOffTmem = kOffBar + 8 * kNumBars;
  static constexpr int kOffProgress = kOffTmem + 4;      // what the softmax warps count
  static constexpr int kOffScales = kOffTmem + 16;       // SC per token: of a tile's tokens
  // Room to start at a multiple of 1024 bytes.  (The array is declared so, and does; the
  // kernel checks that this room is enough.)
  static constexpr int kPad = 512;
  static constexpr int kBytes = kPad + kOffScales + kScaleSlots * kScaleBytes;
  static_assert(kOffScales % 16 == 0, "bulk copies");
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
};

// What the CTA's softmax warps have counted in all (kOffProgress), and one more.
__device__ __forceinline__ uint32_t progress_of(uint32_t count) {
  uint32_t n;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(n) : "r"(count) : "memory");
  return n;
}
__device__ __forceinline__ void count_on(uint32_t count) {
  asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(count) : "memory");
}

// dev::mbar_wait with a bound on standstill instead of time: it runs out where
// kWaitTimeoutNs pass and no softmax warp has counted on.
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, bool& aborted, int* err,
                                          uint32_t count) {
  if (aborted || dev::mbar_try_wait(bar, parity)) return;
  unsigned long long t0 = dev::global_timer_ns();
  uint32_t before = progress_of(count);
  while (!dev::mbar_try_wait(bar, parity)) {
    if (dev::global_timer_ns() - t0 <= dev::kWaitTimeoutNs) continue;
    const uint32_t now = progress_of(count);
    if (now == before) {
      aborted = true;
      atomicOr(err, 2);
      return;
    }
    before = now;
    t0 = dev::global_timer_ns();
  }
}

// A scale of V per token in two factors: a power of two, which V's elements take exactly,
// and the rest in [1, 2), which the weights take before they are rounded.  (The whole of
// it multiplied into the elements rounds each of them, as much as the weights' own
// rounding: 2.6e-3 of the output for 2.1e-3.)  What is no normal number is the first.
__device__ __forceinline__ float scale_power(float s) {
  const uint32_t b = __float_as_uint(s), e = b & 0x7f800000u;
  return e == 0 || e == 0x7f800000u ? s : __uint_as_float(b & 0xff800000u);
}
__device__ __forceinline__ float scale_rest(float s) {
  const uint32_t b = __float_as_uint(s), e = b & 0x7f800000u;
  return e == 0 || e == 0x7f800000u ? 1.f : __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
}

// a * b of two pairs
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace pf

// 32 bytes in one store, a whole sector (32-byte aligned).
__device__ __forceinline__ void store32(void* p, const uint32_t (&x)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// A value of V that is not finite, at a token that some rows of a block see and
// others do not, reaches those others through a weight of 0 (0 * inf is NaN).  So a
// row whose output is not finite is computed again by its warp, over the tokens it
// sees alone (the first `seen` from the item's first tile on, whose entry is
// `entry`), from its reference m and inv = 1 / sum - if such a value stands among
// the others of the block's tiles, up to token `end`.  to: its D outputs, T or fp32.
template <typename T, int D, int SC>
__device__ __forceinline__ void fix_row(const pf::Params& p, int entry, int seen, int end, int head,
                                     int64_t q_row, float scale, float m, float inv, char* to,
                                     bool part, uint32_t count) {
  constexpr int V = D / 32;  // dims of a lane
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  const int lane = threadIdx.x & 31;
  const int64_t token = (int64_t)p.num_kv_heads * D;
  auto row_of = [&](int t) -> const T* {  // K of token t, its V a half page on
    const int e = entry + t / kPageSize, id = p.indices ? __ldg(p.indices + e) : e;
    if (id < 0 || (int64_t)id >= p.num_pages) return nullptr;
    return static_cast<const T*>(p.kv) +
           ((int64_t)id * 2 * kPageSize + t % kPageSize) * token + (int64_t)head * D + lane * V;
  };
  auto read = [&](const T* x, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = dev::to_float(x[i]);
  };
  float x[V];
  bool hidden = false;
#pragma unroll 1
  for (int t = seen; t < end; ++t) {
    const T* k = row_of(t);
    if (k == nullptr) continue;
    read(k + kPageSize * token, x);
#pragma unroll
    for (int i = 0; i < V; ++i) hidden |= !(fabsf(x[i]) < INFINITY);
  }
  if (!__any_sync(0xffffffffu, hidden)) return;
  float q[V], o[V] = {};
  read(static_cast<const T*>(p.q) + q_row + lane * V, q);
#pragma unroll 1
  for (int t = 0; t < seen; ++t) {
    if (t % 64 == 0 && lane == 0) pf::count_on(count);  // others wait for this warp
    const T* k = row_of(t);
    float s = 0.f, v[V] = {};
    if (k != nullptr) {
      read(k, x);
      read(k + kPageSize * token, v);
#pragma unroll
      for (int i = 0; i < V; ++i) s = fmaf(q[i], x[i], s);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if constexpr (SC != kScaleNone) {
      const int64_t at = (int64_t)(entry + t / kPageSize) * p.num_kv_heads + head;
      s *= __ldg(p.k_scales + (SC == kScalePerToken ? at * kPageSize + t % kPageSize : at));
    }
    float w = dev::fast_exp2(fmaf(s, scale, -m));
    if constexpr (SC == kScalePerToken)
      w *= __ldg(p.v_rests + ((int64_t)(entry + t / kPageSize) * p.num_kv_heads + head) *
                                 kPageSize + t % kPageSize);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(w, v[i], o[i]);
  }
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if (part)
      *reinterpret_cast<float2*>(to + (lane * V + i) * 4) = make_float2(o[i] * inv, o[i + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(to + (lane * V + i) * 2) =
          mma::pack2(o[i] * inv, o[i + 1] * inv, kBf16);
  }
}

// SC: K's elements are their scales short (an E4M3 cache's, kScalePerToken or
// kScalePerBlock): the scales multiply the scores, whose precision lse has.  Per token
// they come through a ring of their own, with the rests of V's (scale_rest), which
// multiply the weights; per block, a group of 16 columns, they join the factors of its
// maximum and exponents, read a tile ahead.  (16 requests of 500 rows behind 1024-8192,
// 64 / 8 heads: 1370 us per token, 1113 per block, 1082 per tensor.  K's scales multiplied
// into K's elements, 1070, cost lse 2^-9 of the logits by their rounding to bf16; V's per
// token whole in V's elements, 1239, a quarter more of o's error.  The per-token form's
// softmax is longer by the two factors' loads and products: issue slots are half full
// under it, shared memory a third; loading the factors earlier changed nothing.)
template <typename T, int D, int SC>
__global__ void __launch_bounds__(pf::kThreads, 1)
    fa_prefill_kernel(const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap kv_map,
                      const __grid_constant__ pf::Params p) {
  using namespace pf;
  using namespace tc;
  using S = Smem<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kIdescQK = instr_desc(kBf16, kRows, kTok, 0);
  constexpr uint32_t kIdescPV = instr_desc(kBf16, kRows, D, 1);
  constexpr int kSlots = S::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u;
  if (pad > S::kPad) {
    atomicOr(p.err, 2);
    return;
  }
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = dev::smem_addr(smem), count = sbase + S::kOffProgress;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + kSlots;
  uint64_t* q_full = bars + 2 * kSlots;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_full + 4;
  uint64_t* p_full = q_full + 6;
  uint64_t* o_full = q_full + 10;  // (p_full: [block][half])
  uint64_t* o_empty = q_full + 12;
  uint64_t* v_there = q_full + 14;
  uint64_t* v_clean = q_full + 15;
  uint64_t* sc_full = q_full + 16;
  uint64_t* sc_empty = sc_full + S::kScaleSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffTmem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = p.cta_offsets[blockIdx.x], last = p.cta_offsets[blockIdx.x + 1];
  const int block_tokens = kRows / p.group;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      dev::mbar_init(dev::smem_addr(&kv_full[s]), 1);
      dev::mbar_init(dev::smem_addr(&kv_empty[s]), 1);
    }
    for (int X = 0; X < 2; ++X) {
      dev::mbar_init(dev::smem_addr(&q_full[X]), 1);
      dev::mbar_init(dev::smem_addr(&q_empty[X]), 1);
      dev::mbar_init(dev::smem_addr(&s_full[X]), 1);
      dev::mbar_init(dev::smem_addr(&p_full[2 * X]), 4);
      dev::mbar_init(dev::smem_addr(&p_full[2 * X + 1]), 4);
      dev::mbar_init(dev::smem_addr(&o_full[X]), 1);
      dev::mbar_init(dev::smem_addr(&o_empty[X]), 4);
    }
    dev::mbar_init(dev::smem_addr(v_there), 1);
    dev::mbar_init(dev::smem_addr(v_clean), 1);
    for (int i = 0; i < S::kScaleSlots; ++i) {
      dev::mbar_init(dev::smem_addr(&sc_full[i]), 1);
      dev::mbar_init(dev::smem_addr(&sc_empty[i]), 8);
    }
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(count), "r"(0) : "memory");
    dev::fence_barrier_init();
  }
  if constexpr (SC == kScalePerToken) {
    // what stands behind a tile's last page meets weights of 0, so it has to be finite: 0
    // at first, then what a tile before left there
    for (int i = threadIdx.x; i < S::kScaleSlots * S::kScaleBytes / 4; i += kThreads)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sbase + S::kOffScales + 4 * i), "r"(0)
                   : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     dev::smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;  // S of block X at X * 128, O at 256 + X * 128
  bool aborted = false;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 9) {
      // ------------------------------------------------------------ K and V loads
      if (lane == 0) dev::prefetch_tensormap(&kv_map);
      const int oob = (int)(2 * p.num_pages);  // beyond the last page: zeros
      int n = 0;                               // slots filled
      for (int it = first; it < last; ++it) {
        const Item w = Item::load(p.items, it);
        const int nblk = w.tokens > block_tokens ? 2 : 1;
        const int keys = w.keys(nblk - 1, block_tokens), tiles = w.tiles(nblk - 1, block_tokens);
        const int pages = (min(keys, w.t1 * kTok) + kPageSize - 1) / kPageSize;
        int ids = 0;
        for (int j = 0; j < tiles; ++j) {
          const int page0 = (w.t0 + j) * kPages;
          if (j % (32 / kPages) == 0) {  // the page ids of four tiles
            const int at = page0 + lane;
            ids = oob;
            if (at < pages) {
              const int id = p.indices ? __ldg(p.indices + w.entry + at) : w.entry + at;
              if (id < 0 || (int64_t)id >= p.num_pages) {
                atomicOr(p.err, 1);
              } else {
                ids = 2 * id;
              }
            }
          }
          // lane l: half l % kHalves of the tile's page l / kHalves
          const int id = __shfl_sync(0xffffffffu, ids,
                                     (j * kPages) % 32 + (lane / S::kHalves) % kPages);
          const uint32_t at = (uint32_t)(lane % S::kHalves) * S::kHalf +
                              (uint32_t)(lane / S::kHalves) * (kPageSize * 128);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int s = n % kSlots;
            const uint32_t full = dev::smem_addr(&kv_full[s]);
            pf::mbar_wait(dev::smem_addr(&kv_empty[s]), (uint32_t)(((n / kSlots) & 1) ^ 1),
                          aborted, p.err, count);
            if (lane == 0) dev::mbar_arrive_expect_tx(full, S::kSlotBytes);
            __syncwarp();
            if (lane < kPages * S::kHalves)
              tma_load_4d_plain(sbase + S::kOffRing + s * S::kSlotBytes + at, &kv_map,
                                (lane % S::kHalves) * 64, w.head, 0, id < oob ? id + kv : oob,
                                full);
          }
        }
        aborted = __any_sync(0xffffffffu, aborted);
      }
      // no copy may still be landing when the CTA exits
      if (lane == 0)
        for (int i = n > kSlots ? n - kSlots : 0; i < n; ++i)
          if (!dev::mbar_wait_bounded(dev::smem_addr(&kv_full[i % kSlots]),
                                      (uint32_t)((i / kSlots) & 1)))
            atomicOr(p.err, 2);
    } else if (warp == 11) {
      // ------------------------------------------------------------ Q loads
      if (lane == 0) {
        dev::prefetch_tensormap(&q_map);
        int n[2] = {0, 0};
        for (int it = first; it < last; ++it) {
          const Item w = Item::load(p.items, it);
          for (int X = 0; X < 2; ++X) {
            if (w.tiles(X, block_tokens) == 0) continue;
            const uint32_t full = dev::smem_addr(&q_full[X]);
            pf::mbar_wait(dev::smem_addr(&q_empty[X]), (uint32_t)((n[X] & 1) ^ 1), aborted, p.err,
                          count);
            dev::mbar_arrive_expect_tx(full, S::kQBytes);
            for (int h = 0; h < S::kHalves; ++h)
              tma_load_3d(sbase + X * S::kQBytes + h * (kRows * 128), &q_map, h * 64,
                          w.head * p.group, w.row0 + X * block_tokens, full);
            ++n[X];
          }
        }
        for (int X = 0; X < 2; ++X)
          if (n[X] > 0 &&
              !dev::mbar_wait_bounded(dev::smem_addr(&q_full[X]), (uint32_t)((n[X] - 1) & 1)))
            atomicOr(p.err, 2);
      }
    } else if (warp == 10) {
      // ------------------------------------------------------------ ragged ends
      // V rows of the item's last page behind its last visible token are cleared
      // once the MMA lane has seen the tile arrive (a wait of this warp's own on the
      // ring could not tell a fill from the one two before)
      int n = 0;       // ring slots up to the item's end
      int ragged = 0;  // such items so far
      int sn = 0;      // SC: tiles so far
      for (int it = first; it < last; ++it) {
        const Item w = Item::load(p.items, it);
        const int last_block = w.tokens > block_tokens ? 1 : 0;
        const int keys = w.keys(last_block, block_tokens), all = w.tiles(last_block, block_tokens);
        n += 2 * all;
        if constexpr (SC == kScalePerToken) {  // the item's scales, a tile a slot
          const int pages = (min(keys, w.t1 * kTok) + kPageSize - 1) / kPageSize;
          for (int j = 0; j < all; ++j, ++sn) {
            const int slot = sn % S::kScaleSlots, page = (w.t0 + j) * kPages + lane;
            const uint32_t full = dev::smem_addr(&sc_full[slot]);
            pf::mbar_wait(dev::smem_addr(&sc_empty[slot]),
                          (uint32_t)(((sn / S::kScaleSlots) & 1) ^ 1), aborted, p.err, count);
            const int there = min(kPages, pages - (w.t0 + j) * kPages);
            if (lane == 0) dev::mbar_arrive_expect_tx(full, there * kPageSize * 8);
            __syncwarp();
            if (lane < there) {
              const int64_t at =
                  ((int64_t)(w.entry + page) * p.num_kv_heads + w.head) * kPageSize;
              const uint32_t to =
                  sbase + S::kOffScales + slot * S::kScaleBytes + lane * (kPageSize * 4);
              dev::bulk_load(to, p.k_scales + at, kPageSize * 4, full);
              dev::bulk_load(to + kTok * 4, p.v_rests + at, kPageSize * 4, full);
            }
            __syncwarp();
          }
        }
        if (!w.ragged(keys, all)) continue;
        const int tail = keys % kTok, rows = kPageSize - tail % kPageSize;
        const uint32_t v_addr = sbase + S::kOffRing + (n - 1) % kSlots * S::kSlotBytes;
        pf::mbar_wait(dev::smem_addr(v_there), (uint32_t)(ragged++ & 1), aborted, p.err, count);
        for (int e = lane; e < rows * 8 * S::kHalves; e += 32) {
          const int r = tail + e / (8 * S::kHalves), c = e % (8 * S::kHalves);
          const uint32_t a = v_addr + (c / 8) * S::kHalf + r * 128 + (c % 8) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_addr(v_clean));
      }
    } else if (elect_one()) {
      // ------------------------------------------------------------ MMAs
      // One lane alone.  Between a block's last MMA and the other's first stands one
      // wait, for the weights; the waits for K and V come behind issued MMAs.
      int n = 0;                                 // ring slots consumed by earlier items
      int cleared = 0;                           // ragged items so far
      int item_n[2] = {0, 0}, tile_n[2] = {0, 0};  // items and tiles so far, per block
      const uint64_t q_desc[2] = {smem_desc(sbase, 16, 1024),
                                  smem_desc(sbase + S::kQBytes, 16, 1024)};
      Item next = Item::load(p.items, first);
      for (int it = first; it < last; ++it) {
        const Item w = next;
        next = Item::load(p.items, min(it + 1, last - 1));
        const int tiles[2] = {w.tiles(0, block_tokens), w.tiles(1, block_tokens)};
        const int last_block = w.tokens > block_tokens ? 1 : 0;  // sees the most tiles
        const int keys = w.keys(last_block, block_tokens), all = tiles[last_block];
        const bool ragged = w.ragged(keys, all);
        int slot = n % kSlots, phase = (n / kSlots) & 1;  // of K(j), then V(j), ...
        auto full = [&](int s, int ph) {
          pf::mbar_wait(dev::smem_addr(&kv_full[s]), (uint32_t)ph, aborted, p.err, count);
        };
        auto qk = [&](int X, int j, int s) {
          const uint64_t k_desc = smem_desc(sbase + S::kOffRing + s * S::kSlotBytes, 16, 1024);
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
            umma4(tmem + X * 128, q_desc[X] + h * (kRows * 128 / 16),
                  k_desc + h * (S::kHalf / 16), kIdescQK, h > 0);
          commit_one(&s_full[X]);
          if (X == last_block) commit_one(&kv_empty[s]);
          if (j == tiles[X] - 1) commit_one(&q_empty[X]);
        };
        full(slot, phase);
#pragma unroll
        for (int X = 0; X < 2; ++X) {
          if (tiles[X] == 0) continue;
          pf::mbar_wait(dev::smem_addr(&q_full[X]), (uint32_t)(item_n[X] & 1), aborted, p.err,
                        count);
          fence_after();
          qk(X, 0, slot);
        }
        auto advance = [&] {
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
          }
        };
        auto v_full = [&](int j) {
          full(slot, phase);
          if (ragged && j == all - 1) dev::mbar_arrive(dev::smem_addr(v_there));
        };
        advance();
        v_full(0);
        for (int j = 0; j < all; ++j) {
          const int v_slot = slot;
          const uint64_t v_desc =
              smem_desc(sbase + S::kOffRing + v_slot * S::kSlotBytes, S::kHalf, 1024);
          if (ragged && j == all - 1)
            pf::mbar_wait(dev::smem_addr(v_clean), (uint32_t)(cleared++ & 1), aborted, p.err,
                          count);
          advance();  // to K(j + 1)
          const int k_slot = slot, k_phase = phase;
          advance();  // to V(j + 1)
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (j >= tiles[X]) continue;
            if (j == 0)  // the output of the block's item before has been read
              pf::mbar_wait(dev::smem_addr(&o_empty[X]), (uint32_t)((item_n[X] & 1) ^ 1), aborted,
                            p.err, count);
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // 64 tokens: 32 columns of P
              pf::mbar_wait(dev::smem_addr(&p_full[2 * X + half]), (uint32_t)(tile_n[X] & 1),
                            aborted, p.err, count);
              fence_after();
              umma4_ts(tmem + 256 + X * 128, tmem + X * 128 + half * 32,
                       v_desc + half * (64 * 128 / 16), kIdescPV, j > 0 || half > 0);
            }
            ++tile_n[X];
            if (X == last_block) {
              commit_one(&kv_empty[v_slot]);
              if (j + 1 < all) v_full(j + 1);
            }
            if (j + 1 < tiles[X]) {
              full(k_slot, k_phase);
              qk(X, j + 1, k_slot);
            } else {
              commit_one(&o_full[X]);
            }
          }
        }
        n += 2 * all;
        for (int X = 0; X < 2; ++X) item_n[X] += tiles[X] > 0;
      }
      // TMEM is freed only after the last MMA completed
      for (int X = 0; X < 2; ++X)
        if (item_n[X] > 0 &&
            !dev::mbar_wait_bounded(dev::smem_addr(&o_full[X]), (uint32_t)((item_n[X] - 1) & 1)))
          atomicOr(p.err, 2);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int X = warp / 4, r = threadIdx.x % kRows;
    const uint32_t lane_off = (uint32_t)(32 * (warp % 4)) << 16;
    const uint32_t tS = tmem + X * 128 + lane_off, tO = tmem + 256 + X * 128 + lane_off;
    const int tok = X * block_tokens + r / p.group, g = r % p.group;
    int tile_n = 0, item_n = 0;
    int sn = 0;  // SC: tiles so far, of all blocks
    auto scales_full = [&] {
      pf::mbar_wait(dev::smem_addr(&sc_full[sn % S::kScaleSlots]),
                    (uint32_t)((sn / S::kScaleSlots) & 1), aborted, p.err, count);
    };
    auto scales_read = [&] {
      dev::release_stage(dev::smem_addr(&sc_empty[sn % S::kScaleSlots]), lane);
      ++sn;
    };
    // SC: slots of tiles that this block has no part in are given back unread
    auto skip_scales = [&](const Item& w, int from) {
      const int all =
          SC == kScalePerToken ? w.tiles(w.tokens > block_tokens ? 1 : 0, block_tokens) : 0;
      for (int j = from; j < all; ++j) {
        scales_full();
        scales_read();
      }
    };
    for (int it = first; it < last; ++it) {
      const Item w = Item::load(p.items, it);
      if (X * block_tokens >= w.tokens) {
        skip_scales(w, 0);
        continue;
      }
      const int tiles = w.tiles(X, block_tokens);
      // keys this row sees, from the item's first tile on; the warp's fewest
      const int seen = w.pos0 + tok + 1 - w.t0 * kTok;
      const int fewest = __shfl_sync(0xffffffffu, seen, 0);
      // (kept above 0: 0 times a masked score's -inf would be NaN)
      const float scale =
          fmaxf(p.head_k_scales ? p.scale * __ldg(p.head_k_scales + w.head) : p.scale, 1.2e-38f);
      float m = -INFINITY, d = 0.f;
      // per block: lane l holds the scale of the tile's page l % 8, read a tile ahead
      auto block_scale = [&](int j) {
        const int page = (w.t0 + j) * kPages + lane % kPages;
        return j < tiles && page * kPageSize < w.keys(X, block_tokens)
                   ? __ldg(p.k_scales + (int64_t)(w.entry + page) * p.num_kv_heads + w.head)
                   : 1.f;
      };
      float next_scale = SC == kScalePerBlock ? block_scale(0) : 1.f;
      for (int j = 0; j < tiles; ++j, ++tile_n) {
        const float page_scale = next_scale;
        if constexpr (SC == kScalePerBlock) next_scale = block_scale(j + 1);
        pf::mbar_wait(dev::smem_addr(&s_full[X]), (uint32_t)(tile_n & 1), aborted, p.err, count);
        fence_after();
        float s[kTok];
        {
          uint32_t raw[kTok / 32][32];  // all in flight before the one wait
#pragma unroll
          for (int c = 0; c < kTok / 32; ++c) ld32_start(tS + c * 32, raw[c]);
          ld_wait();
#pragma unroll
          for (int c = 0; c < kTok / 32; ++c) {
            ld32_use(raw[c]);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(raw[c][i]);
          }
        }
        const uint32_t scales_at = sbase + S::kOffScales + sn % S::kScaleSlots * S::kScaleBytes;
        if constexpr (SC == kScalePerToken) {
          scales_full();
#pragma unroll
          for (int i = 0; i < kTok / 4; ++i) {
            float k[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(k[0]), "=f"(k[1]), "=f"(k[2]), "=f"(k[3])
                         : "r"(scales_at + i * 16));
#pragma unroll
            for (int e = 0; e < 4; ++e) s[4 * i + e] *= k[e];
          }
        }
        if (fewest < (j + 1) * kTok) {
          const int valid = seen - j * kTok;
          asm volatile("" ::: "memory");  // a branch: most tiles need no select
#pragma unroll
          for (int i = 0; i < kTok; ++i)
            if (i >= valid) s[i] = -INFINITY;
        }
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float a = s[16 * k];
#pragma unroll
          for (int i = 1; i < 15; i += 2) a = max3(a, s[16 * k + i], s[16 * k + i + 1]);
          m8[k] = fmaxf(a, s[16 * k + 15]);
        }
        float by_page[8];  // factors of the 16-column groups
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          by_page[k] = scale;
          if constexpr (SC == kScalePerBlock) {
            by_page[k] = fmaxf(scale * __shfl_sync(0xffffffffu, page_scale, k), 1.2e-38f);
            m8[k] *= by_page[k];
          }
        }
        const float mt = (SC == kScalePerBlock ? 1.f : scale) *
                         fmaxf(max3(max3(m8[0], m8[1], m8[2]), m8[3], m8[4]),
                               max3(m8[5], m8[6], m8[7]));
        // the reference moves only when the maximum passes it by more than 2^8
        const bool rebase = mt > m + (kRescaleAbove + kBelowScore<T>);
        const float m_new = rebase ? mt - kBelowScore<T> : m;
        const float alpha = m == -INFINITY ? 0.f : dev::fast_exp2(m - m_new);
        if (j > 0 && __any_sync(0xffffffffu, rebase)) {
          // O holds the tiles before j
          const float f = rebase ? alpha : 1.f;
          const bool clear = rebase && m == -INFINITY;  // nothing seen so far
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t v[16];
            ld16u(tO + c * 16, v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[i] = clear ? 0u : __float_as_uint(__uint_as_float(v[i]) * f);
            st16u(tO + c * 16, v);
          }
        }
        if (rebase) {
          d *= alpha;
          m = m_new;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t neg_m2 = f2(-ref, -ref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < kTok / 32; ++c) {
          uint32_t pk[16];
          uint64_t rests[2];  // SC per token: V's, of four columns
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if constexpr (SC == kScalePerToken)
              if (i % 2 == 0)
                asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                             : "=l"(rests[0]), "=l"(rests[1])
                             : "r"(scales_at + kTok * 4 + (32 * c + 2 * i) * 4));
            float x0, x1;
            const float factor = by_page[2 * c + i / 8];
            f2_split(fma2(f2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), f2(factor, factor),
                          neg_m2), x0, x1);
            const float a0 = dev::fast_exp2(x0), a1 = dev::fast_exp2(x1);
            acc[i % 4] = add2(acc[i % 4], f2(a0, a1));
            if constexpr (SC == kScalePerToken) {
              f2_split(mul2(f2(a0, a1), rests[i % 2]), x0, x1);
              pk[i] = mma::pack2(x0, x1, kBf16);
            } else {
              pk[i] = mma::pack2(a0, a1, kBf16);
            }
          }
          st16u(tS + c * 16, pk);
          if (c % 2) {  // half of the weights: P V may begin on them
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) {
              dev::mbar_arrive(dev::smem_addr(&p_full[2 * X + c / 2]));
              if (c / 2) count_on(count);
            }
          }
        }
        if constexpr (SC == kScalePerToken) scales_read();
        float lo, hi;
        f2_split(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), lo, hi);
        d += lo + hi;
      }
      skip_scales(w, tiles);
      // ---- the row's output
      if (tiles > 0) {
        pf::mbar_wait(dev::smem_addr(&o_full[X]), (uint32_t)(item_n & 1), aborted, p.err, count);
        fence_after();
      }
      const bool ok = tok < w.tokens;
      const float v_scale =
          p.head_v_scales ? p.v_scale * __ldg(p.head_v_scales + w.head) : p.v_scale;
      const float inv = d > 0.f || d != d ? v_scale / d : 0.f;
      const float lse = d > 0.f || d != d ? m + log2f(d) : -INFINITY;
      const size_t row = (size_t)(w.row0 + tok) * p.num_qo_heads + (size_t)w.head * p.group + g;
      const size_t part = (size_t)(w.slot < 0 ? 0 : w.slot) * 256 + X * kRows + r;
      uint32_t raw[D / 32][32];
      if (tiles > 0) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) ld32_start(tO + c * 32, raw[c]);
        ld_wait();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) ld32_use(raw[c]);
        fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_addr(&o_empty[X]));
        ++item_n;
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) raw[c][i] = 0u;
      }
      auto value = [&](int i) { return __uint_as_float(raw[i / 32][i % 32]) * inv; };
      // Four lanes trade the 32-byte chunks of their rows, so that a store of theirs
      // fills 128 bytes of one row: a row a lane, every store touched 32 lines.
      const int q4 = lane & 3;
      auto put = [&](uint32_t (&x)[4][8], char* base, int64_t pitch, int at) {
#pragma unroll
        for (int bit = 1; bit <= 2; ++bit)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int lo = bit == 1 ? 2 * i : i, hi = lo + bit;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t t =
                  __shfl_xor_sync(0xffffffffu, (q4 & bit) ? x[lo][e] : x[hi][e], bit);
              if (q4 & bit)
                x[lo][e] = t;
              else
                x[hi][e] = t;
            }
          }
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // chunk q4 of lane r's row
          const int row = __shfl_sync(0xffffffffu, at, (lane & ~3) | r);
          if (row >= 0) store32(base + row * pitch + q4 * 32, x[r]);
        }
      };
      uint64_t odd2 = 0;  // NaN where the row's output is not finite
#pragma unroll
      for (int i = 0; i < D; i += 2)
        odd2 = fma2(f2(__uint_as_float(raw[i / 32][i % 32]),
                       __uint_as_float(raw[i / 32][i % 32 + 1])),
                    0ull, odd2);
      float odd, odd_hi;
      f2_split(odd2, odd, odd_hi);
      odd += odd_hi;
      if (w.slot < 0) {
        // rows of o from the item's first head on, counted in heads
        char* base = reinterpret_cast<char*>(
            static_cast<T*>(p.o) +
            ((size_t)w.row0 * p.num_qo_heads + (size_t)w.head * p.group) * D);
        const int at = ok ? tok * p.num_qo_heads + g : -1;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t x[4][8];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[e / 8][e % 8] = mma::pack2(value(64 * c + 2 * e), value(64 * c + 2 * e + 1), kBf16);
          put(x, base + c * 128, (int64_t)D * 2, at);
        }
      } else {
        char* base = reinterpret_cast<char*>(p.part_o + ((size_t)w.slot * 256 + X * kRows) * D);
        const int at = ok ? r : -1;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[4][8];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e / 8][e % 8] = __float_as_uint(value(32 * c + e));
          put(x, base + c * 128, (int64_t)D * 4, at);
        }
      }
      unsigned again = __ballot_sync(0xffffffffu, ok && odd != odd);
      if (again) {  // (rare: rows are taken one after the other)
        asm volatile("" ::: "memory");
        __syncwarp();
        // the block's tiles may hold tokens that only the other block sees
        const int end = min(w.keys(w.tokens > block_tokens, block_tokens) - w.t0 * kTok,
                            tiles * kTok);
#pragma unroll 1
        while (again) {
          const int l = __ffs(again) - 1;
          again &= again - 1;
          const int t = __shfl_sync(0xffffffffu, tok, l), gl = __shfl_sync(0xffffffffu, g, l);
          const float ml = __shfl_sync(0xffffffffu, m, l), il = __shfl_sync(0xffffffffu, inv, l);
          const int64_t row_l = w.row0 + t, head = (int64_t)w.head * p.group + gl;
          const size_t part_l = (size_t)w.slot * 256 + X * kRows + warp % 4 * 32 + l;
          char* to = w.slot < 0 ? reinterpret_cast<char*>(static_cast<T*>(p.o) +
                                                          (row_l * p.num_qo_heads + head) * D)
                                : reinterpret_cast<char*>(p.part_o + part_l * D);
          fix_row<T, D, SC>(p, w.entry + w.t0 * kPages,
                        max(0, min(w.pos0 + t + 1 - w.t0 * kTok, end)), end, w.head,
                        row_l * p.q_token + head * p.q_head, scale, ml == -INFINITY ? 0.f : ml, il,
                        to, w.slot >= 0, count);
        }
      }
      if (ok) {
        if (w.slot >= 0)
          p.part_lse[part] = lse;
        else if (p.lse)
          p.lse[row] = lse * dev::kLn2;
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 8) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

}  // namespace fadecode
