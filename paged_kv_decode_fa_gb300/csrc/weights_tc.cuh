// Accumulated attention weights of many query rows, on the fifth-generation tensor
// cores (tcgen05); the definition is weights.cu's.
//
// A job is one kv head and up to 256 cached tokens, two blocks of 128; its columns
// are (query row, head of the group), 128 a tile, from the first that sees one of
// the tokens.  S = K Q^T with the tokens on the MMA's M side: a thread owns a token
// (TMEM lane), so the sum over the columns stays in its registers, and only the
// columns' lse come from shared memory, four a load for the whole warp.
//  - warp 9 loads Q tiles (tensor copies, as fa_prefill_kernel's) and their lse;
//  - K, two stages of two tiles, by warp 10's tensor copies; an E4M3 cache's codes are
//    copied aside, and warps 12-19 widen them (exactly) into the same layout;
//  - warp 8, one lane, issues the MMAs into two score buffers a block;
//  - warps 0-3 and 4-7 turn the scores of the two blocks into sums.
// The grid is persistent and nothing waits for a whole CTA between jobs.  Every wait is
// bounded (2 s; a job takes less, by the plan's limit on columns); one that runs out sets
// bit 1 of the device-check word and the CTA drains.
//
// What bounds it.  32 rows of 4 heads over 16 prompts of 2048-8192 tokens, 8 kv heads:
// 36 us from a 16-bit cache (168 MB: 25 us at the copy rate), where a job of one
// tile waits for its K; 45 us from an E4M3 cache (84 MB), 4300 cycles a job of 256
// tokens in which codes, widening, MMAs and sums follow each other.  On the way: 67 us
// with a thread a row reading its codes straight from global memory, 48 with four
// warps widening from shared memory (4600 cycles a job), 53 with eight of 96
// registers (the sums spill).  Widening in integer steps and a bf16 product took
// longer (58-92 us).  Columns' masks inside the sums' one loop doubled it (2460
// cycles a tile, 1140 with two loops).
#pragma once

#include <cuda.h>

#include "decode_mma.cuh"
#include "tcgen05.cuh"

namespace fadecode {
namespace wt {

constexpr int kTok = 128;                 // tokens of a block, columns of a tile
constexpr int kPages = kTok / kPageSize;  // 8
constexpr uint32_t kTmemCols = 512;       // [block][buffer] of 128

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kTok * 128;  // [128][D] in 16 bits
  static constexpr int kQSlots = D == 128 ? 2 : 4;
  static constexpr int kOffK = 0;                      // [stage][block]
  static constexpr int kOffQ = 4 * kTile;
  static constexpr int kOffRaw = kOffQ + kQSlots * kTile;  // a job's codes (E4M3)
  static constexpr int kOffLse = kOffRaw + 2 * kTok * D;
  static constexpr int kOffBar = kOffLse + kQSlots * kTok * 4;
  // q_full, q_empty [slots]; k_full, k_empty [2]; s_full, s_empty [block][buffer];
  // raw_full, raw_empty
  static constexpr int kNumBars = 2 * kQSlots + 4 + 8 + 2;
  static constexpr int kOffTmem = kOffBar + 8 * kNumBars;
  static constexpr int kOffDead = kOffTmem + 16;  // [slot] a tile has columns that add nothing
  static constexpr int kBytes = kOffDead + 4 * kQSlots + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
};

// Warps: 0-7 sums, 8-11 MMAs and loads, 12-19 widening (E4M3).
constexpr int threads(bool e4m3) { return e4m3 ? 640 : 384; }
// Registers a thread with twenty warps: as launched, and as the sums and the others
// share them out.
constexpr int kLaunchRegs = 96, kSumRegs = 136, kOtherRegs = 64;
static_assert(256 * kSumRegs + 384 * kOtherRegs <= 640 * kLaunchRegs,
              "a larger share would be waited for without end");

}  // namespace wt

template <typename T, typename KVT, int D, int SC>
__global__ void __launch_bounds__(wt::threads(!std::is_same<T, KVT>::value), 1)
    fa_weights_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                         const __grid_constant__ CUtensorMap kv_map,
                         const __grid_constant__ WeightsParams p, const int jobs) {
  using namespace wt;
  using namespace tc;
  using S = Smem<D>;
  constexpr bool kE4m3 = !std::is_same<T, KVT>::value;
  constexpr uint32_t kIdesc = instr_desc(std::is_same<T, __nv_bfloat16>::value, kTok, kTok, 0);
  constexpr int kQSlots = S::kQSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = dev::smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + kQSlots;
  uint64_t* k_full = bars + 2 * kQSlots;
  uint64_t* k_empty = k_full + 2;
  uint64_t* s_full = k_full + 4;   // [block][buffer]
  uint64_t* s_empty = k_full + 8;
  uint64_t* raw_full = k_full + 12;
  uint64_t* raw_empty = k_full + 13;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffTmem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool aborted = false;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kQSlots; ++s) {
      dev::mbar_init(dev::smem_addr(&q_full[s]), 1);
      dev::mbar_init(dev::smem_addr(&q_empty[s]), 9);  // the MMAs and eight warps' lse
    }
    for (int s = 0; s < 2; ++s) {
      dev::mbar_init(dev::smem_addr(&k_full[s]), kE4m3 ? 8 : 1);
      dev::mbar_init(dev::smem_addr(&k_empty[s]), 1);
    }
    for (int s = 0; s < 4; ++s) {
      dev::mbar_init(dev::smem_addr(&s_full[s]), 1);
      dev::mbar_init(dev::smem_addr(&s_empty[s]), 4);
    }
    dev::mbar_init(dev::smem_addr(raw_full), 1);
    dev::mbar_init(dev::smem_addr(raw_empty), 8);
    dev::fence_barrier_init();
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
  const uint32_t tmem = *tmem_slot;

  // a job's unit and head, its blocks, and its tiles of columns
  struct Job {
    int row0, rows, entry, pages, pos0, before, h, blocks, columns, t0, t1;
  };
  auto load_job = [&](int j) {
    const int4* up = reinterpret_cast<const int4*>(p.units + j / p.hkv);
    const int4 a = __ldg(up), b = __ldg(up + 1);
    Job w{a.x, a.y, a.z, a.w, b.x, b.y, j % p.hkv, 0, 0, 0, 0};
    w.blocks = w.pages > kPages ? 2 : 1;
    w.columns = w.rows << p.group_log2;
    w.t0 = (max(0, w.pos0 - w.before) << p.group_log2) / kTok;
    w.t1 = (w.columns + kTok - 1) / kTok;
    return w;
  };
  auto page_of = [&](const Job& w, int i) -> int {
    int page = i < w.pages ? __ldg(p.indices + w.entry + i) : -1;
    return page < 0 || (int64_t)page >= p.num_pages ? -1 : page;
  };

  if (warp >= 8) {
    if constexpr (kE4m3) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 9) {
      // -------------------------------------------------------------- Q and lse
      const int tile_tokens = kTok >> p.group_log2;
      int n = 0;
      for (int j = blockIdx.x; j < jobs; j += gridDim.x) {
        const Job w = load_job(j);
        for (int t = w.t0; t < w.t1; ++t, ++n) {
          const int s = n % kQSlots;
          float lse[4];  // -lse of columns lane, lane + 32, ...: before the wait
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = t * kTok + lane + 32 * i;
            const int row = x >> p.group_log2, g = x & ((1 << p.group_log2) - 1);
            lse[i] = x < w.columns ? __ldg(p.lse + (int64_t)(w.row0 + row) * p.hq +
                                           (w.h << p.group_log2) + g) * -1.4426950408889634f
                                   : -INFINITY;
            if (lse[i] == INFINITY) lse[i] = -INFINITY;  // a row that saw nothing: weight 0
          }
          const bool dead = __any_sync(0xffffffffu, lse[0] == -INFINITY || lse[1] == -INFINITY ||
                                                        lse[2] == -INFINITY || lse[3] == -INFINITY);
          dev::mbar_wait(dev::smem_addr(&q_empty[s]), (uint32_t)(((n / kQSlots) & 1) ^ 1), aborted,
                         p.err);
          float* to = reinterpret_cast<float*>(smem + S::kOffLse) + s * kTok;
#pragma unroll
          for (int i = 0; i < 4; ++i) to[lane + 32 * i] = lse[i];
          if (lane == 0) *reinterpret_cast<int*>(smem + S::kOffDead + 4 * s) = dead;
          __syncwarp();
          if (lane == 0) {
            const uint32_t full = dev::smem_addr(&q_full[s]);
            dev::mbar_arrive_expect_tx(full, S::kTile);
            for (int h = 0; h < S::kHalves; ++h)
              tma_load_3d(sbase + S::kOffQ + s * S::kTile + h * (kTok * 128), &q_map, h * 64,
                          w.h << p.group_log2, w.row0 + t * tile_tokens, full);
          }
          __syncwarp();
        }
      }
      if (lane == 0)  // no copy may still be landing when the CTA exits
        for (int i = n > kQSlots ? n - kQSlots : 0; i < n; ++i)
          if (!dev::mbar_wait_bounded(dev::smem_addr(&q_full[i % kQSlots]),
                                      (uint32_t)((i / kQSlots) & 1)))
            atomicOr(p.err, 2);
    } else if (warp == 10) {
      // -------------------------------------------------------------- K
      // from a 16-bit cache into the tiles, from an E4M3 cache its codes
      const int oob = (int)(2 * p.num_pages);  // beyond the last page: zeros
      constexpr int kStages = kE4m3 ? 1 : 2;
      uint64_t* full_bar = kE4m3 ? raw_full : k_full;
      uint64_t* empty_bar = kE4m3 ? raw_empty : k_empty;
      int n = 0;
      for (int j = blockIdx.x; j < jobs; j += gridDim.x, ++n) {
        const Job w = load_job(j);
        const int s = n % kStages;
        const uint32_t full = dev::smem_addr(&full_bar[s]);
        // lane l: half l / 16 of page l % 16
        const int half = lane / (2 * kPages), at = lane % (2 * kPages);
        const int page = page_of(w, at), c3 = page < 0 ? oob : 2 * page;
        dev::mbar_wait(dev::smem_addr(&empty_bar[s]), (uint32_t)(((n / kStages) & 1) ^ 1), aborted,
                       p.err);
        if (lane == 0)
          dev::mbar_arrive_expect_tx(full, w.blocks * (kE4m3 ? kTok * D : S::kTile));
        __syncwarp();
        if (at < w.blocks * kPages) {
          if (kE4m3 && half == 0)
            tma_load_4d_plain(sbase + S::kOffRaw + at * (kPageSize * D), &kv_map, 0, w.h, 0, c3,
                              full);
          if (!kE4m3 && half < S::kHalves)
            tma_load_4d_plain(sbase + S::kOffK + (2 * s + at / kPages) * S::kTile +
                                  half * (kTok * 128) + at % kPages * (kPageSize * 128),
                              &kv_map, half * 64, w.h, 0, c3, full);
        }
        __syncwarp();
      }
      if (lane == 0)
        for (int i = n > kStages ? n - kStages : 0; i < n; ++i)
          if (!dev::mbar_wait_bounded(dev::smem_addr(&full_bar[i % kStages]),
                                      (uint32_t)((i / kStages) & 1)))
            atomicOr(p.err, 2);
    } else if (kE4m3 && warp >= 12) {
      // -------------------------------------------------------------- K, widened
      // A thread widens the codes of one token.  They stand in shared memory by
      // tensor copy: read straight from global memory, a thread a row, they missed L1
      // at every piece.
      const int row = threadIdx.x - 12 * 32, X = row / kTok, r = row % kTok;
      constexpr int kPieces = D / 16;  // 16 codes each
      // piece i of a row stands at i ^ (r % 8), or ^ (r / 2 % 4) in rows of 64 bytes
      const int mix = D == 128 ? r & 7 : r >> 1 & 3;
      int n = 0;
      for (int j = blockIdx.x; j < jobs; j += gridDim.x, ++n) {
        const int s = n & 1;
        const bool active = X < load_job(j).blocks;
        dev::mbar_wait(dev::smem_addr(raw_full), (uint32_t)(n & 1), aborted, p.err);
        uint4 codes[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (active)
            codes[i] =
                *reinterpret_cast<const uint4*>(smem + S::kOffRaw + row * D + (i ^ mix) * 16);
        dev::release_stage(dev::smem_addr(raw_empty), lane);
        dev::mbar_wait(dev::smem_addr(&k_empty[s]), (uint32_t)(((n >> 1) & 1) ^ 1), aborted,
                       p.err);
        if (active) {
          const uint32_t tile = sbase + S::kOffK + (2 * s + X) * S::kTile + r * 128;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const uint32_t in[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
            uint32_t out[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              out[2 * e] = widen2<T>(in[e] & 0xffffu);
              out[2 * e + 1] = widen2<T>(in[e] >> 16);
            }
            // granule g (8 dims) of row r stands at g ^ (r % 8) of its half's 128 bytes
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int g = 2 * i + k;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               tile + (g / 8) * (kTok * 128) + ((g % 8) ^ (r & 7)) * 16),
                           "r"(out[4 * k]), "r"(out[4 * k + 1]), "r"(out[4 * k + 2]),
                           "r"(out[4 * k + 3])
                           : "memory");
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_addr(&k_full[s]));
      }
    } else if (warp == 8) {
      // -------------------------------------------------------------- MMAs
      if (elect_one()) {
        int n = 0, q_n = 0, cnt[2] = {0, 0};
        for (int j = blockIdx.x; j < jobs; j += gridDim.x, ++n) {
          const Job w = load_job(j);
          dev::mbar_wait(dev::smem_addr(&k_full[n & 1]), (uint32_t)((n >> 1) & 1), aborted, p.err);
          for (int t = w.t0; t < w.t1; ++t, ++q_n) {
            const int qs = q_n % kQSlots;
            dev::mbar_wait(dev::smem_addr(&q_full[qs]), (uint32_t)((q_n / kQSlots) & 1), aborted,
                           p.err);
            const uint64_t q_desc = smem_desc(sbase + S::kOffQ + qs * S::kTile, 16, 1024);
#pragma unroll
            for (int X = 0; X < 2; ++X) {
              if (X >= w.blocks) continue;
              const int b = cnt[X] & 1;
              dev::mbar_wait(dev::smem_addr(&s_empty[2 * X + b]),
                             (uint32_t)(((cnt[X] >> 1) & 1) ^ 1), aborted, p.err);
              fence_after();
              ++cnt[X];
              const uint64_t k_desc =
                  smem_desc(sbase + S::kOffK + (2 * (n & 1) + X) * S::kTile, 16, 1024);
#pragma unroll
              for (int h = 0; h < S::kHalves; ++h)
                umma4(tmem + X * 256 + b * 128, k_desc + h * (kTok * 128 / 16),
                      q_desc + h * (kTok * 128 / 16), kIdesc, h > 0);
              commit_one(&s_full[2 * X + b]);
            }
            commit_one(&q_empty[qs]);
          }
          commit_one(&k_empty[n & 1]);
        }
        // TMEM is freed only after the last MMA completed
        if (n > 0 &&
            !dev::mbar_wait_bounded(dev::smem_addr(&k_empty[(n - 1) & 1]),
                                    (uint32_t)(((n - 1) >> 1) & 1)))
          atomicOr(p.err, 2);
      }
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------------- sums
    if constexpr (kE4m3) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int X = warp / 4, r = threadIdx.x % kTok;
    const uint32_t tS = tmem + X * 256 + ((uint32_t)(32 * (warp % 4)) << 16);
    int q_n = 0, cnt = 0;
    // A job's page id and scale are loaded during the jobs before: the chain unit ->
    // page -> scale would stand in front of every tile.
    const int at = X * kTok + r;
    auto id_of = [&](const Job& w, int j) {
      return j < jobs && at / kPageSize < w.pages ? __ldg(p.indices + w.entry + at / kPageSize)
                                                  : -1;
    };
    auto slot_of = [&](int page, int h) {
      return ((int64_t)max(page, 0) * p.hkv + h) * kPageSize + at % kPageSize;
    };
    auto scale_of = [&](int page, int h) {
      if constexpr (SC == kScalePerToken) return __ldg(p.k_scales + slot_of(page, h));
      if constexpr (SC == kScalePerBlock) return __ldg(p.k_scales + slot_of(page, h) / kPageSize);
      return 1.f;
    };
    auto checked = [&](int page) { return (int64_t)page < p.num_pages ? max(page, -1) : -1; };
    const int step = gridDim.x;
    Job w = load_job(blockIdx.x), w1 = load_job(min((int)blockIdx.x + step, jobs - 1));
    int id = id_of(w, blockIdx.x), id1 = id_of(w1, blockIdx.x + step);
    float token_scale = scale_of(checked(id), w.h);
    for (int j = blockIdx.x; j < jobs; j += step) {
      const float scale1 = scale_of(checked(id1), w1.h);
      const Job w2 = load_job(min(j + 2 * step, jobs - 1));
      const int id2 = id_of(w2, j + 2 * step);
      const bool active = X < w.blocks;
      const int pos = w.pos0 + at, page = active ? checked(id) : -1;
      if (active && page < 0 && at / kPageSize < w.pages && r % kPageSize == 0)
        atomicOr(p.err, 1);
      const float scale =
          token_scale * (p.head_k_scales ? p.scale * __ldg(p.head_k_scales + w.h) : p.scale);
      const int64_t slot = slot_of(page, w.h);
      // columns that see this token: from `seen` on (the warp's last token: `warp_seen`)
      const int seen = max(0, pos - w.before) << p.group_log2;
      const int warp_seen = __shfl_sync(0xffffffffu, seen, 31);
      const uint64_t scale2 = f2(scale, scale);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
      for (int t = w.t0; t < w.t1; ++t, ++q_n) {
        const int qs = q_n % kQSlots;
        dev::mbar_wait(dev::smem_addr(&q_full[qs]), (uint32_t)((q_n / kQSlots) & 1), aborted,
                       p.err);
        if (active) {
          const int b = cnt & 1;
          dev::mbar_wait(dev::smem_addr(&s_full[2 * X + b]), (uint32_t)((cnt >> 1) & 1), aborted,
                         p.err);
          fence_after();
          ++cnt;
          const int lo = seen - t * kTok, hi = w.columns - t * kTok;
          const bool whole = warp_seen <= t * kTok &&
                             *reinterpret_cast<const int*>(smem + S::kOffDead + 4 * qs) == 0;
          // 16 columns at a time: the next ones' scores and lse on their way
          const uint32_t lse_at = sbase + S::kOffLse + qs * (kTok * 4);
          const int steps = min(kTok / 16, (hi + 15) / 16);
          uint32_t raw[2][16];
          uint64_t neg[2][8];  // -lse, in pairs
          auto start = [&](int c, int to) {
            ld16_start(tS + b * 128 + c * 16, raw[to]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                           : "=l"(neg[to][2 * i]), "=l"(neg[to][2 * i + 1])
                           : "r"(lse_at + (c * 16 + 4 * i) * 4));
          };
          start(0, 0);
          // (two loops: with the test inside one, every column paid for its compares)
          auto add_up = [&](auto every) {
            constexpr bool all = decltype(every)::value;
#pragma unroll
            for (int c = 0; c < kTok / 16; ++c) {
              if (!all && c >= steps) break;
              ld_wait();
              ld16_use(raw[c & 1]);
              if (c + 1 < kTok / 16 && (all || c + 1 < steps)) start(c + 1, (c + 1) & 1);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float x0, x1;
                f2_split(fma2(f2(__uint_as_float(raw[c & 1][2 * i]),
                                 __uint_as_float(raw[c & 1][2 * i + 1])),
                              scale2, neg[c & 1][i]), x0, x1);
                x0 = dev::fast_exp2(x0);
                x1 = dev::fast_exp2(x1);
                if (!all) {
                  // (columns behind the last have a -lse of -inf too)
                  const int col = 16 * c + 2 * i;
                  float n0, n1;
                  f2_split(neg[c & 1][i], n0, n1);
                  x0 = col >= lo && n0 != -INFINITY ? x0 : 0.f;
                  x1 = col + 1 >= lo && n1 != -INFINITY ? x1 : 0.f;
                }
                acc[i % 4] = add2(acc[i % 4], f2(x0, x1));
              }
            }
          };
          if (whole)
            add_up(std::true_type{});
          else
            add_up(std::false_type{});
          fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(dev::smem_addr(&s_empty[2 * X + b]));
        }
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_addr(&q_empty[qs]));
      }
      float lo, hi;
      f2_split(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), lo, hi);
      // tokens that no row sees (slots behind the request's last) stay
      if (page >= 0 && pos <= w.before + w.rows - 1) atomicAdd(p.weights + slot, lo + hi);
      w = w1;
      w1 = w2;
      id = id1;
      id1 = id2;
      token_scale = scale1;
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
