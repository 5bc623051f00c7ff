// Eviction from a paged KV cache by accumulated attention weight: the calls
// fa_evict_* (declared in include/fa_decode.h).
//
// The definition, per request of L tokens and kv head, n = min(L, keep): kept are the
// last min(recent, n) tokens and, of those before, the n - recent of the largest
// weight (equal weights: the earlier token).  They move, in their order, to the
// request's first n slots: K, V, the weight and an E4M3 cache's scales per token;
// the weights of slots n .. L-1 become 0, so that they can be appended to.
//
// Work.  A cluster of C CTAs (1 to 8) takes one (request, kv head):
//  1. each CTA reads the weights of its share of the tokens, as 32-bit keys in
//     the order of the floats (in shared memory where they fit);
//  2. the key of the last kept token is found eight bits at a time: histograms in
//     shared memory, summed over the cluster, four passes;
//  3. counts of larger and equal keys, summed over the cluster's lower CTAs, give
//     every kept token its rank; the list rank -> token goes to the workspace;
//  4. the rows move a chunk of ranks at a time: all CTAs read the chunk's rows
//     into shared memory, the cluster meets, all write.  A kept token's rank is at
//     most its index, so the chunk's slots lie before every later chunk's rows:
//     one barrier a chunk orders everything, in place, and each row is read
//     and written once.  Rows already in their slots are left.
//
// What bounds it.  64 requests of 2048-8192 tokens kept to 2048 (8 kv heads, head_dim 128,
// bf16), a CTA each: 219-231 us for a first eviction, 1.07 GB moved = 4.6-4.9 TB/s,
// 0.70-0.73 of the copy rate; 24 us of it select, in which no row moves.  One E4M3 request
// of 65536 tokens kept to 8000, eight CTAs a kv head: 49 us, 34 MB (5.1 at the copy rate):
// the cluster's barriers and chains of loads, the border's four passes 11 of them.
// Evicted again and again, the two calls take 129 and 31 us, in which 256 of 2048 and 33
// of 8000 ranks a head move (the recent tokens alone).  Measured so: with 256 threads
// for the long request as well 51 us for 31; ranks looked up a chunk at a time, in front of
// its rows, 54.  In the batch's loop, pieces' addresses by divisions a piece cost 40-60 us,
// a cluster barrier a chunk 15.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <limits>
#include <new>
#include <vector>

#include "decode_kernel.cuh"
#include "fa_decode.h"
#include "staging.h"

namespace fadecode {
namespace {

namespace cg = cooperative_groups;

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Threads of a CTA: many where the CTAs are few.
constexpr int kThreads = 256, kManyThreads = 1024;
constexpr int kMostCtas = 8;              // of a cluster
// Shared memory beside EvictShared: keys, then two stages of rows.  Four CTAs an SM, or
// one with more where there are no more.  And ranks looked up at once.
constexpr int kBuffer = 40 << 10, kBigBuffer = 160 << 10;
constexpr int kRanks = 128, kManyRanks = 512;
constexpr int kBatch = 4;                 // loads of a thread in flight

struct EvictUnit {
  int32_t entry, length, kept, recent;
  int64_t list;  // its first kept token of head 0 in the workspace's lists
  int32_t pad[2];
};
static_assert(sizeof(EvictUnit) == 32, "read as two int4");

struct EvictParams {
  uint8_t* kv;
  float* weights;   // [pages, Hkv, 16]
  float* k_scales;  // [pages, Hkv, 16] or nullptr
  float* v_scales;
  const int32_t* indices;
  const EvictUnit* units;
  int32_t* lists;
  int* err;
  int64_t num_pages;
  int hkv;
  int row_bytes;  // of K (or V) of one token and head
  int buffer;     // bytes of dynamic shared memory
};

// Unsigned order = order of the floats, NaN above all, -0 = 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

template <int kRankInfo>
struct EvictShared {
  int hist[2][256];
  int counts[2];        // kept for sure / equal to the last key, of this CTA
  int warp_counts[2][kManyThreads / 32];
  int digit, above;     // of one pass
  // ranks looked up: the byte offsets of their K rows, from (-1: nothing to move) and
  // to; the slot in the arrays per token; and what moves there: weight, K and V scale
  int64_t src[3][kRankInfo], dst[3][kRankInfo], slot[3][kRankInfo];
  float moved[3][3][kRankInfo];
};

template <int kThreads, int kRankInfo>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    fa_evict_kernel(const EvictParams p) {
  constexpr int kWarps = kThreads / 32;
  using Shared = EvictShared<kRankInfo>;
  extern __shared__ __align__(16) uint8_t shared[];
  Shared& sh = *reinterpret_cast<Shared*>(shared);
  uint8_t* const buffer = shared + (sizeof(Shared) + 15) / 16 * 16;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
  const int job = blockIdx.x / C, h = job % p.hkv, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const EvictUnit u = p.units[job / p.hkv];
  const int L = u.length, n = u.kept, cand = L - u.recent, want = n - u.recent;
  int32_t* list = p.lists + u.list + (int64_t)h * n;

  // The cluster meets: memory written before is seen after.  (A cluster's own barrier
  // waits for every store in flight, also of a cluster of one.)
  auto meet = [&] {
    if (C == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  // a token's slot in the arrays per token; -1 for a page id outside the cache
  auto place = [&](int t) -> int64_t {
    const int page = __ldg(p.indices + u.entry + t / kPageSize);
    if (page < 0 || (int64_t)page >= p.num_pages) {
      atomicOr(p.err, 1);
      return -1;
    }
    return (int64_t)page * kPageSize + t % kPageSize;
  };
  auto token_at = [&](int64_t at) -> int64_t {  // index into [pages, Hkv, 16]
    return ((at / kPageSize) * p.hkv + h) * kPageSize + at % kPageSize;
  };

  // ---- 1. the keys of tokens t0 .. t1 (t0 at a page's start: four tokens a load)
  const int share = ((cand + C - 1) / C + kPageSize - 1) / kPageSize * kPageSize;
  const int t0 = min(c * share, cand), t1 = min(t0 + share, cand);
  uint32_t* keys = reinterpret_cast<uint32_t*>(buffer);
  const bool held = (t1 - t0 + 3) / 4 * 16 <= p.buffer;
  auto read_key = [&](int t) -> uint32_t {
    const int64_t at = place(t);
    return at < 0 ? key_of(0.f) : key_of(p.weights[token_at(at)]);
  };
  if (held) {
    for (int i = t0 + 4 * tid; i < t1; i += 4 * kThreads * kBatch) {
      int64_t at[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int t = i + 4 * kThreads * k;
        at[k] = t < t1 ? place(t) : -1;
      }
      float4 w[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        w[k] = at[k] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                         : *reinterpret_cast<const float4*>(p.weights + token_at(at[k]));
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int t = i + 4 * kThreads * k;
        if (t < t1)  // keys behind t1, of the same page, are not looked at
          *reinterpret_cast<uint4*>(keys + (t - t0)) =
              make_uint4(key_of(w[k].x), key_of(w[k].y), key_of(w[k].z), key_of(w[k].w));
      }
    }
  }
  auto key = [&](int t) { return held ? keys[t - t0] : read_key(t); };
  __syncthreads();

  // ---- 2. the want-th largest key
  uint32_t border = 0xffffffffu;  // keys above it are kept,
  int ties = 0;                   // and the first `ties` of those equal to it
  if (want > 0) {
    uint32_t prefix = 0;
    int left = want;
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      int* hist = sh.hist[pass & 1];
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = t0; i < t1; i += kThreads * kBatch) {
        uint32_t k[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int t = i + b * kThreads + tid;
          k[b] = t < t1 ? key(t) : 0;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const bool in = i + b * kThreads + tid < t1 &&
                          (pass == 0 || (k[b] >> (shift + 8)) == prefix);
          if (!__any_sync(0xffffffffu, in)) continue;
          const int digit = in ? (int)((k[b] >> shift) & 0xff) : 256;
          // equal digits of a warp are counted once (weights crowd few exponents)
          const unsigned same = __match_any_sync(0xffffffffu, digit);
          if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
        }
      }
      meet();
      if (tid < 256) {
        int sum = 0;
        for (int r = 0; r < C; ++r) sum += cluster.map_shared_rank(hist, r)[tid];
        // with the keys of larger digits: a suffix sum over the 256 threads
        int suffix = sum;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
          const int v = __shfl_down_sync(0xffffffffu, suffix, off);
          if (lane + off < 32) suffix += v;
        }
        if (lane == 0) sh.warp_counts[0][warp] = suffix;
        dev::named_barrier(1, 256);
        for (int w = warp + 1; w < 8; ++w) suffix += sh.warp_counts[0][w];
        if (suffix >= left && suffix - sum < left) {
          sh.digit = tid;
          sh.above = suffix - sum;
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | (uint32_t)sh.digit;
      left -= sh.above;
      // (the other histogram is cleared next; this one only after the next meeting)
    }
    border = prefix;
    ties = left;
  }

  // ---- 3. ranks: a warp takes a run of the CTA's tokens
  auto flags = [&](int t, int end, bool* above, bool* equal) {
    const uint32_t k = t < end && want > 0 ? key(t) : 0;
    *above = t < end && want > 0 && k > border;
    *equal = t < end && want > 0 && k == border;
  };
  const int per_warp = ((t1 - t0 + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int w0 = min(t0 + warp * per_warp, t1), w1 = min(w0 + per_warp, t1);
  {
    int a = 0, e = 0;
    for (int i = w0; i < w1; i += 32) {
      bool above, equal;
      flags(i + lane, w1, &above, &equal);
      a += __popc(__ballot_sync(0xffffffffu, above));
      e += __popc(__ballot_sync(0xffffffffu, equal));
    }
    if (lane == 0) {
      sh.warp_counts[0][warp] = a;
      sh.warp_counts[1][warp] = e;
    }
    __syncthreads();
    if (tid < 2) {
      int sum = 0;
      for (int w = 0; w < kWarps; ++w) sum += sh.warp_counts[tid][w];
      sh.counts[tid] = sum;
    }
  }
  meet();
  {
    int a = 0, e = 0;  // kept for sure, and equal to the border, before this warp
    for (int r = 0; r < c; ++r) {
      const int* other = cluster.map_shared_rank(sh.counts, r);
      a += other[0];
      e += other[1];
    }
    for (int w = 0; w < warp; ++w) {
      a += sh.warp_counts[0][w];
      e += sh.warp_counts[1][w];
    }
    const unsigned below = (1u << lane) - 1;
    for (int i = w0; i < w1; i += 32) {
      bool above, equal;
      flags(i + lane, w1, &above, &equal);
      const unsigned ma = __ballot_sync(0xffffffffu, above);
      const unsigned me = __ballot_sync(0xffffffffu, equal);
      const int mine = e + __popc(me & below);
      if (above || (equal && mine < ties))
        list[a + __popc(ma & below) + min(mine, ties)] = i + lane;
      a += __popc(ma);
      e += __popc(me);
    }
  }
  for (int i = c * kThreads + tid; i < u.recent; i += C * kThreads) list[want + i] = cand + i;
  meet();  // the list is whole, and the keys are done with

  // ---- 4. the rows, a chunk of ranks at a time, the next chunk's on their way
  const int rb = p.row_bytes, pieces = 2 * rb / 16;  // 16-byte pieces of a token's K and V
  const int chunk = min(kRankInfo, p.buffer / 2 / (2 * rb));
  const int64_t token_bytes = (int64_t)p.hkv * rb, page_half = kPageSize * token_bytes;
  // a thread moves one piece (a power of two of them) of every so many ranks
  const int piece = tid & (pieces - 1), first_rank = tid / pieces, ranks = kThreads / pieces;
  uint8_t* const base = p.kv + (int64_t)h * rb +
                        (piece * 16 < rb ? piece * 16 : page_half + piece * 16 - rb);
  auto row_of = [&](int64_t at) {
    return at / kPageSize * 2 * page_half + at % kPageSize * token_bytes;
  };
  const int steps = (n + C * chunk - 1) / (C * chunk);
  // The ranks of a few steps are looked up at once, two such groups ahead: the chain
  // list -> page -> weight takes longer than a chunk's rows.
  const int group = kRankInfo / chunk;
  auto count_of = [&](int step) {
    return step < steps ? max(0, min(chunk, n - (step * C + c) * chunk)) : 0;
  };
  // where the ranks of steps g * group .. come from and go to, and what moves
  // beside their rows
  auto look_up = [&](int g) {
    const int s = g % 3;
    for (int e = tid; e < group * chunk; e += kThreads) {
      const int step = g * group + e / chunk, i = e % chunk;
      if (i >= count_of(step)) continue;
      const int rank = (step * C + c) * chunk + i, t = __ldcg(list + rank);
      int64_t src = -1, dst = -1;
      if (t != rank) {
        src = place(t);
        dst = place(rank);
        if (dst < 0) src = -1;
      }
      sh.src[s][e] = src < 0 ? -1 : row_of(src);
      if (src >= 0) {
        sh.dst[s][e] = row_of(dst);
        sh.slot[s][e] = token_at(dst);
        const int64_t at = token_at(src);
        sh.moved[s][0][e] = p.weights[at];
        if (p.k_scales) {
          sh.moved[s][1][e] = p.k_scales[at];
          sh.moved[s][2][e] = p.v_scales[at];
        }
      }
    }
  };
  auto fetch = [&](int step) {
    const int count = count_of(step), s = step / group % 3, first = step % group * chunk;
    const uint32_t to = dev::smem_addr(buffer) + (step & 1) * (p.buffer / 2) + piece * 16;
    for (int i = first_rank; i < count; i += ranks) {
      const int64_t src = sh.src[s][first + i];
      if (src >= 0) dev::cp_async16(to + i * 2 * rb, base + src);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look_up(0);
  look_up(1);
  __syncthreads();
  fetch(0);
  for (int step = 0; step < steps; ++step) {
    fetch(step + 1);
    if (step % group == 0) look_up(step / group + 2);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    // all of the chunk's rows have been read (nothing else is handed over: a
    // thread writes the pieces that it fetched itself)
    if (C == 1)
      __syncthreads();
    else
      asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::
                       : "memory");
    const int count = count_of(step), s = step / group % 3, first = step % group * chunk;
    const uint8_t* from = buffer + (step & 1) * (p.buffer / 2) + piece * 16;
    for (int i = first_rank; i < count; i += ranks)
      if (sh.src[s][first + i] >= 0)
        *reinterpret_cast<uint4*>(base + sh.dst[s][first + i]) =
            *reinterpret_cast<const uint4*>(from + i * 2 * rb);
    for (int i = first + tid; i < first + count; i += kThreads) {
      if (sh.src[s][i] < 0) continue;
      const int64_t at = sh.slot[s][i];
      p.weights[at] = sh.moved[s][0][i];
      if (p.k_scales) {
        p.k_scales[at] = sh.moved[s][1][i];
        p.v_scales[at] = sh.moved[s][2][i];
      }
    }
    __syncthreads();  // the stage is free
  }
  // all weights have been read: those of the freed slots start again at 0
  for (int i = n / 4 * 4 + 4 * (c * kThreads + tid); i < L; i += 4 * C * kThreads) {
    const int64_t at = place(i);
    if (at < 0) continue;
    float* w = p.weights + token_at(at);
    if (i >= n && i + 4 <= L) {
      *reinterpret_cast<float4*>(w) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k >= n && i + k < L) w[k] = 0.f;
    }
  }
}

template <int kRankInfo>
constexpr int evict_shared() {
  return (int)((sizeof(EvictShared<kRankInfo>) + 15) / 16 * 16);
}
static_assert(4 * (evict_shared<kRanks>() + kBuffer + 1024) <= 228 << 10, "four CTAs an SM");
static_assert(evict_shared<kManyRanks>() + kBigBuffer <= 227 << 10, "shared memory per CTA");

struct EvictLayout {
  size_t units, lists, total;
};

// Requests that lose tokens, counted or (with `out`) written; -1 for malformed
// arguments.  *tokens: kept tokens of one kv head, in all; *longest: of one request.
int64_t make_units(const int32_t* indptr, const int32_t* last_page_len, const int32_t* keep,
                   const int32_t* recent, int batch, int heads, EvictUnit* out, int64_t* tokens,
                   int64_t* longest) {
  int64_t units = 0;
  *tokens = *longest = 0;
  for (int i = 0; i < batch; ++i) {
    const int64_t pages = (int64_t)indptr[i + 1] - indptr[i];
    if (pages < 0 || keep[i] < 0 || (recent && recent[i] < 0)) return -1;
    if (pages > 0 && (last_page_len[i] < 1 || last_page_len[i] > kPageSize)) return -1;
    const int64_t len = pages > 0 ? (pages - 1) * kPageSize + last_page_len[i] : 0;
    if (len > std::numeric_limits<int32_t>::max() - kPageSize) return -1;
    if (len <= keep[i]) continue;
    if (out)
      out[units] = EvictUnit{indptr[i], (int32_t)len, keep[i],
                             recent ? std::min(recent[i], keep[i]) : 0, *tokens * heads, {0, 0}};
    ++units;
    *tokens += keep[i];
    *longest = std::max(*longest, len);
  }
  return units;
}

EvictLayout evict_layout(int64_t units, int64_t tokens, int heads) {
  EvictLayout L;
  L.units = kAlign;
  L.lists = align_up(L.units + sizeof(EvictUnit) * (size_t)units);
  L.total = align_up(L.lists + 4 * (size_t)tokens * heads);
  return L;
}

}  // namespace
}  // namespace fadecode

using namespace fadecode;

struct fa_evict_plan_s {
  int device = 0;
  int hkv = 0, row_bytes = 0;
  fa_dtype kv_dtype = FA_DTYPE_BF16;
  const int32_t* indices = nullptr;
  uint8_t* ws = nullptr;
  EvictLayout layout{};
  int64_t units = 0;
  int cluster = 1, buffer = kBuffer, threads = kThreads;
  int shared = evict_shared<kRanks>();
  const void* kernel = reinterpret_cast<const void*>(&fa_evict_kernel<kThreads, kRanks>);
};

extern "C" {

size_t fa_evict_workspace_size(int batch, int64_t total_kept, int num_kv_heads) {
  if (batch < 0 || total_kept < 0 || num_kv_heads <= 0 ||
      total_kept > (int64_t)1 << 40)
    return 0;
  return evict_layout(batch, total_kept, num_kv_heads).total;
}

int fa_evict_plan(const int32_t* indptr_host, const int32_t* indices_dev,
                  const int32_t* last_page_len_host, const int32_t* keep_host,
                  const int32_t* recent_host, int batch, int num_kv_heads, int head_dim,
                  int page_size, fa_dtype kv_dtype, void* workspace_dev, size_t workspace_bytes,
                  void* cuda_stream, fa_evict_plan_t* out_plan) {
  if (!out_plan) return FA_ERR_INVALID_ARG;
  *out_plan = nullptr;
  if (!indptr_host || batch < 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 ||
      (batch > 0 && (!last_page_len_host || !keep_host)) || !workspace_dev ||
      reinterpret_cast<uintptr_t>(workspace_dev) % kAlign)
    return FA_ERR_INVALID_ARG;
  const int es = kv_dtype == FA_DTYPE_F32                                 ? 4
                 : kv_dtype == FA_DTYPE_BF16 || kv_dtype == FA_DTYPE_F16 ? 2
                 : kv_dtype == FA_DTYPE_E4M3                             ? 1
                                                                          : 0;
  if (page_size != kPageSize || (head_dim != 64 && head_dim != 128) || es == 0)
    return FA_ERR_UNSUPPORTED;
  if (indptr_host[0] != 0 || (indptr_host[batch] > 0 && !indices_dev)) return FA_ERR_INVALID_ARG;
  int64_t tokens = 0, longest = 0;
  const int64_t units = make_units(indptr_host, last_page_len_host, keep_host, recent_host, batch,
                                   num_kv_heads, nullptr, &tokens, &longest);
  if (units < 0) return FA_ERR_INVALID_ARG;
  const EvictLayout L = evict_layout(units, tokens, num_kv_heads);
  if (L.total > workspace_bytes) return FA_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  // as many CTAs to a (request, kv head) as fill the SMs four times, none with
  // under a thousand tokens
  int cluster = 1;
  while (cluster < kMostCtas && units * num_kv_heads * cluster * 2 <= 4 * (int64_t)sms &&
         longest >= 1024 * 2 * (int64_t)cluster)
    cluster *= 2;
  if (units * num_kv_heads * cluster > std::numeric_limits<int32_t>::max())
    return FA_ERR_UNSUPPORTED;
  try {
    std::vector<uint8_t> meta(L.lists, 0);
    make_units(indptr_host, last_page_len_host, keep_host, recent_host, batch, num_kv_heads,
               reinterpret_cast<EvictUnit*>(meta.data() + L.units), &tokens, &longest);
    fa_evict_plan_s* plan = new fa_evict_plan_s();
    plan->device = dev;
    plan->hkv = num_kv_heads;
    plan->row_bytes = head_dim * es;
    plan->kv_dtype = kv_dtype;
    plan->indices = indices_dev;
    plan->ws = static_cast<uint8_t*>(workspace_dev);
    plan->layout = L;
    plan->units = units;
    plan->cluster = cluster;
    if (units * num_kv_heads * cluster <= sms) {
      plan->buffer = kBigBuffer;
      plan->threads = kManyThreads;
      plan->shared = evict_shared<kManyRanks>();
      plan->kernel = reinterpret_cast<const void*>(&fa_evict_kernel<kManyThreads, kManyRanks>);
    }
    if (cudaFuncSetAttribute(plan->kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             plan->shared + plan->buffer) !=
            cudaSuccess ||
        upload_async(plan->ws, meta.data(), meta.size(),
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

int fa_evict_run(fa_evict_plan_t plan, void* paged_kv, int64_t num_pages, float* weights,
                 float* k_scales, float* v_scales, void* cuda_stream) {
  if (!plan) return FA_ERR_INVALID_ARG;
  if (plan->units == 0) return FA_OK;
  if (!paged_kv || !weights || num_pages <= 0 || reinterpret_cast<uintptr_t>(paged_kv) % 16 ||
      reinterpret_cast<uintptr_t>(weights) % 16 || reinterpret_cast<uintptr_t>(k_scales) % 4 ||
      reinterpret_cast<uintptr_t>(v_scales) % 4 || (k_scales == nullptr) != (v_scales == nullptr))
    return FA_ERR_INVALID_ARG;
  if (k_scales && plan->kv_dtype != FA_DTYPE_E4M3) return FA_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev != plan->device) return FA_ERR_INVALID_ARG;
  EvictParams p;
  std::memset(&p, 0, sizeof p);
  p.kv = static_cast<uint8_t*>(paged_kv);
  p.weights = weights;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.indices = plan->indices;
  p.units = reinterpret_cast<const EvictUnit*>(plan->ws + plan->layout.units);
  p.lists = reinterpret_cast<int32_t*>(plan->ws + plan->layout.lists);
  p.err = reinterpret_cast<int*>(plan->ws);
  p.num_pages = num_pages;
  p.hkv = plan->hkv;
  p.row_bytes = plan->row_bytes;
  p.buffer = plan->buffer;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3((unsigned)(plan->units * plan->hkv * plan->cluster));
  cfg.blockDim = dim3((unsigned)plan->threads);
  cfg.dynamicSmemBytes = (size_t)(plan->shared + plan->buffer);
  cfg.stream = static_cast<cudaStream_t>(cuda_stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)plan->cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* args[1] = {&p};
  return cudaLaunchKernelExC(&cfg, plan->kernel, args) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_evict_check(fa_evict_plan_t plan, void* cuda_stream, int* flags) {
  if (!plan || !flags) return FA_ERR_INVALID_ARG;
  int word = 0;
  if (take_word(reinterpret_cast<int*>(plan->ws), &word, static_cast<cudaStream_t>(cuda_stream)) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  *flags = word;
  return word ? FA_ERR_DEVICE_CHECK : FA_OK;
}

int fa_evict_plan_destroy(fa_evict_plan_t plan) {
  delete plan;
  return FA_OK;
}

}  // extern "C"
