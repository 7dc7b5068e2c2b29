// pa_evict.cu -- eviction from the paged cache: pa_evict_select chooses, per
// sequence and kv head, which tokens stay (those with the most accumulated
// attention weight), and pa_evict_compact closes the gaps.
//
// Every kv head keeps its own tokens: a page holds each head's slots apart, so
// the j-th kept token of head 0 and of head 1 may be different tokens of the
// text and still share slot j of the block table's pages.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

// ----------------------------------------------------------------- select --

struct SelectParams {
  const int32_t* seq_ids;
  const int32_t* lengths;
  const float* mass;  // [num_seqs][Hkv][max_tokens]
  int32_t* keep;      // [n][Hkv][budget]
  int32_t* kept_lengths;
  int32_t* status;
  int32_t n, num_seqs, Hkv, max_tokens, budget, keep_first, keep_last;
};

constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectSamples = 512;
constexpr int kSelectList = 512;             // keys a warp's list holds
constexpr int kSelectAll = kSelectList * kSelectWarps;  // that many competing tokens need no sample
constexpr int kSelectWords = 2048;           // 32-token words marked at once

// The weights in an integer order: a larger weight has a larger key, -0 and +0
// share one, and NaN comes last (below -infinity).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelectSmem {
  uint32_t list[kSelectAll];   // per warp: keys between the two pivots
  uint32_t marks[kSelectWords][2];  // per word: tokens above the last key, of exactly the last key; then kept tokens, first place
  uint32_t count[2][kSelectWarps][2];
  uint32_t warp_sum[kSelectWarps][2];
  uint32_t pivot[2];
  int overflow;
};

// One warp: a key that `want` of the samples reach, or a few more.
__device__ __forceinline__ uint32_t sample_pivot(const uint32_t* samples, int want, int lane) {
  constexpr int PER = kSelectSamples / 32;
  uint32_t k[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) k[i] = samples[i * 32 + lane];
  uint32_t lo = 0u, hi = 0xffffffffu;  // as many reach lo, fewer reach hi
  while (hi - lo > 1u) {
    const uint32_t mid = lo + (hi - lo) / 2;
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += k[i] >= mid;
    c = static_cast<int>(__reduce_add_sync(0xffffffffu, c));
    if (c >= want) {
      lo = mid;
      if (c <= want + 2) break;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// One CTA per (sequence, kv head).  Of the N tokens between the protected ones
// the m with the largest keys stay; what has to be known is the last key kept
// and how many tokens of exactly that key stay (the lowest indices).
//   1. 512 samples, evenly spaced, give two pivots that enclose the m-th key
//      (3.5 standard deviations of a sample rank to either side).
//   2. One pass over the weights counts the keys from the upper pivot on and those of
//      exactly the lower one, and lists the keys between the two (a few in a
//      hundred; no sample is taken where all fit).
//   3. Bisection over the list, three pivots a step, finds the last key.
//   4. A second pass (from L2) marks kept tokens as bits, 32 to a word; counts
//      over the words place them, in ascending order.
// Where the pivots miss (the m-th key outside, or a warp's list too short, as a
// hostile order can bring about) step 3 bisects over the weights themselves.
// Bound by the read of the weights and the latency of the steps.
__global__ void __launch_bounds__(kSelectThreads, 5) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ SelectSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const int seq = __ldg(p.seq_ids + i), len = __ldg(p.lengths + i);
  int32_t* keep = p.keep + static_cast<size_t>(blockIdx.x) * p.budget;
  const bool bad = seq < 0 || seq >= p.num_seqs || len < 0 || len > p.max_tokens;
  if (h == 0 && tid == 0) {
    if (bad) record_error(p.status, ST_OUT_OF_RANGE);
    if (p.kept_lengths != nullptr) p.kept_lengths[i] = bad ? 0 : min(len, p.budget);
  }
  if (bad || len <= p.budget) {  // everything stays (or nothing, of a bad row)
    for (int j = tid; j < p.budget; j += kSelectThreads) keep[j] = (!bad && j < len) ? j : -1;
    return;
  }
  const float* w = p.mass + (static_cast<size_t>(seq) * p.Hkv + h) * p.max_tokens;
  const int a = p.keep_first, b = len - p.keep_last, N = b - a;  // tokens [a, b) compete
  const int m = p.budget - p.keep_first - p.keep_last;           // 0 <= m < N
  // sums over the CTA of two counts; alternating buffers, so one barrier a sum
  int turn = 0;
  auto sum2 = [&](uint32_t x, uint32_t y) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    turn ^= 1;
    if (lane == 0) {
      sm.count[turn][warp][0] = x;
      sm.count[turn][warp][1] = y;
    }
    __syncthreads();
    x = y = 0u;
#pragma unroll
    for (int k = 0; k < kSelectWarps; ++k) {
      x += sm.count[turn][k][0];
      y += sm.count[turn][k][1];
    }
    return make_uint2(x, y);
  };
  uint32_t last = 0xffffffffu, ties = 0u;  // kept: keys above `last`, and the first `ties` tokens of exactly it
  if (m > 0) {
    uint32_t low = 0u, high = 0xffffffffu;  // no key is that high
    if (N > kSelectAll) {
      for (int k = tid; k < kSelectSamples; k += kSelectThreads)
        sm.list[k] = weight_key(__ldg(w + a + static_cast<int>((static_cast<long long>(2 * k + 1) * N) / (2 * kSelectSamples))));
      __syncthreads();
      if (warp < 2) {
        const float rank = static_cast<float>(m) * kSelectSamples / N;
        const float off = 3.5f * sqrtf(rank * (1.0f - rank / kSelectSamples)) + 2.0f;
        const int want = static_cast<int>(warp == 0 ? rank - off : rank + off + 1.0f);
        uint32_t pivot = warp == 0 ? 0xffffffffu : 0u;
        if (want >= 1 && want <= kSelectSamples) pivot = sample_pivot(sm.list, want, lane);
        if (lane == 0) sm.pivot[warp] = pivot;
      }
      __syncthreads();
      high = sm.pivot[0];
      low = sm.pivot[1];
    }
    if (tid == 0) sm.overflow = 0;
    __syncthreads();
    uint32_t above = 0u, equal = 0u;
    int listed = 0;  // of this warp
    const uint32_t below = (1u << lane) - 1u;
    uint32_t* mine = sm.list + warp * kSelectList;
    constexpr int UNROLL = 8;
    for (int t0 = a + tid; t0 - tid < b; t0 += UNROLL * kSelectThreads) {
      float x[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int t = t0 + u * kSelectThreads;
        x[u] = t < b ? __ldg(w + t) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const bool in = t0 + u * kSelectThreads < b;
        const uint32_t k = weight_key(x[u]);
        above += in && k >= high;
        equal += in && k == low && k < high;
        const bool between = in && k > low && k < high;
        const uint32_t who = __ballot_sync(0xffffffffu, between);
        if (who != 0u) {
          const int at = listed + __popc(who & below);
          if (between && at < kSelectList) mine[at] = k;
          listed += __popc(who);
        }
      }
    }
    if (lane == 0 && listed > kSelectList) sm.overflow = 1;
    const uint2 s = sum2(above, equal);
    const int between = static_cast<int>(sum2(lane == 0 ? listed : 0, 0u).x);
    const int need = m - static_cast<int>(s.x);  // of the keys below `high`
    const bool found = !sm.overflow && need > 0 && need <= between + static_cast<int>(s.y);
    if (found && need > between) {
      last = low;
      ties = need - between;
    } else {
      // the last key lies between two keys, fewer than `want` tokens reach hi, as many or more reach lo: over the
      // listed keys, or (the pivots missed) over all
      uint32_t lo = found ? low : 0u, hi = found ? high : 0xffffffffu;
      const int want = found ? need : m;
      uint32_t k[kSelectAll / kSelectThreads];
#pragma unroll
      for (int e = 0; e < kSelectAll / kSelectThreads; ++e) k[e] = 0u;
      if (found) {
#pragma unroll
        for (int e = 0; e < kSelectAll / kSelectThreads; ++e) {
          const int at = e * 32 + lane;
          if (at < listed) k[e] = mine[at];
        }
      }
      int reach_hi = 0;
      bool done = false;
      while (hi - lo > 1u && !done) {
        const uint32_t step = (hi - lo) / 4;
        uint32_t q[3] = {lo + step, lo + 2 * step, lo + 3 * step};
        if (step == 0u) q[0] = q[1] = q[2] = lo + 1u;
        uint32_t c[3] = {0u, 0u, 0u};
        if (found) {
#pragma unroll
          for (int e = 0; e < kSelectAll / kSelectThreads; ++e)
#pragma unroll
            for (int z = 0; z < 3; ++z) c[z] += k[e] >= q[z];
        } else {
          for (int t = a + tid; t < b; t += kSelectThreads) {
            const uint32_t key = weight_key(__ldg(w + t));
#pragma unroll
            for (int z = 0; z < 3; ++z) c[z] += key >= q[z];
          }
        }
        // listed keys: sums below 2^16, two to a word
        uint2 r;
        int n[3];
        if (found) {
          r = sum2(c[0] | (c[1] << 16), c[2]);
          n[0] = r.x & 0xffffu, n[1] = r.x >> 16, n[2] = r.y;
        } else {
          r = sum2(c[0], c[1]);
          n[0] = r.x, n[1] = r.y;
          n[2] = sum2(c[2], 0u).x;
        }
#pragma unroll
        for (int z = 2; z >= 0; --z) {
          if (n[z] < want) {
            if (q[z] < hi) hi = q[z], reach_hi = n[z];
          } else if (q[z] > lo) {
            lo = q[z];
            if (n[z] == want) done = true;
          }
        }
      }
      if (done) {
        last = lo - 1u;  // exactly those from lo on
      } else {
        last = lo;
        ties = want - reach_hi;
      }
    }
  }
  // ---- marks and places, kSelectWords words of 32 tokens at a time
  uint32_t sel_base = 0u, eq_base = 0u;
  for (int t0 = 0; t0 < len; t0 += kSelectWords * 32) {
    const int words = min(kSelectWords, (len - t0 + 31) / 32);
    __syncthreads();
    for (int w0 = warp; w0 < words; w0 += 4 * kSelectWarps) {
      float x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + (w0 + u * kSelectWarps) * 32 + lane;
        x[u] = t < len ? __ldg(w + t) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int word = w0 + u * kSelectWarps, t = t0 + word * 32 + lane;
        const uint32_t k = weight_key(x[u]);
        const bool competes = t >= a && t < b;
        const uint32_t gt = __ballot_sync(0xffffffffu, t < len && (!competes || k > last));
        const uint32_t eq = __ballot_sync(0xffffffffu, t < len && competes && k == last && ties > 0u);
        if (lane == 0 && word < words) {
          sm.marks[word][0] = gt;
          sm.marks[word][1] = eq;
        }
      }
    }
    __syncthreads();
    constexpr int PER = kSelectWords / kSelectThreads;
    uint32_t gt[PER], eq[PER], ng = 0u, ne = 0u;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int word = tid * PER + e;
      gt[e] = word < words ? sm.marks[word][0] : 0u;
      eq[e] = word < words ? sm.marks[word][1] : 0u;
      ng += __popc(gt[e]);
      ne += __popc(eq[e]);
    }
    uint32_t ig = ng, ie = ne;  // inclusive over the warp, then the warps before
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, ig, off), y = __shfl_up_sync(0xffffffffu, ie, off);
      if (lane >= off) ig += x, ie += y;
    }
    if (lane == 31) {
      sm.warp_sum[warp][0] = ig;
      sm.warp_sum[warp][1] = ie;
    }
    __syncthreads();
    uint32_t all_g = 0u, all_e = 0u;
    uint32_t pg = ig - ng, pe = ie - ne;
#pragma unroll
    for (int k = 0; k < kSelectWarps; ++k) {
      const uint32_t x = sm.warp_sum[k][0], y = sm.warp_sum[k][1];
      if (k < warp) pg += x, pe += y;
      all_g += x;
      all_e += y;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int word = tid * PER + e;
      // of the ties before this word `ties` at most were kept; of its own, the first of what is left
      const uint32_t before = min(eq_base + pe, ties), left = ties - before;
      uint32_t take = eq[e];
      if (__popc(take) > left) take = left == 0u ? 0u : take & (0xffffffffu >> (31 - __fns(take, 0, left)));
      if (word < words) {
        sm.marks[word][0] = gt[e] | take;
        sm.marks[word][1] = sel_base + pg + before - min(eq_base, ties);
      }
      pg += __popc(gt[e]);
      pe += __popc(eq[e]);
    }
    sel_base += all_g + min(eq_base + all_e, ties) - min(eq_base, ties);
    eq_base += all_e;
    __syncthreads();
    for (int word = warp; word < words; word += kSelectWarps) {
      const uint32_t sel = sm.marks[word][0];
      if ((sel >> lane) & 1u) keep[sm.marks[word][1] + __popc(sel & ((1u << lane) - 1u))] = t0 + word * 32 + lane;
    }
  }
}

// ---------------------------------------------------------------- compact --

struct CompactParams {
  unsigned char* pool[2];  // K, V
  float* mass;             // may be NULL
  const int32_t* seq_ids;
  const int32_t* dst_seq_ids;  // NULL: in place
  const int32_t* lengths;
  const int32_t* keep;
  const int32_t* block_tables;
  int32_t* status;
  int32_t n, num_seqs, max_blocks, num_pages, P, Hkv, row_bytes, budget;
};

constexpr int kCompactThreads = 256;
constexpr int kCompactUnroll = 4;

// The physical page of token t of a sequence, or -1 after recording an error.
__device__ __forceinline__ int page_of(const CompactParams& p, const int32_t* table, int t) {
  const int page = __ldg(table + t / p.P);
  if (page >= 0 && page < p.num_pages) return page;
  record_error(p.status, ST_OUT_OF_RANGE);
  return -1;
}

// keep[j] if it is a token of the sequence above the one before it (the order
// that moving in place relies on), else -1 after recording an error.
__device__ __forceinline__ int kept_token(const CompactParams& p, const int32_t* keep, int j, int len) {
  const int t = __ldg(keep + j), before = j > 0 ? __ldg(keep + j - 1) : -1;
  if (t >= 0 && t < len && t > before) return t;
  record_error(p.status, ST_OUT_OF_RANGE);
  return -1;
}

// One CTA per (sequence, kv head, K | V | weights).  The kept tokens move in
// order, a tile at a time: every thread loads its pieces of the tile, the CTA
// meets, and the tile is stored.  Kept tokens ascend, so the j-th comes from a
// token t >= j: a tile's stores reach only slots that earlier tiles and this
// one read, never a later tile's, and the move is safe in place.
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ CompactParams p) {
  const int operands = p.mass != nullptr ? 3 : 2;
  const int op = blockIdx.x % operands;
  const int unit = blockIdx.x / operands;
  const int i = unit / p.Hkv, h = unit % p.Hkv, tid = threadIdx.x;
  const int src = __ldg(p.seq_ids + i), dst = p.dst_seq_ids != nullptr ? __ldg(p.dst_seq_ids + i) : src;
  const int len = __ldg(p.lengths + i);
  if (src < 0 || src >= p.num_seqs || dst < 0 || dst >= p.num_seqs || len < 0 || len > p.max_blocks * p.P) {
    if (h == 0 && op == 0 && tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
    return;
  }
  const int count = min(len, p.budget);
  const int32_t* keep = p.keep + static_cast<size_t>(unit) * p.budget;
  if (op == 2) {
    const size_t T = static_cast<size_t>(p.max_blocks) * p.P;
    const float* from = p.mass + (static_cast<size_t>(src) * p.Hkv + h) * T;
    float* to = p.mass + (static_cast<size_t>(dst) * p.Hkv + h) * T;
    for (int j0 = 0; j0 < count; j0 += kCompactThreads * kCompactUnroll) {
      float v[kCompactUnroll];
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int j = j0 + u * kCompactThreads + tid;
        const int t = j < count ? kept_token(p, keep, j, len) : -1;
        v[u] = t >= 0 ? from[t] : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int j = j0 + u * kCompactThreads + tid;
        if (j < count) to[j] = v[u];
      }
    }
    for (int j = count + tid; j < len; j += kCompactThreads) to[j] = 0.0f;
    return;
  }
  const int32_t* from_table = p.block_tables + static_cast<size_t>(src) * p.max_blocks;
  const int32_t* to_table = p.block_tables + static_cast<size_t>(dst) * p.max_blocks;
  unsigned char* pool = p.pool[op];
  const int pieces = p.row_bytes / 16, rows = kCompactThreads / pieces;  // rows moved side by side
  const int piece = tid % pieces, r = tid / pieces;
  auto address = [&](int page, int t) {
    return pool + ((static_cast<size_t>(page) * p.Hkv + h) * p.P + t % p.P) * p.row_bytes + piece * 16;
  };
  for (int j0 = 0; j0 < count; j0 += rows * kCompactUnroll) {
    uint4 v[kCompactUnroll];
    unsigned char* to[kCompactUnroll];
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u) {
      const int j = j0 + u * rows + r;
      to[u] = nullptr;
      if (j >= count) continue;
      const int t = kept_token(p, keep, j, len);
      const int page = t >= 0 ? page_of(p, from_table, t) : -1;
      const int to_page = page_of(p, to_table, j);
      if (page < 0 || to_page < 0) continue;
      v[u] = *reinterpret_cast<const uint4*>(address(page, t));
      to[u] = address(to_page, j);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCompactUnroll; ++u)
      if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = v[u];
  }
}

}  // namespace pa

using pa::aligned;
using pa::cuda_fail;
using pa::fail;

extern "C" {

pa_status pa_evict_select(int32_t n, const int32_t* seq_ids, const int32_t* lengths, const float* mass,
                          int32_t num_seqs, int32_t num_kv_heads, int32_t max_tokens, int32_t budget,
                          int32_t keep_first, int32_t keep_last, int32_t* keep, int32_t* kept_lengths,
                          int32_t* status_dev, void* stream) {
  if (n < 0) return fail(PA_ERR_INVALID_ARG, "n %d < 0", n);
  if (num_seqs <= 0 || num_kv_heads <= 0 || max_tokens <= 0)
    return fail(PA_ERR_INVALID_ARG, "num_seqs, num_kv_heads and max_tokens must be positive");
  if (max_tokens > (1 << 30)) return fail(PA_ERR_UNSUPPORTED, "max_tokens %d > 2^30", max_tokens);
  if (budget <= 0) return fail(PA_ERR_INVALID_ARG, "budget %d must be positive", budget);
  if (keep_first < 0 || keep_last < 0 || static_cast<int64_t>(keep_first) + keep_last > budget)
    return fail(PA_ERR_INVALID_ARG, "keep_first %d and keep_last %d must be non-negative and fit in the budget %d",
                keep_first, keep_last, budget);
  if (n == 0) return PA_OK;
  if (!seq_ids || !lengths || !mass || !keep) return fail(PA_ERR_INVALID_ARG, "select: a device pointer is NULL");
  const int64_t units = static_cast<int64_t>(n) * num_kv_heads;
  if (units > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "%lld (sequence, kv head) pairs in one call", (long long)units);
  pa::SelectParams p{};
  p.seq_ids = seq_ids;
  p.lengths = lengths;
  p.mass = mass;
  p.keep = keep;
  p.kept_lengths = kept_lengths;
  p.status = status_dev;
  p.n = n;
  p.num_seqs = num_seqs;
  p.Hkv = num_kv_heads;
  p.max_tokens = max_tokens;
  p.budget = budget;
  p.keep_first = keep_first;
  p.keep_last = keep_last;
  pa::select_kernel<<<static_cast<unsigned>(units), pa::kSelectThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  pa::count_launch();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "select launch");
}

pa_status pa_evict_compact(const pa_pool* pool, int32_t n, const int32_t* seq_ids, const int32_t* dst_seq_ids,
                           const int32_t* lengths, const int32_t* keep, int32_t budget, const int32_t* block_tables,
                           int32_t num_seqs, int32_t max_blocks_per_seq, float* mass, int32_t* status_dev,
                           void* stream) {
  if (pool == nullptr) return fail(PA_ERR_INVALID_ARG, "pool is NULL");
  if (n < 0) return fail(PA_ERR_INVALID_ARG, "n %d < 0", n);
  if (num_seqs <= 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID_ARG, "num_seqs and max_blocks_per_seq must be positive");
  const pa_pool_desc& d = pool->desc;
  if (static_cast<int64_t>(max_blocks_per_seq) * d.page_size > 0x7fffffff)
    return fail(PA_ERR_UNSUPPORTED, "a block-table row of %d pages of %d tokens", max_blocks_per_seq, d.page_size);
  if (budget <= 0) return fail(PA_ERR_INVALID_ARG, "budget %d must be positive", budget);
  if (n == 0) return PA_OK;
  if (!seq_ids || !lengths || !keep || !block_tables) return fail(PA_ERR_INVALID_ARG, "compact: a device pointer is NULL");
  const int64_t units = static_cast<int64_t>(n) * d.num_kv_heads * (mass != nullptr ? 3 : 2);
  if (units > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "%lld units of work in one call", (long long)units);
  pa::CompactParams p{};
  p.pool[0] = static_cast<unsigned char*>(pool->k);
  p.pool[1] = static_cast<unsigned char*>(pool->v);
  p.mass = mass;
  p.seq_ids = seq_ids;
  p.dst_seq_ids = dst_seq_ids;
  p.lengths = lengths;
  p.keep = keep;
  p.block_tables = block_tables;
  p.status = status_dev;
  p.n = n;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.num_pages = d.num_pages;
  p.P = d.page_size;
  p.Hkv = d.num_kv_heads;
  p.row_bytes = d.head_dim * static_cast<int>(pa::elt_bytes(d.kv_dtype));
  p.budget = budget;
  pa::compact_kernel<<<static_cast<unsigned>(units), pa::kCompactThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  pa::count_launch();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "compact launch");
}

}  // extern "C"
