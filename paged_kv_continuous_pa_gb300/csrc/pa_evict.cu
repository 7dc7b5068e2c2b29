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

constexpr int kSelectNarrow = 256, kSelectWide = 1024;         // threads of a CTA
constexpr int kSelectSamples = 512;                         // or twice as many
constexpr int kSelectSlots = 32;                            // weights a thread can list
constexpr int kSelectGroups = 512;                          // groups of 128 tokens marked at once
constexpr int kSelectBinBits = 11;
constexpr int kSelectBins = 1 << kSelectBinBits;
constexpr int kSelectBatch = 4;                             // groups a warp loads at once

// The weights in an integer order: a larger weight has a larger key, -0 and +0
// share one, and NaN comes last (0, below -infinity).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_weight(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

template <int THREADS>
struct SelectSmem {
  float list[kSelectSlots][THREADS];  // weights between the two pivots, a column to a thread
  union {
    uint32_t bins[kSelectBins];
    struct {
      // a group's tokens by lane (four consecutive ones each): kept outright, equal to the last weight
      uint32_t above[kSelectGroups][4], equal[kSelectGroups][4];
    };
  };
  uint32_t before[kSelectGroups][2];  // kept tokens and ties before a group
  int pick[3], gathered;
  uint32_t count[2][THREADS / 32][2];
  uint32_t warp_sum[THREADS / 32][2];
  float pivot[2];
  int overflow;
};

// One warp: a key that `want` of the 32 PER samples reach, or a few more.
template <int PER>
__device__ __forceinline__ uint32_t sample_pivot(const float* samples, int want, int lane) {
  uint32_t k[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) k[i] = weight_key(samples[i * 32 + lane]);
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

// kSelectBatch groups of 128 tokens for a warp, `stride` tokens apart, four tokens
// to a lane: x[u][e] is token t0 + u * stride + e (0 behind `len`).  One uniform
// branch around all loads, so that none waits for another.
__device__ __forceinline__ void load_groups(const float* w, bool vec, int t0, int stride, int len, float (&x)[kSelectBatch][4]) {
  if (vec && t0 + (kSelectBatch - 1) * stride + 4 <= len) {
#pragma unroll
    for (int u = 0; u < kSelectBatch; ++u) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + t0 + u * stride));
      x[u][0] = v.x, x[u][1] = v.y, x[u][2] = v.z, x[u][3] = v.w;
    }
  } else {
#pragma unroll
    for (int u = 0; u < kSelectBatch; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + u * stride + e;
        x[u][e] = t < len ? __ldg(w + t) : 0.0f;
      }
  }
}

// One CTA per (sequence, kv head).  Of the N tokens between the protected ones
// the m with the largest weights stay; what has to be known is the last weight
// kept and how many tokens of exactly that weight stay (the lowest indices).
//   1. 512 samples, four to each of 128 evenly spaced places (44 us at 64 x 32768
//      tokens; 512 places, each a memory access of its own, 47.5), give two pivots
//      that enclose the m-th weight (3.5 standard deviations of a sample rank to
//      either side).
//   2. One pass counts the weights from the upper pivot on and lists those between
//      the two (a few in a hundred; no sample is taken where all fit).
//   3. A histogram of the listed keys, over their range, finds the bin of the last
//      one; its few keys are ranked by counting (or it is the next range).
//   4. A second pass (from L2) marks the kept tokens as bits; counts over groups of
//      128 tokens place them, in ascending order, a group to a thread where few
//      stay (2048 of 32768: 45 us, a group to a warp 47), else to a warp (28000 of
//      32768: 65 us against 145).
// Where the pivots miss (the m-th weight outside, or a thread's list too short,
// as a hostile order can bring about) step 3 goes over the weights themselves.
// Bound by the latency of the steps, of which a CTA's are in a row: 64 x 8 rows of
// 32768 take 45 us (67 MB read from memory and again from L2: 1.5 TB/s), a third of
// it the first pass, a quarter the second, a fifth the samples; 1024 threads to a
// CTA bring long rows' passes down (16 x 8 rows of 131072: 166 to 43 us).
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int WARPS = THREADS / 32;
  constexpr int ALL = kSelectSlots * THREADS;  // that many competing tokens need no sample
  extern __shared__ __align__(16) unsigned char select_smem[];
  SelectSmem<THREADS>& sm = *reinterpret_cast<SelectSmem<THREADS>*>(select_smem);
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
    for (int j = tid; j < p.budget; j += THREADS) keep[j] = (!bad && j < len) ? j : -1;
    return;
  }
  const float* w = p.mass + (static_cast<size_t>(seq) * p.Hkv + h) * p.max_tokens;
  const bool vec = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
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
    for (int k = 0; k < WARPS; ++k) {
      x += sm.count[turn][k][0];
      y += sm.count[turn][k][1];
    }
    return make_uint2(x, y);
  };
  // kept: keys above `last`, and of the `equals` tokens (0: not counted) of exactly it the first `ties`
  uint32_t last = 0xffffffffu, ties = 0u, equals = 0u;
  if (m > 0) {
    float low = -INFINITY, high = INFINITY;
    if (N > ALL) {
      float* samples = sm.list[0];
      // ranks to either side of the m-th weight's among s samples
      auto margin = [&](int s) {
        const float share = static_cast<float>(m) / N;
        return 3.5f * sqrtf(s * share * (1.0f - share)) + 2.0f;
      };
      // a thread lists 2 margin / samples of its N / THREADS weights: twice the samples where that would come near the
      // room it has (budgets in the middle, long rows)
      const bool twice = 2.0f * margin(kSelectSamples) * N > 0.375f * kSelectSlots * kSelectSamples * THREADS;
      const int count = twice ? 2 * kSelectSamples : kSelectSamples;
      for (int k = tid; k < count; k += THREADS) {
        // four samples, four tokens apart, to a place: N > 2^13, so the last place is at least 16 tokens from b
        const int at = static_cast<int>((static_cast<long long>(2 * (k / 4) + 1) * N) / (count / 2));
        samples[k] = __ldg(w + a + at + k % 4 * 4);
      }
      __syncthreads();
      if (warp < 2) {
        const float rank = static_cast<float>(m) * count / N, off = margin(count);
        const int want = static_cast<int>(warp == 0 ? rank - off : rank + off + 1.0f);
        uint32_t pivot = 0u;
        if (want >= 1 && want <= count)
          pivot = twice ? sample_pivot<2 * kSelectSamples / 32>(samples, want, lane) : sample_pivot<kSelectSamples / 32>(samples, want, lane);
        // no pivot, or a NaN: every number
        if (lane == 0) sm.pivot[warp] = pivot == 0u ? (warp == 0 ? INFINITY : -INFINITY) : key_weight(pivot);
      }
      __syncthreads();
      high = sm.pivot[0];
      low = sm.pivot[1];
    }
    if (tid == 0) sm.overflow = 0;
    __syncthreads();
    uint32_t from_high = 0u;
    int listed = 0;  // of this thread
    constexpr int STRIDE = WARPS * 128;
    // four comparisons and a store in predicates, no branch: a weight between the pivots goes to the next
    // slot, or the last one over and over (which `overflow` reports)
    auto list4 = [&](const float(&x)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        from_high += x[e] >= high;
        const bool in = x[e] > low && x[e] < high;
        if (in) sm.list[min(listed, kSelectSlots - 1)][tid] = x[e];
        listed += in;
      }
    };
    // a batch's loads are on their way while the one before is listed
    auto batch = [&](int g0, const float(&x)[kSelectBatch][4], float(&next)[kSelectBatch][4]) {
      const int t0 = g0 + warp * 128 + lane * 4, ahead = g0 + kSelectBatch * STRIDE;
      if (ahead < b) load_groups(w, vec, t0 + kSelectBatch * STRIDE, STRIDE, b, next);
      if (g0 >= a && ahead <= b) {
#pragma unroll
        for (int u = 0; u < kSelectBatch; ++u) list4(x[u]);
      } else {
#pragma unroll
        for (int u = 0; u < kSelectBatch; ++u) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t0 + u * STRIDE + e;
            y[e] = t >= a && t < b ? x[u][e] : NAN;  // NaN: in no comparison
          }
          list4(y);
        }
      }
    };
    const int g_first = a / 128 * 128;
    float x[kSelectBatch][4], y[kSelectBatch][4];
    load_groups(w, vec, g_first + warp * 128 + lane * 4, STRIDE, b, x);
    for (int g0 = g_first; g0 < b; g0 += 2 * kSelectBatch * STRIDE) {
      batch(g0, x, y);
      if (g0 + kSelectBatch * STRIDE < b) batch(g0 + kSelectBatch * STRIDE, y, x);
    }
    if (listed > kSelectSlots) sm.overflow = 1;
    const uint2 s = sum2(from_high, listed);
    const int between = static_cast<int>(s.y), need = m - static_cast<int>(s.x);  // of the weights below `high`
    bool found = !sm.overflow && need > 0 && low < high;
    bool at_low = false;
    if (found && need > between) {
      // weights equal to `low` come next (many equal ones, or -infinity), then, behind -infinity, NaNs
      uint32_t same = 0u;
      for (int t = a + tid; t < b; t += THREADS) same += __ldg(w + t) == low;
      const int n = static_cast<int>(sum2(same, 0u).x);
      at_low = need <= between + n || low == -INFINITY;
      if (at_low) {
        last = need <= between + n ? weight_key(low) : 0u;
        ties = need <= between + n ? need - between : need - between - n;
      } else {
        found = false;
      }
    }
    if (!at_low) {
      // the last key kept lies in [lo, hi): `ahead` keys (fewer than `want`) reach hi, `want` or more reach lo; of
      // the listed weights, or (the pivots missed) of all
      uint32_t lo = found ? weight_key(low) : 0u, hi = found ? weight_key(high) : 0xffffffffu;
      const int want = found ? need : m;
      int ahead = 0;
      auto each_key = [&](auto f) {
        if (found)
          for (int e = 0; e < listed; ++e) f(weight_key(sm.list[e][tid]));
        else
          for (int t = a + tid; t < b; t += THREADS) f(weight_key(__ldg(w + t)));
      };
      for (bool more = true; more;) {
        // a histogram of the range's keys, and the bin that holds the last one
        const int shift = max(0, 32 - __clz(hi - 1u - lo) - kSelectBinBits);
        __syncthreads();
        for (int k = tid; k < kSelectBins; k += THREADS) sm.bins[k] = 0u;
        if (tid == 0) sm.gathered = 0;
        __syncthreads();
        each_key([&](uint32_t key) {
          if (key >= lo && key < hi) atomicAdd(&sm.bins[(key - lo) >> shift], 1u);
        });
        __syncthreads();
        constexpr int PER = kSelectBins / THREADS;  // a thread's bins, from the top down
        uint32_t n[PER], sum = 0u;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          n[k] = sm.bins[kSelectBins - 1 - (tid * PER + k)];
          sum += n[k];
        }
        uint32_t upto = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        if (lane == 31) sm.warp_sum[warp][0] = upto;
        __syncthreads();
        int before = ahead + static_cast<int>(upto - sum);
#pragma unroll
        for (int k = 0; k < WARPS; ++k)
          if (k < warp) before += static_cast<int>(sm.warp_sum[k][0]);
        if (before < want && before + static_cast<int>(sum) >= want) {
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            if (before < want && before + static_cast<int>(n[k]) >= want) {
              sm.pick[0] = kSelectBins - 1 - (tid * PER + k);
              sm.pick[1] = before;
              sm.pick[2] = static_cast<int>(n[k]);
              break;
            }
            before += static_cast<int>(n[k]);
          }
        }
        __syncthreads();
        lo += static_cast<uint32_t>(sm.pick[0]) << shift;
        if (hi - lo > (1u << shift)) hi = lo + (1u << shift);
        ahead = sm.pick[1];
        const int held = sm.pick[2];  // keys in [lo, hi)
        if (hi - lo == 1u) {
          last = lo;
          ties = want - ahead;
          equals = held;
          more = false;
        } else if (held <= 32) {
          // few enough to rank by counting, in every warp
          each_key([&](uint32_t key) {
            // (the bins are read: room for 32, which weights that change during the call could pass)
            if (key >= lo && key < hi) sm.bins[min(atomicAdd(&sm.gathered, 1), 32)] = key;
          });
          __syncthreads();
          const uint32_t key = lane < held ? sm.bins[lane] : 0u;
          int above = 0, same = 0;
          for (int k = 0; k < held; ++k) {
            const uint32_t other = __shfl_sync(0xffffffffu, key, k);
            above += other > key;
            same += other == key;
          }
          const bool mine = lane < held && ahead + above < want && ahead + above + same >= want;
          const int who = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
          last = __shfl_sync(0xffffffffu, key, who);
          ties = want - ahead - __shfl_sync(0xffffffffu, above, who);
          equals = __shfl_sync(0xffffffffu, same, who);
          more = false;
        }
      }
    }
  }
  // ---- marks and places, kSelectGroups groups of 128 tokens at a time.  Kept: weights from `from` on, and the
  // first `ties` equal to `edge`.  The key 0 is the NaNs': every number stays, and `ties` of them; no weight has
  // the key 0xffffffff: none stays.  (The number behind an edge has the next key; behind infinity comes a NaN,
  // which nothing reaches.)
  const bool numbers = last == 0u, none = last == 0xffffffffu;
  const bool whole = !numbers && equals > 0u && ties == equals;  // every token of the last weight stays
  if (whole) ties = 0u;
  const float edge = numbers || none ? NAN : key_weight(last);
  const float from = numbers || none ? NAN : key_weight(whole ? last : last + 1u);
  uint32_t kept_base = 0u, tie_base = 0u;
  for (int c0 = 0; c0 < len; c0 += kSelectGroups * 128) {
    const int groups = min(kSelectGroups, (len - c0 + 127) / 128);
    __syncthreads();
    auto mark = [&](int g0, const float(&x)[kSelectBatch][4], float(&next)[kSelectBatch][4]) {
      const int t0 = c0 + g0 * 128 + lane * 4, ahead = g0 + kSelectBatch * WARPS;
      if (ahead < groups) load_groups(w, vec, c0 + ahead * 128 + lane * 4, WARPS * 128, len, next);
#pragma unroll
      for (int u = 0; u < kSelectBatch; ++u) {
        const int g = g0 + u * WARPS, t = t0 + u * WARPS * 128;
        uint32_t gt[4], eq[4] = {0u, 0u, 0u, 0u};
        if (c0 + g * 128 >= a && c0 + g * 128 + 128 <= b && !numbers) {  // the whole group competes
#pragma unroll
          for (int e = 0; e < 4; ++e) gt[e] = __ballot_sync(0xffffffffu, x[u][e] >= from);
          if (ties > 0u) {
#pragma unroll
            for (int e = 0; e < 4; ++e) eq[e] = __ballot_sync(0xffffffffu, x[u][e] == edge);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool competes = t + e >= a && t + e < b;
            const bool more = numbers ? x[u][e] == x[u][e] : x[u][e] >= from;
            const bool same = numbers ? x[u][e] != x[u][e] : x[u][e] == edge;
            gt[e] = __ballot_sync(0xffffffffu, t + e < len && (!competes || more));
            eq[e] = __ballot_sync(0xffffffffu, competes && same && ties > 0u);
          }
        }
        if (lane == 0 && g < groups) {
          *reinterpret_cast<uint4*>(sm.above[g]) = make_uint4(gt[0], gt[1], gt[2], gt[3]);
          *reinterpret_cast<uint4*>(sm.equal[g]) = make_uint4(eq[0], eq[1], eq[2], eq[3]);
        }
      }
    };
    float x[kSelectBatch][4], y[kSelectBatch][4];
    if (warp < groups) load_groups(w, vec, c0 + warp * 128 + lane * 4, WARPS * 128, len, x);
    for (int g0 = warp; g0 < groups; g0 += 2 * kSelectBatch * WARPS) {
      mark(g0, x, y);
      if (g0 + kSelectBatch * WARPS < groups) mark(g0 + kSelectBatch * WARPS, y, x);
    }
    __syncthreads();
    // kept tokens and ties before each group: PER groups to a thread
    constexpr int PER = (kSelectGroups + THREADS - 1) / THREADS;
    uint32_t ng[PER], ne[PER], sg = 0u, se = 0u;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int g = tid * PER + k;
      ng[k] = ne[k] = 0u;
      if (g < groups) {
        const uint4 x = *reinterpret_cast<const uint4*>(sm.above[g]), y = *reinterpret_cast<const uint4*>(sm.equal[g]);
        ng[k] = __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w);
        ne[k] = __popc(y.x) + __popc(y.y) + __popc(y.z) + __popc(y.w);
      }
      sg += ng[k];
      se += ne[k];
    }
    uint32_t ig = sg, ie = se;  // inclusive over the warp, then the warps before
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
    uint32_t all_g = 0u, all_e = 0u, pg = ig - sg, pe = ie - se;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const uint32_t x = sm.warp_sum[k][0], y = sm.warp_sum[k][1];
      if (k < warp) pg += x, pe += y;
      all_g += x;
      all_e += y;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int g = tid * PER + k;
      if (g < groups) {
        sm.before[g][0] = kept_base + pg + min(tie_base + pe, ties) - min(tie_base, ties);
        sm.before[g][1] = tie_base + pe;
      }
      pg += ng[k];
      pe += ne[k];
    }
    const uint32_t kept_now = all_g + min(tie_base + all_e, ties) - min(tie_base, ties);
    kept_base += kept_now;
    tie_base += all_e;
    // no more than the budget is marked, unless the weights change between the passes: then nothing is written behind it
    if (kept_base > static_cast<uint32_t>(p.budget)) return;
    __syncthreads();
    if (kept_now > static_cast<uint32_t>(groups) * 16) {
      // many stay: a group to a warp, four tokens to a lane, whose stores lie together
      const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
      for (int g = warp; g < groups; g += WARPS) {
        const uint4 x = *reinterpret_cast<const uint4*>(sm.above[g]);
        uint32_t keep_bits = ((x.x >> lane) & 1u) | ((x.y >> lane) & 1u) << 1 | ((x.z >> lane) & 1u) << 2 | ((x.w >> lane) & 1u) << 3;
        uint32_t at = sm.before[g][0] + __popc(x.x & below) + __popc(x.y & below) + __popc(x.z & below) + __popc(x.w & below);
        if (ties > 0u) {
          const uint4 y = *reinterpret_cast<const uint4*>(sm.equal[g]);
          const uint32_t tie0 = sm.before[g][1];
          uint32_t tie = tie0 + __popc(y.x & below) + __popc(y.y & below) + __popc(y.z & below) + __popc(y.w & below);
          at += min(tie, ties) - min(tie0, ties);  // ties of the lanes before that stayed
          const uint32_t eq[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t same = (eq[e] >> lane) & 1u;
            if (same && tie < ties) keep_bits |= 1u << e;
            tie += same;
          }
        }
        const int t = c0 + g * 128 + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((keep_bits >> e) & 1u) keep[at++] = t + e;
      }
      continue;
    }
    // few stay: a group to a thread, which goes over the lanes that marked something (four tokens a step)
    for (int g = tid; g < groups; g += THREADS) {
      const uint4 x = *reinterpret_cast<const uint4*>(sm.above[g]);
      uint4 y = make_uint4(0u, 0u, 0u, 0u);
      int32_t* out = keep + sm.before[g][0];
      uint32_t left = 0u;  // ties that may still stay
      if (ties > sm.before[g][1]) {
        left = ties - sm.before[g][1];
        y = *reinterpret_cast<const uint4*>(sm.equal[g]);
      }
      for (uint32_t any = x.x | x.y | x.z | x.w | y.x | y.y | y.z | y.w; any != 0u; any &= any - 1u) {
        const int l = __ffs(any) - 1, t = c0 + g * 128 + l * 4;
        const uint32_t kept[4] = {x.x, x.y, x.z, x.w}, tied[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bool stays = (kept[e] >> l) & 1u;
          if (left > 0u && ((tied[e] >> l) & 1u)) {
            stays = true;
            --left;
          }
          if (stays) *out++ = t + e;
        }
      }
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
  int32_t stripes;  // CTAs that share a (sequence, kv head, K | V), a column of 16-byte pieces each
};

constexpr int kCompactThreads = 256;
constexpr int kCompactUnroll = 4;
constexpr int kCompactCtas = 304;
constexpr int kCompactBlock = 1024;  // kept tokens looked up at once

// keep[j] if it is a token of the sequence above the one before it and not below
// its own place, else -1 after recording an error.  Moving in place relies on both:
// an ascending list has keep[j] >= j throughout, but behind a step back a neighbour's
// comparison holds again while the tokens' slots may have been overwritten.
__device__ __forceinline__ int kept_token(const CompactParams& p, const int32_t* keep, int j, int len) {
  const int t = __ldg(keep + j), before = j > 0 ? __ldg(keep + j - 1) : -1;
  if (t >= j && t < len && t > before) return t;
  record_error(p.status, ST_OUT_OF_RANGE);
  return -1;
}

// 16 bytes that another thread of the CTA may overwrite later: an ordinary load
// (never through the read-only path), not kept in L1.
__device__ __forceinline__ uint4 load_piece(const unsigned char* a) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(a)
               : "memory");
  return v;
}

// One CTA per (sequence, kv head, K | V, stripe), and one per (sequence, kv head)
// for the weights.  The kept tokens move in order, a tile at a time: every thread
// loads its pieces of the tile, the CTA meets, and the tile is stored.  The
// j-th comes from a token t >= j (`kept_token`): a tile's stores reach only
// slots that earlier tiles and this one read, never a later tile's, and the move
// is safe in place -- also with the next tile's loads on their way before the
// stores.  Stripes of a row are independent of one another; they fill the GPU
// where the sequences alone would not.
// Bound by the read and the write of the kept rows: 1024 of up to 8192 tokens of 64
// sequences x 8 heads (bf16, D 128: 556 MB) take 98 us, 5.7 TB/s of scattered
// 256-byte rows.  Four CTAs to an SM with four pieces to a thread; more pieces or
// fewer CTAs took 98 to 125.  Stripes, until there are two CTAs to an SM: one
// sequence of 8192 kept tokens 39 us, without them 92; 16 of 2048 47 us, without
// 55, until there are four CTAs 54.
__global__ void __launch_bounds__(kCompactThreads, 4) compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ long long from[kCompactBlock], to[kCompactBlock];  // byte offsets of a kept token's row (from -1: not moved)
  const int per_head = 2 * p.stripes;
  const int rows_ctas = p.n * p.Hkv * per_head, tid = threadIdx.x;
  const bool weights = static_cast<int>(blockIdx.x) >= rows_ctas;
  const int unit = weights ? blockIdx.x - rows_ctas : blockIdx.x / per_head;
  const int op = blockIdx.x / p.stripes % 2, stripe = blockIdx.x % p.stripes;  // of K and V
  const int i = unit / p.Hkv, h = unit % p.Hkv;
  const int src = __ldg(p.seq_ids + i), dst = p.dst_seq_ids != nullptr ? __ldg(p.dst_seq_ids + i) : src;
  const int len = __ldg(p.lengths + i);
  if (src < 0 || src >= p.num_seqs || dst < 0 || dst >= p.num_seqs || len < 0 || len > p.max_blocks * p.P) {
    if (tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
    return;
  }
  const int count = min(len, p.budget);
  const int32_t* keep = p.keep + static_cast<size_t>(unit) * p.budget;
  if (weights) {
    const size_t T = static_cast<size_t>(p.max_blocks) * p.P;
    const float* from_w = p.mass + (static_cast<size_t>(src) * p.Hkv + h) * T;
    float* to_w = p.mass + (static_cast<size_t>(dst) * p.Hkv + h) * T;
    for (int j0 = 0; j0 < count; j0 += kCompactThreads * kCompactUnroll) {
      float v[kCompactUnroll];
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int j = j0 + u * kCompactThreads + tid;
        const int t = j < count ? kept_token(p, keep, j, len) : -1;
        v[u] = t >= 0 ? from_w[t] : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int j = j0 + u * kCompactThreads + tid;
        if (j < count) to_w[j] = v[u];
      }
    }
    for (int j = count + tid; j < len; j += kCompactThreads) to_w[j] = 0.0f;
    return;
  }
  const int32_t* from_table = p.block_tables + static_cast<size_t>(src) * p.max_blocks;
  const int32_t* to_table = p.block_tables + static_cast<size_t>(dst) * p.max_blocks;
  unsigned char* pool = p.pool[op];
  const int lg_p = 31 - __clz(p.P);
  const int pieces = p.row_bytes / 16 / p.stripes, rows = kCompactThreads / pieces;  // rows moved side by side
  const int r = tid / pieces, offset = (stripe * pieces + tid % pieces) * 16;
  const unsigned char* base = pool + offset;
  auto row_offset = [&](int page, int t) {
    return static_cast<long long>((((static_cast<size_t>(page) * p.Hkv + h) << lg_p) + (t & (p.P - 1))) * p.row_bytes);
  };
  for (int b0 = 0; b0 < count; b0 += kCompactBlock) {
    const int n = min(count - b0, kCompactBlock);
    __syncthreads();
    for (int k = tid; k < n; k += kCompactThreads) {
      const int j = b0 + k, t = kept_token(p, keep, j, len);
      const int page = t >= 0 ? __ldg(from_table + (t >> lg_p)) : -1;
      const int to_page = __ldg(to_table + (j >> lg_p));
      bool moves = page >= 0 && page < p.num_pages && to_page >= 0 && to_page < p.num_pages;
      if (t >= 0 && !moves) record_error(p.status, ST_OUT_OF_RANGE);
      if (t == j && src == dst) moves = false;  // in its place already
      from[k] = moves ? row_offset(page, t) : -1;
      to[k] = moves ? row_offset(to_page, j) : 0;
    }
    __syncthreads();
    const int step = rows * kCompactUnroll;
    uint4 now[kCompactUnroll], next[kCompactUnroll];
    auto load = [&](int k0, uint4(&v)[kCompactUnroll]) {
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int k = k0 + u * rows;
        v[u] = load_piece(base + (k < n ? max(from[k], 0ll) : 0ll));  // (a row that is not moved: any valid address)
      }
    };
    load(r, now);
    for (int k0 = r; k0 - r < n; k0 += step) {
      if (k0 - r + step < n) load(k0 + step, next);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) {
        const int k = k0 + u * rows;
        if (k < n && from[k] >= 0) *reinterpret_cast<uint4*>(const_cast<unsigned char*>(base) + to[k]) = now[u];
      }
#pragma unroll
      for (int u = 0; u < kCompactUnroll; ++u) now[u] = next[u];
    }
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
  // (a row's CTAs read its slot and length at different times)
  if (kept_lengths != nullptr && (kept_lengths == lengths || kept_lengths == seq_ids))
    return fail(PA_ERR_INVALID_ARG, "kept_lengths may not be lengths or seq_ids");
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
  // Long rows take CTAs of 1024 threads, shorter ones where there is at most one to an SM.  Measured, us narrow / wide
  // (8 kv heads, 2048 kept): 16 x 32768 22.8 / 27.0, 16 x 49152 28.2 / 24.9, 64 x 65536 74 / 108, 64 x 131072 275 / 156.
  const bool wide = max_tokens > (units <= 152 ? 1 << 15 : 1 << 16);
  static std::atomic<unsigned long long> done_wide{0}, done{0};
  constexpr size_t wide_smem = sizeof(pa::SelectSmem<pa::kSelectWide>), smem = sizeof(pa::SelectSmem<pa::kSelectNarrow>);
  cudaError_t e = wide ? pa::allow_dynamic_smem(pa::select_kernel<pa::kSelectWide>, done_wide, wide_smem)
                       : pa::allow_dynamic_smem(pa::select_kernel<pa::kSelectNarrow>, done, smem);
  if (e != cudaSuccess) return cuda_fail(e, "select shared memory");
  const dim3 grid(static_cast<unsigned>(units));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = wide ? pa::launch_kernel(pa::select_kernel<pa::kSelectWide>, grid, dim3(pa::kSelectWide), wide_smem, s, false, p)
           : pa::launch_kernel(pa::select_kernel<pa::kSelectNarrow>, grid, dim3(pa::kSelectNarrow), smem, s, false, p);
  pa::count_launch();
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
  if (d.kv_dtype == PA_INT4) return fail(PA_ERR_UNSUPPORTED, "compact: a 4-bit pool");
  if (static_cast<int64_t>(max_blocks_per_seq) * d.page_size > (1 << 30))  // (tokens and steps beyond stay int32)
    return fail(PA_ERR_UNSUPPORTED, "a block-table row of %d pages of %d tokens", max_blocks_per_seq, d.page_size);
  if (budget <= 0) return fail(PA_ERR_INVALID_ARG, "budget %d must be positive", budget);
  if (n == 0) return PA_OK;
  if (!seq_ids || !lengths || !keep || !block_tables) return fail(PA_ERR_INVALID_ARG, "compact: a device pointer is NULL");
  const int row_bytes = d.head_dim * static_cast<int>(pa::elt_bytes(d.kv_dtype));
  const int64_t heads = static_cast<int64_t>(n) * d.num_kv_heads;
  // stripes of 64 bytes and more (what a memory access moves) until there are about two CTAs to an SM
  int stripes = 1;
  while (heads * 2 * stripes < pa::kCompactCtas && row_bytes / stripes > 64) stripes *= 2;
  const int64_t units = heads * (2 * stripes + (mass != nullptr ? 1 : 0));
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
  p.row_bytes = row_bytes;
  p.stripes = stripes;
  p.budget = budget;
  pa::compact_kernel<<<static_cast<unsigned>(units), pa::kCompactThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  pa::count_launch();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "compact launch");
}

}  // extern "C"
