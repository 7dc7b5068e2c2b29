// pa_beam.cu -- beam search around the paged cache: pa_beam_select chooses the
// best continuations over beams x vocabulary from raw logits, and
// pa_beam_reorder gives each beam its parent's cache.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

constexpr int kMaxBeams = 32;
constexpr int kMaxBeamOut = 64;

// ----------------------------------------------------------------- select --

struct BeamParams {
  const void* logits;
  int64_t row_stride;
  const float* scores;
  const int32_t* finished;  // may be NULL
  int32_t* parents;
  int32_t* tokens;
  float* out_scores;
  // workspace, per segment of a row: its best (logit, token) keys, best first (0: none), its sum of
  // exponentials and the maximum they are relative to
  uint64_t* segment_keys;  // [rows][segments][n_out]
  float* segment_sum;      // [rows][segments]
  float* segment_max;      // [rows][segments]
  int32_t groups, beams, vocab, segments, n_out, end_token;
  int32_t merge_warps;  // warps of the merge that have room for a row's keys
};

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamVecs = 8;                                        // 16-byte vectors a thread holds
constexpr int kBeamChunkBytes = kBeamThreads * kBeamVecs * 16;      // of a row, held at once
constexpr int kBeamSegment = 4;                                     // chunks of a CTA's part of a row
constexpr int kMaxVocab = 1 << 20;
static_assert(kMaxVocab <= 32 * kBeamSegment * kBeamChunkBytes / 4, "a row has at most 32 segments");
constexpr size_t kBeamListBytes = 32 * 1024;  // keys the merge holds at once (a row has 32 segments at most, n_out 64 of each)
constexpr size_t kBeamMaxSmem = 96 * 1024;

__host__ __device__ constexpr int beam_chunk(bool bf16) { return kBeamChunkBytes / (bf16 ? 2 : 4); }

// A logit and its token as one integer: larger logits first, then lower
// tokens; -0 and +0 are one value.  NaN and -infinity are never asked for (0).
__device__ __forceinline__ uint32_t logit_order(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t cand_key(uint32_t order, int token) {
  return (static_cast<uint64_t>(order) << 32) | (0xffffffffu - static_cast<uint32_t>(token));
}
__device__ __forceinline__ float cand_logit(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int cand_token(uint64_t key) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)); }

// 16 bytes of a row from an address `off` bytes behind a 16-byte boundary, shifted
// together from the two aligned vectors that hold them, the second read only
// where it holds an element of the row (left: the row's bytes from here on), so
// that no aligned 16 bytes without one is touched.
__device__ __forceinline__ uint4 load_row_vec(const unsigned char* src, int off, int64_t left) {
  const uint4* at = reinterpret_cast<const uint4*>(src - off);
  const uint4 a = __ldcs(at);
  uint4 b = make_uint4(0u, 0u, 0u, 0u);
  if (left > 16 - off) b = __ldcs(at + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int sh = 8 * (off & 3);
  uint32_t r[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int s = 0; s < 4; ++s)  // the same word offset for the whole row: a uniform choice
    if (off / 4 == s) {
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = __funnelshift_r(w[s + k], s + k + 1 < 8 ? w[s + k + 1] : 0u, sh);
    }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Element e of a held vector.
template <bool BF16>
__device__ __forceinline__ float vec_logit(const uint4& v, int e) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (BF16) return (e & 1) ? bf16hi(w[e / 2]) : bf16lo(w[e / 2]);
  return __uint_as_float(w[e]);
}

// A held vector whose elements from `left` on are behind the row: those become -infinity.
template <bool BF16>
__device__ __forceinline__ uint4 cut_vec(uint4 v, int left) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      if (2 * k >= left) w[k] = (w[k] & 0xffff0000u) | 0xff80u;
      if (2 * k + 1 >= left) w[k] = (w[k] & 0x0000ffffu) | 0xff800000u;
    } else {
      if (k >= left) w[k] = 0xff800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The largest element of a vector (NaN only if nothing else is there).
template <bool BF16>
__device__ __forceinline__ float vec_max(const uint4& v) {
  if constexpr (BF16) {
    const uint32_t m = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
    return fmaxf(bf16lo(m), bf16hi(m));
  } else {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
}

// One warp: a bound that at least `want` of the (distinct, or zero) keys list[0, n)
// reach, and no more than 2 * want; 1 where fewer than `want` reach lo.
__device__ __forceinline__ uint64_t bound_keys(const uint64_t* list, int n, int want, uint64_t lo, uint64_t hi, int lane) {
  auto reach = [&](uint64_t bound) {
    int c = 0;
    for (int i = lane; i < n; i += 32) c += list[i] >= bound;
    return static_cast<int>(__reduce_add_sync(0xffffffffu, c));
  };
  int at_lo = reach(lo);
  if (at_lo < want) return 1ull;
  while (at_lo > 2 * want && hi - lo > 1ull) {  // reach(lo) >= want > reach(hi)
    const uint64_t mid = lo + (hi - lo) / 2;
    const int c = reach(mid);
    if (c >= want) lo = mid, at_lo = c;
    else hi = mid;
  }
  return lo;
}

// One CTA per segment of a row (four chunks of 32 KB).  A chunk is held in
// registers from one read; the SM's other CTAs compute while it arrives.
//   * log-sum-exp: every thread keeps its own maximum and sum; they meet once, at
//     the segment's end.
//   * the n_out best: only threads whose largest logit of the chunk beats the
//     n_out-th best so far look for candidates.  Where those are more than
//     2 n_out (the first chunk, or an ascending row), a value that n_out of the
//     threads' bests reach, and at most twice as many, bounds them first: the n_out-th
//     best of the chunk is at least that.  It is found by bisection; among equal
//     bests the lowest tokens set it.  Candidates are ranked by counting.
//
// Bound by the read of the logits and by the pauses in it: a CTA asks for its next
// chunk when the one before is summed and ranked (DRAM 54% busy, issue slots 34%, special
// functions 13%; warps wait for loads, then at barriers).  512 rows
// of 131071 f32 logits (268 MB) take 56 us, 4.8 TB/s, the merge behind it 6 more.
// Four CTAs to an SM: 64 us for the pair, three 71, five 79.
template <bool BF16>
__global__ void __launch_bounds__(kBeamThreads, 4) beam_select_kernel(const __grid_constant__ BeamParams p) {
  constexpr int V = BF16 ? 8 : 4;  // elements of a vector
  constexpr int ELT = BF16 ? 2 : 4;
  constexpr int CHUNK = beam_chunk(BF16);
  constexpr int PER = kBeamThreads / 32;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ uint64_t list[];  // the best so far and a chunk's candidates, then [n_out] for their ranking
  __shared__ float red_sum[kBeamWarps], red_max[kBeamWarps];
  __shared__ uint32_t best_order[kBeamThreads];
  __shared__ int best_token[kBeamThreads];
  __shared__ uint32_t bound_order;
  __shared__ int bound_need, bound_token, found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.segments, segment = blockIdx.x % p.segments;
  const int K = p.n_out;
  if (p.finished != nullptr && __ldg(p.finished + row) != 0) return;  // its logits do not matter
  uint64_t* ranked = list + K + 2 * K * (CHUNK / kBeamThreads);
  const unsigned char* src = static_cast<const unsigned char*>(p.logits) + static_cast<size_t>(row) * p.row_stride * ELT;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
  // A whole chunk of an aligned row (the common case) as eight plain loads: one uniform branch for all of
  // them, so that none waits for another.
  auto load = [&](int base, uint4(&v)[kBeamVecs]) {
    const int n = p.vocab - base;
    const unsigned char* at = src + static_cast<size_t>(base + tid * V) * ELT;
    if (off == 0 && n >= CHUNK) {
#pragma unroll
      for (int i = 0; i < kBeamVecs; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(at + i * kBeamThreads * 16));
    } else {
#pragma unroll
      for (int i = 0; i < kBeamVecs; ++i) {
        const int e0 = (i * kBeamThreads + tid) * V;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (e0 < n) v[i] = load_row_vec(at + i * kBeamThreads * 16, off, static_cast<int64_t>(n - e0) * ELT);
        if (e0 + V > n) v[i] = cut_vec<BF16>(v[i], n - e0);
      }
    }
  };
  const int begin = segment * kBeamSegment * CHUNK, end = min(p.vocab, begin + kBeamSegment * CHUNK);
  uint4 v[kBeamVecs];
  if (tid == 0) found = 0;
  float run_max = -INFINITY, run_sum = 0.0f;  // this thread's, over the segment
  int held = 0;                               // entries of the list, sorted: the best so far
  float least = -INFINITY;                    // the n_out-th of them, once there are as many
  for (int base = begin; base < end; base += CHUNK) {
    load(base, v);
    if (base + CHUNK >= end) griddep_launch_dependents();  // the merge may be launched; it waits for all of this
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBeamVecs; ++i) top = fmaxf(top, vec_max<BF16>(v[i]));
    best_order[tid] = logit_order(top);
    const int many = __syncthreads_count(top > least);
    // a candidate is above `bv`, or equal to it with a token of at most `bt` in the chunk
    float bv = least;
    int bt = -1;
    if (many > 2 * K) {
      if (warp == 0) {
        uint32_t o[PER], most = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          o[i] = best_order[i * 32 + lane];
          most = max(most, o[i]);
        }
        auto reach = [&](uint32_t bound) {
          int c = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) c += o[i] >= bound;
          return static_cast<int>(__reduce_add_sync(0xffffffffu, c));
        };
        uint32_t lo = logit_order(least) + 1u, hi = __reduce_max_sync(0xffffffffu, most) + 1u;
        int at_lo = many;  // reach(lo) >= K > reach(hi) all along
        if (K <= 32) {
          // every lane has a best that reaches the smallest of the lanes' largest
          const uint32_t first = __reduce_min_sync(0xffffffffu, most);
          if (first > lo) at_lo = reach(lo = first);
        }
        while (at_lo > 2 * K && hi - lo > 1u) {
          const uint32_t mid = lo + (hi - lo) / 2;
          const int c = reach(mid);
          if (c >= K) lo = mid, at_lo = c;
          else hi = mid;
        }
        const int above = at_lo > 2 * K ? reach(lo + 1u) : K;
        if (lane == 0) {
          bound_order = lo;
          bound_need = K - above;  // of the equal bests: so many, those with the lowest tokens (0: all)
        }
      }
      __syncthreads();
      const uint32_t bo = bound_order;
      bv = cand_logit(static_cast<uint64_t>(bo) << 32);
      bt = CHUNK;
      if (bo <= 0x00800000u) bv = -3.402823466e38f;  // below every finite logit's key: all of them
      if (bound_need > 0) {
        int first = CHUNK;  // this thread's first token of exactly the bound
        if (logit_order(top) == bo) {
#pragma unroll
          for (int i = kBeamVecs - 1; i >= 0; --i)
#pragma unroll
            for (int e = V - 1; e >= 0; --e)
              if (vec_logit<BF16>(v[i], e) == bv) first = (i * kBeamThreads + tid) * V + e;
        }
        best_token[tid] = first;
        __syncthreads();
        if (warp == 0) {
          int t[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) t[i] = best_token[i * 32 + lane];
          int a = 0, b = CHUNK - 1;
          while (a < b) {
            const int mid = (a + b) / 2;
            int c = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) c += t[i] <= mid;
            if (static_cast<int>(__reduce_add_sync(0xffffffffu, c)) >= bound_need) b = mid;
            else a = mid + 1;
          }
          if (lane == 0) bound_token = a;
        }
        __syncthreads();
        bt = bound_token;
      }
    }
    // at most 2 n_out threads find anything: the list has room for all that they hold
    if (many > 0 && (top > bv || (top == bv && bt >= 0))) {
#pragma unroll
      for (int i = 0; i < kBeamVecs; ++i) {
        if (!(vec_max<BF16>(v[i]) >= bv)) continue;
        const int e0 = (i * kBeamThreads + tid) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x = vec_logit<BF16>(v[i], e);
          if (x > bv || (x == bv && e0 + e <= bt)) list[atomicAdd(&found, 1)] = cand_key(logit_order(x), base + e0 + e);
        }
      }
    }
    // the exponentials against the thread's maximum (0 where it holds none, so that a NaN still shows)
    {
      const float m = fmaxf(run_max, top), ref = m == -INFINITY ? 0.0f : m;
      if (m > run_max) {
        run_sum = __fmul_rn(run_sum, ex2(__fmul_rn(__fsub_rn(run_max, m), kLog2e)));
        run_max = m;
      }
      float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < kBeamVecs; ++i)
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 d = __fadd2_rn(make_float2(vec_logit<BF16>(v[i], e), vec_logit<BF16>(v[i], e + 1)), make_float2(-ref, -ref));
          const float2 t = __fmul2_rn(d, make_float2(kLog2e, kLog2e));
          part = __fadd2_rn(part, make_float2(ex2(t.x), ex2(t.y)));
        }
      run_sum = __fadd_rn(run_sum, __fadd_rn(part.x, part.y));
    }
    if (many > 0) {
      __syncthreads();
      const int total = found;
      for (int c = tid; c < total; c += kBeamThreads) {
        const uint64_t key = list[c];
        int rank = 0;
        for (int o = 0; o < total; ++o) rank += list[o] > key;
        if (rank < K) ranked[rank] = key;
      }
      __syncthreads();
      held = min(total, K);
      for (int c = tid; c < held; c += kBeamThreads) list[c] = ranked[c];
      if (tid == 0) found = held;
      if (held == K) least = cand_logit(ranked[K - 1]);
      __syncthreads();
    }
  }
  // the segment's maximum and sum
  float m = run_max;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) red_max[warp] = m;
  __syncthreads();
  m = red_max[0];
#pragma unroll
  for (int w = 1; w < kBeamWarps; ++w) m = fmaxf(m, red_max[w]);
  float sum = run_max == m ? run_sum : __fmul_rn(run_sum, ex2(__fmul_rn(__fsub_rn(run_max, m), kLog2e)));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, off));
  if (lane == 0) red_sum[warp] = sum;
  __syncthreads();
  const size_t at = static_cast<size_t>(row) * p.segments + segment;
  if (tid == 0) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kBeamWarps; w += 2) s = __fadd_rn(s, __fadd_rn(red_sum[w], red_sum[w + 1]));
    p.segment_sum[at] = s;
    p.segment_max[at] = m == -INFINITY ? 0.0f : m;
  }
  for (int c = tid; c < K; c += kBeamThreads) p.segment_keys[at * K + c] = c < held ? list[c] : 0ull;
}

// A score (finite) as an integer of the same order, above 0.
__device__ __forceinline__ uint64_t score_key(double s) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(s == 0.0 ? 0.0 : s));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double score_of(uint64_t key) {
  return __longlong_as_double(static_cast<long long>((key >> 63) ? (key & ~(1ull << 63)) : ~key));
}

// One CTA per group.  A warp takes a row: the log-sum-exp over its segments,
// and its n_out best out of their lists (a bound, then ranks by counting what
// reaches it).  Then the beams' candidates by score in 64 bits: each beam's
// descend, so a candidate's rank is a sum of binary searches.  Latency: about 8
// us alone, part of it hidden behind the segments' launch (its programmatic
// dependent); a logarithm per warp instead of one per lane cost 15 us at 47 groups of 14.
__global__ void __launch_bounds__(kBeamThreads) beam_merge_kernel(const __grid_constant__ BeamParams p) {
  extern __shared__ uint64_t list[];  // a warp each: [segments][n_out] keys, [2 n_out] candidates; then the scores
  __shared__ int found;
  __shared__ int row_kind[kMaxBeams];  // 0: no continuation, 1: by its logits, 2: finished
  __shared__ float row_max[kMaxBeams];
  __shared__ double row_log[kMaxBeams];  // the sum of exponentials, then its logarithm
  const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = p.n_out, per_row = p.segments * K, total = p.beams * K;
  uint64_t* keys = list + static_cast<size_t>(warp) * (per_row + 2 * K);
  uint64_t* cand = keys + per_row;
  uint64_t* score = list + static_cast<size_t>(p.merge_warps) * (per_row + 2 * K);  // [beams][n_out] logit keys, then score keys, 0: none
  int* token = reinterpret_cast<int*>(score + total);
  if (tid == 0) found = 0;
  bool waited = false;
  for (int b = warp; b < p.beams && warp < p.merge_warps; b += p.merge_warps) {
    const size_t row = static_cast<size_t>(g) * p.beams + b;
    const float cum = __ldg(p.scores + row);
    const bool ended = p.finished != nullptr && __ldg(p.finished + row) != 0;
    for (int k = lane; k < K; k += 32) score[b * K + k] = 0ull;
    if (lane == 0) row_kind[b] = ended && isfinite(cum) ? 2 : 0;
    __syncwarp();
    if (!waited) griddep_wait();  // the segments' results
    waited = true;
    if (ended) continue;
    const uint64_t* from = p.segment_keys + row * per_row;
    const float* cs = p.segment_sum + row * p.segments;
    const float* cm = p.segment_max + row * p.segments;
    // a row has at most 32 segments: one to a lane
    const float part = lane < p.segments ? __ldcg(cs + lane) : 0.0f;
    const float ref = lane < p.segments ? __ldcg(cm + lane) : 0.0f;
    for (int c = lane; c < per_row; c += 32) keys[c] = __ldcg(from + c);
    __syncwarp();
    uint64_t most = lane < p.segments ? keys[lane * K] : 0ull;           // the best of all
    uint64_t least = lane < p.segments ? keys[lane * K + K - 1] : 0ull;  // the largest n_out-th of a segment
    float m = part != 0.0f ? ref : -INFINITY;                            // NaN sums among them
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      const uint64_t a = __shfl_xor_sync(0xffffffffu, most, off), z = __shfl_xor_sync(0xffffffffu, least, off);
      most = a > most ? a : most;
      least = z > least ? z : least;
    }
    double s = part != 0.0f ? static_cast<double>(part) * static_cast<double>(expf(__fsub_rn(ref, m))) : 0.0;
    for (int off = 1; off < p.segments; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s = __shfl_sync(0xffffffffu, s, 0);
    if (!isfinite(m) || !(s > 0.0) || !isfinite(s) || !isfinite(cum) || most == 0ull) continue;
    if (lane == 0) {
      row_kind[b] = 1;
      row_max[b] = m;
      row_log[b] = s;
    }
    const uint64_t bound = bound_keys(keys, per_row, K, least > 0ull ? least : 1ull, most + 1ull, lane);
    int n = 0;
    for (int c0 = 0; c0 < per_row; c0 += 32) {
      const uint64_t key = c0 + lane < per_row ? keys[c0 + lane] : 0ull;
      const unsigned in = __ballot_sync(0xffffffffu, key >= bound);
      const int at = n + __popc(in & ((1u << lane) - 1u));
      if (key >= bound && at < 2 * K) cand[at] = key;
      n = min(n + __popc(in), 2 * K);  // (2 n_out at most, unless another call writes this workspace)
    }
    __syncwarp();
    for (int c = lane; c < n; c += 32) {
      const uint64_t key = cand[c];
      int rank = 0;
#pragma unroll 4
      for (int o = 0; o < n; ++o) rank += cand[o] > key;
      if (rank < K) score[b * K + rank] = key;
    }
    __syncwarp();
  }
  __syncthreads();
  // FP64 goes through the SM a lane or two at a time: one warp takes the logarithms of all rows
  if (tid < p.beams && row_kind[tid] == 1) row_log[tid] = log(row_log[tid]);
  __syncthreads();
  for (int c = tid; c < total; c += kBeamThreads) {
    const int b = c / K;
    const uint64_t key = score[c];
    const double cum = __ldg(p.scores + static_cast<size_t>(g) * p.beams + b);
    if (key != 0ull) {
      // the logit below the maximum first: exact where both are large
      score[c] = score_key(cum + ((static_cast<double>(cand_logit(key)) - static_cast<double>(row_max[b])) - row_log[b]));
      token[c] = cand_token(key);
    } else if (row_kind[b] == 2 && c == b * K) {
      score[c] = score_key(cum);
      token[c] = p.end_token;
    }
  }
  __syncthreads();
  int valid = 0, top_step = 1;
  while (2 * top_step <= K) top_step *= 2;
  for (int b = warp; b < p.beams; b += kBeamWarps)
    for (int k = lane; k < K; k += 32) {
      const uint64_t s = score[b * K + k];
      if (s == 0ull) continue;
      ++valid;
      int rank = k;  // the better ones of its own beam
#pragma unroll 4
      for (int o = 0; o < p.beams; ++o) {
        // those of beam o that come first: better, or as good in a lower beam
        const uint64_t* other = score + o * K;
        const uint64_t edge = s + (o < b ? 0ull : 1ull);
        int at = 0;
        for (int step = top_step; step > 0; step >>= 1)
          if (at + step <= K && other[at + step - 1] >= edge) at += step;
        rank += o == b ? 0 : at;
      }
      if (rank >= K) continue;
      const size_t at = static_cast<size_t>(g) * K + rank;
      p.parents[at] = b;
      p.tokens[at] = token[b * K + k];
      p.out_scores[at] = static_cast<float>(score_of(s));
    }
  if (valid > 0) atomicAdd(&found, valid);
  __syncthreads();
  for (int c = found + tid; c < K; c += kBeamThreads) {
    p.parents[static_cast<size_t>(g) * K + c] = -1;
    p.tokens[static_cast<size_t>(g) * K + c] = -1;
    p.out_scores[static_cast<size_t>(g) * K + c] = -INFINITY;
  }
}

// ---------------------------------------------------------------- reorder --

struct ReorderParams {
  unsigned char* pool[2];
  const int32_t* seq_ids;  // [groups][beams]
  const int32_t* parents;  // [groups][beams]
  const int32_t* lengths;  // [groups]
  int32_t* block_tables;
  unsigned char* state;  // may be NULL
  int64_t state_row_bytes;
  int32_t* status;
  int32_t groups, beams, num_seqs, max_blocks, num_pages, P, Hkv, row_bytes;
};

constexpr int kReorderThreads = 256;

// One value of every beam, permuted in place: all reads before any write, so
// no beam's old value is lost.  T is what one thread moves of each beam.
template <typename T, int B, typename Address>
__device__ __forceinline__ void permute(int beams, const int* parent, Address address) {
  T v[B];
#pragma unroll
  for (int b = 0; b < B; ++b)
    if (b < beams && parent[b] != b) v[b] = *address(parent[b]);
#pragma unroll
  for (int b = 0; b < B; ++b)
    if (b < beams && parent[b] != b) *address(b) = v[b];
}

// Grid (pieces of work, groups).  A thread takes one element of the group's
// state -- a block-table column of whole pages, 16 bytes of the unfinished
// page of K or V, or one word of a state row -- for all beams.  Every CTA
// checks the whole group first, so a bad group is left as it was by all.  B (4, 8,
// 16 or 32, the least that holds the beams) registers hold the values on their way.
// Bound by the rows moved: 64 groups of 8 beams with half a page of 64 tokens and
// a 32 KB state row each (147 MB) take 26 us, 5.6 TB/s; 1 x 4 beams are latency, 3 us.
template <int B>
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ int seq[kMaxBeams], parent[kMaxBeams], tail_page[kMaxBeams];
  const int g = blockIdx.y, tid = threadIdx.x;
  const int len = __ldg(p.lengths + g);
  bool bad = len < 0 || len > p.max_blocks * p.P;
  const int whole = bad ? 0 : len / p.P, tail = bad ? 0 : len % p.P;
  if (tid < p.beams) {
    const int s = __ldg(p.seq_ids + static_cast<size_t>(g) * p.beams + tid);
    int from = __ldg(p.parents + static_cast<size_t>(g) * p.beams + tid);
    if (from == -1) from = tid;  // no parent: the beam keeps its own cache
    seq[tid] = s;
    parent[tid] = from;
    bad |= s < 0 || s >= p.num_seqs || from < 0 || from >= p.beams;
    tail_page[tid] = -1;
    if (!bad && tail > 0) {
      tail_page[tid] = p.block_tables[static_cast<size_t>(s) * p.max_blocks + whole];
      bad |= tail_page[tid] < 0 || tail_page[tid] >= p.num_pages;
    }
  }
  __syncthreads();
  // two beams in one slot, or with one unfinished page, cannot have their own contents
  for (int c = tid; c < p.beams * p.beams; c += kReorderThreads) {
    const int x = c / p.beams, y = c % p.beams;
    if (x < y) bad |= seq[x] == seq[y] || (tail > 0 && tail_page[x] == tail_page[y]);
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kReorderThreads + tid;
  if (item < whole) {
    permute<int32_t, B>(p.beams, parent, [&](int b) {
      return p.block_tables + static_cast<size_t>(seq[b]) * p.max_blocks + item;
    });
  }
  const int pieces = p.row_bytes / 16;
  const int64_t per_pool = static_cast<int64_t>(p.Hkv) * tail * pieces;
  if (item < 2 * per_pool) {
    unsigned char* pool = p.pool[item >= per_pool];
    const int64_t i = item >= per_pool ? item - per_pool : item;
    const int h = static_cast<int>(i / (tail * pieces)), off = static_cast<int>(i % (tail * pieces));
    permute<uint4, B>(p.beams, parent, [&](int b) {
      return reinterpret_cast<uint4*>(pool + (static_cast<size_t>(tail_page[b]) * p.Hkv + h) * p.P * p.row_bytes) + off;
    });
  }
  if (p.state != nullptr && item < p.state_row_bytes / 4) {
    permute<uint32_t, B>(p.beams, parent, [&](int b) {
      return reinterpret_cast<uint32_t*>(p.state + static_cast<size_t>(seq[b]) * p.state_row_bytes) + item;
    });
  }
}

}  // namespace pa

using pa::aligned;
using pa::cuda_fail;
using pa::fail;

namespace {

bool beam_sizes_ok(int32_t beams, int32_t vocab, int32_t n_out) {
  return beams >= 1 && beams <= pa::kMaxBeams && vocab >= 1 && vocab <= pa::kMaxVocab && n_out >= 1 &&
         n_out <= pa::kMaxBeamOut;
}

int32_t beam_segments(int32_t vocab, bool bf16) {
  const int segment = pa::kBeamSegment * pa::beam_chunk(bf16);
  return (vocab + segment - 1) / segment;
}

// The workspace's parts.
size_t beam_layout(int32_t n_groups, int32_t beams, int32_t n_out, int32_t segments, void* base, pa::BeamParams* p) {
  const size_t rows = static_cast<size_t>(n_groups) * beams;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return static_cast<unsigned char*>(base) + at;
  };
  p->segment_keys = reinterpret_cast<uint64_t*>(take(rows * segments * n_out * sizeof(uint64_t)));
  p->segment_sum = reinterpret_cast<float*>(take(rows * segments * sizeof(float)));
  p->segment_max = reinterpret_cast<float*>(take(rows * segments * sizeof(float)));
  return off;
}

}  // namespace

extern "C" {

size_t pa_beam_workspace_bytes(int32_t n_groups, int32_t beams, int32_t vocab, int32_t n_out) {
  if (n_groups <= 0 || !beam_sizes_ok(beams, vocab, n_out)) return 0;
  pa::BeamParams p{};
  return beam_layout(n_groups, beams, n_out, beam_segments(vocab, false), nullptr, &p);  // f32 rows have the most segments
}

pa_status pa_beam_select(int32_t n_groups, int32_t beams, int32_t vocab, const void* logits, pa_dtype logits_dtype,
                         int64_t row_stride, const float* scores, const int32_t* finished, int32_t end_token,
                         int32_t n_out, int32_t* parents, int32_t* tokens, float* out_scores, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (n_groups < 0) return fail(PA_ERR_INVALID_ARG, "n_groups %d < 0", n_groups);
  if (beams < 1 || vocab < 1 || n_out < 1)
    return fail(PA_ERR_INVALID_ARG, "beams %d, vocab %d and n_out %d must be positive", beams, vocab, n_out);
  if (!beam_sizes_ok(beams, vocab, n_out))
    return fail(PA_ERR_UNSUPPORTED, "beams %d > %d, n_out %d > %d or vocab %d > %d", beams, pa::kMaxBeams, n_out,
                pa::kMaxBeamOut, vocab, pa::kMaxVocab);
  if (logits_dtype != PA_F32 && logits_dtype != PA_BF16)
    return fail(PA_ERR_INVALID_ARG, "logits dtype must be f32 or bf16");
  if (row_stride < vocab) return fail(PA_ERR_INVALID_ARG, "row stride %lld < vocab %d", (long long)row_stride, vocab);
  const bool bf16 = logits_dtype == PA_BF16;
  const int32_t segments = beam_segments(vocab, bf16);
  if (static_cast<int64_t>(n_groups) * beams * segments > 0x7fffffff)
    return fail(PA_ERR_UNSUPPORTED, "%d groups of %d beams in one call", n_groups, beams);
  if (n_groups == 0) return PA_OK;
  if (!logits || !scores || !parents || !tokens || !out_scores)
    return fail(PA_ERR_INVALID_ARG, "beam select: a device pointer is NULL");
  if (!aligned(logits, pa::elt_bytes(logits_dtype))) return fail(PA_ERR_INVALID_ARG, "logits are misaligned");
  const size_t need = pa_beam_workspace_bytes(n_groups, beams, vocab, n_out);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PA_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need,
                workspace == nullptr ? static_cast<size_t>(0) : workspace_bytes);
  if (!aligned(workspace, 256)) return fail(PA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  pa::BeamParams p{};
  beam_layout(n_groups, beams, n_out, segments, workspace, &p);
  p.logits = logits;
  p.row_stride = row_stride;
  p.scores = scores;
  p.finished = finished;
  p.parents = parents;
  p.tokens = tokens;
  p.out_scores = out_scores;
  p.groups = n_groups;
  p.beams = beams;
  p.vocab = vocab;
  p.segments = segments;
  p.n_out = n_out;
  p.end_token = end_token;
  // the best so far (twice) and a chunk's candidates: 2 n_out threads at most, all their elements
  const size_t smem = sizeof(uint64_t) * n_out * (2 + 2 * (pa::beam_chunk(bf16) / pa::kBeamThreads));
  const size_t row_bytes = sizeof(uint64_t) * (static_cast<size_t>(segments) + 2) * n_out;
  p.merge_warps = static_cast<int32_t>(
      std::min<size_t>({static_cast<size_t>(pa::kBeamWarps), static_cast<size_t>(beams), pa::kBeamListBytes / row_bytes}));
  const size_t merge_smem = p.merge_warps * row_bytes + static_cast<size_t>(beams) * n_out * (sizeof(double) + sizeof(int));
  static std::atomic<unsigned long long> done_f32{0}, done_bf16{0}, done_merge{0};
  cudaError_t e = bf16 ? pa::allow_dynamic_smem(pa::beam_select_kernel<true>, done_bf16, pa::kBeamMaxSmem)
                       : pa::allow_dynamic_smem(pa::beam_select_kernel<false>, done_f32, pa::kBeamMaxSmem);
  if (e == cudaSuccess) e = pa::allow_dynamic_smem(pa::beam_merge_kernel, done_merge, pa::kBeamMaxSmem);
  if (e != cudaSuccess) return cuda_fail(e, "beam select shared memory");
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(n_groups) * beams * segments));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = bf16 ? pa::launch_kernel(pa::beam_select_kernel<true>, grid, dim3(pa::kBeamThreads), smem, s, false, p)
           : pa::launch_kernel(pa::beam_select_kernel<false>, grid, dim3(pa::kBeamThreads), smem, s, false, p);
  pa::count_launch();
  if (e != cudaSuccess) return cuda_fail(e, "beam select launch");
  e = pa::launch_kernel(pa::beam_merge_kernel, dim3(n_groups), dim3(pa::kBeamThreads), merge_smem, s, true, p);
  pa::count_launch();
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "beam merge launch");
}

pa_status pa_beam_reorder(const pa_pool* pool, int32_t n_groups, int32_t beams, const int32_t* seq_ids,
                          const int32_t* parents, const int32_t* lengths, int32_t* block_tables, int32_t num_seqs,
                          int32_t max_blocks_per_seq, void* state, size_t state_row_bytes, int32_t* status_dev,
                          void* stream) {
  if (pool == nullptr) return fail(PA_ERR_INVALID_ARG, "pool is NULL");
  if (n_groups < 0) return fail(PA_ERR_INVALID_ARG, "n_groups %d < 0", n_groups);
  if (beams < 1) return fail(PA_ERR_INVALID_ARG, "beams %d must be positive", beams);
  if (beams > pa::kMaxBeams) return fail(PA_ERR_UNSUPPORTED, "beams %d > %d", beams, pa::kMaxBeams);
  if (n_groups > 65535) return fail(PA_ERR_UNSUPPORTED, "n_groups %d > 65535", n_groups);
  if (num_seqs <= 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID_ARG, "num_seqs and max_blocks_per_seq must be positive");
  const pa_pool_desc& d = pool->desc;
  if (static_cast<int64_t>(max_blocks_per_seq) * d.page_size > 0x7fffffff)
    return fail(PA_ERR_UNSUPPORTED, "a block-table row of %d pages of %d tokens", max_blocks_per_seq, d.page_size);
  if (state != nullptr && (state_row_bytes == 0 || state_row_bytes % 4 != 0 || !aligned(state, 4)))
    return fail(PA_ERR_INVALID_ARG, "state rows must be 4-byte aligned and a positive multiple of 4 bytes");
  if (n_groups == 0) return PA_OK;
  if (!seq_ids || !parents || !lengths || !block_tables)
    return fail(PA_ERR_INVALID_ARG, "reorder: a device pointer is NULL");
  pa::ReorderParams p{};
  p.pool[0] = static_cast<unsigned char*>(pool->k);
  p.pool[1] = static_cast<unsigned char*>(pool->v);
  p.seq_ids = seq_ids;
  p.parents = parents;
  p.lengths = lengths;
  p.block_tables = block_tables;
  p.state = static_cast<unsigned char*>(state);
  p.state_row_bytes = static_cast<int64_t>(state_row_bytes);
  p.status = status_dev;
  p.groups = n_groups;
  p.beams = beams;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.num_pages = d.num_pages;
  p.P = d.page_size;
  p.Hkv = d.num_kv_heads;
  p.row_bytes = d.head_dim * static_cast<int>(pa::elt_bytes(d.kv_dtype));
  // items of the longest kind of work: an unfinished page holds at most P - 1 tokens
  int64_t items = std::max<int64_t>(max_blocks_per_seq, 2ll * p.Hkv * (p.P - 1) * (p.row_bytes / 16));
  if (state != nullptr) items = std::max<int64_t>(items, p.state_row_bytes / 4);
  const int64_t blocks = (items + pa::kReorderThreads - 1) / pa::kReorderThreads;
  if (blocks > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "state rows of %zu bytes", state_row_bytes);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(n_groups));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (beams <= 4)
    pa::reorder_kernel<4><<<grid, pa::kReorderThreads, 0, s>>>(p);
  else if (beams <= 8)
    pa::reorder_kernel<8><<<grid, pa::kReorderThreads, 0, s>>>(p);
  else if (beams <= 16)
    pa::reorder_kernel<16><<<grid, pa::kReorderThreads, 0, s>>>(p);
  else
    pa::reorder_kernel<32><<<grid, pa::kReorderThreads, 0, s>>>(p);
  pa::count_launch();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "reorder launch");
}

}  // extern "C"
