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

constexpr int kSelectThreads = 1024;

// The weights in an integer order: a larger weight has a larger key, -0 and +0
// share one, and NaN comes last (below -infinity).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, kv head).  The tokens between the protected first and
// last ones are searched by radix: four passes over 8 bits of the key fix the
// key of the last token kept and how many tokens of exactly that key stay (the
// lowest indices); one more pass writes the kept indices in ascending order.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_eq[32], warp_sel[32];
  __shared__ uint32_t sh_prefix, sh_need;
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
  const int a = p.keep_first, b = len - p.keep_last;  // tokens [a, b) compete
  const uint32_t m = p.budget - p.keep_first - p.keep_last;
  uint32_t prefix = 0u, mask = 0u, need = m;
  if (m > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0u;
      __syncthreads();
      for (int t = a + tid; t < b; t += kSelectThreads) {
        const uint32_t k = weight_key(w[t]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t above = 0u;
        int bin = 255;
        while (bin > 0 && above + hist[bin] < need) above += hist[bin--];
        sh_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
        sh_need = need - above;
      }
      __syncthreads();
      prefix = sh_prefix;
      need = sh_need;
      mask |= 255u << shift;
    }
  }
  // ascending output: per block of tokens, ranks among the tokens of the last key and among the kept
  uint32_t eq_base = 0u, sel_base = 0u;
  const uint32_t below = (1u << lane) - 1u;
  for (int t0 = 0; t0 < len; t0 += kSelectThreads) {
    const int t = t0 + tid;
    bool sel = false, eq = false;
    if (t < len) {
      if (t < a || t >= b) {
        sel = true;
      } else if (m > 0) {
        const uint32_t k = weight_key(w[t]);
        sel = k > prefix;
        eq = k == prefix;
      }
    }
    const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) warp_eq[warp] = __popc(eqs);
    __syncthreads();
    uint32_t rank = eq_base, eq_all = 0u;
    for (int i2 = 0; i2 < 32; ++i2) {
      if (i2 < warp) rank += warp_eq[i2];
      eq_all += warp_eq[i2];
    }
    if (eq) sel = rank + __popc(eqs & below) < need;
    const uint32_t sels = __ballot_sync(0xffffffffu, sel);
    if (lane == 0) warp_sel[warp] = __popc(sels);
    __syncthreads();
    uint32_t at = sel_base, sel_all = 0u;
    for (int i2 = 0; i2 < 32; ++i2) {
      if (i2 < warp) at += warp_sel[i2];
      sel_all += warp_sel[i2];
    }
    if (sel) keep[at + __popc(sels & below)] = t;
    eq_base += eq_all;
    sel_base += sel_all;
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
