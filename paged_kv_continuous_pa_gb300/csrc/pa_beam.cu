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
  uint64_t* cand;   // [rows][n_out] best (logit, token) of each row, best first; 0: none
  double* norm;     // [rows] log-sum-exp; NaN: the row has no candidates
  int32_t groups, beams, vocab, n_out, end_token;
};

constexpr int kBeamThreads = 512;

// A logit and its token as one integer: larger logits first, then lower
// tokens; -0 and +0 are one value.  NaN and -infinity are never asked for (0).
__device__ __forceinline__ uint64_t cand_key(float x, int token) {
  if (!(x > -INFINITY)) return 0ull;
  const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<uint64_t>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(token));
}
__device__ __forceinline__ float cand_logit(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int cand_token(uint64_t key) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)); }

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <bool BF16>
__device__ __forceinline__ float logit_at(const BeamParams& p, size_t i) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.logits)[i]) << 16);
  else
    return static_cast<const float*>(p.logits)[i];
}

// One CTA per beam: the row's log-sum-exp, then its n_out best logits, one
// scan of the row for each.
template <bool BF16>
__global__ void __launch_bounds__(kBeamThreads) beam_row_kernel(const __grid_constant__ BeamParams p) {
  __shared__ double red_sum[kBeamThreads / 32];
  __shared__ float red_max[kBeamThreads / 32];
  __shared__ uint64_t red_key[kBeamThreads / 32];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.finished != nullptr && __ldg(p.finished + row) != 0) return;
  const size_t base = static_cast<size_t>(row) * p.row_stride;
  float top = -INFINITY;
  bool nan = false;
  for (int v = tid; v < p.vocab; v += kBeamThreads) {
    const float x = logit_at<BF16>(p, base + v);
    nan |= x != x;
    top = fmaxf(top, x);
  }
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) red_max[warp] = top;
  nan = __syncthreads_or(nan);
  top = red_max[0];
  for (int w = 1; w < kBeamThreads / 32; ++w) top = fmaxf(top, red_max[w]);
  const bool dead = nan || !(fabsf(top) < INFINITY);
  float part = 0.0f;
  for (int v = tid; v < p.vocab && !dead; v += kBeamThreads) part += expf(logit_at<BF16>(p, base + v) - top);
  double sum = part;
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) red_sum[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < kBeamThreads / 32; ++w) s += red_sum[w];
    p.norm[row] = dead ? static_cast<double>(NAN) : static_cast<double>(top) + log(s);
  }
  uint64_t last = ~0ull;
  for (int k = 0; k < p.n_out; ++k) {
    uint64_t best = 0ull;
    for (int v = tid; v < p.vocab && !dead; v += kBeamThreads) {
      const uint64_t key = cand_key(logit_at<BF16>(p, base + v), v);
      if (key < last) best = max_u64(best, key);
    }
    for (int off = 16; off > 0; off >>= 1) best = max_u64(best, __shfl_xor_sync(0xffffffffu, best, off));
    __syncthreads();
    if (lane == 0) red_key[warp] = best;
    __syncthreads();
    for (int w = 0; w < kBeamThreads / 32; ++w) best = max_u64(best, red_key[w]);
    last = best;
    if (tid == 0) p.cand[static_cast<size_t>(row) * p.n_out + k] = best;
  }
}

// One CTA per group: scores of the beams' candidates in 64 bits, each
// candidate's rank by counting the better ones, the n_out best written.
__global__ void __launch_bounds__(256) beam_merge_kernel(const __grid_constant__ BeamParams p) {
  extern __shared__ double score[];  // [beams * n_out]
  const int g = blockIdx.x, tid = threadIdx.x;
  const int total = p.beams * p.n_out;
  for (int c = tid; c < total; c += 256) {
    const int row = g * p.beams + c / p.n_out, k = c % p.n_out;
    const double cum = __ldg(p.scores + row);
    double s = -INFINITY;
    if (p.finished != nullptr && __ldg(p.finished + row) != 0) {
      if (k == 0) s = cum;
    } else {
      const uint64_t key = p.cand[static_cast<size_t>(row) * p.n_out + k];
      if (key != 0ull) s = cum + (static_cast<double>(cand_logit(key)) - p.norm[row]);
    }
    score[c] = isfinite(s) ? s : static_cast<double>(-INFINITY);
  }
  for (int k = tid; k < p.n_out; k += 256) {
    p.parents[static_cast<size_t>(g) * p.n_out + k] = -1;
    p.tokens[static_cast<size_t>(g) * p.n_out + k] = -1;
    p.out_scores[static_cast<size_t>(g) * p.n_out + k] = -INFINITY;
  }
  __syncthreads();
  for (int c = tid; c < total; c += 256) {
    const double s = score[c];
    if (!(s > -INFINITY)) continue;
    int rank = 0;
    for (int o = 0; o < total; ++o) rank += score[o] > s || (score[o] == s && o < c);
    if (rank >= p.n_out) continue;
    const int row = g * p.beams + c / p.n_out;
    const bool ended = p.finished != nullptr && __ldg(p.finished + row) != 0;
    const size_t at = static_cast<size_t>(g) * p.n_out + rank;
    p.parents[at] = c / p.n_out;
    p.tokens[at] = ended ? p.end_token : cand_token(p.cand[static_cast<size_t>(row) * p.n_out + c % p.n_out]);
    p.out_scores[at] = static_cast<float>(s);
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
// checks the whole group first, so a bad group is left as it was by all.
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
  return beams >= 1 && beams <= pa::kMaxBeams && vocab >= 1 && n_out >= 1 && n_out <= pa::kMaxBeamOut;
}

}  // namespace

extern "C" {

size_t pa_beam_workspace_bytes(int32_t n_groups, int32_t beams, int32_t vocab, int32_t n_out) {
  if (n_groups <= 0 || !beam_sizes_ok(beams, vocab, n_out)) return 0;
  const size_t rows = static_cast<size_t>(n_groups) * beams;
  const size_t need = rows * n_out * sizeof(uint64_t) + rows * sizeof(double);
  return (need + 255) / 256 * 256;
}

pa_status pa_beam_select(int32_t n_groups, int32_t beams, int32_t vocab, const void* logits, pa_dtype logits_dtype,
                         int64_t row_stride, const float* scores, const int32_t* finished, int32_t end_token,
                         int32_t n_out, int32_t* parents, int32_t* tokens, float* out_scores, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (n_groups < 0) return fail(PA_ERR_INVALID_ARG, "n_groups %d < 0", n_groups);
  if (beams < 1 || vocab < 1 || n_out < 1)
    return fail(PA_ERR_INVALID_ARG, "beams %d, vocab %d and n_out %d must be positive", beams, vocab, n_out);
  if (beams > pa::kMaxBeams || n_out > pa::kMaxBeamOut)
    return fail(PA_ERR_UNSUPPORTED, "beams %d > %d or n_out %d > %d", beams, pa::kMaxBeams, n_out, pa::kMaxBeamOut);
  if (logits_dtype != PA_F32 && logits_dtype != PA_BF16)
    return fail(PA_ERR_INVALID_ARG, "logits dtype must be f32 or bf16");
  if (row_stride < vocab) return fail(PA_ERR_INVALID_ARG, "row stride %lld < vocab %d", (long long)row_stride, vocab);
  if (static_cast<int64_t>(n_groups) * beams > 0x7fffffff)
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
  const size_t rows = static_cast<size_t>(n_groups) * beams;
  p.logits = logits;
  p.row_stride = row_stride;
  p.scores = scores;
  p.finished = finished;
  p.parents = parents;
  p.tokens = tokens;
  p.out_scores = out_scores;
  p.cand = static_cast<uint64_t*>(workspace);
  p.norm = reinterpret_cast<double*>(p.cand + rows * n_out);
  p.groups = n_groups;
  p.beams = beams;
  p.vocab = vocab;
  p.n_out = n_out;
  p.end_token = end_token;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (logits_dtype == PA_BF16)
    pa::beam_row_kernel<true><<<static_cast<unsigned>(rows), pa::kBeamThreads, 0, s>>>(p);
  else
    pa::beam_row_kernel<false><<<static_cast<unsigned>(rows), pa::kBeamThreads, 0, s>>>(p);
  pa::count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "beam select launch");
  pa::beam_merge_kernel<<<n_groups, 256, sizeof(double) * beams * n_out, s>>>(p);
  pa::count_launch();
  e = cudaGetLastError();
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
