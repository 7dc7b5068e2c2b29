// pa_mass.cu -- pa_attention_mass: the attention weight that every cached key
// receives from a step's queries, accumulated per sequence and kv head.
//
// For row r (sequence s, position p), kv head h and its G query heads,
//     mass[s][h][t] += sum_g exp(scale q[r][g] . K_s[t] - lse[r][g]),  t = 0..p
// with lse the log-sum-exp of the row's own scores: the weights pa_attention
// gives the values, without the values.
#include <algorithm>
#include <cmath>

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

struct MassParams {
  const void* k_pool;
  const void* q;
  const int32_t* seq_ids;
  const int32_t* positions;
  const int32_t* block_tables;
  float* mass;  // [num_seqs][Hkv][max_blocks * P]
  int32_t* status;
  int32_t n_rows, num_seqs, max_blocks, num_pages, P, Hq, Hkv, D;
  int32_t q_is_bf16, kv_type, head_scales;
  float qk_scale_log2_h[kMaxHeadScales];  // softmax scale * log2(e) * k scale
  int32_t n_chunks;
  int32_t chunk_begin[kMaxChunks];
  int32_t chunk_end[kMaxChunks];
};

constexpr int kMassThreads = 256;
constexpr int kMassWarps = kMassThreads / 32;

__device__ __forceinline__ float k_element(const MassParams& p, size_t i) {
  if (p.kv_type == KV_F32) return static_cast<const float*>(p.k_pool)[i];
  if (p.kv_type == KV_BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.k_pool)[i]) << 16);
  return e4m3x2_to_float2(static_cast<const uint8_t*>(p.k_pool)[i]).x;
}

// One CTA per (row, kv head); the rows of a chunk share one sequence's sums, so
// the CTA of the chunk's first row takes them all, in order.  Two passes over
// the row's keys, a warp to a key: the maximum and the sum of the weights, then
// the weights.
__global__ void __launch_bounds__(kMassThreads) mass_kernel(const __grid_constant__ MassParams p) {
  __shared__ float qs[8][128];
  __shared__ float red[kMassWarps][8][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hkv, G = p.Hq / p.Hkv;
  const int first = blockIdx.x / p.Hkv;
  int last = first + 1;
  for (int c = 0; c < p.n_chunks; ++c)
    if (first >= p.chunk_begin[c] && first < p.chunk_end[c]) {
      if (first != p.chunk_begin[c]) return;
      last = p.chunk_end[c];
    }
  // the rows (consecutive positions of one sequence) and every page they reach
  const int seq = __ldg(p.seq_ids + first), pos0 = __ldg(p.positions + first);
  const int end = last - first - 1 + pos0;  // the last row's position
  bool bad = seq < 0 || seq >= p.num_seqs || pos0 < 0 || end >= p.max_blocks * p.P;
  const int32_t* table = p.block_tables + static_cast<size_t>(bad ? 0 : seq) * p.max_blocks;
  if (!bad) {
    for (int r = tid; r < last - first; r += kMassThreads)
      bad |= __ldg(p.seq_ids + first + r) != seq || __ldg(p.positions + first + r) != pos0 + r;
    for (int j = tid; j <= end / p.P; j += kMassThreads) {
      const int page = __ldg(table + j);
      bad |= page < 0 || page >= p.num_pages;
    }
  }
  if (__syncthreads_or(bad)) {  // the rows add nothing
    if (tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
    return;
  }
  for (int row = first; row < last; ++row) {
    const int pos = pos0 + row - first;
    for (int i = tid; i < G * p.D; i += kMassThreads) {
      const size_t at = (static_cast<size_t>(row) * p.Hq + static_cast<size_t>(h) * G) * p.D + i;
      const float x = p.q_is_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.q)[at]) << 16)
                                  : static_cast<const float*>(p.q)[at];
      qs[i / p.D][i % p.D] = x * p.qk_scale_log2_h[PA_HEAD(p, h)];
    }
    __syncthreads();
    float m[8], l[8];
    for (int g = 0; g < 8; ++g) m[g] = -INFINITY, l[g] = 0.0f;
    float* sums = p.mass + (static_cast<size_t>(seq) * p.Hkv + h) * (static_cast<size_t>(p.max_blocks) * p.P);
    for (int pass = 0; pass < 2; ++pass) {
      for (int t = warp; t <= pos; t += kMassWarps) {
        const size_t k0 = ((static_cast<size_t>(__ldg(table + t / p.P)) * p.Hkv + h) * p.P + t % p.P) * p.D;
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int d = lane; d < p.D; d += 32) {
          const float k = k_element(p, k0 + d);
          for (int g = 0; g < G; ++g) s[g] = fmaf(qs[g][d], k, s[g]);
        }
        float w = 0.0f;
        for (int g = 0; g < G; ++g) {
          for (int off = 16; off > 0; off >>= 1) s[g] += __shfl_xor_sync(0xffffffffu, s[g], off);
          if (pass == 0) {
            const float top = fmaxf(m[g], s[g]);
            l[g] = l[g] * ex2(m[g] - top) + ex2(s[g] - top);
            m[g] = top;
          } else {
            w += ex2(s[g] - m[g]) / l[g];
          }
        }
        if (pass == 1 && lane == 0) sums[t] += w;
      }
      if (pass == 0) {
        if (lane == 0)
          for (int g = 0; g < 8; ++g) red[warp][g][0] = m[g], red[warp][g][1] = l[g];
        __syncthreads();
        for (int g = 0; g < 8; ++g) {
          float top = -INFINITY, sum = 0.0f;
          for (int w = 0; w < kMassWarps; ++w) top = fmaxf(top, red[w][g][0]);
          for (int w = 0; w < kMassWarps; ++w)
            if (red[w][g][1] > 0.0f) sum += red[w][g][1] * ex2(red[w][g][0] - top);
          m[g] = top;
          l[g] = sum;
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace pa

using pa::aligned;
using pa::cuda_fail;
using pa::fail;

extern "C" {

size_t pa_attention_mass_workspace_bytes(const pa_pool* pool, int32_t n_rows, int32_t num_q_heads,
                                         int32_t max_blocks_per_seq, const pa_chunk* chunks, int32_t n_chunks) {
  (void)pool, (void)n_rows, (void)num_q_heads, (void)max_blocks_per_seq, (void)chunks, (void)n_chunks;
  return 0;
}

pa_status pa_attention_mass(const pa_pool* pool, int32_t n_rows, const void* q, pa_dtype q_dtype, int32_t num_q_heads,
                            const int32_t* seq_ids, const int32_t* positions, const int32_t* block_tables,
                            int32_t num_seqs, int32_t max_blocks_per_seq, const pa_chunk* chunks, int32_t n_chunks,
                            float softmax_scale, float* mass, void* workspace, size_t workspace_bytes,
                            int32_t* status_dev, void* stream) {
  if (pool == nullptr) return fail(PA_ERR_INVALID_ARG, "pool is NULL");
  const pa_pool_desc& d = pool->desc;
  pa_status st = pa::check_rows(d, n_rows, q_dtype, num_q_heads, num_seqs, max_blocks_per_seq, chunks, n_chunks);
  if (st != PA_OK) return st;
  if (static_cast<int64_t>(max_blocks_per_seq) * d.page_size > 0x7fffffff)
    return fail(PA_ERR_UNSUPPORTED, "a block-table row of %d pages of %d tokens", max_blocks_per_seq, d.page_size);
  if (n_rows == 0) return PA_OK;
  if (!q || !seq_ids || !positions || !block_tables || !mass)
    return fail(PA_ERR_INVALID_ARG, "attention mass: a device pointer is NULL");
  if (!aligned(q, 16) || !aligned(mass, 16)) return fail(PA_ERR_INVALID_ARG, "q / mass must be 16-byte aligned");
  const int64_t units = static_cast<int64_t>(n_rows) * d.num_kv_heads;
  if (units > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "%lld (row, kv head) pairs in one call", (long long)units);
  (void)workspace, (void)workspace_bytes;
  const double sm = softmax_scale > 0.f ? static_cast<double>(softmax_scale) : 1.0 / std::sqrt(static_cast<double>(d.head_dim));
  pa::MassParams p{};
  p.k_pool = pool->k;
  p.q = q;
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.block_tables = block_tables;
  p.mass = mass;
  p.status = status_dev;
  p.n_rows = n_rows;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.num_pages = d.num_pages;
  p.P = d.page_size;
  p.Hq = num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.D = d.head_dim;
  p.q_is_bf16 = q_dtype == PA_BF16;
  p.kv_type = static_cast<int32_t>(d.kv_dtype);
  p.head_scales = pool->head_scales ? 1 : 0;
  for (int h = 0; h < (pool->head_scales ? d.num_kv_heads : 1); ++h) {
    const double ks = d.kv_dtype == PA_FP8_E4M3 ? static_cast<double>(pool->head_scales ? pool->k_scale_h[h] : d.k_scale) : 1.0;
    p.qk_scale_log2_h[h] = static_cast<float>(sm * ks * 1.4426950408889634073599246810018921);  // log2(e)
  }
  p.n_chunks = n_chunks;
  for (int c = 0; c < n_chunks; ++c) {
    p.chunk_begin[c] = chunks[c].row_begin;
    p.chunk_end[c] = chunks[c].row_begin + chunks[c].n_rows;
  }
  pa::mass_kernel<<<static_cast<unsigned>(units), pa::kMassThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  pa::count_launch();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "attention mass launch");
}

}  // extern "C"
