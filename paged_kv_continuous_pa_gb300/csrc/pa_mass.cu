// pa_mass.cu -- pa_attention_mass: argument checks, launch geometry and
// dispatch (the kernels are in pa_mass.cuh).
#include <algorithm>
#include <cmath>

#include "pa_host.h"
#include "pa_mass.cuh"

using pa::aligned;
using pa::cuda_fail;
using pa::fail;

namespace {

// Key ranges, key blocks and the chunks' places in the workspace, from sizes alone.
size_t plan_chunks(const pa_pool_desc& d, int32_t hq, int32_t max_blocks, const pa_chunk* chunks, int32_t n_chunks,
                   pa::MassParams* p) {
  const int64_t keys = static_cast<int64_t>(max_blocks) * d.page_size;
  p->n_splits = static_cast<int32_t>((keys + pa::kMassSplitKeys - 1) / pa::kMassSplitKeys);
  p->n_blocks = static_cast<int32_t>((keys + pa::kMassBlockKeys - 1) / pa::kMassBlockKeys);
  int64_t pairs = 0;
  for (int c = 0; c < n_chunks; ++c) {
    p->chunk_begin[c] = chunks[c].row_begin;
    p->chunk_end[c] = chunks[c].row_begin + chunks[c].n_rows;
    p->chunk_stats[c] = pairs;
    pairs += static_cast<int64_t>(chunks[c].n_rows) * hq * p->n_splits;
  }
  p->n_chunks = n_chunks;
  return (static_cast<size_t>(pairs) * sizeof(float2) + 255) / 256 * 256;
}

}  // namespace

extern "C" {

size_t pa_attention_mass_workspace_bytes(const pa_pool* pool, int32_t n_rows, int32_t num_q_heads,
                                         int32_t max_blocks_per_seq, const pa_chunk* chunks, int32_t n_chunks) {
  if (pool == nullptr || pa::check_rows(pool->desc, n_rows, PA_BF16, num_q_heads, 1, max_blocks_per_seq, chunks,
                                        n_chunks) != PA_OK)
    return 0;
  pa::MassParams p{};
  return plan_chunks(pool->desc, num_q_heads, max_blocks_per_seq, chunks, n_chunks, &p);
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
  const size_t need = plan_chunks(d, num_q_heads, max_blocks_per_seq, chunks, n_chunks, &p);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(PA_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need,
                  workspace == nullptr ? static_cast<size_t>(0) : workspace_bytes);
    if (!aligned(workspace, 256)) return fail(PA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    p.ws_stats = static_cast<float2*>(workspace);
  }
  int64_t in_chunks = 0;
  for (int c = 0; c < n_chunks; ++c) in_chunks += chunks[c].n_rows;
  // A row's cluster: by the block table's width, never by the batch, so that a
  // row's sums are taken in the same order whatever else the call holds.
  const int64_t keys = static_cast<int64_t>(max_blocks_per_seq) * d.page_size;
  p.cluster = 1;
  while (p.cluster < pa::kMassMaxCluster && keys > static_cast<int64_t>(p.cluster) * pa::kMassClusterKeys) p.cluster *= 2;
  const int G = num_q_heads / d.num_kv_heads;
  const int64_t room = (static_cast<int64_t>(pa::kMassScoreBytes) / (G * 4) - 36) / 32 * 32;  // keys whose scores fit
  const int64_t share = ((keys + 15) / 16 + p.cluster - 1) / p.cluster * 16;
  p.score_keys = static_cast<int32_t>(std::min(room, share));
  if (static_cast<int64_t>(n_rows) * d.num_kv_heads * p.cluster > 0x7fffffff)
    return fail(PA_ERR_UNSUPPORTED, "%d rows of %d kv heads in one call", n_rows, d.num_kv_heads);
  const bool rows = in_chunks < n_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (d.kv_dtype) {
    case PA_F32: e = pa::launch_mass_f32(p, rows, s); break;
    case PA_BF16: e = pa::launch_mass_bf16(p, rows, s); break;
    default: e = pa::launch_mass_e4m3(p, rows, s); break;
  }
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "attention mass launch");
}

}  // extern "C"
