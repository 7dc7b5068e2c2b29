// pa_mass.cu -- pa_attention_mass: argument checks, launch geometry and
// dispatch (the kernels are in pa_mass.cuh).
#include <algorithm>
#include <cmath>

#include "pa_host.h"
#include "pa_mass.cuh"

namespace pa {

// A CTA per chunk: whether its rows are consecutive positions of one sequence
// within the table, and every page that they reach a page of the pool.
__global__ void __launch_bounds__(256) chunk_check_kernel(const __grid_constant__ MassParams p) {
  griddep_launch_dependents();  // the statistics may be launched; they wait for this
  const int c = blockIdx.x, tid = threadIdx.x;
  const int row0 = p.chunk_begin[c], rows = p.chunk_end[c] - row0;
  const int seq = __ldg(p.seq_ids + row0), pos0 = __ldg(p.positions + row0);
  bool bad = seq < 0 || seq >= p.num_seqs || pos0 < 0 || pos0 > p.max_blocks * p.P - rows;
  if (!bad) {
    const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks;
    for (int r = tid; r < rows; r += 256)
      bad |= __ldg(p.seq_ids + row0 + r) != seq || __ldg(p.positions + row0 + r) != pos0 + r;
    for (int j = tid; j <= (pos0 + rows - 1) / p.P; j += 256) {
      const int page = __ldg(table + j);
      bad |= page < 0 || page >= p.num_pages;
    }
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    if (bad) record_error(p.status, ST_OUT_OF_RANGE);
    p.ws_head[c] = make_int2(bad ? -1 : seq, pos0);
    p.ws_whole[c] = 0;
  }
}

}  // namespace pa

using pa::aligned;
using pa::cuda_fail;
using pa::fail;

namespace {

// Key ranges, key blocks and the chunks' places in the workspace, from sizes alone.
size_t plan_chunks(const pa_pool_desc& d, int32_t hq, int32_t max_blocks, const pa_chunk* chunks, int32_t n_chunks,
                   void* workspace, pa::MassParams* p) {
  const int64_t keys = static_cast<int64_t>(max_blocks) * d.page_size;
  auto cut = [&](int64_t n) { return static_cast<int32_t>((keys + n - 1) / n); };
  p->n_splits = cut(pa::kMassSplitKeys);
  p->n_blocks = cut(pa::kMassBlockKeys);
  const int R = pa::kMassSlots / (hq / d.num_kv_heads);
  int64_t pairs = 0;
  for (int c = 0; c < n_chunks; ++c) {
    p->chunk_begin[c] = chunks[c].row_begin;
    p->chunk_end[c] = chunks[c].row_begin + chunks[c].n_rows;
    p->chunk_tiles[c] = (chunks[c].n_rows + R - 1) / R;
    const int64_t slots = static_cast<int64_t>(p->chunk_tiles[c]) * pa::kMassSlots * d.num_kv_heads;
    p->chunk_part[c] = pairs;
    pairs += slots * p->n_splits;
  }
  p->n_chunks = n_chunks;
  if (n_chunks == 0) return 0;
  static_assert(pa::kMaxChunks * (sizeof(int2) + sizeof(int32_t)) <= 256, "the chunks' heads");
  p->ws_head = static_cast<int2*>(workspace);
  p->ws_whole = reinterpret_cast<int32_t*>(p->ws_head + pa::kMaxChunks);
  p->ws_part = reinterpret_cast<float2*>(static_cast<unsigned char*>(workspace) + 256);
  return 256 + static_cast<size_t>(pairs) * sizeof(float2);
}

// The chunks' columns: a look at the chunks, statistics over key ranges, then the weights.
template <typename Launch>
cudaError_t launch_chunks(const pa::MassParams& p, Launch launch, cudaStream_t s) {
  pa::chunk_check_kernel<<<p.n_chunks, 256, 0, s>>>(p);
  pa::count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch(p, pa::MASS_CHUNK_STATS, s);
  if (e == cudaSuccess) e = launch(p, pa::MASS_CHUNK_WEIGHTS, s);
  return e;
}

}  // namespace

extern "C" {

size_t pa_attention_mass_workspace_bytes(const pa_pool* pool, int32_t n_rows, int32_t num_q_heads,
                                         int32_t max_blocks_per_seq, const pa_chunk* chunks, int32_t n_chunks) {
  if (pool == nullptr || pa::check_rows(pool->desc, n_rows, PA_BF16, num_q_heads, 1, max_blocks_per_seq, chunks,
                                        n_chunks) != PA_OK)
    return 0;
  pa::MassParams p{};
  return plan_chunks(pool->desc, num_q_heads, max_blocks_per_seq, chunks, n_chunks, nullptr, &p);
}

pa_status pa_attention_mass(const pa_pool* pool, int32_t n_rows, const void* q, pa_dtype q_dtype, int32_t num_q_heads,
                            const int32_t* seq_ids, const int32_t* positions, const int32_t* block_tables,
                            int32_t num_seqs, int32_t max_blocks_per_seq, const pa_chunk* chunks, int32_t n_chunks,
                            float softmax_scale, float* mass, void* workspace, size_t workspace_bytes,
                            int32_t* status_dev, void* stream) {
  if (pool == nullptr) return fail(PA_ERR_INVALID_ARG, "pool is NULL");
  const pa_pool_desc& d = pool->desc;
  if (d.kv_dtype == PA_INT4) return fail(PA_ERR_UNSUPPORTED, "attention mass: a 4-bit pool");
  pa_status st = pa::check_rows(d, n_rows, q_dtype, num_q_heads, num_seqs, max_blocks_per_seq, chunks, n_chunks);
  if (st != PA_OK) return st;
  if (static_cast<int64_t>(max_blocks_per_seq) * d.page_size > (1 << 30))  // (positions and steps beyond stay int32)
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
  const size_t need = plan_chunks(d, num_q_heads, max_blocks_per_seq, chunks, n_chunks, workspace, &p);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(PA_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need,
                  workspace == nullptr ? static_cast<size_t>(0) : workspace_bytes);
    if (!aligned(workspace, 256)) return fail(PA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  int64_t in_chunks = 0;
  for (int c = 0; c < n_chunks; ++c) in_chunks += chunks[c].n_rows;
  // A row's cluster: by the block table's width, never by the batch, so that a
  // row's sums are taken in the same order whatever else the call holds.  4096
  // keys to a CTA (512 ragged rows of up to 2662 keys in one CTA each: 225 us, in
  // CTAs of 2048 keys 255, of 1024 358), so 8 CTAs from 16385 keys on; 16 from 65537
  // on (one row of 131072 keys: 59 us with 16, 160 with 8; at 16 rows of 65536,
  // 364 with 16 and 335 with 8).  The price is paid by short rows under wide tables: the
  // 512 ragged rows take 236 us with a table of 2662 tokens, 270 with 8192, 627 with 32768,
  // 1432 with 131072.
  const int64_t keys = static_cast<int64_t>(max_blocks_per_seq) * d.page_size;
  p.cluster = 1;
  while (p.cluster < 8 && keys > static_cast<int64_t>(p.cluster) * pa::kMassClusterKeys) p.cluster *= 2;
  if (keys > static_cast<int64_t>(pa::kMassMaxCluster) * pa::kMassClusterKeys) p.cluster = pa::kMassMaxCluster;
  const int G = num_q_heads / d.num_kv_heads;
  const int64_t room = (static_cast<int64_t>(pa::kMassScoreBytes) / (G * 4) - 36) / 32 * 32;  // keys whose scores fit
  // a CTA's share of the longest row, in the kernel's steps (at most four 16-key tiles)
  const int64_t share = ((keys + 15) / 16 + p.cluster * 4 - 1) / (p.cluster * 4) * 64;
  p.score_keys = static_cast<int32_t>(std::min(room, share));
  if (static_cast<int64_t>(n_rows) * d.num_kv_heads * p.cluster > 0x7fffffff)
    return fail(PA_ERR_UNSUPPORTED, "%d rows of %d kv heads in one call", n_rows, d.num_kv_heads);
  p.wait_limit = pa::wait_limit();
  p.debug_stall = pa::debug_stall();
  if (n_chunks > 0 && d.kv_dtype == PA_BF16 && q_dtype == PA_BF16) {  // the tile path
    st = pa::encode_tile_maps(const_cast<pa_pool*>(pool));
    if (st == PA_OK) st = pa::encode_query_map(&p.qmap, q, n_rows, num_q_heads, d.head_dim, G);
    if (st != PA_OK) return st;
    p.kmap = pool->kmap;
  }
  auto launch = d.kv_dtype == PA_F32 ? pa::launch_mass_f32 : d.kv_dtype == PA_BF16 ? pa::launch_mass_bf16 : pa::launch_mass_e4m3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (in_chunks < n_rows) e = launch(p, pa::MASS_ROWS, s);
  if (e == cudaSuccess && n_chunks > 0) e = launch_chunks(p, launch, s);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "attention mass launch");
}

}  // extern "C"
