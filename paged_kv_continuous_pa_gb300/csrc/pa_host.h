// pa_host.h -- host-side pieces shared by the files that implement the C ABI:
// the pool object, error reporting and small checks.  Internal.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include "../../include/pa.h"
#include "pa_kernels.h"

struct pa_pool {
  pa_pool_desc desc;
  bool head_scales;  // fp8 scales per kv head (pa_pool_set_head_scales)
  float k_scale_h[pa::kMaxHeadScales], v_scale_h[pa::kMaxHeadScales];
  void* k;
  void* v;
  std::mutex maps;       // held while they are encoded: threads may make a pool's first calls at once
  std::atomic<bool> tile_maps_ready;  // kmap / vmap encoded (on first use by the tile paths)
  std::atomic<bool> dec_maps_ready;   // kmap_dec / vmap_dec encoded (on first use by tensor-core decode units)
  CUtensorMap kmap;      // 2-D views of the pools for tensor-map copies
  CUtensorMap vmap;
  CUtensorMap kmap_dec;
  CUtensorMap vmap_dec;
};

namespace pa {

// Set the calling thread's pa_last_error() text and return `st`.
pa_status fail(pa_status st, const char* fmt, ...);
pa_status cuda_fail(cudaError_t e, const char* what);

// The checks of a call's rows that pa_attention, pa_step and pa_attention_mass share.
pa_status check_rows(const pa_pool_desc& d, int32_t n_rows, pa_dtype q_dtype, int32_t num_q_heads, int32_t num_seqs,
                     int32_t max_blocks_per_seq, const pa_chunk* chunks, int32_t n_chunks);

// The pool's tensor maps for the tile paths (bf16), encoded on first use.
pa_status encode_tile_maps(pa_pool* pool);
// bf16 queries [n_rows][hq][head_dim] as a 3-D tensor, 128-byte swizzle, boxes of
// 64 elements x `group` heads x 128 / group rows.
pa_status encode_query_map(CUtensorMap* map, const void* q, int32_t n_rows, int32_t hq, int32_t head_dim, int32_t group);

// Process-wide settings, each read once per call.
uint32_t wait_limit();
int32_t debug_stall();

inline size_t elt_bytes(pa_dtype t) { return t == PA_F32 ? 4 : t == PA_BF16 ? 2 : 1; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace pa
