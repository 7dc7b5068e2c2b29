// pa_mass.cuh -- the kernels of pa_attention_mass: the attention weight that
// every cached key receives from a step's queries, accumulated per sequence and
// kv head.  For row r (sequence s, position p), kv head h and its G query heads,
//     mass[s][h][t] += sum_g exp(scale q[r][g] . K_s[t] - lse[r][g]),  t = 0..p
// with lse the log-sum-exp of the row's own scores.  Scores live in the log2
// domain; a row's weights need its maximum and sum over all keys first.
//
// Rows outside the chunks (`mass_row_kernel`): one cluster of CTAs per (row, kv
// head).  K is read from memory once, straight into tensor-core fragments (but for
// keys whose scores find no room); the scores wait in shared memory while the cluster's CTAs exchange their (max,
// sum) pairs, then become weights.
// Chunks: the (row, head) pairs of a kv head are columns that share the keys.
// `chunk_check_kernel` looks the chunks over, `chunk_stats_kernel` finds every
// column's (max, sum) over ranges of keys, `chunk_weights_kernel` merges the
// ranges, recomputes the scores key block by key block and sums the weights over
// the columns: each key has one owner, which adds once.  (bf16 queries over a bf16 pool: the same steps on the tile path,
// pa_mass_tiles.cuh.)
// No atomic decides an order: the same rows give the same bits in any batch.
#pragma once

#include <cooperative_groups.h>

#include "pa_decode_mma.cuh"

namespace pa {

constexpr int kMassThreads = 256;
constexpr int kMassWarps = kMassThreads / 32;
constexpr int kMassSplitKeys = 1024;  // keys per range of the chunks' first launch (and of the tile path's last)
constexpr int kMassLongKeys = 256;    // ... of that one for chunks of more than kMassLongTiles column tiles
constexpr int kMassLongTiles = 8;
constexpr int kMassBlockKeys = 512;   // keys per CTA of their last launch
constexpr int kMassSlots = 128;       // columns of a chunk come in tiles of 128 / G rows, 128 slots each
constexpr int kMassClusterKeys = 4096;             // keys per CTA that a row's cluster aims at
constexpr int kMassMaxCluster = 16;
constexpr size_t kMassScoreBytes = 104 * 1024;     // shared memory for a CTA's scores (two CTAs to an SM)

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
  int32_t cluster;      // CTAs per (row, kv head) of the rows' launch
  int32_t score_keys;   // keys per CTA whose scores fit in shared memory (a multiple of 16)
  uint32_t wait_limit;  // microseconds (tile path)
  int32_t debug_stall;  // tile path: also wait on a barrier nothing completes
  int32_t n_chunks;
  int32_t chunk_begin[kMaxChunks];
  int32_t chunk_end[kMaxChunks];
  int32_t chunk_cta[kMaxChunks + 1];   // prefix sums of CTAs per chunk (set per launch)
  int32_t chunk_tiles[kMaxChunks];     // tiles of 128 / G rows
  int32_t n_splits, n_blocks;          // of the longest row: key ranges, key blocks
  int64_t chunk_part[kMaxChunks];      // offset of a chunk in ws_part, in pairs
  int2* ws_head;                       // per chunk its sequence (-1: the chunk adds nothing) and first position
  int32_t* ws_whole;                   // per chunk: whether whole operands gave a column its sum (`in_parts`)
  float2* ws_part;                     // (max, sum) per chunk [Hkv][n_splits][tiles][128]
  CUtensorMap kmap;                    // tile path: the pool as [num_pages * Hkv * P][D], boxes of 64 x min(P, 64)
  CUtensorMap qmap;                    // tile path: q as [n_rows][Hq][D], boxes of 128 / G rows x G heads x 64
};

// The slot of a column (head col % G of row col / G) among its chunk's tiles.
__device__ __forceinline__ int column_slot(int col, int G) {
  const int r = col / G, R = kMassSlots / G;
  return r / R * kMassSlots + r % R * G + col % G;
}

// ------------------------------------------------------------- fragments --
//
// A warp scores 16 keys x 8 columns with mma.m16n8k16: A = K, lane (g4, t4)
// holding pieces of key rows g4 and g4 + 8, B = the queries.  The order of the
// D products of a dot product is free, so a lane takes whole 16-byte pieces of
// its rows (piece t4 + 4 i) and feeds them to the MMAs as they are; the query
// fragments follow the same order.
//   bf16 K  as it is; an f32 query enters as three bf16 parts (24 bits), a bf16 one as one
//   e4m3 K  exactly as f16; the query as f16 after a power-of-two scaling per column that puts
//           its largest element in [2^14, 2^15): one part for bf16, two (22 bits) for f32
//   f32 K   as three bf16 parts, with the query's parts; products below 2^-24 are left out

template <int KVT, int D, bool QB>
struct MassGeom {
  static constexpr int ELT = KvElt<KVT>::bytes;
  static constexpr int RB = D * ELT;        // bytes of a K row
  static constexpr int EP = 16 / ELT;       // elements of a piece
  static constexpr int NPT = RB / 64;       // pieces a lane holds of a row
  static constexpr int STEPS = D / 16;      // MMA k-steps
  static constexpr int MT = RB < 256 ? 256 / RB : 1;  // 16-key tiles a warp of a row's cluster loads at once (4 KB)
  static constexpr int KP = KVT == KV_F32 ? 3 : 1;
  static constexpr int QP = QB ? 1 : (KVT == KV_E4M3 ? 2 : 3);
};

__device__ __forceinline__ void mass_mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two floats as bf16 pairs: the leading part, and what it leaves (in place).
__device__ __forceinline__ uint32_t take_bf16(float& x, float& y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  x = __fsub_rn(x, __low2float(h));
  y = __fsub_rn(y, __high2float(h));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t take_f16(float& x, float& y) {
  const __half2 h = __floats2half2_rn(x, y);
  x = __fsub_rn(x, __low2float(h));
  y = __fsub_rn(y, __high2float(h));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A column's query as B fragments, and the factor that turns its dot products
// into log2-domain scores.  `row` < 0: an empty column (zeros).
template <int KVT, int D, bool QB>
struct QueryFrag {
  using Geo = MassGeom<KVT, D, QB>;
  uint32_t b[Geo::QP][Geo::STEPS][2];

  // The column of lane group g4 (head `head` of row `row`); returns its factor.
  __device__ __forceinline__ float load(const MassParams& p, int row, int head, float scale, int t4) {
    float x[Geo::STEPS][4];
    const size_t base = row < 0 ? 0 : (static_cast<size_t>(row) * p.Hq + head) * D;
#pragma unroll
    for (int i = 0; i < Geo::NPT; ++i)
#pragma unroll
      for (int j = 0; j < Geo::EP / 4; ++j) {
        float(&e)[4] = x[i * (Geo::EP / 4) + j];
        const size_t at = base + (t4 + 4 * i) * Geo::EP + 4 * j;
        if (row < 0) {
          e[0] = e[1] = e[2] = e[3] = 0.0f;
        } else if constexpr (QB) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + at));
          e[0] = bf16lo(w.x), e[1] = bf16hi(w.x), e[2] = bf16lo(w.y), e[3] = bf16hi(w.y);
        } else {
          const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at));
          e[0] = w.x, e[1] = w.y, e[2] = w.z, e[3] = w.w;
        }
      }
    if constexpr (KVT == KV_E4M3) {
      float top = 0.0f;
#pragma unroll
      for (int s = 0; s < Geo::STEPS; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(x[s][k]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the power of two that puts `top` in [2^14, 2^15); none for a column of zeros or one that is not finite
      const int e = (top > 0.0f && top < INFINITY) ? 14 - ilogbf(top) : 0;
#pragma unroll
      for (int s = 0; s < Geo::STEPS; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[s][k] = scalbnf(x[s][k], e);
      scale = scalbnf(scale, -e);
    }
#pragma unroll
    for (int part = 0; part < Geo::QP; ++part)
#pragma unroll
      for (int s = 0; s < Geo::STEPS; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          b[part][s][k] = KVT == KV_E4M3 ? take_f16(x[s][2 * k], x[s][2 * k + 1]) : take_bf16(x[s][2 * k], x[s][2 * k + 1]);
    return scale;
  }
};

// A lane's pieces of the two key rows it holds of a 16-key tile.
template <int KVT, int D, bool QB>
struct KeyFrag {
  using Geo = MassGeom<KVT, D, QB>;
  uint4 lo[Geo::NPT], hi[Geo::NPT];  // rows g4 and g4 + 8

  // rows: the tile's first key row (16 consecutive slots of one page)
  __device__ __forceinline__ void load(const unsigned char* rows, int g4, int t4) {
    const unsigned char* r = rows + static_cast<size_t>(g4) * Geo::RB + t4 * 16;
#pragma unroll
    for (int i = 0; i < Geo::NPT; ++i) {
      lo[i] = ldg_stream(r + 64 * i);
      hi[i] = ldg_stream(r + 8 * Geo::RB + 64 * i);
    }
  }
  __device__ __forceinline__ static uint4 ldg_stream(const unsigned char* a) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(a));
    return v;
  }

  // c[n] += K . Q of NT column groups
  template <int NT>
  __device__ __forceinline__ void score(const QueryFrag<KVT, D, QB> (&q)[NT], float (&c)[NT][4]) const {
#pragma unroll
    for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
#pragma unroll
    for (int i = 0; i < Geo::NPT; ++i) {
      const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w}, hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
      if constexpr (KVT == KV_BF16) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a[4] = {lw[2 * j], hw[2 * j], lw[2 * j + 1], hw[2 * j + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int part = 0; part < Geo::QP; ++part)
              mass_mma_bf16(c[n], a, q[n].b[part][2 * i + j][0], q[n].b[part][2 * i + j][1]);
        }
      } else if constexpr (KVT == KV_E4M3) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {e4m3x2_to_f16x2(lw[j], true), e4m3x2_to_f16x2(hw[j], true),
                                 e4m3x2_to_f16x2(lw[j], false), e4m3x2_to_f16x2(hw[j], false)};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int part = 0; part < Geo::QP; ++part)
              mma_f16_16816(c[n], a, q[n].b[part][4 * i + j][0], q[n].b[part][4 * i + j][1]);
        }
      } else {
        float l[4], h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) l[k] = __uint_as_float(lw[k]), h[k] = __uint_as_float(hw[k]);
#pragma unroll
        for (int kp = 0; kp < Geo::KP; ++kp) {
          const uint32_t a[4] = {take_bf16(l[0], l[1]), take_bf16(h[0], h[1]), take_bf16(l[2], l[3]),
                                 take_bf16(h[2], h[3])};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int part = 0; part < Geo::QP; ++part)
              if (kp + part < 3) mass_mma_bf16(c[n], a, q[n].b[part][i][0], q[n].b[part][i][1]);
        }
      }
    }
  }
};

// A lane's running (maximum, sum) of one column, over the keys that it sees.
struct ColumnStat {
  float m, l;
  // N scores more (log2 domain); a NaN among them makes the sum NaN
  template <int N>
  __device__ __forceinline__ void add(const float (&s)[N]) {
    float top = m;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, s[i]);
    if (top > m) {
      l = __fmul_rn(l, ex2(__fsub_rn(m, top)));
      m = top;
    }
    const float ref = m == -INFINITY ? 0.0f : m;  // every score so far is -infinity: weights 0
    float w = ex2(__fsub_rn(s[0], ref));
#pragma unroll
    for (int i = 1; i < N; ++i) w = __fadd_rn(w, ex2(__fsub_rn(s[i], ref)));
    l = __fadd_rn(l, w);
  }
  // (scale: of maxima in another measure than log2)
  __device__ __forceinline__ void merge(float om, float ol, float scale = 1.0f) {
    const float top = fmaxf(m, om);
    const float a = m == top ? 1.0f : ex2(__fmul_rn(__fsub_rn(m, top), scale)), b = om == top ? 1.0f : ex2(__fmul_rn(__fsub_rn(om, top), scale));
    l = __fadd_rn(__fmul_rn(l, a), __fmul_rn(ol, b));
    m = top;
  }
};

// ----------------------------------------------- operands outside their parts --
//
// Parts of a value cannot stand for an infinity (what is left of it is inf - inf, and a
// zero part times infinity is NaN too), nor for an f32 above the largest bf16, which
// rounds to one.  A dot product with such an operand comes out right or NaN, and its
// column's sum then NaN: a lane that finds its share of one so takes the scores again
// from the operands themselves, in FP32, until the sum is NaN once more.  Other
// columns keep their bits, and where no sum is NaN nothing is added to the loops (a
// test of every score took 1923 us instead of 1335 for the windows of f32 queries below).
// Keys and queries of one bf16 part need none of this, nor e4m3 keys (no
// infinities; a query that is not finite has no weights at all).
template <int KVT, bool QB>
__host__ __device__ constexpr bool in_parts() { return KVT == KV_F32 || (KVT == KV_BF16 && !QB); }

template <int KVT, int D, bool QB>
__device__ float whole_dot(const MassParams& p, const int32_t* table, int h, int t, int row, int head) {
  const int lg_p = 31 - __clz(p.P), page = __ldg(table + (t >> lg_p));
  if (page < 0 || page >= p.num_pages) return 0.0f;  // a row that adds nothing
  const size_t k0 = (((static_cast<size_t>(page) * p.Hkv + h) << lg_p) + (t & (p.P - 1))) * D;
  const size_t q0 = (static_cast<size_t>(row) * p.Hq + head) * D;
  float s = 0.0f;
#pragma unroll 4
  for (int d = 0; d < D; ++d) {
    const float k = KVT == KV_F32 ? __ldg(static_cast<const float*>(p.k_pool) + k0 + d)
                                  : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p.k_pool) + k0 + d)) << 16);
    const float q = QB ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p.q) + q0 + d)) << 16)
                       : __ldg(static_cast<const float*>(p.q) + q0 + d);
    s = fmaf(q, k, s);
  }
  return s;
}

// One column's log2-domain scores of keys t and t + 8 (-infinity where its row, at position pos, does not see them).
template <int KVT, int D, bool QB>
__device__ __noinline__ float2 whole_scores(const MassParams& p, const int32_t* table, int h, int t, int pos, int row, int head) {
  const float f = p.qk_scale_log2_h[PA_HEAD(p, h)];
  return make_float2(t <= pos ? __fmul_rn(whole_dot<KVT, D, QB>(p, table, h, t, row, head), f) : -INFINITY,
                     t + 8 <= pos ? __fmul_rn(whole_dot<KVT, D, QB>(p, table, h, t + 8, row, head), f) : -INFINITY);
}

// The tensor-map-free address of token t's K row of kv head h (t % 16 == 0), or
// of page 0 where the page id is out of range (`bad` is set then).
template <int RB>
__device__ __forceinline__ const unsigned char* key_rows(const MassParams& p, int page, int h, int t, int lg_p, bool& bad) {
  if (page < 0 || page >= p.num_pages) {
    bad = true;
    page = 0;
  }
  return static_cast<const unsigned char*>(p.k_pool) +
         (((static_cast<size_t>(page) * p.Hkv + h) << lg_p) + (t & ((1 << lg_p) - 1))) * RB;
}

__device__ __forceinline__ bool mass_row_in_chunk(const MassParams& p, int row) {
  for (int c = 0; c < p.n_chunks; ++c)
    if (row >= p.chunk_begin[c] && row < p.chunk_end[c]) return true;
  return false;
}

// ------------------------------------------------------------------ rows --

// Stride between the heads' score rows: 4 banks apart, so that the four lanes
// that hold a key's columns write to different banks.
__host__ __device__ constexpr int score_stride(int keys) { return (keys + 31) / 32 * 32 + 4; }

// One cluster per (row, kv head).  The row's 16-key tiles are dealt to the CTAs
// in contiguous shares of its own length, and within a CTA to the warps in
// turn, MT at a time (4 KB of K, 8 KB with f32); the loads of a warp's next tiles
// in flight while it scores one's.
//
// Bound by the one read of K: 512 ragged rows of up to 2662 keys (16 query heads
// over 8, bf16) take 226 us, 6.5 TB/s; 32 rows of 32768 keys (32 heads over 8,
// e4m3) 217 us, 5.0 TB/s: there the loads' latency shows (DRAM 62% busy, issue slots
// 36%, most warps waiting for K), with 4 KB of K ahead for each of an SM's 16 warps and
// more to do between two loads.  f32 queries over bf16 take 309 us for the ragged
// rows, f32 pools 535 (bf16 queries) and 608.  A weight costs one exponential
// per score twice (the running sum, the weight); the score itself is kept, not
// recomputed, as far as the CTA's room goes: 104 KB, 3744 keys of 7 query heads and 3264
// of 8.  Keys beyond are read and scored a second time (64 rows of 4000 to 4096
// keys: 98 us with 4 query heads, 170 with 7, 188 with 8).  4 KB of K to a warp's step, in one CTA: 225 us; 16-key tiles one by
// one in CTAs of 2048 keys: 256.  Few short rows (4 of up to 900 keys) are latency: 6 us.
template <int KVT, int D, bool QB>
__global__ void __launch_bounds__(kMassThreads, MassGeom<KVT, D, QB>::RB > 256 ? 1 : 2) mass_row_kernel(const __grid_constant__ MassParams p) {
  using Geo = MassGeom<KVT, D, QB>;
  extern __shared__ float scores[];  // [G][score_stride(score_keys)]
  __shared__ float2 warp_stat[kMassWarps][8];
  __shared__ float2 cta_stat[8];
  __shared__ int cta_bad, cta_whole;
  __shared__ float2 row_stat[8];  // (maximum, 1 / sum) of the whole row
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x % p.cluster, unit = blockIdx.x / p.cluster;
  const int h = unit % p.Hkv, row = unit / p.Hkv;
  if (mass_row_in_chunk(p, row)) return;  // the whole cluster leaves
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
  const int G = p.Hq / p.Hkv, lg_p = 31 - __clz(p.P);
  const int seq = __ldg(p.seq_ids + row), pos = __ldg(p.positions + row);
  if (seq < 0 || seq >= p.num_seqs || pos < 0 || pos >= p.max_blocks * p.P) {
    if (rank == 0 && tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
    return;
  }
  constexpr int MT = Geo::MT;
  const int tiles = (pos + 16) / 16, share = (tiles + p.cluster * MT - 1) / (p.cluster * MT) * MT;
  const int tile0 = min(tiles, rank * share), mine = min(tiles, tile0 + share) - tile0;  // this CTA's tiles
  const int stride = score_stride(p.score_keys);
  const int32_t* table = p.block_tables + static_cast<size_t>(seq) * p.max_blocks;
  if (tid == 0) cta_bad = cta_whole = 0;

  QueryFrag<KVT, D, QB> q[1];
  const float factor = q[0].load(p, g4 < G ? row : -1, h * G + g4, p.qk_scale_log2_h[PA_HEAD(p, h)], t4);
  // this lane's columns are 2 t4 and 2 t4 + 1: their factors sit in the lanes of those groups
  const float f0 = __shfl_sync(0xffffffffu, factor, 8 * t4), f1 = __shfl_sync(0xffffffffu, factor, 8 * t4 + 4);
  __syncthreads();

  bool bad = false;
  // the warp's k-th MT tiles start at the CTA's tile (warp + 8 k) MT; page ids of the next 32 tiles, one to a lane
  int pages = 0;
  auto load = [&](int k, KeyFrag<KVT, D, QB>(&f)[MT]) {
    if (k % (32 / MT) == 0) {
      const int t = (tile0 + (warp + (k + lane / MT) * kMassWarps) * MT + lane % MT) * 16;
      pages = t <= pos ? __ldg(table + (t >> lg_p)) : 0;
    }
#pragma unroll
    for (int s = 0; s < MT; ++s) {
      const int page = __shfl_sync(0xffffffffu, pages, k % (32 / MT) * MT + s);
      f[s].load(key_rows<Geo::RB>(p, page, h, (tile0 + (warp + k * kMassWarps) * MT + s) * 16, lg_p, bad), g4, t4);
    }
  };
  // log2-domain scores of a 16-key tile (-infinity behind the row's position)
  auto scores_of = [&](const KeyFrag<KVT, D, QB>& f, int t0, float (&c)[4]) {
    float raw[1][4];
    f.score(q, raw);
    c[0] = __fmul_rn(raw[0][0], f0), c[1] = __fmul_rn(raw[0][1], f1);
    c[2] = __fmul_rn(raw[0][2], f0), c[3] = __fmul_rn(raw[0][3], f1);
    if (t0 + 15 > pos) {
      if (t0 + g4 > pos) c[0] = c[1] = -INFINITY;
      if (t0 + g4 + 8 > pos) c[2] = c[3] = -INFINITY;
    }
  };
  ColumnStat st0{-INFINITY, 0.0f}, st1{-INFINITY, 0.0f};
  const int count = mine > warp * MT ? (mine - warp * MT + kMassWarps * MT - 1) / (kMassWarps * MT) : 0;  // of this warp
  auto step = [&](int k, KeyFrag<KVT, D, QB>(&now)[MT], KeyFrag<KVT, D, QB>(&next)[MT]) {
    if (k + 1 < count) load(k + 1, next);
    float even[2 * MT], odd[2 * MT];  // columns 2 t4 and 2 t4 + 1
#pragma unroll
    for (int s = 0; s < MT; ++s) {
      const int local = (warp + k * kMassWarps) * MT + s;
      float c[4];
      scores_of(now[s], (tile0 + local) * 16, c);
      even[2 * s] = c[0], even[2 * s + 1] = c[2];
      odd[2 * s] = c[1], odd[2 * s + 1] = c[3];
      if (local * 16 < p.score_keys) {
        float* z = scores + 2 * t4 * stride + local * 16 + g4;
        if (2 * t4 < G) z[0] = c[0], z[8] = c[2];
        if (2 * t4 + 1 < G) z[stride] = c[1], z[stride + 8] = c[3];
      }
    }
    st0.add(even);
    st1.add(odd);
  };
  KeyFrag<KVT, D, QB> x[MT], y[MT];
  if (count > 0) load(0, x);
  for (int k = 0; k < count; k += 2) {
    step(k, x, y);
    if (k + 1 < count) step(k + 1, y, x);
  }
  if constexpr (in_parts<KVT, QB>()) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // this lane's share of a column
      ColumnStat& st = k == 0 ? st0 : st1;
      if (2 * t4 + k >= G || st.l == st.l) continue;
      st = ColumnStat{-INFINITY, 0.0f};
#pragma unroll 1
      for (int i = 0; i < count * MT && st.l == st.l; ++i) {
        const int local = (warp + i / MT * kMassWarps) * MT + i % MT;
        const float2 c = whole_scores<KVT, D, QB>(p, table, h, (tile0 + local) * 16 + g4, pos, row, h * G + 2 * t4 + k);
        if (local * 16 < p.score_keys) {
          float* z = scores + (2 * t4 + k) * stride + local * 16 + g4;
          z[0] = c.x, z[8] = c.y;
        }
        const float two[2] = {c.x, c.y};
        st.add(two);
      }
      if (st.l == st.l) cta_whole = 1;
    }
    __syncwarp();
  }
  // (max, sum) of each column: over the lanes of a warp, the warps, the CTAs
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    st0.merge(__shfl_xor_sync(0xffffffffu, st0.m, off), __shfl_xor_sync(0xffffffffu, st0.l, off));
    st1.merge(__shfl_xor_sync(0xffffffffu, st1.m, off), __shfl_xor_sync(0xffffffffu, st1.l, off));
  }
  if (g4 == 0) {
    warp_stat[warp][2 * t4] = make_float2(st0.m, st0.l);
    warp_stat[warp][2 * t4 + 1] = make_float2(st1.m, st1.l);
  }
  if (bad) cta_bad = 1;
  __syncthreads();
  if (tid < 8) {
    ColumnStat s{-INFINITY, 0.0f};
    for (int w = 0; w < kMassWarps; ++w) s.merge(warp_stat[w][tid].x, warp_stat[w][tid].y);
    cta_stat[tid] = make_float2(s.m, s.l);
  }
  cluster.sync();
  int any_bad = 0;
  if (tid < 8) {
    ColumnStat s{-INFINITY, 0.0f};
    for (int r = 0; r < p.cluster; ++r) {
      const float2 o = cluster.map_shared_rank(cta_stat, r)[tid];
      any_bad |= *cluster.map_shared_rank(&cta_bad, r);
      s.merge(o.x, o.y);
    }
    row_stat[tid] = make_float2(s.m, __fdiv_rn(1.0f, s.l));
  }
  __syncwarp();
  cluster.barrier_arrive();  // this CTA has read the others'
  if (__syncthreads_or(any_bad)) {  // a page out of range: the row adds nothing
    if (rank == 0 && tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
  } else {
    float* sums = p.mass + (static_cast<size_t>(seq) * p.Hkv + h) * (static_cast<size_t>(p.max_blocks) << lg_p);
    const int first = tile0 * 16, stored = min(min(mine * 16, p.score_keys), pos + 1 - first);
    float2 rs[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) rs[g] = row_stat[g];
    for (int t = tid; t < stored; t += kMassThreads) {
      float w = 0.0f;
#pragma unroll
      for (int g = 0; g < 8; ++g)
        if (g < G) w = fmaf(ex2(__fsub_rn(scores[g * stride + t], rs[g].x)), rs[g].y, w);
      atomicAdd(sums + first + t, w);  // one writer a key: the order of additions is the calls'
    }
    // keys whose scores found no room: scored again
    const float2 r0 = row_stat[2 * t4], r1 = row_stat[2 * t4 + 1];
    for (int local = p.score_keys / 16 + warp; local < mine; local += kMassWarps) {
      const int t0 = (tile0 + local) * 16;
      KeyFrag<KVT, D, QB> f;
      f.load(key_rows<Geo::RB>(p, __ldg(table + (t0 >> lg_p)), h, t0, lg_p, bad), g4, t4);
      float c[4];
      scores_of(f, t0, c);
      if constexpr (in_parts<KVT, QB>()) {
        if (cta_whole) {
#pragma unroll 1
          for (int k = 0; k < 2 && 2 * t4 + k < G; ++k) {
            const float2 w = whole_scores<KVT, D, QB>(p, table, h, t0 + g4, pos, row, h * G + 2 * t4 + k);
            if (k == 0) c[0] = w.x, c[2] = w.y;
            else c[1] = w.x, c[3] = w.y;
          }
        }
      }
      float w0 = 0.0f, w1 = 0.0f;
      if (2 * t4 < G) {
        w0 = __fmul_rn(ex2(__fsub_rn(c[0], r0.x)), r0.y);
        w1 = __fmul_rn(ex2(__fsub_rn(c[2], r0.x)), r0.y);
      }
      if (2 * t4 + 1 < G) {
        w0 = fmaf(ex2(__fsub_rn(c[1], r1.x)), r1.y, w0);
        w1 = fmaf(ex2(__fsub_rn(c[3], r1.x)), r1.y, w1);
      }
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        w0 = __fadd_rn(w0, __shfl_xor_sync(0xffffffffu, w0, off));
        w1 = __fadd_rn(w1, __shfl_xor_sync(0xffffffffu, w1, off));
      }
      if (t4 == 0 && t0 + g4 <= pos) atomicAdd(sums + t0 + g4, w0);
      if (t4 == 0 && t0 + g4 + 8 <= pos) atomicAdd(sums + t0 + g4 + 8, w1);
    }
  }
  __syncwarp();
  cluster.barrier_wait();  // no CTA leaves while another may read its (max, sum)
}

// ---------------------------------------------------------------- chunks --

// A chunk as the launches see it: its rows (consecutive positions of one
// sequence, checked by the launch before) and its columns, column c being head
// c % G of row c / G.
struct ChunkView {
  int rows, row0, seq, pos0, last;  // last: the last row's position
  const int32_t* table;

  // false for a chunk that adds nothing
  __device__ __forceinline__ bool open(const MassParams& p, int c) {
    const int2 head = __ldcg(p.ws_head + c);
    row0 = p.chunk_begin[c];
    rows = p.chunk_end[c] - row0;
    seq = head.x;
    pos0 = head.y;
    last = pos0 + rows - 1;
    table = p.block_tables + static_cast<size_t>(max(seq, 0)) * p.max_blocks;
    return seq >= 0;
  }
};

// A column's (maximum, 1 / sum) over the key ranges that a row at `pos` sees,
// merged in ascending order: slot `slot` of the chunk's tile `tile`.  (The tile path's maxima are scores as the
// MMAs give them, to be scaled.)
__device__ __forceinline__ float2 column_stat(const MassParams& p, int c, int h, int tile, int slot,
                                              int pos, float scale = 1.0f) {
  const size_t stride = static_cast<size_t>(p.chunk_tiles[c]) * kMassSlots;
  const float2* s = p.ws_part + p.chunk_part[c] + static_cast<size_t>(h) * p.n_splits * stride +
                    static_cast<size_t>(tile) * kMassSlots + slot;
  const int n = pos / kMassSplitKeys + 1;
  ColumnStat st{-INFINITY, 0.0f};
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float2 o = __ldcg(s + k * stride);
    st.merge(o.x, o.y, scale);
  }
  return make_float2(st.m, __fdiv_rn(1.0f, st.l));
}

// A lane's share of key t's weight (columns 2 t4 and 2 t4 + 1 of every 8) from whole operands.
template <int KVT, int D, bool QB>
__device__ __noinline__ float whole_weight(const MassParams& p, const ChunkView& v, int c, int h, int t, int t4) {
  const int G = p.Hq / p.Hkv;
  float w = 0.0f;
#pragma unroll 1
  for (int i = max(0, t - v.pos0) * G / 8 * 2; w == w; ++i) {  // no row before that one sees the key
    const int col = i / 2 * 8 + 2 * t4 + i % 2, row = col / G, pos = v.pos0 + row;
    if (i / 2 * 8 >= v.rows * G) break;
    if (row >= v.rows || pos < t) continue;
    const int slot = column_slot(col, G);
    const float2 z = column_stat(p, c, h, slot / kMassSlots, slot % kMassSlots, pos);
    w = fmaf(ex2(__fsub_rn(whole_scores<KVT, D, QB>(p, v.table, h, t, pos, v.row0 + row, h * G + col % G).x, z.x)), z.y, w);
  }
  return w;
}

// A CTA's columns, in groups of 8: a warp prepares a group's query fragments for
// all, in shared memory, and a key tile meets NT groups at a time (held to about
// 64 registers of fragments).
template <int KVT, int D, bool QB>
struct ChunkGeom {
  using Geo = MassGeom<KVT, D, QB>;
  static constexpr int NT = Geo::QP == 1 ? 4 : Geo::QP == 2 ? 2 : 1;
  static constexpr int GROUPS = Geo::QP == 3 ? 4 : 8;
  static constexpr int COLS = 8 * GROUPS;
  static constexpr int VECS = Geo::QP * Geo::STEPS * 2 / 4;  // 16-byte vectors of a lane's fragments
  static constexpr bool AHEAD = Geo::RB <= 256;              // room for the next key tile's fragments
  static_assert(GROUPS <= kMassWarps && GROUPS % NT == 0, "a warp prepares a group");
};

template <int KVT, int D, bool QB>
struct ChunkQueries {
  using Cg = ChunkGeom<KVT, D, QB>;
  uint4 frag[Cg::GROUPS][Cg::VECS][32];
  float factor[Cg::COLS];

  // Each of the first warps prepares its group of the columns from col0 on; the caller meets before and behind.
  __device__ __forceinline__ void prepare(const MassParams& p, const ChunkView& v, int h, int col0, int cols, int G, int warp, int g4, int t4) {
    if (warp >= Cg::GROUPS) return;
    const int col = col0 + 8 * warp + g4;
    QueryFrag<KVT, D, QB> q;
    const float f = q.load(p, col < cols ? v.row0 + col / G : -1, h * G + col % G, p.qk_scale_log2_h[PA_HEAD(p, h)], t4);
    if (t4 == 0) factor[8 * warp + g4] = f;
    const uint32_t* b = &q.b[0][0][0];
#pragma unroll
    for (int i = 0; i < Cg::VECS; ++i) frag[warp][i][4 * g4 + t4] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
  }
  __device__ __forceinline__ void get(int group, int lane, QueryFrag<KVT, D, QB>& q) const {
    uint32_t* b = &q.b[0][0][0];
#pragma unroll
    for (int i = 0; i < Cg::VECS; ++i) {
      const uint4 x = frag[group][i][lane];
      b[4 * i] = x.x, b[4 * i + 1] = x.y, b[4 * i + 2] = x.z, b[4 * i + 3] = x.w;
    }
  }
};

// The warp-level launches serve f32 and e4m3 pools and f32 queries; bf16 queries
// over bf16 pools have the tile path.  Eight windows of 64 rows over 4k-16k keys (32
// heads over 8) take 545 us with an e4m3 pool (f32 queries 700), 1305 with f32
// queries over a bf16 one, 1229 with bf16 queries over an f32 one, 2649 with f32
// both.  Bound by latency, not by a unit (issue slots 30% to 48% busy, tensor pipe 23% to
// 48%, DRAM 3% to 5%): 8 or 16 warps to an SM, for their fragments' registers, and in each a
// chain of conversions, MMAs and exponentials.  Fragments prepared by every warp for
// itself took twice the time.
//
// First launch: one CTA per (chunk, kv head, key range, column block).  The
// CTA's warps take the range's 16-key tiles in turn.
template <int KVT, int D, bool QB>
__global__ void __launch_bounds__(kMassThreads) chunk_stats_kernel(const __grid_constant__ MassParams p) {
  using Geo = MassGeom<KVT, D, QB>;
  using Cg = ChunkGeom<KVT, D, QB>;
  __shared__ ChunkQueries<KVT, D, QB> sq;
  __shared__ float2 warp_stat[kMassWarps][Cg::COLS];
  int c = 0;
  while (c + 1 < p.n_chunks && static_cast<int>(blockIdx.x) >= p.chunk_cta[c + 1]) ++c;
  const int local = blockIdx.x - p.chunk_cta[c];
  const int h = local % p.Hkv, split = (local / p.Hkv) % p.n_splits, block = local / p.Hkv / p.n_splits;
  const int G = p.Hq / p.Hkv, lg_p = 31 - __clz(p.P);
  ChunkView v;
  if (!v.open(p, c)) return;
  const int cols = v.rows * G, col0 = block * Cg::COLS, col_end = min(cols, col0 + Cg::COLS);
  const int key0 = split * kMassSplitKeys;
  const int top = v.pos0 + (col_end - 1) / G;  // the last key any of the columns sees
  const int key_end = min(top + 1, key0 + kMassSplitKeys);
  if (key0 >= key_end) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
  sq.prepare(p, v, h, col0, cols, G, warp, g4, t4);
  int lim[Cg::GROUPS][2];  // last key of the lane's columns
  ColumnStat st[Cg::GROUPS][2];
#pragma unroll
  for (int n = 0; n < Cg::GROUPS; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      lim[n][k] = v.pos0 + (col0 + 8 * n + 2 * t4 + k) / G;
      st[n][k] = ColumnStat{-INFINITY, 0.0f};
    }
  __syncthreads();
  bool bad = false;
  auto load = [&](int t0, KeyFrag<KVT, D, QB>& a) {
    if (t0 < key_end) a.load(key_rows<Geo::RB>(p, __ldg(v.table + (t0 >> lg_p)), h, t0, lg_p, bad), g4, t4);
  };
  auto step = [&](int t0, KeyFrag<KVT, D, QB>& now, KeyFrag<KVT, D, QB>& next) {
    if (t0 >= key_end) return;
    if (Cg::AHEAD) load(t0 + kMassWarps * 16, next);
    else load(t0, now);
#pragma unroll
    for (int n0 = 0; n0 < Cg::GROUPS; n0 += Cg::NT) {
      if (col0 + 8 * n0 >= cols) break;
      QueryFrag<KVT, D, QB> q[Cg::NT];
#pragma unroll
      for (int n = 0; n < Cg::NT; ++n) sq.get(n0 + n, lane, q[n]);
      float s[Cg::NT][4];
      now.score(q, s);
#pragma unroll
      for (int n = 0; n < Cg::NT; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(sq.factor + 8 * (n0 + n) + 2 * t4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float fk = k == 0 ? f.x : f.y;
          const float z[2] = {t0 + g4 <= lim[n0 + n][k] ? __fmul_rn(s[n][k], fk) : -INFINITY,
                              t0 + g4 + 8 <= lim[n0 + n][k] ? __fmul_rn(s[n][2 + k], fk) : -INFINITY};
          st[n0 + n][k].add(z);
        }
      }
    }
  };
  KeyFrag<KVT, D, QB> x, y;
  if (Cg::AHEAD) load(key0 + warp * 16, x);
  for (int t0 = key0 + warp * 16; t0 < key_end; t0 += 2 * kMassWarps * 16) {
    step(t0, x, y);
    step(t0 + kMassWarps * 16, y, x);
  }
  if constexpr (in_parts<KVT, QB>()) {
#pragma unroll
    for (int n = 0; n < Cg::GROUPS; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // this lane's share of a column
        const int col = col0 + 8 * n + 2 * t4 + k;
        if (col >= cols || st[n][k].l == st[n][k].l) continue;
        ColumnStat again{-INFINITY, 0.0f};
#pragma unroll 1
        for (int t0 = key0 + warp * 16; t0 < key_end && again.l == again.l; t0 += kMassWarps * 16) {
          const float2 z = whole_scores<KVT, D, QB>(p, v.table, h, t0 + g4, lim[n][k], v.row0 + col / G, h * G + col % G);
          const float two[2] = {z.x, z.y};
          again.add(two);
        }
        st[n][k] = again;
        if (again.l == again.l) p.ws_whole[c] = 1;
      }
    __syncwarp();
  }
#pragma unroll
  for (int n = 0; n < Cg::GROUPS; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        st[n][k].merge(__shfl_xor_sync(0xffffffffu, st[n][k].m, off), __shfl_xor_sync(0xffffffffu, st[n][k].l, off));
      if (g4 == 0) warp_stat[warp][8 * n + 2 * t4 + k] = make_float2(st[n][k].m, st[n][k].l);
    }
  __syncthreads();
  if (tid < Cg::COLS && col0 + tid < cols) {
    ColumnStat s{-INFINITY, 0.0f};
    for (int w = 0; w < kMassWarps; ++w) s.merge(warp_stat[w][tid].x, warp_stat[w][tid].y);
    p.ws_part[p.chunk_part[c] + (static_cast<size_t>(h) * p.n_splits + split) * p.chunk_tiles[c] * kMassSlots +
              column_slot(col0 + tid, G)] = make_float2(s.m, s.l);
  }
}

// Last launch: one CTA per (chunk, kv head, block of 512 keys).  A warp has four
// 16-key tiles of them and goes over the columns that see the block, a CTA's
// groups of columns at a time.
template <int KVT, int D, bool QB>
__global__ void __launch_bounds__(kMassThreads) chunk_weights_kernel(const __grid_constant__ MassParams p) {
  using Geo = MassGeom<KVT, D, QB>;
  using Cg = ChunkGeom<KVT, D, QB>;
  constexpr int TILES = kMassBlockKeys / (16 * kMassWarps);
  __shared__ ChunkQueries<KVT, D, QB> sq;
  __shared__ float2 stat[Cg::COLS];
  const int h = blockIdx.x % p.Hkv, block = (blockIdx.x / p.Hkv) % p.n_blocks, c = blockIdx.x / p.Hkv / p.n_blocks;
  const int G = p.Hq / p.Hkv, lg_p = 31 - __clz(p.P);
  ChunkView v;
  if (!v.open(p, c)) return;
  const int key0 = block * kMassBlockKeys;
  if (key0 > v.last) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
  const int cols = v.rows * G;
  bool bad = false;
  auto tile_at = [&](int i) { return key0 + (i * kMassWarps + warp) * 16; };
  auto load = [&](int i, KeyFrag<KVT, D, QB>& a) {
    const int t0 = tile_at(i);
    if (t0 <= v.last) a.load(key_rows<Geo::RB>(p, __ldg(v.table + (t0 >> lg_p)), h, t0, lg_p, bad), g4, t4);
  };
  float w0[TILES], w1[TILES];  // keys g4 and g4 + 8 of each tile
#pragma unroll
  for (int i = 0; i < TILES; ++i) w0[i] = w1[i] = 0.0f;
  // columns before the first row that sees key0 see none of the block
  for (int col0 = max(0, key0 - v.pos0) * G / Cg::COLS * Cg::COLS; col0 < cols; col0 += Cg::COLS) {
    __syncthreads();
    sq.prepare(p, v, h, col0, cols, G, warp, g4, t4);
    const int mine = tid - (kMassThreads - Cg::COLS);  // the last warps look the statistics up
    if (mine >= 0 && col0 + mine < cols) {
      const int slot = column_slot(col0 + mine, G);
      stat[mine] = column_stat(p, c, h, slot / kMassSlots, slot % kMassSlots, v.pos0 + (col0 + mine) / G);
    }
    __syncthreads();
    const int top = v.pos0 + (min(cols, col0 + Cg::COLS) - 1) / G;  // the last key that any of the columns sees
    if (tile_at(0) > top) continue;
    KeyFrag<KVT, D, QB> a[2];
    if (Cg::AHEAD) load(0, a[0]);
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int t0 = tile_at(i);
      if (t0 > top) break;
      if (!Cg::AHEAD) load(i, a[0]);
      else if (i + 1 < TILES) load(i + 1, a[(i + 1) & 1]);
#pragma unroll 1
      for (int n0 = 0; n0 < Cg::GROUPS && col0 + 8 * n0 < cols; n0 += Cg::NT) {
        QueryFrag<KVT, D, QB> q[Cg::NT];
#pragma unroll
        for (int n = 0; n < Cg::NT; ++n) sq.get(n0 + n, lane, q[n]);
        float s[Cg::NT][4];
        a[Cg::AHEAD ? i & 1 : 0].score(q, s);
#pragma unroll
        for (int n = 0; n < Cg::NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int at = 8 * (n0 + n) + 2 * t4 + k, col = col0 + at;
            if (col < cols) {
              const int lim = v.pos0 + col / G;
              const float f = sq.factor[at];
              const float2 z = stat[at];
              if (t0 + g4 <= lim) w0[i] = fmaf(ex2(__fsub_rn(__fmul_rn(s[n][k], f), z.x)), z.y, w0[i]);
              if (t0 + g4 + 8 <= lim) w1[i] = fmaf(ex2(__fsub_rn(__fmul_rn(s[n][2 + k], f), z.x)), z.y, w1[i]);
            }
          }
      }
    }
  }
  if constexpr (in_parts<KVT, QB>()) {
    if (__ldcg(p.ws_whole + c) != 0) {
#pragma unroll
      for (int i = 0; i < TILES; ++i) {
        if (w0[i] != w0[i]) w0[i] = whole_weight<KVT, D, QB>(p, v, c, h, tile_at(i) + g4, t4);
        if (w1[i] != w1[i]) w1[i] = whole_weight<KVT, D, QB>(p, v, c, h, tile_at(i) + g4 + 8, t4);
      }
      __syncwarp();
    }
  }
  float* sums = p.mass + (static_cast<size_t>(v.seq) * p.Hkv + h) * (static_cast<size_t>(p.max_blocks) << lg_p);
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    const int t0 = tile_at(i);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      w0[i] = __fadd_rn(w0[i], __shfl_xor_sync(0xffffffffu, w0[i], off));
      w1[i] = __fadd_rn(w1[i], __shfl_xor_sync(0xffffffffu, w1[i], off));
    }
    if (t4 == 0 && t0 + g4 <= v.last) atomicAdd(sums + t0 + g4, w0[i]);
    if (t4 == 0 && t0 + g4 + 8 <= v.last) atomicAdd(sums + t0 + g4 + 8, w1[i]);
  }
}

// -------------------------------------------------------------- launches --

// More than 8 CTAs to a cluster have to be allowed, once per device.
template <typename Kernel>
cudaError_t allow_wide_clusters(Kernel kernel, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// The tensor-core tile launches (bf16 queries and pool): the columns'
// statistics, or with `weights` the weights.
cudaError_t launch_mass_tiles(const MassParams& p, bool weights, cudaStream_t stream);

// What one call to a launcher runs, in this order.
enum MassLaunch { MASS_ROWS, MASS_CHUNK_STATS, MASS_CHUNK_WEIGHTS };

template <int KVT, int D, bool QB>
cudaError_t launch_mass_inst(const MassParams& p0, MassLaunch what, cudaStream_t stream) {
  MassParams p = p0;
  const int G = p.Hq / p.Hkv;
  if (what == MASS_ROWS) {
    const size_t smem = static_cast<size_t>(G) * score_stride(p.score_keys) * sizeof(float);
    static std::atomic<unsigned long long> smem_done{0};
    const cudaError_t e = allow_dynamic_smem(mass_row_kernel<KVT, D, QB>, smem_done, kMassScoreBytes);
    if (e != cudaSuccess) return e;
    if (p.cluster > 8) {
      static std::atomic<unsigned long long> wide_done{0};
      const cudaError_t w = allow_wide_clusters(mass_row_kernel<KVT, D, QB>, wide_done);
      if (w != cudaSuccess) return w;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.n_rows) * p.Hkv * p.cluster);
    cfg.blockDim = dim3(kMassThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(p.cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, mass_row_kernel<KVT, D, QB>, p);
  }
  if constexpr (KVT == KV_BF16 && QB) {
    return launch_mass_tiles(p, what == MASS_CHUNK_WEIGHTS, stream);
  } else {
    constexpr int COLS = ChunkGeom<KVT, D, QB>::COLS;
    long long ctas = 0;
    for (int c = 0; c < p.n_chunks; ++c) {
      p.chunk_cta[c] = static_cast<int32_t>(ctas);
      const long long cols = static_cast<long long>(p.chunk_end[c] - p.chunk_begin[c]) * G;
      ctas += (cols + COLS - 1) / COLS * p.Hkv * p.n_splits;
      if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    }
    p.chunk_cta[p.n_chunks] = static_cast<int32_t>(ctas);
    const long long blocks = static_cast<long long>(p.n_chunks) * p.Hkv * p.n_blocks;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (what == MASS_CHUNK_STATS)
      chunk_stats_kernel<KVT, D, QB><<<static_cast<unsigned>(ctas), kMassThreads, 0, stream>>>(p);
    else
      chunk_weights_kernel<KVT, D, QB><<<static_cast<unsigned>(blocks), kMassThreads, 0, stream>>>(p);
    count_launch();
    return cudaGetLastError();
  }
}

template <int KVT>
cudaError_t launch_mass_dispatch(const MassParams& p, MassLaunch what, cudaStream_t stream) {
  if (p.D == 64) return p.q_is_bf16 ? launch_mass_inst<KVT, 64, true>(p, what, stream) : launch_mass_inst<KVT, 64, false>(p, what, stream);
  return p.q_is_bf16 ? launch_mass_inst<KVT, 128, true>(p, what, stream) : launch_mass_inst<KVT, 128, false>(p, what, stream);
}

// One translation unit per K dtype.
cudaError_t launch_mass_f32(const MassParams& p, MassLaunch what, cudaStream_t stream);
cudaError_t launch_mass_bf16(const MassParams& p, MassLaunch what, cudaStream_t stream);
cudaError_t launch_mass_e4m3(const MassParams& p, MassLaunch what, cudaStream_t stream);

}  // namespace pa
