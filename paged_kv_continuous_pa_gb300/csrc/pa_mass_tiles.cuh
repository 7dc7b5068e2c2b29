// pa_mass_tiles.cuh -- the chunks' launches of pa_attention_mass on the
// 5th-generation tensor cores (bf16 queries and pool, chunks of at least
// kMinTileRows rows).
//
// A chunk's columns for kv head h are its (row, query head) pairs, 128 / G rows
// to a tile of 128 columns.
//   mass_tile_kernel<D, false>: per (tile, key range) every column's maximum and
//     sum.  S = Q K^T with the tile's queries in tensor memory and key tiles of 128
//     streamed; a thread owns a column (one lane of S) and goes over the keys.
//   mass_tile_kernel<D, true>: per range of kMassRangeKeys keys the weights.
//     S^T = K Q^T with a tile's queries and their statistics resident and the key
//     tiles streamed; a thread owns a key (one lane of S^T) and sums the weights of
//     the columns, tile after tile in order, in an accumulator that only it
//     writes.  One addition to the buffer per key.
// Both run ten warps: eight turn scores into sums (two groups of four, taking
// key tiles in turn), one issues the copies, one the MMAs; they meet at
// mbarriers only.  Three S buffers in tensor memory and three key tiles in
// shared memory keep the tensor pipe fed while the exponentials run.
//
// The scores are computed twice (a weight needs its column's sum over all
// keys first): 4 D operations and two exponentials per visible (row, head, key).
// Every wait is bounded; a call that gives up adds nothing and reports it.
#pragma once

#include "pa_mass.cuh"
#include "pa_prefill.cuh"

namespace pa {

constexpr int kMtThreads = 320;   // eight score warps, a copy warp, an MMA warp
constexpr int kMtKeys = 128;      // keys of a key tile
constexpr int kMtBuffers = 3;     // S buffers, and key tiles in shared memory
constexpr int kMtCopyWarp = 8, kMtMmaWarp = 9;

template <int D, bool W>
struct MassTileSmem {  // byte offsets from a 1024-byte aligned base
  static constexpr int NH = D / 64;            // 64-element halves of the head dim
  static constexpr int HALF = kMtKeys * 128;   // one half of a tile of 128 rows
  static constexpr int TILE = NH * HALF;
  static constexpr int Q_OFF = kMtBuffers * TILE;                // W: two query tiles
  static constexpr int STAT_OFF = Q_OFF + (W ? 2 * TILE : 0);    // W: their statistics, [max x 128][1 / sum x 128]
  static constexpr int ACC_OFF = STAT_OFF + (W ? 2 * 1024 : 0);  // W: a sum per key of the range; else the second group's (max, sum)
  static constexpr int BAR_OFF = ACC_OFF + (W ? kMassRangeKeys * 4 : 1024);
  static constexpr int TMEM_OFF = BAR_OFF + 15 * 8;
  static constexpr int PID_OFF = BAR_OFF + 128;
  static constexpr int PIDS = (W ? kMassRangeKeys : kMassSplitKeys) / 16;
  static constexpr int BYTES = PID_OFF + PIDS * 4 + 1024;        // slack for aligning the base
};

enum {
  MT_KF0 = 0,   // key tile in buffer 0 / 1 / 2 landed
  MT_SD0 = 3,   // S buffer 0 / 1 / 2 computed (its key tile is free)
  MT_SE0 = 6,   // S buffer 0 / 1 / 2 read by its four warps
  MT_QF0 = 9,   // query tile and statistics 0 / 1 landed
  MT_QE0 = 11,  // query tile 0 / 1 done with by the eight score warps
  MT_STALL = 13,
  MT_COUNT = 14
};

// 3-D tiled load of the box at (x, y, z); x * element size a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_3d(void* dst_smem, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// Key tile `tile` (keys key0 + 128 tile ..) by the lanes of one warp: a box of
// min(P, 64) keys x 64 elements per page piece and head-dim half.
template <int D>
__device__ __forceinline__ void mass_load_keys(const CUtensorMap* map, unsigned char* dst, uint64_t* bar,
                                               const int32_t* ybase, int jp0, int t0, int lg_p, int lane) {
  constexpr int NH = D / 64;
  const int lg_br = lg_p < 6 ? lg_p : 6;
  if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(kMtKeys * D * 2));
  __syncwarp();
  if (lane < (kMtKeys >> lg_br) * NH) {
    const int k = lane / NH, half = lane % NH;
    const int t = t0 + (k << lg_br);
    tc::tma_load_2d(dst + half * (kMtKeys * 128) + (k << lg_br) * 128, map, half * 64,
                    ybase[(t >> lg_p) - jp0] + (t & ((1 << lg_p) - 1)), bar);
  }
}

template <int D, bool W>
__global__ void __launch_bounds__(kMtThreads, 1) mass_tile_kernel(const __grid_constant__ MassParams p) {
  using S = MassTileSmem<D, W>;
  constexpr uint32_t kTmemQ = kMtBuffers * kMtKeys;  // W false: the queries, behind the S buffers
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S::BAR_OFF);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + S::TMEM_OFF);
  int32_t* pids = reinterpret_cast<int32_t*>(sm + S::PID_OFF);  // tensor-map rows of the pages
  float* acc = reinterpret_cast<float*>(sm + S::ACC_OFF);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.Hq / p.Hkv, R = kMtKeys / G, lg_p = 31 - __clz(p.P);

  int c = 0;
  while (c + 1 < p.n_chunks && static_cast<int>(blockIdx.x) >= p.chunk_cta[c + 1]) ++c;
  const int local = blockIdx.x - p.chunk_cta[c];
  const int h = local % p.Hkv, part = local / p.Hkv;
  const int split = W ? 0 : part % p.n_splits, tile = W ? 0 : part / p.n_splits;
  ChunkView v;
  const bool ok_chunk = v.open(p, c);
  const int key0 = W ? part * kMassRangeKeys : split * kMassSplitKeys;  // the CTA's first key
  const int row_end = W ? v.rows : min(v.rows, (tile + 1) * R);
  const int last = v.pos0 + row_end - 1;  // the last key that a row of the CTA sees
  if (!ok_chunk || key0 > last) {
    if (warp == 0) tc::tmem_relinquish();
    return;
  }
  const int nk = min((W ? kMassRangeKeys : kMassSplitKeys) / kMtKeys, (last - key0) / kMtKeys + 1);  // key tiles
  // W: the query tiles that see key0, and how many of the key tiles tile `q` sees
  const int q_first = W ? max(0, key0 - v.pos0) / R : tile, q_count = W ? (v.rows + R - 1) / R - q_first : 1;
  auto tiles_of = [&](int q) { return W ? min(nk, (v.pos0 + min(v.rows, (q + 1) * R) - 1 - key0) / kMtKeys + 1) : nk; };

  if (warp == 0) tc::tmem_alloc(tslot, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < MT_COUNT; ++i)
      mbar_init(&bar[i], i >= MT_SE0 && i < MT_SE0 + 3 ? 4 : (i == MT_QE0 || i == MT_QE0 + 1) ? 8 : 1);
    fence_barrier_init();
    tc::prefetch_tensormap(&p.kmap);
    if (W) tc::prefetch_tensormap(&p.qmap);
  }
  const int jp0 = key0 / p.P, jp_last = (key0 + nk * kMtKeys - 1) / p.P;
  for (int jp = jp0 + tid; jp <= jp_last; jp += kMtThreads) {
    int pid = jp <= v.last / p.P ? __ldg(v.table + jp) : __ldg(v.table + jp0);  // past the chunk: any valid page (masked)
    pids[jp - jp0] = (pid * p.Hkv + h) << lg_p;
  }
  if (W)
    for (int i = tid; i < kMassRangeKeys; i += kMtThreads) acc[i] = 0.0f;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = *tslot;
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int m = (warp & 3) * 32 + lane;  // this thread's lane of S
  if constexpr (!W) {
    // the queries into tensor memory: lane m holds column m of the tile (row m / G, head m % G)
    if (warp < 4) {
      uint32_t w[D / 2];
      const int r = tile * R + m / G;
      if (m < R * G && r < v.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                          (static_cast<size_t>(v.row0 + r) * p.Hq + h * G + m % G) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 x = __ldg(src + i);
          w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 2; ++i) w[i] = 0u;
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        tc::tmem_st16(tb + lane_base + kTmemQ + i * 16, *reinterpret_cast<uint32_t(*)[16]>(&w[16 * i]));
      tc::tmem_wait_st();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  }

  PrefillIssueLog log;
  bool wok = !p.debug_stall || mbar_wait(&bar[MT_STALL], 0, p.wait_limit);  // the stall runs out
  wok = __all_sync(0xffffffffu, wok);
  const float scale = p.qk_scale_log2_h[PA_HEAD(p, h)];
  auto wait = [&](int b, int use) { return __all_sync(0xffffffffu, mbar_wait(&bar[b], use & 1, p.wait_limit)); };

  if (warp == kMtCopyWarp) {
    // ---- copies: key tile j into buffer j % 3 once S(j - 3) is computed; the next query tile a few
    // key tiles into the current one, once the score warps are done with the one before
    auto load_queries = [&](int q) {
      const int b = q & 1;
      if (q >= 2 && !wait(MT_QE0 + b, (q >> 1) - 1)) return false;
      if (lane == 0) {
        log.issue(MT_QF0 + b);
        mbar_arrive_expect_tx(&bar[MT_QF0 + b], static_cast<uint32_t>(S::NH * R * G * 128 + 1024));
        for (int half = 0; half < S::NH; ++half)
          tma_load_3d(sm + S::Q_OFF + b * S::TILE + half * S::HALF, &p.qmap, half * 64, h * G, v.row0 + (q_first + q) * R,
                      &bar[MT_QF0 + b]);
        bulk_g2s(sm + S::STAT_OFF + b * 1024,
                 p.ws_stat + p.chunk_stat[c] + (static_cast<size_t>(h) * p.chunk_tiles[c] + q_first + q) * 256, 1024u,
                 &bar[MT_QF0 + b], l2_policy_evict_last());
      }
      __syncwarp();
      return true;
    };
    if (W && wok) wok = load_queries(0);
    int j = 0;
    for (int q = 0; q < q_count && wok; ++q) {
      const int n = tiles_of(q_first + q);
      for (int kt = 0; kt < n && wok; ++kt, ++j) {
        if (j >= kMtBuffers) wok = wait(MT_SD0 + j % kMtBuffers, j / kMtBuffers - 1);
        if (!wok) break;
        if (lane == 0) log.issue(MT_KF0 + j % kMtBuffers);
        mass_load_keys<D>(&p.kmap, sm + (j % kMtBuffers) * S::TILE, &bar[MT_KF0 + j % kMtBuffers], pids, jp0,
                          key0 + kt * kMtKeys, lg_p, lane);
        if (W && kt == min(n - 1, kMtBuffers) && q + 1 < q_count) wok = load_queries(q + 1);
      }
    }
  } else if (warp == kMtMmaWarp) {
    // ---- MMAs: S(j) into buffer j % 3 once its four warps have read S(j - 3) and key tile j has landed
    constexpr uint32_t idesc = tc::idesc_bf16_f32(kMtKeys, kMtKeys, false);
    int j = 0;
    for (int q = 0; q < q_count && wok; ++q) {
      if (W) wok = wait(MT_QF0 + (q & 1), q >> 1);
      const int n = tiles_of(q_first + q);
      for (int kt = 0; kt < n && wok; ++kt, ++j) {
        const int b = j % kMtBuffers;
        if (j >= kMtBuffers) wok = wait(MT_SE0 + b, j / kMtBuffers - 1);
        wok = wok && wait(MT_KF0 + b, j / kMtBuffers);
        if (!wok) break;
        if (lane == 0) {
          tc::fence_after_sync();
          const unsigned char* K = sm + b * S::TILE;
          const unsigned char* Q = sm + S::Q_OFF + (q & 1) * S::TILE;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int off = (kk / 4) * S::HALF + (kk % 4) * 32;
            const uint64_t kd = tc::smem_desc(K + off, 16, 1024);
            if constexpr (W)
              tc::mma_bf16(tb + b * kMtKeys, kd, tc::smem_desc(Q + off, 16, 1024), idesc, kk > 0);
            else
              tc::mma_bf16_ts(tb + b * kMtKeys, tb + kTmemQ + kk * 8, kd, idesc, kk > 0);
          }
          tc::mma_commit(&bar[MT_SD0 + b]);
          log.issue(MT_SD0 + b);
        }
        __syncwarp();
      }
    }
  } else {
    const int group = warp >> 2;  // takes the key tiles kt with kt % 2 == group
    float m_ref = -INFINITY, l_run = 0.0f;
    const int my_row = min(tile * R + m / G, v.rows - 1);  // W false: this thread's column
    int j = 0;
    for (int q = 0; q < q_count && wok; ++q) {
      if (W) wok = wait(MT_QF0 + (q & 1), q >> 1);
      const int n = tiles_of(q_first + q);
      for (int kt = 0; kt < n && wok; ++kt, ++j) {
        if ((kt & 1) != group) continue;
        const int b = j % kMtBuffers, t0 = key0 + kt * kMtKeys;
        wok = wait(MT_SD0 + b, j / kMtBuffers);
        if (!wok) break;
        tc::fence_after_sync();
        const uint32_t col = tb + lane_base + b * kMtKeys;
        if constexpr (!W) {
          // keys of the tile that the column sees: the first `seen`
          const int seen = v.pos0 + my_row - t0 + 1;
          const bool edge = v.pos0 + tile * R - t0 + 1 < kMtKeys;  // some column of the tile sees less than all
#pragma unroll 1
          for (int i0 = 0; i0 < kMtKeys; i0 += 32) {
            float s[32];
            tc::tmem_ld32(col + i0, s);
            if (edge) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i0 + i >= seen) s[i] = -INFINITY;
            }
            float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
            const float mx = __fmul_rn(fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])), scale);
            if (mx > __fadd_rn(m_ref, kRescaleSlack)) {
              l_run = __fmul_rn(l_run, ex2(__fsub_rn(m_ref, mx)));
              m_ref = mx;
            }
            const float neg = m_ref == -INFINITY ? 0.0f : -m_ref;
            float2 ls[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) ls[i] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 t = __ffma2_rn(make_float2(s[i], s[i + 1]), make_float2(scale, scale), make_float2(neg, neg));
              ls[(i / 2) & 3] = __fadd2_rn(ls[(i / 2) & 3], make_float2(ex2(t.x), ex2(t.y)));
            }
            const float2 u = __fadd2_rn(__fadd2_rn(ls[0], ls[1]), __fadd2_rn(ls[2], ls[3]));
            l_run = __fadd_rn(l_run, __fadd_rn(u.x, u.y));
          }
        } else {
          const float* stat = reinterpret_cast<const float*>(sm + S::STAT_OFF + (q & 1) * 1024);
          const int row0 = (q_first + q) * R, cols = min(R, v.rows - row0) * G;
          // columns that see this thread's key: from `from` on (rows at or behind the key's position)
          const int from = max(0, t0 + m - (v.pos0 + row0)) * G;
          const bool edge = t0 + kMtKeys - 1 > v.pos0 + row0 || cols < kMtKeys;
          float2 w2 = make_float2(0.0f, 0.0f);
          // two columns' weights; in an edge tile those that do not see the key (or are none) are left
          // out whole, so that nothing of theirs reaches it
          auto add = [&](float x, float y, int i, float mx, float my, float ix, float iy) {
            const float2 t = __ffma2_rn(make_float2(x, y), make_float2(scale, scale), make_float2(-mx, -my));
            float2 e = make_float2(ex2(t.x), ex2(t.y));
            if (edge) {
              if (i < from || i >= cols) e.x = ix = 0.0f;
              if (i + 1 < from || i + 1 >= cols) e.y = iy = 0.0f;
            }
            w2 = __ffma2_rn(e, make_float2(ix, iy), w2);
          };
#pragma unroll 1
          for (int i0 = 0; i0 < cols; i0 += 32) {
            float s[32];
            tc::tmem_ld32(col + i0, s);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 M = *reinterpret_cast<const float4*>(stat + i0 + i);
              const float4 I = *reinterpret_cast<const float4*>(stat + kMtKeys + i0 + i);
              add(s[i], s[i + 1], i0 + i, M.x, M.y, I.x, I.y);
              add(s[i + 2], s[i + 3], i0 + i + 2, M.z, M.w, I.z, I.w);
            }
          }
          acc[kt * kMtKeys + m] = __fadd_rn(acc[kt * kMtKeys + m], __fadd_rn(w2.x, w2.y));
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[MT_SE0 + b]);
      }
      if (W && wok && lane == 0) mbar_arrive(&bar[MT_QE0 + (q & 1)]);
    }
    if constexpr (!W) {
      if (group == 1) {
        acc[m] = m_ref;
        acc[kMtKeys + m] = l_run;
      }
    }
    if constexpr (!W) {
      // the two groups' shares of the keys, group 0 first (the score warps meet)
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (group == 0 && wok) {
        ColumnStat s{m_ref, l_run};
        s.merge(acc[m], acc[kMtKeys + m]);
        if (m < R * G && tile * R + m / G < v.rows)
          p.ws_part[p.chunk_part[c] + ((static_cast<size_t>(h) * p.n_splits + split) * p.chunk_tiles[c] + tile) * kMtKeys + m] =
              make_float2(s.m, s.l);
      }
    }
  }
  const bool ok = __syncthreads_and(wok);
  if (!ok) {
    // every copy and MMA in flight finishes before its memory is given back
    if (lane == 0 && (warp == kMtCopyWarp || warp == kMtMmaWarp)) {
      for (int b = 0; b < MT_COUNT; ++b)
        if ((log.pending >> b) & 1u) mbar_wait(&bar[b], ((log.parity >> b) & 1u) ^ 1u, kDrainWaitLimit);
    }
    if (tid == 0) record_error(p.status, ST_TIMEOUT);
  } else if (W) {
    float* sums = p.mass + (static_cast<size_t>(v.seq) * p.Hkv + h) * (static_cast<size_t>(p.max_blocks) << lg_p) + key0;
    for (int i = tid; i < nk * kMtKeys && key0 + i <= last; i += kMtThreads) atomicAdd(sums + i, acc[i]);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, kTmemCols);
  }
}

template <int D, bool W>
cudaError_t launch_mass_tile_inst(const MassParams& p, long long ctas, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_done{0};
  const cudaError_t e = allow_dynamic_smem(mass_tile_kernel<D, W>, smem_done, MassTileSmem<D, W>::BYTES);
  if (e != cudaSuccess) return e;
  mass_tile_kernel<D, W><<<static_cast<unsigned>(ctas), kMtThreads, MassTileSmem<D, W>::BYTES, stream>>>(p);
  count_launch();
  return cudaGetLastError();
}

}  // namespace pa
