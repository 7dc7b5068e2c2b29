// pa_mass_tiles.cuh -- the chunks' launches of pa_attention_mass on the
// 5th-generation tensor cores (bf16 queries and pool).  Eight windows of 2 rows
// over 4k-16k keys take 100 us here and 250 with the warp-level MMAs of the other
// types' launches, of 64 rows 134 us here.
//
// A chunk's columns for kv head h are its (row, query head) pairs, 128 / G rows
// to a tile of 128 columns; a CTA works on two tiles at a time, so that a key
// tile brought to shared memory serves 256 columns.
//   mass_tile_kernel<D, false>: per (two tiles, kMassSplitKeys keys) every column's maximum
//     and sum.  S = Q K^T with the tiles' queries resident in shared memory and key
//     tiles of 128 streamed; a thread owns a column (one lane of S) and goes over
//     the keys.
//   mass_tile_kernel<D, true>: per range of as many keys, or of 256 for a chunk of more
//     than eight column tiles, the weights.
//     S^T = K Q^T, queries and key tiles alike, the columns' log2-sum-exps beside the
//     queries; a thread owns a key (one lane of S^T) and sums the weights of the
//     columns.  Each group of warps has accumulators of its own; they are
//     joined in order at the end.  One addition to the buffer per key.
// Both run one CTA per SM that goes through its share of the units, so that the
// copies of the next unit run while the scores of this one are summed, with 15
// warps: twelve turn scores into sums (three groups of four, each with its S
// buffer in tensor memory), one issues the copies, two the MMAs; they meet at
// mbarriers only.
//
// The scores are computed twice (a weight needs its column's sum over all
// keys first): 4 D operations and two exponentials per visible (row, head, key).
// Eight windows of 64 rows over 4k-16k keys (32 heads over 8): 134 us with cold
// caches (127 among other calls), of which 62 to 64 are the statistics' and 70 the
// weights' (each alone; 43 GFLOP each).  A CTA takes 1850 and 2030 cycles to a step
// of 128 keys x 128 columns, which needs 512 of
// the tensor pipe and, at 32 exponentials a cycle, 512 of the special functions'.
// No unit is busy: tensor pipe 26% and 24%, special functions 28% and 25%, issue
// slots 41% and 32%.  Bound by latency: three score warps to a scheduler, which
// mostly wait for their own results, for S from tensor memory and (weights) at the
// barriers around the columns' statistics.  One MMA warp for both column tiles took
// 139 us where two took 121 (inputs in L2); a CTA per unit 147; S buffers of 64
// columns, two to a group, 212; key ranges of 512 / 2048 keys instead of 1024: 133 / 127.
// Every wait is bounded; a call that gives up reports it, and adds nothing more.
#pragma once

#include <algorithm>
#include <type_traits>

#include "pa_mass.cuh"
#include "pa_prefill.cuh"

namespace pa {

constexpr int kMtKeys = 128;      // keys of a key tile, columns of a column tile
constexpr int kMtBuffers = 3;     // S buffers, each with a group of four score warps
constexpr int kMtKeyBufs = 4;     // key tiles in shared memory
// Scores (log2 domain) up to which the weights take a column's log2-sum-exp as one number, rounded twice by half a
// step of at most 2^-14: a weight is then off by up to 2^-14 ln 2 = 4e-5 of itself.  (As one number for all, scores of
// 1e6 gave columns whose weights summed to 1.01, of 1e8 to millions.)
constexpr float kMtNear = 1024.0f;
constexpr int kMtScoreWarps = 4 * kMtBuffers;
constexpr int kMtCopyWarp = kMtScoreWarps, kMtMmaWarp = kMtCopyWarp + 1;  // ... two MMA warps
constexpr int kMtThreads = 32 * (kMtMmaWarp + 2);

enum {
  MT_KF0 = 0,                          // key tile in buffer b landed
  MT_KE0 = MT_KF0 + kMtKeyBufs,        // ... read by its MMAs
  MT_SD0 = MT_KE0 + kMtKeyBufs,        // S buffer b computed
  MT_SE0 = MT_SD0 + kMtBuffers,        // ... read by its four warps
  MT_QF0 = MT_SE0 + kMtBuffers,        // queries of column tile 0 / 1 landed
  MT_QE0 = MT_QF0 + 2,                 // ... read by their MMAs
  MT_DRAIN0 = MT_QE0 + 2,              // after a failure: all of MMA warp 0's / 1's MMAs done
  MT_STALL = MT_DRAIN0 + 2,
  MT_COUNT
};

template <int D, bool W>
struct MassTileSmem {  // byte offsets from a 1024-byte aligned base
  static constexpr int NH = D / 64;            // 64-element halves of the head dim
  static constexpr int HALF = kMtKeys * 128;   // one half of a tile of 128 rows
  static constexpr int TILE = NH * HALF;
  static constexpr int Q_OFF = kMtKeyBufs * TILE;                // two query tiles
  static constexpr int STAT_OFF = Q_OFF + 2 * TILE;              // W: of their columns minus the log2-sum-exp, then (for
                                                                 // far scores) the maximum and minus log2 of the sum
  static constexpr int ACC_OFF = STAT_OFF + (W ? 6 * kMtKeys * 4 : 0);  // per group: W a sum per key; else (max, sum) of two tiles
  static constexpr int ACC = W ? kMassSplitKeys : 4 * kMtKeys;   // floats of a group
  static constexpr int BAR_OFF = ACC_OFF + kMtBuffers * ACC * 4;
  static constexpr int TMEM_OFF = BAR_OFF + MT_COUNT * 8;
  static constexpr int HEAD_OFF = BAR_OFF + 256;                 // the chunks
  static constexpr int BYTES = HEAD_OFF + kMaxChunks * 16 + 1024;  // slack for aligning the base
  static_assert(MT_COUNT * 8 + 8 <= 256 && BYTES <= 227 * 1024, "shared memory");
};

// 32 columns of this warp's lanes from tensor memory, without waiting ...
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// ... and the wait for every load started; r is read only behind it.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// f(first column, its 32 columns) over the first `cols` columns of an S buffer,
// the next 32 on their way while f runs.
template <typename F>
__device__ __forceinline__ void over_columns(uint32_t taddr, int cols, F f) {
  uint32_t a[32], b[32];
  tmem_ld32_start(taddr, a);
#pragma unroll
  for (int i0 = 0; i0 < kMtKeys; i0 += 64) {
    if (i0 >= cols) break;
    tmem_ld32_wait(a);
    if (i0 + 32 < cols) tmem_ld32_start(taddr + i0 + 32, b);
    f(i0, a);
    if (i0 + 32 >= cols) break;
    tmem_ld32_wait(b);
    if (i0 + 64 < cols) tmem_ld32_start(taddr + i0 + 64, a);
    f(i0 + 32, b);
  }
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
      : "r"(taddr)
      : "memory");
}

// A key's weights of a column tile whose scores are far from zero, summed over the columns from `from` on: 2^((score -
// maximum) scale - log2 sum), the steps of the statistics, so that a column's weights sum to 1 whatever its scores.
// (Rarely run, and small, so as to leave the registers of the loop around it alone.)
__device__ __forceinline__ float far_weight(uint32_t taddr, int from, int cols, const float* maximum, const float* lg, float scale) {
  float w = 0.0f;
#pragma unroll 1
  for (int i0 = 0; i0 < cols; i0 += 8) {
    float y[8];
    tmem_ld8(taddr + i0, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float z = fmaf(__fsub_rn(y[j], maximum[i0 + j]), scale, lg[i0 + j]);
      if (i0 + j >= from && i0 + j < cols) w = __fadd_rn(w, ex2(z));
    }
  }
  return w;
}

// 3-D tiled load of the box at (x, y, z); x * element size a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_3d(void* dst_smem, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// A piece of work: for a kv head of a chunk two column tiles and a range of
// keys (W false), or a range of keys and every column tile that sees it (W).
struct MassUnit {
  int chunk, h, row0, rows, seq, pos0, last;  // last: the last key that a row of the unit sees
  int key0, nk;                               // first key, key tiles (0: nothing to do)
  int t_first, t_end, split;                  // column tiles
  const int32_t* table;
};

template <int D, bool W>
__global__ void __launch_bounds__(kMtThreads, 1) mass_tile_kernel(const __grid_constant__ MassParams p) {
  using S = MassTileSmem<D, W>;
  constexpr uint32_t kTmemCols = 512;  // the S buffers (384; a power of two)
  // Keys of a unit: 1024, or, of the weights of a chunk with many column tiles to go through, 256.  By the chunk
  // alone, so that its sums do not depend on the batch.  us with 1024 / 256: 13 chunks of 396 rows x 6 heads (19
  // tiles) 190 / 98, one of 512 x 32 over 8 (16 tiles) 113 / 77, eight of 256 x 32 over 8 (8 tiles) 413 / 528.
  auto range_of = [&](int c) { return W && p.chunk_tiles[c] > kMassLongTiles ? kMassLongKeys : kMassSplitKeys; };
  static_assert(kMtBuffers * kMtKeys <= kTmemCols, "tensor memory");
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S::BAR_OFF);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + S::TMEM_OFF);
  int32_t* failed = reinterpret_cast<int32_t*>(sm + S::TMEM_OFF + 4);
  int4* heads = reinterpret_cast<int4*>(sm + S::HEAD_OFF);  // per chunk: sequence, first position, units before and of it
  float* acc = reinterpret_cast<float*>(sm + S::ACC_OFF);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.Hq / p.Hkv, R = kMtKeys / G, lg_p = 31 - __clz(p.P);

  if (warp == 0) tc::tmem_alloc(tslot, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < MT_COUNT; ++i)
      mbar_init(&bar[i], i >= MT_SE0 && i < MT_SE0 + kMtBuffers   ? 5u  // a group's warps, and the other MMA warp
                         : i >= MT_KE0 && i < MT_KE0 + kMtKeyBufs ? 2u  // the MMA warps
                                                                  : 1u);
    *failed = 0;
    fence_barrier_init();
    tc::prefetch_tensormap(&p.kmap);
    tc::prefetch_tensormap(&p.qmap);
  }
  if (W)
    for (int i = tid; i < kMtBuffers * S::ACC; i += kMtThreads) acc[i] = 0.0f;
  griddep_wait();  // the chunks' heads, and (W) their columns' statistics, from the launches before
  if (!W) griddep_launch_dependents();
  if (tid == 0) {
    int before = 0;
    for (int c = 0; c < p.n_chunks; ++c) {
      const int2 hd = __ldcg(p.ws_head + c);
      const int rows = p.chunk_end[c] - p.chunk_begin[c];
      int units = 0;  // a chunk that adds nothing has none
      if (hd.x >= 0) units = p.Hkv * ((hd.y + rows - 1) / range_of(c) + 1) * (W ? 1 : (p.chunk_tiles[c] + 1) / 2);
      heads[c] = make_int4(hd.x, hd.y, before, units);
      before += units;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = *tslot;
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int m = (warp & 3) * 32 + lane;  // this thread's lane of S
  const int4 end_head = heads[p.n_chunks - 1];
  const int total = end_head.z + end_head.w;

  // unit i; every role goes through the same units, and in each through the same steps: per two column tiles
  // the key tiles, per key tile the column tiles that see it
  auto unit_at = [&](int i) {
    MassUnit x;
    int c = 0;
    while (c + 1 < p.n_chunks && i >= heads[c + 1].z) ++c;
    const int4 hd = heads[c];
    const int local = i - hd.z;
    x.chunk = c;
    x.h = local % p.Hkv;
    x.row0 = p.chunk_begin[c];
    x.rows = p.chunk_end[c] - x.row0;
    x.seq = hd.x;
    x.pos0 = hd.y;
    x.table = p.block_tables + static_cast<size_t>(x.seq) * p.max_blocks;
    const int range = range_of(c), ranges = (x.pos0 + x.rows - 1) / range + 1, part = local / p.Hkv;
    x.split = part % ranges;
    x.key0 = x.split * range;
    const int pair = part / ranges;
    const int row_end = W ? x.rows : min(x.rows, (2 * pair + 2) * R);
    x.last = x.pos0 + row_end - 1;
    x.nk = x.key0 > x.last ? 0 : min(range / kMtKeys, (x.last - x.key0) / kMtKeys + 1);
    x.t_first = W ? max(0, x.key0 - x.pos0) / R : 2 * pair;
    x.t_end = (row_end + R - 1) / R;
    return x;
  };
  // how many of a unit's key tiles column tile t sees
  auto tiles_seen = [&](const MassUnit& x, int t) {
    const int end = x.pos0 + min(x.rows, (t + 1) * R) - 1;  // the last key that the column tile sees
    return t < x.t_end && end >= x.key0 ? min(x.nk, (end - x.key0) / kMtKeys + 1) : 0;
  };

  PrefillIssueLog log;  // of the copies
  bool wok = !p.debug_stall || mbar_wait(&bar[MT_STALL], 0, p.wait_limit);  // the stall runs out
  wok = __all_sync(0xffffffffu, wok);
  // A barrier's use-th phase.  Every waiter of a phase has seen the one before it, or the phase cannot
  // begin without it: none mistakes an older phase of the same parity for its own.
  auto wait = [&](int b, int use) { return __all_sync(0xffffffffu, mbar_wait(&bar[b], use & 1, p.wait_limit)); };

  if (warp == kMtCopyWarp) {
    // ---- copies: key tile k into buffer k % 4 once the MMAs of key tile k - 4 are done
    int k = 0, q_use[2] = {0, 0};
    const int lg_br = lg_p < 6 ? lg_p : 6;  // rows of a box: a page, or a 64-key part of a larger page
    const bool copies = lane < (kMtKeys >> lg_br) * S::NH;
    for (int i = blockIdx.x; i < total && wok; i += gridDim.x) {
      const MassUnit x = unit_at(i);
      // the tensor-map row of this lane's box of key tile kt (keys past the chunk: its last page's, masked later)
      auto box_row = [&](int kt) {
        const int t = x.key0 + kt * kMtKeys + (lane / S::NH << lg_br);
        const int page = copies ? __ldg(x.table + (min(t, x.pos0 + x.rows - 1) >> lg_p)) : 0;
        return ((page * p.Hkv + x.h) << lg_p) + (t & (p.P - 1));
      };
      int row = x.nk > 0 ? box_row(0) : 0;
      for (int t = x.t_first; t < x.t_end && x.nk > 0 && wok; t += 2) {
        const int n = max(tiles_seen(x, t), tiles_seen(x, t + 1));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (t + half >= x.t_end || !wok) continue;
          if (q_use[half] > 0) wok = wait(MT_QE0 + half, q_use[half] - 1);
          if (!wok) continue;
          ++q_use[half];
          if (lane == 0) {
            log.issue(MT_QF0 + half);
            mbar_arrive_expect_tx(&bar[MT_QF0 + half], static_cast<uint32_t>(S::NH * R * G * 128));
            for (int j = 0; j < S::NH; ++j)
              tma_load_3d(sm + S::Q_OFF + half * S::TILE + j * S::HALF, &p.qmap, j * 64, x.h * G,
                          x.row0 + (t + half) * R, &bar[MT_QF0 + half]);
          }
          __syncwarp();
        }
        for (int kt = 0; kt < n && wok; ++kt, ++k) {
          const int b = k % kMtKeyBufs;
          if (k >= kMtKeyBufs) wok = wait(MT_KE0 + b, k / kMtKeyBufs - 1);
          if (!wok) break;
          if (lane == 0) {
            log.issue(MT_KF0 + b);
            mbar_arrive_expect_tx(&bar[MT_KF0 + b], static_cast<uint32_t>(kMtKeys * D * 2));
          }
          __syncwarp();
          if (copies) {
            const int piece = lane / S::NH, half = lane % S::NH;
            tc::tma_load_2d(sm + b * S::TILE + half * S::HALF + (piece << lg_br) * 128, &p.kmap, half * 64, row,
                            &bar[MT_KF0 + b]);
          }
          row = box_row(kt + 1 < n ? kt + 1 : 0);  // the next key tile's, looked up while this one's buffer fills
        }
      }
    }
  } else if (warp >= kMtMmaWarp) {
    // ---- MMAs: step u into S buffer u % 3 once its four warps have read step u - 3.  One MMA warp has the first
    // column tile of two, one the second (issuing a tile's MMAs holds a warp about as long as they run, so one's
    // waits go beside the other's MMAs).  Both go through all steps: at the other's step a warp only adds its
    // arrival to the buffer's barrier, so that no phase of it passes that one of the two has not seen.
    const int my_half = warp - kMtMmaWarp;
    constexpr uint32_t idesc = tc::idesc_bf16_f32(kMtKeys, kMtKeys, false);
    // descriptors of the first key and query tiles: others lie a constant number of 16-byte units away
    const uint64_t k_desc = tc::smem_desc(sm, 16, 1024), q_desc = tc::smem_desc(sm + S::Q_OFF, 16, 1024);
    int k = 0, u = 0, q_use = 0;
    for (int i = blockIdx.x; i < total && wok; i += gridDim.x) {
      const MassUnit x = unit_at(i);
      for (int t = x.t_first; t < x.t_end && x.nk > 0 && wok; t += 2) {
        const int n0 = tiles_seen(x, t), n1 = tiles_seen(x, t + 1), n = max(n0, n1);
        if (t + my_half < x.t_end) wok = wait(MT_QF0 + my_half, q_use++);
        for (int kt = 0; kt < n && wok; ++kt, ++k) {
          const int kb = k % kMtKeyBufs;
          wok = wait(MT_KF0 + kb, k / kMtKeyBufs);
          for (int half = 0; half < 2 && wok; ++half) {
            if (kt >= (half ? n1 : n0)) continue;
            const int b = u % kMtBuffers;
            if (u >= kMtBuffers) wok = wait(MT_SE0 + b, u / kMtBuffers - 1);
            if (!wok) break;
            if (lane == 0 && half != my_half) mbar_arrive(&bar[MT_SE0 + b]);
            if (lane == 0 && half == my_half) {
              tc::fence_after_sync();
              const uint64_t kd = k_desc + kb * (S::TILE / 16), qd = q_desc + half * (S::TILE / 16);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const int off = ((kk / 4) * S::HALF + (kk % 4) * 32) / 16;
                // W: lanes are keys and columns columns; else the other way round
                tc::mma_bf16(tb + b * kMtKeys, (W ? kd : qd) + off, (W ? qd : kd) + off, idesc, kk > 0);
              }
              tc::mma_commit(&bar[MT_SD0 + b]);
            }
            __syncwarp();
            ++u;
          }
          if (wok && lane == 0) {
            tc::mma_commit(&bar[MT_KE0 + kb]);
            if (kt == n - 1 && t + my_half < x.t_end) tc::mma_commit(&bar[MT_QE0 + my_half]);
          }
          __syncwarp();
        }
      }
    }
  } else {
    const int group = warp >> 2;  // takes the steps u with u % 3 == group, and S buffer `group`
    const float scale = p.qk_scale_log2_h[0];  // bf16 pools have no head scales
    int u = 0;
    auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(kMtScoreWarps * 32) : "memory"); };
    auto meet_or = [](bool mine) {  // ... and whether it holds for any of them
      uint32_t any;
      asm volatile("{ .reg .pred p, q; setp.ne.u32 q, %1, 0; bar.red.or.pred p, 1, %2, q; selp.u32 %0, 1, 0, p; }"
                   : "=r"(any)
                   : "r"(static_cast<uint32_t>(mine)), "n"(kMtScoreWarps * 32)
                   : "memory");
      return any != 0;
    };
    // The score warps meet the same number of times whatever a wait of theirs does (`wok` guards the waits).
    for (int i = blockIdx.x; i < total; i += gridDim.x) {
      const MassUnit x = unit_at(i);
      if (x.nk == 0) continue;
      // the group's place in this unit: by the unit's own steps, so that its sums do not depend on the units before
      float* const mine = acc + (group + kMtBuffers - u % kMtBuffers) % kMtBuffers * S::ACC;
      // W false: this thread's columns, the maximum of the scores as the MMAs give them.  A score enters as its
      // distance from it, times the scale: a product from which the scaled maximum is taken in one step (unrounded
      // against rounded) is off by half a step of that, which a large one makes any number.  (62 us for the windows
      // above, in one step 59.)
      float m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
      for (int t = x.t_first; t < x.t_end; t += 2) {
        const int n0 = tiles_seen(x, t), n1 = tiles_seen(x, t + 1), n = max(n0, n1);
        bool far = false;  // W: a column of the two tiles has scores beyond kMtNear
        if constexpr (W) {
          // every column's maximum and sum, of the two tiles, a column to a thread
          if (t > x.t_first) meet();  // the tiles before are done with
          if (tid < 2 * kMtKeys) {
            const int col = tid % kMtKeys, r = (t + tid / kMtKeys) * R + col / G;
            float m = 0.0f, lg = 0.0f;
            if (col < R * G && r < x.rows) {
              const float2 st = column_stat(p, x.chunk, x.h, t + tid / kMtKeys, col, x.pos0 + r, scale);
              m = st.x;
              lg = log2f(st.y);  // (y is one over the sum)
            }
            float* stat = reinterpret_cast<float*>(sm + S::STAT_OFF) + tid;
            const float y = __fmul_rn(m, scale);
            stat[0] = __fsub_rn(lg, y);
            stat[2 * kMtKeys] = m;
            stat[4 * kMtKeys] = lg;
            far = fabsf(y) > kMtNear && fabsf(y) < INFINITY;  // (a column without a finite maximum has no weights)
          }
          far = meet_or(far);
        }
        for (int kt = 0; kt < n && wok; ++kt) {
          for (int half = 0; half < 2 && wok; ++half) {
            if (kt >= (half ? n1 : n0)) continue;
            const int use = u++;
            if (use % kMtBuffers != group) continue;
            const int t0 = x.key0 + kt * kMtKeys;
            wok = wait(MT_SD0 + group, use / kMtBuffers);
            if (!wok) break;
            tc::fence_after_sync();
            const uint32_t col = tb + lane_base + group * kMtKeys;
            if constexpr (!W) {
              // keys of the tile that the column sees: the first `seen`
              const int seen = x.pos0 + min((t + half) * R + m / G, x.rows - 1) - t0 + 1;
              const bool edge = x.pos0 + (t + half) * R - t0 + 1 < kMtKeys;  // some column of the tile sees less than all
              float mr = half ? m_ref[1] : m_ref[0], lr = half ? l_run[1] : l_run[0];
              over_columns(col, kMtKeys, [&](int i0, uint32_t(&y)[32]) {
                float s[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(y[j]);
                if (edge) {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (i0 + j >= seen) s[j] = -INFINITY;
                }
                float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int j = 4; j < 32; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], s[j]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                if (__fmul_rn(__fsub_rn(mx, mr), scale) > kRescaleSlack) {
                  lr = __fmul_rn(lr, ex2(__fmul_rn(__fsub_rn(mr, mx), scale)));
                  mr = mx;
                }
                const float neg = mr == -INFINITY ? 0.0f : -mr;
                float2 ls[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) ls[j] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  const float2 z = __fmul2_rn(__fadd2_rn(make_float2(s[j], s[j + 1]), make_float2(neg, neg)), make_float2(scale, scale));
                  ls[(j / 2) & 3] = __fadd2_rn(ls[(j / 2) & 3], make_float2(ex2(z.x), ex2(z.y)));
                }
                const float2 z = __fadd2_rn(__fadd2_rn(ls[0], ls[1]), __fadd2_rn(ls[2], ls[3]));
                lr = __fadd_rn(lr, __fadd_rn(z.x, z.y));
              });
              if (half) m_ref[1] = mr, l_run[1] = lr;
              else m_ref[0] = mr, l_run[0] = lr;
            } else {
              const float* stat = reinterpret_cast<const float*>(sm + S::STAT_OFF) + half * kMtKeys;
              const int first_row = (t + half) * R, cols = min(R, x.rows - first_row) * G;
              // columns that see this thread's key: from `from` on (rows at or behind the key's position)
              const int from = max(0, t0 + m - (x.pos0 + first_row)) * G;
              float2 w2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
              // four columns' weights 2^(score - log2-sum-exp); in an edge tile those that do not see the key
              // (or are none) are left out whole, so that nothing of theirs reaches it
              auto add4 = [&](auto edge, const uint32_t(&y)[32], int i0, int j) {
                const float4 z = *reinterpret_cast<const float4*>(stat + i0 + j);
                const float2 sc = make_float2(scale, scale);
                const float2 z0 = __ffma2_rn(make_float2(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), sc, make_float2(z.x, z.y));
                const float2 z1 = __ffma2_rn(make_float2(__uint_as_float(y[j + 2]), __uint_as_float(y[j + 3])), sc, make_float2(z.z, z.w));
                float2 e0 = make_float2(ex2(z0.x), ex2(z0.y)), e1 = make_float2(ex2(z1.x), ex2(z1.y));
                if constexpr (decltype(edge)::value) {
                  const int k = i0 + j;
                  if (k < from || k >= cols) e0.x = 0.0f;
                  if (k + 1 < from || k + 1 >= cols) e0.y = 0.0f;
                  if (k + 2 < from || k + 2 >= cols) e1.x = 0.0f;
                  if (k + 3 < from || k + 3 >= cols) e1.y = 0.0f;
                }
                w2[0] = __fadd2_rn(w2[0], e0);
                w2[1] = __fadd2_rn(w2[1], e1);
              };
              if (far)
                w2[0].x = far_weight(col, from, cols, stat + 2 * kMtKeys, stat + 4 * kMtKeys, scale);
              else if (t0 + kMtKeys - 1 > x.pos0 + first_row || cols < kMtKeys)
                over_columns(col, cols, [&](int i0, uint32_t(&y)[32]) {
#pragma unroll
                  for (int j = 0; j < 32; j += 4) add4(std::true_type(), y, i0, j);
                });
              else
                over_columns(col, kMtKeys, [&](int i0, uint32_t(&y)[32]) {
#pragma unroll
                  for (int j = 0; j < 32; j += 4) add4(std::false_type(), y, i0, j);
                });
              const float2 w = __fadd2_rn(w2[0], w2[1]);
              mine[kt * kMtKeys + m] = __fadd_rn(mine[kt * kMtKeys + m], __fadd_rn(w.x, w.y));
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[MT_SE0 + group]);
          }
        }
      }
      if (!wok) *failed = 1;
      if constexpr (!W) {
        meet();  // the unit before is merged (a group without a step of this one gets here early)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          mine[half * 2 * kMtKeys + m] = m_ref[half];
          mine[half * 2 * kMtKeys + kMtKeys + m] = l_run[half];
        }
      }
      meet();
      if (*failed) continue;  // adds nothing more
      if constexpr (!W) {
        // the groups' shares of the keys, merged in order
        const int half = group, row = (x.t_first + half) * R + m / G;
        if (group < 2 && m < R * G && row < x.rows) {
          ColumnStat s{-INFINITY, 0.0f};
#pragma unroll
          for (int k = 0; k < kMtBuffers; ++k)
            s.merge(acc[k * S::ACC + half * 2 * kMtKeys + m], acc[k * S::ACC + half * 2 * kMtKeys + kMtKeys + m], scale);
          p.ws_part[p.chunk_part[x.chunk] +
                    ((static_cast<size_t>(x.h) * p.n_splits + x.split) * p.chunk_tiles[x.chunk] + x.t_first + half) * kMtKeys + m] =
              make_float2(s.m, s.l);
        }
      } else {
        // the groups' sums of each key, in order; the accumulators are empty again for the next unit (whose
        // score warps meet before they add)
        float* sums = p.mass + (static_cast<size_t>(x.seq) * p.Hkv + x.h) * (static_cast<size_t>(p.max_blocks) << lg_p) + x.key0;
        for (int j = tid; j < x.nk * kMtKeys; j += kMtScoreWarps * 32) {
          float w = acc[j];
          acc[j] = 0.0f;
#pragma unroll
          for (int k = 1; k < kMtBuffers; ++k) {
            w = __fadd_rn(w, acc[k * S::ACC + j]);
            acc[k * S::ACC + j] = 0.0f;
          }
          if (x.key0 + j <= x.last) atomicAdd(sums + j, w);
        }
      }
    }
  }
  const bool ok = __syncthreads_and(wok);
  if (!ok) {
    // every copy and MMA in flight finishes before its memory is given back
    if (lane == 0 && warp == kMtCopyWarp) log.drain(bar, MT_COUNT);
    if (lane == 0 && warp >= kMtMmaWarp) {
      tc::mma_commit(&bar[MT_DRAIN0 + warp - kMtMmaWarp]);
      mbar_wait(&bar[MT_DRAIN0 + warp - kMtMmaWarp], 0, kDrainWaitLimit);
    }
    if (tid == 0) record_error(p.status, ST_TIMEOUT);
    if (!W && tid < p.n_chunks) p.ws_head[tid].x = -1;  // no weights without the statistics
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, kTmemCols);
  }
}

template <int D, bool W>
cudaError_t launch_mass_tile_inst(const MassParams& p, long long units, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_done{0};
  static std::atomic<long long> resident[64];
  const long long ctas = resident_ctas(mass_tile_kernel<D, W>, resident, smem_done, kMtThreads, MassTileSmem<D, W>::BYTES);
  if (ctas <= 0) return cudaErrorInvalidConfiguration;
  count_launch();
  return launch_kernel(mass_tile_kernel<D, W>, dim3(static_cast<unsigned>(std::min(units, ctas))), dim3(kMtThreads),
                       MassTileSmem<D, W>::BYTES, stream, true, p);
}

}  // namespace pa
