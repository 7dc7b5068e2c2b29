// pa_mass_tiles.cuh -- the chunks' launches of pa_attention_mass on the
// 5th-generation tensor cores (bf16 queries and pool, chunks of at least
// kMinTileRows rows).
//
// A chunk's columns for kv head h are its (row, query head) pairs, 128 / G rows
// to a tile of 128 columns; a CTA works on two tiles at a time, so that a key
// tile brought to shared memory serves 256 columns.
//   mass_tile_kernel<D, false>: per (two tiles, key range) every column's maximum
//     and sum.  S = Q K^T with the tiles' queries in tensor memory and key tiles of
//     128 streamed; a thread owns a column (one lane of S) and goes over the keys.
//   mass_tile_kernel<D, true>: per range of kMassRangeKeys keys the weights.
//     S^T = K Q^T with two tiles' queries and their statistics resident and the key
//     tiles streamed; a thread owns a key (one lane of S^T) and sums the weights of
//     the columns.  Each group of warps has accumulators of its own; they are
//     joined in order at the end.  One addition to the buffer per key.
// Both run 14 warps: twelve turn scores into sums (three groups of four, each with
// its S buffer in tensor memory), one issues the copies, one the MMAs; they meet
// at mbarriers only.
//
// The scores are computed twice (a weight needs its column's sum over all
// keys first): 4 D operations and two exponentials per visible (row, head, key).
// Every wait is bounded; a call that gives up adds nothing and reports it.
#pragma once

#include <type_traits>

#include "pa_mass.cuh"
#include "pa_prefill.cuh"

namespace pa {

constexpr int kMtKeys = 128;      // keys of a key tile, columns of a column tile
constexpr int kMtBuffers = 3;     // S buffers, each with a group of four score warps
constexpr int kMtKeyBufs = 4;     // key tiles in shared memory
constexpr int kMtScoreWarps = 4 * kMtBuffers;
constexpr int kMtCopyWarp = kMtScoreWarps, kMtMmaWarp = kMtCopyWarp + 1;
constexpr int kMtThreads = 32 * (kMtMmaWarp + 1);

enum {
  MT_KF0 = 0,                          // key tile in buffer b landed
  MT_KE0 = MT_KF0 + kMtKeyBufs,        // ... read by its MMAs
  MT_SD0 = MT_KE0 + kMtKeyBufs,        // S buffer b computed
  MT_SE0 = MT_SD0 + kMtBuffers,        // ... read by its four warps
  MT_QF0 = MT_SE0 + kMtBuffers,        // queries of column tile 0 / 1 landed
  MT_QE0 = MT_QF0 + 2,                 // ... done with by the score warps
  MT_STALL = MT_QE0 + 2,
  MT_COUNT
};

template <int D, bool W>
struct MassTileSmem {  // byte offsets from a 1024-byte aligned base
  static constexpr int NH = D / 64;            // 64-element halves of the head dim
  static constexpr int HALF = kMtKeys * 128;   // one half of a tile of 128 rows
  static constexpr int TILE = NH * HALF;
  static constexpr int Q_OFF = kMtKeyBufs * TILE;                // W: two query tiles
  static constexpr int STAT_OFF = Q_OFF + (W ? 2 * TILE : 0);    // W: their statistics, [max x 128][1 / sum x 128]
  static constexpr int ACC_OFF = STAT_OFF + (W ? 2 * 1024 : 0);  // per group: W a sum per key; else (max, sum) of two tiles
  static constexpr int ACC = W ? kMassRangeKeys : 4 * kMtKeys;   // floats of a group
  static constexpr int BAR_OFF = ACC_OFF + kMtBuffers * ACC * 4;
  static constexpr int TMEM_OFF = BAR_OFF + MT_COUNT * 8;
  static constexpr int PID_OFF = BAR_OFF + 256;
  static constexpr int PIDS = (W ? kMassRangeKeys : kMassSplitKeys) / 16;
  static constexpr int BYTES = PID_OFF + PIDS * 4 + 1024;        // slack for aligning the base
  static_assert(MT_COUNT * 8 + 4 <= 256 && BYTES <= 227 * 1024, "shared memory");
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
  constexpr uint32_t kTmemQ = kMtBuffers * kMtKeys;  // W false: the two query tiles, behind the S buffers
  constexpr uint32_t kTmemCols = 512;
  static_assert(kTmemQ + D <= kTmemCols, "tensor memory");
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
  if (!W) griddep_launch_dependents();  // the weights' CTAs may be launched; what they read of this launch they wait for
  const int local = blockIdx.x - p.chunk_cta[c];
  const int h = local % p.Hkv, part = local / p.Hkv;
  const int split = W ? 0 : part % p.n_splits, first_tile = W ? 0 : part / p.n_splits * 2;
  ChunkView v;
  const bool ok_chunk = v.open(p, c);
  const int key0 = W ? part * kMassRangeKeys : split * kMassSplitKeys;  // the CTA's first key
  const int row_end = W ? v.rows : min(v.rows, (first_tile + 2) * R);
  const int last = v.pos0 + row_end - 1;  // the last key that a row of the CTA sees
  if (!ok_chunk || key0 > last) {
    if (warp == 0) tc::tmem_relinquish();
    if (W) griddep_wait();  // no CTA of a dependent launch ends before the launch it depends on
    return;
  }
  const int nk = min((W ? kMassRangeKeys : kMassSplitKeys) / kMtKeys, (last - key0) / kMtKeys + 1);  // key tiles
  // The CTA's column tiles [t_first, t_end), two at a time, and how many of its key tiles a column tile sees.
  // All roles go through the same steps: per two tiles the key tiles, per key tile the column tiles that see it.
  const int t_end = (row_end + R - 1) / R, t_first = W ? max(0, key0 - v.pos0) / R : first_tile;
  auto tiles_seen = [&](int t) {
    const int end = v.pos0 + min(v.rows, (t + 1) * R) - 1;  // the last key that the column tile sees
    return t < t_end && end >= key0 ? min(nk, (end - key0) / kMtKeys + 1) : 0;
  };

  if (warp == 0) tc::tmem_alloc(tslot, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < MT_COUNT; ++i)
      mbar_init(&bar[i], i >= MT_SE0 && i < MT_SE0 + kMtBuffers ? 4u                // a group's warps
                         : i >= MT_QE0 && i < MT_QE0 + 2        ? kMtScoreWarps : 1u);
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
    for (int i = tid; i < kMtBuffers * S::ACC; i += kMtThreads) acc[i] = 0.0f;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = *tslot;
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int m = (warp & 3) * 32 + lane;  // this thread's lane of S
  if constexpr (!W) {
    // the queries into tensor memory: lane m holds column m of a tile (row m / G, head m % G)
    if (warp < 8) {
      uint32_t w[D / 2];
      const int half = warp >> 2, r = (first_tile + half) * R + m / G;
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
        tc::tmem_st16(tb + lane_base + kTmemQ + half * (D / 2) + i * 16, *reinterpret_cast<uint32_t(*)[16]>(&w[16 * i]));
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
  // A barrier's use-th phase.  Every waiter of a phase has seen the one before it, or the phase cannot
  // begin without it: none mistakes an older phase of the same parity for its own.
  auto wait = [&](int b, int use) { return __all_sync(0xffffffffu, mbar_wait(&bar[b], use & 1, p.wait_limit)); };

  if (warp == kMtCopyWarp) {
    // ---- copies: key tile k into buffer k % 4 once the MMAs of key tile k - 4 are done
    int k = 0;
    for (int t = t_first, pair = 0; t < t_end && wok; t += 2, ++pair) {
      const int n0 = tiles_seen(t), n1 = tiles_seen(t + 1), n = max(n0, n1);
      if (W) {
        for (int half = 0; half < 2 && t + half < t_end && wok; ++half) {
          if (pair > 0) wok = wait(MT_QE0 + half, pair - 1);
          if (!wok) break;
          if (lane == 0) {
            log.issue(MT_QF0 + half);
            mbar_arrive_expect_tx(&bar[MT_QF0 + half], static_cast<uint32_t>(S::NH * R * G * 128));
            for (int i = 0; i < S::NH; ++i)
              tma_load_3d(sm + S::Q_OFF + half * S::TILE + i * S::HALF, &p.qmap, i * 64, h * G, v.row0 + (t + half) * R,
                          &bar[MT_QF0 + half]);
          }
          __syncwarp();
        }
      }
      for (int kt = 0; kt < n && wok; ++kt, ++k) {
        const int b = k % kMtKeyBufs;
        if (k >= kMtKeyBufs) wok = wait(MT_KE0 + b, k / kMtKeyBufs - 1);
        if (!wok) break;
        if (lane == 0) log.issue(MT_KF0 + b);
        mass_load_keys<D>(&p.kmap, sm + b * S::TILE, &bar[MT_KF0 + b], pids, jp0, key0 + kt * kMtKeys, lg_p, lane);
      }
    }
  } else if (warp == kMtMmaWarp) {
    // ---- MMAs: step u into S buffer u % 3 once its four warps have read step u - 3
    constexpr uint32_t idesc = tc::idesc_bf16_f32(kMtKeys, kMtKeys, false);
    // descriptors of the first key and query tiles: others lie a constant number of 16-byte units away
    const uint64_t k_desc = tc::smem_desc(sm, 16, 1024), q_desc = tc::smem_desc(sm + S::Q_OFF, 16, 1024);
    int k = 0, u = 0;
    for (int t = t_first, pair = 0; t < t_end && wok; t += 2, ++pair) {
      const int n0 = tiles_seen(t), n1 = tiles_seen(t + 1), n = max(n0, n1);
      if (W) wok = wait(MT_QF0, pair) && (t + 1 >= t_end || wait(MT_QF0 + 1, pair));
      for (int kt = 0; kt < n && wok; ++kt, ++k) {
        const int kb = k % kMtKeyBufs;
        wok = wait(MT_KF0 + kb, k / kMtKeyBufs);
        for (int half = 0; half < 2 && wok; ++half) {
          if (kt >= (half ? n1 : n0)) continue;
          const int b = u % kMtBuffers;
          if (u >= kMtBuffers) wok = wait(MT_SE0 + b, u / kMtBuffers - 1);
          if (!wok) break;
          if (lane == 0) {
            tc::fence_after_sync();
            const uint64_t kd = k_desc + kb * (S::TILE / 16), qd = q_desc + half * (S::TILE / 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int off = ((kk / 4) * S::HALF + (kk % 4) * 32) / 16;
              if constexpr (W)
                tc::mma_bf16(tb + b * kMtKeys, kd + off, qd + off, idesc, kk > 0);
              else
                tc::mma_bf16_ts(tb + b * kMtKeys, tb + kTmemQ + half * (D / 2) + kk * 8, kd + off, idesc, kk > 0);
            }
            tc::mma_commit(&bar[MT_SD0 + b]);
            log.issue(MT_SD0 + b);
          }
          __syncwarp();
          ++u;
        }
        if (wok && lane == 0) {
          tc::mma_commit(&bar[MT_KE0 + kb]);
          log.issue(MT_KE0 + kb);
        }
        __syncwarp();
      }
    }
  } else {
    const int group = warp >> 2;  // takes the steps u with u % 3 == group, and S buffer `group`
    float* mine = acc + group * S::ACC;
    float m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};  // W false: this thread's columns
    if (W) griddep_wait();  // the first launch's results
    int u = 0;
    for (int t = t_first, pair = 0; t < t_end; t += 2, ++pair) {
      const int n0 = tiles_seen(t), n1 = tiles_seen(t + 1), n = max(n0, n1);
      if constexpr (W) {
        // every column's (maximum, 1 / sum) of the two tiles, its key ranges merged in ascending order, a
        // column to a thread (the score warps meet: the tiles before are done with)
        if (pair > 0) asm volatile("bar.sync 1, %0;" ::"n"(kMtScoreWarps * 32) : "memory");
        if (tid < 2 * kMtKeys) {
          const int col = tid % kMtKeys, r = (t + tid / kMtKeys) * R + col / G;
          float2 z = make_float2(0.0f, 0.0f);
          if (col < R * G && r < v.rows) z = column_stat(p, c, h, t + tid / kMtKeys, col, v.pos0 + r);
          float* stat = reinterpret_cast<float*>(sm + S::STAT_OFF + tid / kMtKeys * 1024);
          stat[col] = z.x;
          stat[kMtKeys + col] = z.y;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kMtScoreWarps * 32) : "memory");
      }
      for (int kt = 0; kt < n && wok; ++kt) {
        for (int half = 0; half < 2 && wok; ++half) {
          if (kt >= (half ? n1 : n0)) continue;
          const int use = u++;
          if (use % kMtBuffers != group) continue;
          const int t0 = key0 + kt * kMtKeys;
          wok = wait(MT_SD0 + group, use / kMtBuffers);
          if (!wok) break;
          tc::fence_after_sync();
          const uint32_t col = tb + lane_base + group * kMtKeys;
          if constexpr (!W) {
            // keys of the tile that the column sees: the first `seen`
            const int seen = v.pos0 + min((t + half) * R + m / G, v.rows - 1) - t0 + 1;
            const bool edge = v.pos0 + (t + half) * R - t0 + 1 < kMtKeys;  // some column of the tile sees less than all
            float mr = half ? m_ref[1] : m_ref[0], lr = half ? l_run[1] : l_run[0];
            over_columns(col, kMtKeys, [&](int i0, uint32_t(&x)[32]) {
              float s[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(x[i]);
              if (edge) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i0 + i >= seen) s[i] = -INFINITY;
              }
              float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
              for (int i = 4; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
              const float mx = __fmul_rn(fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])), scale);
              if (mx > __fadd_rn(mr, kRescaleSlack)) {
                lr = __fmul_rn(lr, ex2(__fsub_rn(mr, mx)));
                mr = mx;
              }
              const float neg = mr == -INFINITY ? 0.0f : -mr;
              float2 ls[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) ls[i] = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 z = __ffma2_rn(make_float2(s[i], s[i + 1]), make_float2(scale, scale), make_float2(neg, neg));
                ls[(i / 2) & 3] = __fadd2_rn(ls[(i / 2) & 3], make_float2(ex2(z.x), ex2(z.y)));
              }
              const float2 z = __fadd2_rn(__fadd2_rn(ls[0], ls[1]), __fadd2_rn(ls[2], ls[3]));
              lr = __fadd_rn(lr, __fadd_rn(z.x, z.y));
            });
            if (half) m_ref[1] = mr, l_run[1] = lr;
            else m_ref[0] = mr, l_run[0] = lr;
          } else {
            const float* stat = reinterpret_cast<const float*>(sm + S::STAT_OFF + half * 1024);
            const int row0 = (t + half) * R, cols = min(R, v.rows - row0) * G;
            // columns that see this thread's key: from `from` on (rows at or behind the key's position)
            const int from = max(0, t0 + m - (v.pos0 + row0)) * G;
            float2 w2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            // four columns' weights; in an edge tile those that do not see the key (or are none) are left
            // out whole, so that nothing of theirs reaches it
            auto add4 = [&](auto edge, const uint32_t(&x)[32], int i0, int i) {
              const float4 M = *reinterpret_cast<const float4*>(stat + i0 + i);
              float4 I = *reinterpret_cast<const float4*>(stat + kMtKeys + i0 + i);
              const float2 sc = make_float2(scale, scale);
              const float2 z0 = __ffma2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sc, make_float2(-M.x, -M.y));
              const float2 z1 = __ffma2_rn(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), sc, make_float2(-M.z, -M.w));
              float2 e0 = make_float2(ex2(z0.x), ex2(z0.y)), e1 = make_float2(ex2(z1.x), ex2(z1.y));
              if constexpr (decltype(edge)::value) {
                const int j = i0 + i;
                if (j < from || j >= cols) e0.x = I.x = 0.0f;
                if (j + 1 < from || j + 1 >= cols) e0.y = I.y = 0.0f;
                if (j + 2 < from || j + 2 >= cols) e1.x = I.z = 0.0f;
                if (j + 3 < from || j + 3 >= cols) e1.y = I.w = 0.0f;
              }
              w2[0] = __ffma2_rn(e0, make_float2(I.x, I.y), w2[0]);
              w2[1] = __ffma2_rn(e1, make_float2(I.z, I.w), w2[1]);
            };
            if (t0 + kMtKeys - 1 > v.pos0 + row0 || cols < kMtKeys)
              over_columns(col, cols, [&](int i0, uint32_t(&x)[32]) {
#pragma unroll
                for (int i = 0; i < 32; i += 4) add4(std::true_type(), x, i0, i);
              });
            else
              over_columns(col, kMtKeys, [&](int i0, uint32_t(&x)[32]) {
#pragma unroll
                for (int i = 0; i < 32; i += 4) add4(std::false_type(), x, i0, i);
              });
            const float2 w = __fadd2_rn(w2[0], w2[1]);
            mine[kt * kMtKeys + m] = __fadd_rn(mine[kt * kMtKeys + m], __fadd_rn(w.x, w.y));
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[MT_SE0 + group]);
        }
      }
      if (W && wok && lane == 0) {
        mbar_arrive(&bar[MT_QE0]);
        if (t + 1 < t_end) mbar_arrive(&bar[MT_QE0 + 1]);
      }
    }
    if constexpr (!W) {
      // the groups' shares of the keys, merged in order (the score warps meet)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        mine[half * 2 * kMtKeys + m] = m_ref[half];
        mine[half * 2 * kMtKeys + kMtKeys + m] = l_run[half];
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kMtScoreWarps * 32) : "memory");
      const int half = group, row = (first_tile + half) * R + m / G;
      if (group < 2 && wok && m < R * G && row < v.rows) {
        ColumnStat s{-INFINITY, 0.0f};
#pragma unroll
        for (int k = 0; k < kMtBuffers; ++k)
          s.merge(acc[k * S::ACC + half * 2 * kMtKeys + m], acc[k * S::ACC + half * 2 * kMtKeys + kMtKeys + m]);
        p.ws_part[p.chunk_part[c] +
                  ((static_cast<size_t>(h) * p.n_splits + split) * p.chunk_tiles[c] + first_tile + half) * kMtKeys + m] =
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
    for (int i = tid; i < nk * kMtKeys && key0 + i <= last; i += kMtThreads) {
      float w = acc[i];
#pragma unroll
      for (int k = 1; k < kMtBuffers; ++k) w = __fadd_rn(w, acc[k * S::ACC + i]);
      atomicAdd(sums + i, w);
    }
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
  count_launch();
  return launch_kernel(mass_tile_kernel<D, W>, dim3(static_cast<unsigned>(ctas)), dim3(kMtThreads),
                       MassTileSmem<D, W>::BYTES, stream, W, p);
}

}  // namespace pa
