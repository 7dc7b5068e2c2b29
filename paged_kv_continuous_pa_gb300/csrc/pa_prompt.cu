// pa_prompt.cu -- causal attention over whole prompts packed one behind the other
// (pa_prompt_attention), on tcgen05 tiles.
//
//   out_i = sum_{j <= i} exp2(s_ij - m_i) v_j / sum_{j <= i} exp2(s_ij - m_i),   s_ij = scale log2(e) q_i . k_j
//
// One pass over the keys with a running reference m_i: it moves only when a score passes it by
// 2^8, so that the accumulator is seldom rescaled and a row's maximum is only joined over its four
// lanes then.
//
// What bounds it: the two matrix products, 4 D flops for each (query head, query, key).
// One CTA per SM goes through units of work.  A unit is two query tiles of 128 rows that
// read the same keys: two query heads of one kv head at the same positions where the
// head group is even, else two neighbouring ranges of 128 positions of one head.  While
// the softmax of one tile runs, the tensor core works for the other.
//   warps 0-7, 8-15  softmax and output of tile A, B: 16 rows to a warp, a row in four lanes (so that a row is one
//                    warp's, and four warps of a scheduler hide each other's latencies); while they wait for the scores
//                    of a block with masked keys they look over its values
//   warp 16          takes the units and loads: queries and 128-key tiles of K and V through a ring (TMA)
//   warps 18, 19     issue the MMAs of tile A, B:  S = Q K^T (smem x smem), O += P V (TMEM x smem).  A whole warp goes
//                    through that code and one lane's instructions are predicated on: beside 16 busy warps an MMA
//                    of 128 x 128 x 16 was issued every 44 clocks so, every 52 in a branch of an elected lane, every 84
//                    in one of lane 0, and it takes the tensor core 64 (one prompt of 16384: 1532 -> 1308 us)
// Tensor memory: S of A and B (128 columns each, the first and the second 64 keys of a block apart), the weights P over
// their S as bf16, O of A and B.  A weight is rounded to bf16 (off by 2^-8 of itself at most) as the product with V takes it; the
// sum l of a row's weights is taken before, in FP32.  The chunk tiles of pa_prefill.cuh take two parts (2^-16) for half as
// many MMAs again, which are what bounds this kernel; results are off by 2.0e-3 of their norm with one, and the output's
// rounding alone makes 1.6e-3 of it.
//
// Masked keys.  Only the block on a tile's diagonal has any (keys behind the
// sequence's end are behind every row's diagonal too).  A masked key's weight is 0,
// but 0 times an infinite or NaN value is NaN, so 0 is put in the
// place of such values in shared memory; a row that does attend to one gets it added at the end.
//
// Order.  A launch of one CTA lists the tiles, and the CTAs take units from the list as they get free.  Longest
// first over all sequences ends with short units, but sends every sequence's keys through L2 once for each range of
// positions: 64 prompts of 64 to 2662 tokens (356 MB of keys and values) read 2.96 GB from DRAM and took 631 us.  So
// sequences come in groups whose keys and values are 16 MB, longest sequences first, and within a
// group the longest tiles first: 523 us (526 with 32 MB, 538 with 64, 520 with 8, where one prompt of 16384 took 1395 instead
// of 1280).  A unit that is taken before the last one's end is near goes to a CTA that is late already
// (128 instead of 102 us for 8192 tokens of 8 heads).  Few units need no list (9.6 -> 8.2 us for 77 tokens).
//
// Measured: 1276 to 1400 us for one prompt of 16384 with 32 heads over 8 (the clock under the power
// limit decides), 84 to 92% of what the products alone take at the measured matrix rate; 523 us for the 64 prompts (338 us of
// products, 13% more on the diagonals' masked halves, and a unit's own start and end).
#include <algorithm>
#include <cmath>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int kPrTile = 128;     // rows of a query tile, keys of a block
constexpr int kPrSoftmaxThreads = 512;
constexpr int kPrThreads = kPrSoftmaxThreads + 128;
constexpr int kPrGroups = 64, kPrBins = 64;  // of sequences, and of positions in a group, when the tiles are ordered
constexpr int kPrLengths = 1024;             // of the sequences' lengths
constexpr int64_t kPrGroupBytes = 16 << 20;
constexpr int kPrPlanThreads = 1024;
// registers of a softmax thread and of the others; their sum over the CTA is what it is launched with
constexpr int kPrRegs = 96, kPrSoftmaxRegs = 104, kPrOtherRegs = 64;
static_assert(kPrSoftmaxThreads * kPrSoftmaxRegs + 128 * kPrOtherRegs <= kPrThreads * kPrRegs, "register split");

struct PromptParams {
  const int32_t* row_starts;
  int32_t* n_tiles;      // workspace: number of tiles listed, number of units taken from the list
  int4* tiles;           // workspace: first row and end of the sequence, position of the tile
  int32_t* groups;       // workspace: each sequence's group
  const uint16_t* v;
  int64_t v_stride;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int32_t n_rows, n_seqs, Hq, G, group_rows;
  int32_t listed;        // the units are taken from the list (else unit i is CTA i's)
  int32_t tile_rows;     // positions of a unit: 128 (two heads) or 256
  float scale_log2;
  uint32_t wait_limit;
  int32_t debug_stall;
  CUtensorMap qmap, kmap, vmap;  // [rows][heads][D], boxes of 64 elements x 1 head x 128 rows
};

// Exclusive sums over the values of the CTA's threads, and (in sums[31]) their total.
__device__ __forceinline__ int prompt_scan(int x, int32_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, own = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int z = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += z;
    }
    sums[lane] = y;
  }
  __syncthreads();
  return x - own + (warp > 0 ? sums[warp - 1] : 0);
}

// The tiles of all sequences in the order in which they are dealt out: by groups of sequences, the longest
// sequences first, and in a group the longest tiles first (to within a 64th of the group's longest).
__global__ void __launch_bounds__(kPrPlanThreads) prompt_plan_kernel(const __grid_constant__ PromptParams p) {
  __shared__ int32_t hist[kPrGroups * kPrBins];
  __shared__ int32_t rows[kPrLengths], longest[kPrGroups], sums[32];
  static_assert(kPrGroups * kPrBins == 4 * kPrPlanThreads && kPrLengths == kPrPlanThreads, "bins of a thread");
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kPrGroups * kPrBins; i += kPrPlanThreads) hist[i] = 0;
  rows[tid] = 0;
  if (tid < kPrGroups) longest[tid] = 0;
  bool bad = false;
  for (int s = tid; s <= p.n_seqs; s += kPrPlanThreads) {
    const int a = p.row_starts[s];
    bad |= a < 0 || a > p.n_rows || (s > 0 && p.row_starts[s - 1] > a);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      record_error(p.status, ST_OUT_OF_RANGE);
      p.n_tiles[0] = 0;
    }
    return;
  }
  auto shift_of = [](int length, int bins) {
    int shift = 0;
    while ((length / kPrTile) >> shift >= bins) ++shift;
    return shift;
  };
  const bool grouped = p.n_rows > p.group_rows;
  if (grouped) {
    // rows of longer sequences before a sequence's own say which group it is in
    const int shift = shift_of(p.n_rows, kPrLengths);
    auto bin_of = [&](int length) { return kPrLengths - 1 - ((length / kPrTile) >> shift); };
    for (int s = tid; s < p.n_seqs; s += kPrPlanThreads) {
      const int length = p.row_starts[s + 1] - p.row_starts[s];
      atomicAdd(&rows[bin_of(length)], length);
    }
    __syncthreads();
    rows[tid] = prompt_scan(rows[tid], sums);
    __syncthreads();
    for (int s = tid; s < p.n_seqs; s += kPrPlanThreads) {
      const int length = p.row_starts[s + 1] - p.row_starts[s];
      const int group = min(kPrGroups - 1, atomicAdd(&rows[bin_of(length)], length) / p.group_rows);  // (empty ones may lie behind the last)
      p.groups[s] = group;
      atomicMax(&longest[group], length);
    }
    __syncthreads();
  }
  auto place_of = [&](int s, int& shift) {  // the bin of a sequence's first tile
    const int group = grouped ? p.groups[s] : 0;
    shift = shift_of(grouped ? longest[group] : p.n_rows, kPrBins);
    return group * kPrBins + kPrBins - 1;
  };
  for (int s = warp; s < p.n_seqs; s += kPrPlanThreads / 32) {
    const int length = p.row_starts[s + 1] - p.row_starts[s];
    int shift;
    const int first = place_of(s, shift);
    for (int64_t pos = static_cast<int64_t>(lane) * p.tile_rows; pos < length; pos += 32ll * p.tile_rows)
      atomicAdd(&hist[first - ((static_cast<int>(pos) / kPrTile) >> shift)], 1);
  }
  __syncthreads();
  int4 n = *reinterpret_cast<const int4*>(hist + 4 * tid);
  const int before = prompt_scan(n.x + n.y + n.z + n.w, sums);
  *reinterpret_cast<int4*>(hist + 4 * tid) = make_int4(before, before + n.x, before + n.x + n.y, before + n.x + n.y + n.z);
  if (tid == 0) {
    p.n_tiles[0] = sums[31];
    p.n_tiles[1] = 0;  // units taken
  }
  __syncthreads();
  for (int s = warp; s < p.n_seqs; s += kPrPlanThreads / 32) {
    const int begin = p.row_starts[s], end = p.row_starts[s + 1];
    int shift;
    const int first = place_of(s, shift);
    for (int64_t pos = static_cast<int64_t>(lane) * p.tile_rows; pos < end - begin; pos += 32ll * p.tile_rows)
      p.tiles[atomicAdd(&hist[first - ((static_cast<int>(pos) / kPrTile) >> shift)], 1)] = make_int4(begin, end, static_cast<int>(pos), 0);
  }
}

__device__ __forceinline__ void pr_load_3d(void* dst_smem, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// The wait of a barrier that is not passed yet.
__device__ __forceinline__ bool pr_wait(uint64_t* bar, uint32_t parity, uint32_t limit, int32_t* status) {
  if (mbar_wait(bar, parity, limit)) return true;
  record_error(status, ST_TIMEOUT);
  return false;
}

// Waits for every load of tensor memory started; r is read only behind it.
__device__ __forceinline__ void pr_ld_wait(float* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                 "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
                 "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                 "+f"(r[30]), "+f"(r[31])
               :
               : "memory");
}

// 64 columns of 16 lanes, without waiting: lane 4 g + c of the warp gets columns 8 i + 2c, + 1 of rows g (r[4i], r[4i + 1]) and g + 8.
__device__ __forceinline__ void pr_ld16x64(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
// 32 columns of two 16-bit numbers each, in the same places: w[2i] of row g, w[2i + 1] of row g + 8.
__device__ __forceinline__ void pr_st16x32(uint32_t taddr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}
// 16 columns of 16 lanes, rows g and g + 8 multiplied in place (few registers: it is seldom done).
__device__ __forceinline__ void pr_scale16x16(uint32_t taddr, float f0, float f1) {
  float r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] *= (i & 2) ? f1 : f0;
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(r[0]), "f"(r[1]),
               "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}

__device__ __forceinline__ uint32_t pr_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Two numbers at a time: a * b + c and a + b.
__device__ __forceinline__ uint64_t pr_two(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void pr_split(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t pr_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pr_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float pr_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Four words of each of a quad's lanes transposed: lane c gets word c of its lanes in order.
__device__ __forceinline__ void pr_transpose4(uint32_t (&w)[4], int c) {
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    const bool up = (c & d) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + d], d);
      if (up)
        w[i] = got;
      else
        w[i + d] = got;
    }
  }
}

// One lane of a converged warp, the same one each time, as a number that is 0 elsewhere.
__device__ __forceinline__ uint32_t pr_elect() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(one));
  return one;
}
// D[tmem] (+)= A B and a commit, by the lane where `one` is not 0: the warp stays together, so that operands
// are worked out once for all of it.
__device__ __forceinline__ void pr_mma(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 e, %5, 0;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u), "r"(one)
      : "memory");
}
__device__ __forceinline__ void pr_mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 e, %5, 0;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u), "r"(one)
      : "memory");
}
__device__ __forceinline__ void pr_commit(uint32_t one, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(one)
      : "memory");
}

template <int D>
struct PromptSmem {  // byte offsets from the base, which is 1024-byte aligned (no static shared memory lies before it)
  static constexpr int NH = D / 64;
  static constexpr int HALF = kPrTile * 128;       // 64 elements of 128 rows
  static constexpr int TILE = NH * HALF;
  static constexpr int STAGES = D == 128 ? 5 : 8;  // tiles of K and V in the ring
  static constexpr int RING = 2 * TILE;            // behind the two query tiles
  static constexpr int BAR = RING + STAGES * TILE;
  static constexpr int BYTES = BAR + 640;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

// A unit: the tiles' positions, heads and numbers of key blocks.  (No arrays: they would be indexed by a tile.)
struct PromptUnit {
  int begin, end;  // rows of the sequence
  int pos_a, pos_b, head_a, head_b, blocks_a, blocks_b;
  int n;           // blocks of the longer tile
};

// A place in the ring: its slot and the parity of its turn.
template <int STAGES>
struct PromptRing {
  int slot = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next() {
    if (++slot == STAGES) {
      slot = 0;
      turn ^= 1u;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using S = PromptSmem<D>;
  enum {
    FULL = 0,                    // K / V tile landed
    EMPTY = FULL + S::STAGES,    // ... read by its MMAs
    QF = EMPTY + S::STAGES,      // queries of tile A / B landed
    QE = QF + 2,                 // ... read by the unit's MMAs
    SF = QE + 2,                 // scores of tile A / B for the first / second 64 keys of a block
    PF = SF + 4,                 // ... their weights (the scores are read, O may be added to)
    PV = PF + 4,                 // O of tile A / B is complete
    PL = PV + 2,                 // ... holds all but the unit's last 64 keys
    // the values of a block with masked keys are looked over: in turn, as the look may be a unit ahead of the
    // MMAs, and a unit has at most two such blocks
    VOK = PL + 2,
    VIN = VOK + 4,               // its load is under way (the ring's slot has come to this tile)
    DRAIN = VIN + 4,
    UF = DRAIN + 2,              // a unit was taken, in turn
    UE = UF + 4,                 // ... every warp knows it
    STALL = UE + 4,
    COUNT
  };
  // A unit is announced when every warp knows the one four before it (UE), so a tile's warps may write the flag of unit
  // k + 4 while one of the other tile's has yet to read that of unit k: five are in use, in a ring of eight.
  constexpr int FLAGS = 8;
  constexpr int UNITS = (COUNT * 8 + 4 + 4 * FLAGS + 15) / 16 * 16;  // behind the barriers, the tensor memory's address and the flags
  static_assert(UNITS + 64 <= S::BYTES - S::BAR, "barriers");
  extern __shared__ __align__(1024) unsigned char sm[];
  if ((smem_addr(sm) & 1023u) != 0) {  // (the swizzled tiles would be read at other places than they were written)
    if (threadIdx.x == 0) record_error(p.status, ST_LAUNCH);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + S::BAR + COUNT * 8);
  volatile int32_t* odd_values = reinterpret_cast<volatile int32_t*>(tslot + 1);  // entry k % FLAGS is k + 1: values of unit k were put to 0
  volatile int4* taken = reinterpret_cast<volatile int4*>(sm + S::BAR + UNITS);  // entry k % 4: unit k's tile and, in w, its head (-1: no unit)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (warp == 0) tc::tmem_alloc(tslot, 512);
  if (tid >= 32 && tid < 32 + COUNT) {
    const int i = tid - 32;
    mbar_init(&bar[i], i >= UE && i < UE + 4 ? 18u : (i >= PF && i < PF + 4) || (i >= VOK && i < VOK + 4) ? 8u : i >= EMPTY && i < QF ? 2u : 1u);
    if (i < FLAGS) odd_values[i] = 0;
    fence_barrier_init();
  }
  if (tid == kPrSoftmaxThreads + 32) {
    tc::prefetch_tensormap(&p.qmap);
    tc::prefetch_tensormap(&p.kmap);
    tc::prefetch_tensormap(&p.vmap);
  }
  // The first unit is the CTA's own (the loading warp finds it; without a list, beside the set-up).
  const bool two_heads = p.tile_rows == kPrTile;
  const int per_tile = two_heads ? p.Hq / 2 : p.Hq;
  int units = 0, u = blockIdx.x;
  int4 tile = make_int4(0, 0, 0, 0);
  if (warp == 16 && !p.listed) {
    // a lane to a sequence; tiles in the sequences' order
    const int begin = lane < p.n_seqs ? p.row_starts[lane] : 0, end = lane < p.n_seqs ? p.row_starts[lane + 1] : 0;
    if (__any_sync(0xffffffffu, begin < 0 || end > p.n_rows || end < begin)) {
      if (lane == 0) record_error(p.status, ST_OUT_OF_RANGE);
    } else {
      const int own = (end - begin + p.tile_rows - 1) / p.tile_rows;
      int upto = own;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      units = __shfl_sync(0xffffffffu, upto, 31) * per_tile;
      const int i = u / per_tile;
      const int from = __popc(__ballot_sync(0xffffffffu, upto <= i)) & 31;  // (32: no unit for this CTA)
      tile = make_int4(__shfl_sync(0xffffffffu, begin, from), __shfl_sync(0xffffffffu, end, from),
                       (i - __shfl_sync(0xffffffffu, upto - own, from)) * p.tile_rows, 0);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_wait();  // the list of tiles
  const uint32_t tb = *tslot;
  if (warp == 16 && p.listed) {
    units = p.n_tiles[0] * per_tile;
    if (u < units) tile = __ldcg(p.tiles + u / per_tile);
  }

  auto wait = [&](int b, uint32_t parity) { return mbar_test(&bar[b], parity) || pr_wait(&bar[b], parity, p.wait_limit, p.status); };
  auto describe = [&](PromptUnit& x, int begin, int end, int pos, int h) {
    x.begin = begin;
    x.end = end;
    x.pos_a = pos;
    x.n = x.blocks_a = pos / kPrTile + 1;
    x.blocks_b = 0;
    if (two_heads) {
      x.head_a = 2 * h;
      x.head_b = 2 * h + 1;
      x.pos_b = pos;
      x.blocks_b = x.n;
    } else {
      x.head_a = x.head_b = h;
      x.pos_b = pos + kPrTile;
      if (x.pos_b < end - begin) x.n = x.blocks_b = x.blocks_a + 1;
    }
  };
  // The k-th unit of this CTA, for a whole warp; false behind the last, and where the wait for it ran out.
  auto unit_at = [&](int k, PromptUnit& x, bool& ok) {
    ok = __all_sync(0xffffffffu, wait(UF + (k & 3), (k >> 2) & 1));
    if (!ok) return false;
    const int begin = taken[k & 3].x, end = taken[k & 3].y, pos = taken[k & 3].z, h = taken[k & 3].w;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[UE + (k & 3)]);
    if (h < 0) return false;
    describe(x, begin, end, pos, h);
    return true;
  };

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrOtherRegs));
    if (warp == 16 && lane == 0) {
      // ---- loads
      PromptRing<S::STAGES> at;
      int items = 0, checked = 0, done_a = 0, done_b = 0;  // tiles of K and V, those to be looked over, query tiles issued so far
      bool ok = !p.debug_stall || wait(STALL, 0);  // (runs out by construction)
      PromptUnit x{};
      auto queries = [&](int t, int& done, int pos, int head) {
        if (done > 0 && !wait(QE + t, (done - 1) & 1)) return false;
        mbar_arrive_expect_tx(&bar[QF + t], S::TILE);
        for (int hf = 0; hf < S::NH; ++hf)
          pr_load_3d(sm + t * S::TILE + hf * S::HALF, &p.qmap, hf * 64, head, x.begin + pos, &bar[QF + t]);
        ++done;
        return true;
      };
      auto keys = [&](const CUtensorMap* map, int kv_head, int j) {
        if (items >= S::STAGES && !wait(EMPTY + at.slot, at.turn ^ 1u)) return false;
        mbar_arrive_expect_tx(&bar[FULL + at.slot], S::TILE);
        for (int hf = 0; hf < S::NH; ++hf)
          pr_load_3d(sm + S::RING + at.slot * S::TILE + hf * S::HALF, map, hf * 64, kv_head, x.begin + j * kPrTile,
                     &bar[FULL + at.slot]);
        ++items;
        at.next();
        return true;
      };
      for (int k = 0; ok; ++k) {
        if (k >= 4) ok = wait(UE + (k & 3), ((k >> 2) - 1) & 1);
        if (!ok) break;
        taken[k & 3].x = tile.x;
        taken[k & 3].y = tile.y;
        taken[k & 3].z = tile.z;
        taken[k & 3].w = u < units ? u % per_tile : -1;
        mbar_arrive(&bar[UF + (k & 3)]);
        if (u >= units) break;
        describe(x, tile.x, tile.y, tile.z, u % per_tile);
        const int kv_head = x.head_a / p.G;
        for (int j = 0; ok && j < x.n; ++j) {
          if (j == x.n - 1) u = p.listed ? static_cast<int>(gridDim.x) + atomicAdd(p.n_tiles + 1, 1) : units;  // the next one
          ok = keys(&p.kmap, kv_head, j);
          if (ok && j == 0)  // (these keys need not wait for the last unit's queries to be done with)
            ok = queries(0, done_a, x.pos_a, x.head_a) && (x.blocks_b == 0 || queries(1, done_b, x.pos_b, x.head_b));
          ok = ok && keys(&p.vmap, kv_head, j);
          if (ok && j >= x.blocks_a - 1) mbar_arrive(&bar[VIN + (checked++ & 3)]);
        }
        if (u < units) tile = __ldcg(p.tiles + u / per_tile);
      }
      if (!ok) {  // what is in flight lands before the shared memory is given up
        for (int i = max(0, items - S::STAGES); i < items; ++i)
          mbar_wait(&bar[FULL + i % S::STAGES], (i / S::STAGES) & 1, kDrainWaitLimit);
        if (done_a > 0) mbar_wait(&bar[QF], (done_a - 1) & 1, kDrainWaitLimit);
        if (done_b > 0) mbar_wait(&bar[QF + 1], (done_b - 1) & 1, kDrainWaitLimit);
      }
    } else if (warp >= 18) {
      // ---- MMAs of tile t.  A block's scores are two products of 64 keys with a place of their own each: while
      // the weights of one are computed the tensor core has the other, and the same place's next scores come
      // right behind its product with V.  (Products of 128 keys into one place take 2048 clocks a pair of tiles
      // instead of 2560, as their operands come from shared memory at its full rate, but wait for the weights and the
      // weights for them: 3500 clocks.)
      constexpr uint32_t id_qk = tc::idesc_bf16_f32(kPrTile, 64, false);
      constexpr uint32_t id_pv = tc::idesc_bf16_f32(kPrTile, D, true);
      const int t = warp - 18;
      const uint32_t ts = tb + t * 128, to = ts + 256;
      PromptRing<S::STAGES> at;
      uint32_t q_turn = 0, p_turn = 0;
      int checked = 0;
      bool ok = true;
      PromptUnit x{};
      const uint32_t one = pr_elect();
      auto wait_all = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
      auto arrive = [&](int b) {
        if (lane == 0) mbar_arrive(&bar[b]);
      };
      // Matrix descriptors differ in their address alone (the lower 14 bits, in 16 bytes).
      const uint64_t k_desc = tc::smem_desc(sm, 16, 1024), v_desc = tc::smem_desc(sm, S::HALF, 1024);
      const uint32_t hi = static_cast<uint32_t>(k_desc >> 32);
      const uint32_t q_lo = static_cast<uint32_t>(k_desc) + t * (S::TILE >> 4);
      const uint32_t k_lo = static_cast<uint32_t>(k_desc) + (S::RING >> 4), v_lo = static_cast<uint32_t>(v_desc) + (S::RING >> 4);
      auto desc = [&](uint32_t lo) { return static_cast<uint64_t>(hi) << 32 | lo; };
      // the next tile of the ring (a tile that is not used is waited for, too: a turn that is missed looks like the next but one)
      auto take = [&](int& slot) {
        slot = at.slot;
        const bool got = wait_all(FULL + at.slot, at.turn);
        at.next();
        return got;
      };
      auto skip = [&](int& slot) {
        slot = at.slot;
        at.next();
      };
      auto qk = [&](int slot, int half) {
        const uint32_t kt = k_lo + slot * (S::TILE >> 4) + half * ((64 * 128) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * S::HALF + (kk % 4) * 32) >> 4;
          pr_mma(one, ts + 64 * half, desc(q_lo + off), desc(kt + off), id_qk, kk > 0);
        }
        pr_commit(one, &bar[SF + 2 * t + half]);
      };
      auto pv = [&](int slot, int half, bool first) {
        if (!wait_all(PF + 2 * t + half, p_turn)) return false;
        tc::fence_after_sync();
        const uint32_t vt = v_lo + slot * (S::TILE >> 4) + half * ((64 * 128) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          pr_mma_ts(one, to, ts + 64 * half + kk * 8, desc(vt + kk * (2048 >> 4)), id_pv, !first || kk > 0);
        return true;
      };
      for (int k = 0; ok && unit_at(k, x, ok); ++k) {
        const int n = t == 0 ? x.blocks_a : x.blocks_b;
        int slot, next = 0;
        ok = take(slot) && (n == 0 || wait_all(QF + t, q_turn));
        if (!ok) break;
        if (n > 0) {
          q_turn ^= 1u;
          qk(slot, 0);
          qk(slot, 1);
          if (n == 1) pr_commit(one, &bar[QE + t]);
        } else {
          arrive(EMPTY + slot);
        }
        for (int j = 0; j < x.n; ++j) {
          if (j < n) {
            skip(slot);
            if (j + 1 < n)
              skip(next);
            else if (j + 1 < x.n)
              ok = take(next);
          } else {
            ok = take(slot) && (j + 1 == x.n || take(next));
          }
          if (ok && j >= x.blocks_a - 1) {
            ok = wait_all(VOK + (checked & 3), (checked >> 2) & 1);
            ++checked;
          }
          if (!ok) break;
          if (j >= n) {  // no block of this tile
            arrive(EMPTY + slot);
            if (j + 1 < x.n) arrive(EMPTY + next);
            continue;
          }
          ok = pv(slot, 0, j == 0);
          if (!ok) break;
          if (j + 1 < n) qk(next, 0);
          if (j + 1 == n) pr_commit(one, &bar[PL + t]);
          ok = pv(slot, 1, false);
          if (!ok) break;
          p_turn ^= 1u;
          if (j + 1 < n) qk(next, 1);
          if (j + 1 == n && j + 1 < x.n) arrive(EMPTY + next);
          if (j + 2 == n) pr_commit(one, &bar[QE + t]);
          if (j + 1 == n) pr_commit(one, &bar[PV + t]);
        }
      }
      if (!ok) {  // every MMA issued is done before the tensor memory is given up
        pr_commit(one, &bar[DRAIN + t]);
        mbar_wait(&bar[DRAIN + t], 0, kDrainWaitLimit);
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrSoftmaxRegs));
    // ---- softmax and output of tile t: rows r0 and r0 + 8, columns 8 i + 2 c, + 1
    const int t = warp >> 3, c = lane & 3;
    const int r0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1) + (lane >> 2);
    const uint32_t ts = tb + (static_cast<uint32_t>(r0 - (lane >> 2)) << 16) + t * 128, to = ts + 256;
    const uint64_t scale2 = pr_two(p.scale_log2, p.scale_log2);
    uint32_t s_turn = 0, o_turn = 0;
    int items = 0, checked = 0;  // tiles of K and V, and those looked over, of all units so far
    const bool leader = (warp & 7) == 0;
    auto landed = [&](int item) { return wait(FULL + item % S::STAGES, (item / S::STAGES) & 1); };
    auto release = [&](int item) {
      if (leader && lane == 0) mbar_arrive(&bar[EMPTY + item % S::STAGES]);
    };
    bool ok = true;
    PromptUnit x{};
    // Values of block `block` (the ring's tile `item`): infinities and NaN become 0.
    auto look_over = [&](int item, int k) {
      const int slot = item % S::STAGES;
      if (!__all_sync(0xffffffffu, wait(VIN + (checked & 3), (checked >> 2) & 1) && wait(FULL + slot, (item / S::STAGES) & 1)))
        return false;
      uint4* tile = reinterpret_cast<uint4*>(sm + S::RING + slot * S::TILE);
      bool found = false;
#pragma unroll 4
      for (int i = tid & 255; i < S::TILE / 16; i += 256) {
        const uint4 w = tile[i];
        auto odd = [](uint32_t a) { return ((a & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };  // exponent of all ones
        if (odd(w.x) | odd(w.y) | odd(w.z) | odd(w.w)) {
          auto clean = [&](uint32_t a) {
            const uint32_t o = odd(a);
            return a & ~((o & 0x8000u ? 0xffffu : 0u) | (o & 0x80000000u ? 0xffff0000u : 0u));
          };
          tile[i] = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
          found = true;
        }
      }
      if (found) odd_values[k & (FLAGS - 1)] = k + 1;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[VOK + (checked & 3)]);
      return true;
    };
    for (int k = 0; ok && unit_at(k, x, ok); ++k) {
      const int n = t == 0 ? x.blocks_a : x.blocks_b;
      const bool two_looks = x.blocks_b > x.blocks_a;  // each tile's warps look over the values of its own diagonal
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
      for (int j = 0; j < n; ++j, s_turn ^= 1u) {
        if (j == n - 1 && (t == 0 || two_looks)) {
          checked += t;
          ok = look_over(items + 2 * j + 1, k);
          checked -= t;
          if (!ok) break;
        }
        for (int half = 0; half < 2; ++half) {  // 64 keys
          ok = __all_sync(0xffffffffu, wait(SF + 2 * t + half, s_turn));
          if (!ok) break;
          tc::fence_after_sync();
          if (half == 0 && leader) {  // what the issuer needs behind these weights
            ok = __all_sync(0xffffffffu, landed(items + 2 * j + 1) && (j + 1 == n || landed(items + 2 * j + 2)));
            if (!ok) break;
          }
          if (half == 1) {  // the block's scores are complete, and with them the last block's product with V
            release(items + 2 * j);
            if (j > 0) release(items + 2 * j - 1);
          }
          const uint32_t at = ts + 64 * half;
          float s[32];
          pr_ld16x64(at, s);
          pr_ld_wait(s);
          if (j == n - 1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int column = 64 * half + 8 * (i >> 2) + 2 * c + (i & 1);
              s[i] = column > r0 + ((i & 2) ? 8 : 0) ? -INFINITY : s[i];
            }
          }
          float top0 = fmaxf(s[0], s[1]), top1 = fmaxf(s[2], s[3]);
#pragma unroll
          for (int i = 4; i < 32; i += 4) {
            top0 = pr_max3(top0, s[i], s[i + 1]);
            top1 = pr_max3(top1, s[i + 2], s[i + 3]);
          }
          if (__any_sync(0xffffffffu, (top0 - m0) * p.scale_log2 > kRescaleSlack || (top1 - m1) * p.scale_log2 > kRescaleSlack)) {
#pragma unroll
            for (int d = 1; d < 4; d *= 2) {
              top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, d));
              top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, d));
            }
            const bool move0 = (top0 - m0) * p.scale_log2 > kRescaleSlack, move1 = (top1 - m1) * p.scale_log2 > kRescaleSlack;
            if (j > 0 || half > 0) {
              // The products with V so far come first.  The next scores were issued behind the last of them.
              const bool got = half == 0    ? wait(SF + 2 * t + 1, s_turn)
                               : j + 1 < n ? wait(SF + 2 * t, s_turn ^ 1u)
                                           : wait(PL + t, o_turn);
              ok = __all_sync(0xffffffffu, got);
              if (!ok) break;
              tc::fence_after_sync();
              const float f0 = move0 ? ex2((m0 - top0) * p.scale_log2) : 1.0f, f1 = move1 ? ex2((m1 - top1) * p.scale_log2) : 1.0f;
              l0 *= f0;
              l1 *= f1;
#pragma unroll 1
              for (int d = 0; d < D; d += 16) pr_scale16x16(to + d, f0, f1);
              tc::tmem_wait_st();
            }
            if (move0) m0 = top0;
            if (move1) m1 = top1;
          }
          const float shift0 = m0 == -INFINITY ? 0.0f : -m0 * p.scale_log2, shift1 = m1 == -INFINITY ? 0.0f : -m1 * p.scale_log2;
          const uint64_t shifts[2] = {pr_two(shift0, shift0), pr_two(shift1, shift1)};
          uint64_t sum[2] = {0ull, 0ull};
          uint32_t w[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            float a, b;
            pr_split(pr_fma2(pr_two(s[2 * q], s[2 * q + 1]), scale2, shifts[q & 1]), a, b);
            a = ex2(a);
            b = ex2(b);
            sum[q & 1] = pr_add2(sum[q & 1], pr_two(a, b));
            w[q] = pr_pack(a, b);
          }
          pr_st16x32(at, w);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[PF + 2 * t + half]);
          float a, b;
          pr_split(sum[0], a, b);
          l0 += a + b;
          pr_split(sum[1], a, b);
          l1 += a + b;
        }
        if (!ok) break;
      }
      if (!ok) break;
      items += 2 * x.n;
      checked += two_looks ? 2 : 1;
      if (n == 0) continue;
      // ---- output
      ok = __all_sync(0xffffffffu, wait(PV + t, o_turn));
      if (!ok) break;
      o_turn ^= 1u;
      release(items - 2 * x.n + 2 * n - 1);
      tc::fence_after_sync();
#pragma unroll
      for (int d = 1; d < 4; d *= 2) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      const int row0 = x.begin + (t == 0 ? x.pos_a : x.pos_b) + r0, row1 = row0 + 8, head = t == 0 ? x.head_a : x.head_b;
      const bool odd = odd_values[k & (FLAGS - 1)] == k + 1;
      const float inv0 = __fdiv_rn(1.0f, l0), inv1 = __fdiv_rn(1.0f, l1);
      uint16_t* out0 = p.out + (static_cast<int64_t>(row0) * p.Hq + head) * D;
      uint16_t* out1 = out0 + static_cast<int64_t>(8) * p.Hq * D;
#pragma unroll 1
      for (int half = 0; half < D / 64; ++half) {
        float o[32];
        pr_ld16x64(to + 64 * half, o);
        pr_ld_wait(o);
        if (odd) {  // the values that were put to 0 and a row attends to
          for (int key = x.begin + (x.blocks_a - 1) * kPrTile; key <= min(row1, x.end - 1); ++key) {
            const uint16_t* v = p.v + key * p.v_stride + (head / p.G) * D + 64 * half + 2 * c;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float a = __uint_as_float(static_cast<uint32_t>(v[8 * (i >> 2) + (i & 1)]) << 16);
              if (!(fabsf(a) < INFINITY) && key <= ((i & 2) ? row1 : row0)) o[i] += a;
            }
          }
        }
        // 8 elements to a lane: the quad's lanes hold two of each of four octets
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w0[4], w1[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* y = o + 4 * (4 * q + i);
            w0[i] = pr_pack(y[0] * inv0, y[1] * inv0);
            w1[i] = pr_pack(y[2] * inv1, y[3] * inv1);
          }
          pr_transpose4(w0, c);
          pr_transpose4(w1, c);
          const int d0 = 64 * half + 32 * q + 8 * c;
          if (row0 < x.end) *reinterpret_cast<uint4*>(out0 + d0) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
          if (row1 < x.end) *reinterpret_cast<uint4*>(out1 + d0) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        }
      }
      if (p.lse != nullptr && c == 0) {
        auto store = [&](int row, float m, float l) {
          if (row < x.end)
            p.lse[static_cast<int64_t>(row) * p.Hq + head] =
                l > 0.0f ? 0.69314718055994531f * fmaf(m, p.scale_log2, log2f(l)) : l == 0.0f ? -INFINITY : l;
        };
        store(row0, m0, l0);
        store(row1, m1, l1);
      }
      tc::fence_before_sync();  // O is read before the next unit's weights are announced
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tb, 512);
}

template <int D>
cudaError_t launch_prompt(const PromptParams& p, unsigned grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_dynamic_smem(prompt_kernel<D>, done, PromptSmem<D>::BYTES);
  if (e != cudaSuccess) return e;
  // the register split waits for what the CTA was not launched with
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_acquire) == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, prompt_kernel<D>);
    if (e != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_release);
  }
  if (regs.load(std::memory_order_acquire) != kPrRegs) return cudaErrorInvalidKernelImage;
  if (p.listed) {
    prompt_plan_kernel<<<1, kPrPlanThreads, 0, stream>>>(p);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  e = launch_kernel(prompt_kernel<D>, dim3(grid), dim3(kPrThreads), PromptSmem<D>::BYTES, stream, p.listed != 0, p);
  count_launch();
  return e;
}

}  // namespace pa

using pa::aligned;
using pa::cuda_fail;
using pa::fail;

namespace {

// Whether a unit is two heads at the same positions (else two ranges of one head).
bool two_heads(int32_t hq, int32_t hkv) { return hq / hkv % 2 == 0; }

int64_t most_tiles(int32_t n_rows, int32_t n_seqs, int32_t hq, int32_t hkv) {
  return n_rows / (two_heads(hq, hkv) ? pa::kPrTile : 2 * pa::kPrTile) + static_cast<int64_t>(n_seqs);
}

pa_status check_prompt(int32_t n_rows, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t head_dim) {
  if (n_rows < 0 || n_seqs < 0) return fail(PA_ERR_INVALID_ARG, "n_rows %d or n_seqs %d < 0", n_rows, n_seqs);
  if (hkv <= 0 || hq <= 0 || hq % hkv != 0)
    return fail(PA_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of num_kv_heads %d", hq, hkv);
  if (head_dim != 64 && head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", head_dim);
  if (most_tiles(n_rows, n_seqs, hq, hkv) * hq > 0x7fffffff - 1024)
    return fail(PA_ERR_UNSUPPORTED, "%d rows of %d query heads in one call", n_rows, hq);
  return PA_OK;
}

pa_status check_rows16(const char* name, const void* base, int64_t stride, int64_t elements) {
  if (base == nullptr) return fail(PA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(base, 16)) return fail(PA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride < elements || stride % 8 != 0 || stride >= (1ll << 38))
    return fail(PA_ERR_INVALID_ARG, "%s rows of %lld elements, %lld apart: a multiple of 8, at least a row", name,
                (long long)elements, (long long)stride);
  return PA_OK;
}

}  // namespace

extern "C" {

size_t pa_prompt_workspace_bytes(int32_t n_rows, int32_t n_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim) {
  if (check_prompt(n_rows, n_seqs, num_q_heads, num_kv_heads, head_dim) != PA_OK) return 0;
  return 256 + static_cast<size_t>(most_tiles(n_rows, n_seqs, num_q_heads, num_kv_heads)) * sizeof(int4) +
         static_cast<size_t>(n_seqs) * sizeof(int32_t);
}

pa_status pa_prompt_attention(int32_t n_rows, int32_t n_seqs, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride, pa_dtype dtype, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, const int32_t* row_starts, float softmax_scale,
                              void* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* status_dev,
                              void* stream) {
  pa_status st = check_prompt(n_rows, n_seqs, num_q_heads, num_kv_heads, head_dim);
  if (st != PA_OK) return st;
  if (dtype != PA_F32 && dtype != PA_BF16) return fail(PA_ERR_INVALID_ARG, "prompt attention takes bf16 rows");
  if (dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "prompt attention takes bf16 rows");
  if (n_rows == 0 || n_seqs == 0) return PA_OK;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim, kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  st = check_rows16("q", q, q_stride, q_row);
  if (st == PA_OK) st = check_rows16("k", k, k_stride, kv_row);
  if (st == PA_OK) st = check_rows16("v", v, v_stride, kv_row);
  if (st == PA_OK) st = check_rows16("out", out, q_row, q_row);
  if (st != PA_OK) return st;
  if (row_starts == nullptr) return fail(PA_ERR_INVALID_ARG, "row_starts is NULL");
  const size_t need = pa_prompt_workspace_bytes(n_rows, n_seqs, num_q_heads, num_kv_heads, head_dim);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PA_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need,
                workspace == nullptr ? static_cast<size_t>(0) : workspace_bytes);
  if (!aligned(workspace, 256)) return fail(PA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const double scale = softmax_scale > 0.f ? static_cast<double>(softmax_scale) : 1.0 / std::sqrt(static_cast<double>(head_dim));
  pa::PromptParams p{};
  p.row_starts = row_starts;
  p.n_tiles = static_cast<int32_t*>(workspace);
  p.tiles = reinterpret_cast<int4*>(static_cast<unsigned char*>(workspace) + 256);
  p.groups = reinterpret_cast<int32_t*>(p.tiles + most_tiles(n_rows, n_seqs, num_q_heads, num_kv_heads));
  p.v = static_cast<const uint16_t*>(v);
  p.v_stride = v_stride;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = status_dev;
  p.n_rows = n_rows;
  p.n_seqs = n_seqs;
  p.Hq = num_q_heads;
  p.G = num_q_heads / num_kv_heads;
  p.tile_rows = two_heads(num_q_heads, num_kv_heads) ? pa::kPrTile : 2 * pa::kPrTile;
  // rows whose keys and values fill a group's share of L2, at most kPrGroups groups
  const int64_t share = pa::kPrGroupBytes / (4 * kv_row);
  p.group_rows = static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>({share, (static_cast<int64_t>(n_rows) + pa::kPrGroups - 1) / pa::kPrGroups, 1}), 0x7fffffff));
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634073599246810018921);
  p.wait_limit = pa::wait_limit();
  p.debug_stall = pa::debug_stall();
  struct { CUtensorMap* map; const void* base; int64_t stride; int32_t heads; } maps[3] = {
      {&p.qmap, q, q_stride, num_q_heads}, {&p.kmap, k, k_stride, num_kv_heads}, {&p.vmap, v, v_stride, num_kv_heads}};
  for (auto& m : maps) {
    const int64_t dims[3] = {head_dim, m.heads, n_rows}, strides[3] = {1, head_dim, m.stride};
    const uint32_t box[3] = {64, 1, static_cast<uint32_t>(pa::kPrTile)};
    st = pa::encode_map_16bit(m.map, m.base, 3, dims, strides, box);
    if (st != PA_OK) return st;
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "prompt attention");
  const int64_t units = most_tiles(n_rows, n_seqs, num_q_heads, num_kv_heads) * (p.tile_rows == pa::kPrTile ? num_q_heads / 2 : num_q_heads);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(sms, units));
  // A CTA for each unit needs no list: its warp finds the unit among up to 32 sequences.
  p.listed = units > sms || n_seqs > 32;
  e = head_dim == 128 ? pa::launch_prompt<128>(p, grid, static_cast<cudaStream_t>(stream))
                      : pa::launch_prompt<64>(p, grid, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "prompt attention launch");
}

}  // extern "C"
