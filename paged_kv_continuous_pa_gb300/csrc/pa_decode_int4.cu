// pa_decode_int4.cu -- attention over 4-bit K/V pools: value(c) = step * c + low with a
// (step, low) pair per token and kv head.
//
// One CTA per (row, split, kv head), as over the other pools; its warps take the split's
// 32-token stages in turn, each through a ring of its own of bulk copies, and are merged
// at the end in a fixed order.  The ranges never touch the products' inner loops:
//   q . K[t]  = step_t (q . c_t) + low_t sum(q)
//   sum_t p_t V[t] = sum_t (p_t step_t) c_t + sum_t p_t low_t
// so codes go into the tensor cores as they are.  A code becomes a bf16 number by placing its bits in
// the mantissa of 16.0 (0x4180 | c << 3 is 16 + c): a shift and one logic operation for two
// codes.  For K the 16 stays, and 16 step sum(q) is subtracted from the score; for V, whose
// sums run over thousands of tokens and cancel, 24 is subtracted first (c - 8, exact), and
// sum p (low + 8 step) is added: the accumulators then hold no offset larger than the result.
//
// m16n8k16 products, bf16 operands, FP32 sums.  The 16 rows are the kv head's G <= 8 query
// heads twice: rows g + 8 carry what rows g lack.  Scores of f32 queries: rows g the upper, rows
// g + 8 the middle eight bits, and a second product for the lower ones.  Weights: w = p step as
// bf16 and, in rows g + 8, the bf16 of the rest (16 bits in all).
//   B of scores (K): lane 4 n + c holds words 4c.. of token n's row, so the k index of an MMA is a
//   permutation of head elements, the same one in A (the queries, prepared once).
//   B of outputs (V): lane 4 n + c holds words of tokens 2c, 2c + 1, 2c + 8, 2c + 9; byte permutes pair
//   two tokens' codes, and n is a permutation of head elements undone at the end.
//
// What bounds it: the read of D + 8 bytes per token and kv head at HBM rate, with the
// conversions close behind (about 270 warp instructions for 16 tokens at D = 128, where
// HBM brings them in 90 clocks).
#include "pa_decode_mma.cuh"

namespace pa {

constexpr int kI4Warps = 4;
constexpr int kI4Stages = 4;   // ring slots of a warp
constexpr int kI4Tokens = 32;  // tokens of a stage

template <int D>
struct I4Geom {
  static constexpr int ROW = D / 2;                      // bytes of a token's codes
  static constexpr int K = 0, V = kI4Tokens * ROW;       // offsets in a stage
  static constexpr int KR = 2 * kI4Tokens * ROW, VR = KR + kI4Tokens * 4;
  static constexpr int STAGE = VR + kI4Tokens * 4;
  static constexpr int NW = D / 64;                      // 32-bit words of V to a lane and token
  static constexpr size_t RING = static_cast<size_t>(kI4Warps) * kI4Stages * STAGE;
};

struct I4Header {
  uint64_t full[kI4Warps][kI4Stages];
  uint64_t stall;              // never completed: the injected-stall test waits here
  int32_t bad;                 // a page id was out of range or a wait gave up
  int32_t last;                // this CTA merges the splits of its (row, kv head)
  int32_t pid[kMaxUnitPages];
};

template <int D>
__host__ __device__ constexpr size_t i4_smem() {
  return (sizeof(I4Header) + 127) / 128 * 128 + I4Geom<D>::RING;
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes s and s + 4 of a word (or code s of two tokens' halves) as bf16 16 + c.
template <int S>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t moved = S == 0 ? w << 3 : w >> (4 * S - 3);
  return (moved & 0x00780078u) | 0x41804180u;
}

__device__ __forceinline__ uint32_t minus24(uint32_t x) {  // 16 + c -> c - 8, exact
  const uint32_t c = 0xc1c0c1c0u;  // bf16 -24, twice
  const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float2 range_of(uint32_t w) {  // (step, low)
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ float bf16_round(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// Stage n of a warp (tokens t0 .. of the unit's pages) into its ring slot: pieces of 32 tokens or
// of one page; pages behind the unit's last are left out (their slots are masked).
template <int D>
__device__ __forceinline__ void i4_issue(const AttnParams& p, const I4Header* hdr, unsigned char* st, uint64_t* bar, int t0,
                                         int j0, int npg, int h, int lg_p) {
  using Geo = I4Geom<D>;
  const int P = 1 << lg_p, piece = min(P, kI4Tokens);
  const uint64_t policy = l2_policy_evict_first();
  int pieces = 0;
  for (int i = 0; i < kI4Tokens / piece; ++i) pieces += ((t0 + i * piece) >> lg_p) - j0 < npg ? 1 : 0;
  mbar_arrive_expect_tx(bar, static_cast<uint32_t>(pieces * piece * (2 * Geo::ROW + 8)));
  for (int i = 0; i < pieces; ++i) {
    const int t = t0 + i * piece;
    const int64_t token = (static_cast<int64_t>(hdr->pid[(t >> lg_p) - j0]) * p.Hkv + h) * P + (t & (P - 1));
    const int at = i * piece;
    bulk_g2s(st + Geo::K + at * Geo::ROW, static_cast<const unsigned char*>(p.k_pool) + token * Geo::ROW, piece * Geo::ROW, bar, policy);
    bulk_g2s(st + Geo::KR + at * 4, static_cast<const unsigned char*>(p.k_ranges) + token * 4, piece * 4, bar, policy);
    bulk_g2s(st + Geo::V + at * Geo::ROW, static_cast<const unsigned char*>(p.v_pool) + token * Geo::ROW, piece * Geo::ROW, bar, policy);
    bulk_g2s(st + Geo::VR + at * 4, static_cast<const unsigned char*>(p.v_ranges) + token * 4, piece * 4, bar, policy);
  }
}

template <int D, bool QF32>
struct I4State {
  uint32_t qa[D / 16][QF32 ? 4 : 2];  // A of scores: (row g, row g + 8) x k halves; bf16 queries leave rows g + 8 zero
  uint32_t ql[QF32 ? D / 16 : 1][2];  // the lower part of f32 queries
  float qsum;                         // sum of the row's query
  float m, l;                         // running reference (log2 domain) and this lane's part of the sum
  float fix;                          // this lane's part of sum p (low + 8 step)
  float o[I4Geom<D>::NW][8][4];
};

// One stage: scores of 32 tokens, the softmax update, the outputs.
template <int D, bool QF32>
__device__ __forceinline__ void i4_stage(I4State<D, QF32>& st, const unsigned char* sm, int n_valid, float scale, int lane) {
  using Geo = I4Geom<D>;
  const int g = lane >> 2, c = lane & 3;
  float s[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
    uint32_t w[D / 32];
    const unsigned char* row = sm + Geo::K + (8 * u + g) * Geo::ROW;
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * c);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(row + 8 * c);
      w[0] = x.x; w[1] = x.y;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t b[4] = {codes_bf16<0>(w[i]), codes_bf16<1>(w[i]), codes_bf16<2>(w[i]), codes_bf16<3>(w[i])};
#pragma unroll
      for (int sp = 0; sp < 2; ++sp) {
        const int k = 2 * i + sp;
        if constexpr (QF32) {
          mma_bf16_16816(s[u], st.qa[k], b[2 * sp], b[2 * sp + 1]);
          const uint32_t lo[4] = {st.ql[k][0], 0u, st.ql[k][1], 0u};
          mma_bf16_16816(s[u], lo, b[2 * sp], b[2 * sp + 1]);
        } else {
          const uint32_t a[4] = {st.qa[k][0], 0u, st.qa[k][1], 0u};
          mma_bf16_16816(s[u], a, b[2 * sp], b[2 * sp + 1]);
        }
      }
    }
  }
  // scores in the log2 domain, tokens 8u + 2c + i
  float mx = -INFINITY;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint2 rw = *reinterpret_cast<const uint2*>(sm + Geo::KR + (8 * u + 2 * c) * 4);
    const float2 r0 = range_of(rw.x), r1 = range_of(rw.y);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float step = i == 0 ? r0.x : r1.x, low = i == 0 ? r0.y : r1.y;
      const float dot = QF32 ? s[u][i] + s[u][2 + i] : s[u][i];
      const float x = fmaf(step, dot, fmaf(-16.0f, step, low) * st.qsum) * scale;
      s[u][i] = 8 * u + 2 * c + i < n_valid ? x : -INFINITY;
      mx = fmaxf(mx, s[u][i]);
    }
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  // the reference moves only when a score passes it by kRescaleSlack (weights stay below 2^8)
  const bool move = mx - st.m > kRescaleSlack;
  if (__any_sync(0xffffffffu, move)) {
    const float f = move ? ex2(st.m - mx) : 1.0f;  // (the first time: 2^-inf)
    if (move) st.m = mx;
    st.l *= f;
    st.fix *= f;
#pragma unroll
    for (int i = 0; i < Geo::NW; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        st.o[i][j][0] *= f;
        st.o[i][j][1] *= f;
        st.o[i][j][2] *= f;
        st.o[i][j][3] *= f;
      }
  }
  const float m = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
  for (int half = 0; half < 2; ++half) {  // 16 tokens each
    uint32_t a[4];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int u = 2 * half + v;
      const uint2 rw = *reinterpret_cast<const uint2*>(sm + Geo::VR + (8 * u + 2 * c) * 4);
      const float2 r0 = range_of(rw.x), r1 = range_of(rw.y);
      float w[2], rest[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float step = i == 0 ? r0.x : r1.x, low = i == 0 ? r0.y : r1.y;
        const bool valid = 8 * u + 2 * c + i < n_valid;
        const float e = ex2(s[u][i] - m);
        st.l += e;
        st.fix = valid ? fmaf(e, fmaf(8.0f, step, low), st.fix) : st.fix;  // (ranges of unused slots may be anything)
        const float x = valid ? e * step : 0.0f;
        w[i] = x;
        rest[i] = x - bf16_round(x);
      }
      a[2 * v] = pack_bf16x2(w[0], w[1]);
      a[2 * v + 1] = pack_bf16x2(rest[0], rest[1]);
    }
    uint32_t x[4][Geo::NW];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9 of the 16
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const unsigned char* row = sm + Geo::V + (16 * half + 2 * c + (t & 1) + 8 * (t >> 1)) * Geo::ROW;
      if constexpr (D == 128) {
        const uint2 y = *reinterpret_cast<const uint2*>(row + 8 * g);
        x[t][0] = y.x;
        x[t][1] = y.y;
      } else {
        x[t][0] = *reinterpret_cast<const uint32_t*>(row + 4 * g);
      }
    }
#pragma unroll
    for (int i = 0; i < Geo::NW; ++i) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // codes 4q .. 4q + 3 of the word
        const uint32_t z0 = __byte_perm(x[0][i], x[1][i], q == 0 ? 0x5410 : 0x7632);
        const uint32_t z1 = __byte_perm(x[2][i], x[3][i], q == 0 ? 0x5410 : 0x7632);
        mma_bf16_16816(st.o[i][4 * q + 0], a, minus24(codes_bf16<0>(z0)), minus24(codes_bf16<0>(z1)));
        mma_bf16_16816(st.o[i][4 * q + 1], a, minus24(codes_bf16<1>(z0)), minus24(codes_bf16<1>(z1)));
        mma_bf16_16816(st.o[i][4 * q + 2], a, minus24(codes_bf16<2>(z0)), minus24(codes_bf16<2>(z1)));
        mma_bf16_16816(st.o[i][4 * q + 3], a, minus24(codes_bf16<3>(z0)), minus24(codes_bf16<3>(z1)));
      }
    }
  }
}

template <int D, bool QF32>
__global__ void __launch_bounds__(32 * kI4Warps, 3) decode_int4_kernel(const __grid_constant__ AttnParams p) {
  using Geo = I4Geom<D>;
  constexpr int THREADS = 32 * kI4Warps;
  extern __shared__ __align__(128) unsigned char smem[];
  I4Header* hdr = reinterpret_cast<I4Header*>(smem);
  unsigned char* rings = smem + (sizeof(I4Header) + 127) / 128 * 128;

  const int unit = static_cast<int>(blockIdx.x);
  const int h = unit % p.Hkv;
  const int rest = unit / p.Hkv;
  const int split = rest % p.max_splits;
  const int row = unit_row(p, rest / p.max_splits);
  if (row >= p.n_rows) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int G = p.Hq / p.Hkv;
  const size_t out_row = static_cast<size_t>(row) * p.Hq + static_cast<size_t>(h) * G;
  const bool q_bf16 = p.q_is_bf16 != 0;
  const int seq = __ldg(p.seq_ids + row), pos = __ldg(p.positions + row), P = p.P;
  if (seq < 0 || seq >= p.num_seqs || pos < 0 || pos >= static_cast<long long>(p.max_blocks) * P) {
    if (split == 0) {
      for (int i = tid; i < G * D; i += THREADS) store_out(p.out, q_bf16, out_row * D + i, 0.0f);
      if (tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
    }
    return;
  }
  const int L = pos + 1, nsplit = (L - 1) / p.split_tokens + 1;
  if (split >= nsplit) return;
  const int t_begin = split * p.split_tokens, t_end = min(L, t_begin + p.split_tokens);
  const int lg_p = 31 - __clz(P);
  const int j0 = t_begin >> lg_p, npg = ((t_end - 1) >> lg_p) + 1 - j0;
  const int nstage = (t_end - t_begin + kI4Tokens - 1) / kI4Tokens;

  if (tid == 0) {
    for (int w = 0; w < kI4Warps; ++w)
      for (int s = 0; s < kI4Stages; ++s) mbar_init(&hdr->full[w][s], 1);
    mbar_init(&hdr->stall, 1);
    hdr->bad = 0;
    hdr->last = 0;
    fence_barrier_init();
  }
  bool bad_page = false;
  for (int i = tid; i < npg && i < kMaxUnitPages; i += THREADS) {
    const int pid = __ldg(p.block_tables + static_cast<size_t>(seq) * p.max_blocks + j0 + i);
    bad_page |= pid < 0 || pid >= p.num_pages;
    hdr->pid[i] = pid;
  }
  bool bad = __syncthreads_or(bad_page) != 0;
  if (bad && tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
  griddep_wait();  // the rows that a preceding append stores

  // warp w takes stages w, w + kI4Warps, ..
  unsigned char* ring = rings + static_cast<size_t>(warp) * kI4Stages * Geo::STAGE;
  const int mine = bad || warp >= nstage ? 0 : (nstage - warp + kI4Warps - 1) / kI4Warps;
  auto issue = [&](int n) {
    i4_issue<D>(p, hdr, ring + (n % kI4Stages) * Geo::STAGE, &hdr->full[warp][n % kI4Stages],
                t_begin + (warp + n * kI4Warps) * kI4Tokens, j0, npg, h, lg_p);
  };
  if (lane == 0)
    for (int n = 0; n < min(mine, kI4Stages); ++n) issue(n);

  I4State<D, QF32> st;
  st.m = -INFINITY;
  st.l = st.fix = st.qsum = 0.0f;
#pragma unroll
  for (int i = 0; i < Geo::NW; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) st.o[i][j][0] = st.o[i][j][1] = st.o[i][j][2] = st.o[i][j][3] = 0.0f;
  {
    // k-step (word i, sp) of lane c: elements e + 2 sp + {0, 4} and e + 2 sp + 1 + {0, 4}, e = (D / 4) c + 8 i
    const size_t base = (out_row + (g < G ? g : 0)) * D + (D / 4) * c;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q[j] = g < G ? load_q(p.q, !QF32, base + 8 * i + j) : 0.0f;
        st.qsum += q[j];
      }
#pragma unroll
      for (int sp = 0; sp < 2; ++sp)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float x = q[2 * sp + hf], y = q[2 * sp + hf + 4];
          if constexpr (QF32) {
            const float x1 = x - bf16_round(x), y1 = y - bf16_round(y);
            const float x2 = x1 - bf16_round(x1), y2 = y1 - bf16_round(y1);
            st.qa[2 * i + sp][2 * hf] = pack_bf16x2(x, y);
            st.qa[2 * i + sp][2 * hf + 1] = pack_bf16x2(x1, y1);
            st.ql[2 * i + sp][hf] = pack_bf16x2(x2, y2);
          } else {
            st.qa[2 * i + sp][hf] = pack_bf16x2(x, y);
          }
        }
    }
    st.qsum += __shfl_xor_sync(0xffffffffu, st.qsum, 1);
    st.qsum += __shfl_xor_sync(0xffffffffu, st.qsum, 2);
  }

  int gave_up = -1;
  for (int n = 0; n < mine; ++n) {
    const int s = n % kI4Stages;
    bool got = mbar_wait(&hdr->full[warp][s], (n / kI4Stages) & 1, p.wait_limit);
    if (p.debug_stall) got = got && mbar_wait(&hdr->stall, 0, p.wait_limit);  // runs out by construction
    if (!__all_sync(0xffffffffu, got)) {
      gave_up = n;
      if (lane == 0) {
        record_error(p.status, ST_TIMEOUT);
        hdr->bad = 1;
      }
      break;
    }
    const int t0 = t_begin + (warp + n * kI4Warps) * kI4Tokens;
    i4_stage<D, QF32>(st, ring + s * Geo::STAGE, min(kI4Tokens, t_end - t0), p.qk_scale_log2_h[0], lane);
    __syncwarp();
    if (lane == 0 && n + kI4Stages < mine) {
      fence_proxy_async();
      issue(n + kI4Stages);
    }
  }
  if (gave_up >= 0 && lane == 0)  // copies in flight land before the ring is used again
    for (int n = gave_up; n < min(gave_up + kI4Stages, mine); ++n)
      mbar_wait(&hdr->full[warp][n % kI4Stages], (n / kI4Stages) & 1, kDrainWaitLimit);

  // the lanes' parts of a row's sums, then the warps' states in shared memory
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    st.l += __shfl_xor_sync(0xffffffffu, st.l, d);
    st.fix += __shfl_xor_sync(0xffffffffu, st.fix, d);
  }
  __syncthreads();  // every ring is read
  bad = bad || hdr->bad != 0;
  float* acc = reinterpret_cast<float*>(rings);    // [warps][G][D]
  float* ml = acc + kI4Warps * G * D;              // [warps][G][2]
  if (g < G) {
#pragma unroll
    for (int i = 0; i < Geo::NW; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k)  // accumulator column 2c + k: word (D / 64)(2c + k) + i of the row
          acc[(warp * G + g) * D + 8 * (Geo::NW * (2 * c + k) + i) + j] = st.o[i][j][k] + st.o[i][j][2 + k] + st.fix;
    if (c == 0) {
      ml[(warp * G + g) * 2] = st.m;
      ml[(warp * G + g) * 2 + 1] = st.l;
    }
  }
  __syncthreads();
  const int ring_bytes = static_cast<int>(Geo::RING);
#define PA_FINISH(GG)                                                                                                \
  case GG:                                                                                                           \
    decode_finish<D, GG, KV_F32, kI4Warps, THREADS>(p, bad, &hdr->last, acc, ml, out_row, row, h, split, nsplit, q_bf16, \
                                                    ring_bytes);                                                    \
    break;
  switch (G) {
    PA_FINISH(1)
    PA_FINISH(2)
    PA_FINISH(3)
    PA_FINISH(4)
    PA_FINISH(5)
    PA_FINISH(6)
    PA_FINISH(7)
    PA_FINISH(8)
  }
#undef PA_FINISH
}

template <int D, bool QF32>
cudaError_t launch_int4_inst(const AttnParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t ea = allow_dynamic_smem(decode_int4_kernel<D, QF32>, done, i4_smem<D>());
  if (ea != cudaSuccess) return ea;
  const long long units = static_cast<long long>(p.n_unit_rows) * p.max_splits * p.Hkv;
  if (units <= 0) return cudaSuccess;
  if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const cudaError_t e = launch_kernel(decode_int4_kernel<D, QF32>, dim3(static_cast<unsigned>(units)),
                                      dim3(32 * kI4Warps), i4_smem<D>(), stream, p.dependent != 0, p);
  count_launch();
  return e;
}

cudaError_t launch_decode_int4(const AttnParams& p, cudaStream_t stream) {
  if (p.D == 128) return p.q_is_bf16 ? launch_int4_inst<128, false>(p, stream) : launch_int4_inst<128, true>(p, stream);
  if (p.D == 64) return p.q_is_bf16 ? launch_int4_inst<64, false>(p, stream) : launch_int4_inst<64, true>(p, stream);
  return cudaErrorNotSupported;
}

}  // namespace pa
