// pa_decode_int4.cu -- attention over 4-bit K/V pools: value(c) = step * c + low with a
// (step, low) pair per token and kv head.
//
// One CTA per (row, split, kv head), as over the other pools; its warps take the split's
// 32-token stages in turn, each through a ring of its own of 16-byte asynchronous copies (bulk copies take
// their addresses from uniform registers, so eight small ones cost a warp 80 instructions a stage, these 25), and
// are merged at the end in a fixed order.  The ranges never touch the products' inner loops:
//   q . K[t]  = step_t (q . c_t) + low_t sum(q)
//   sum_t p_t V[t] = sum_t (p_t step_t) (c_t - 8) + sum_t p_t (low_t + 8 step_t)
//
// A code needs no conversion: the f16 number with the bits 0x000c is c 2^-24, 0x00c0 is c 2^-20 (subnormal
// numbers run on into the first normal ones), and the tensor cores take them at full rate.  So one shift and four
// masks turn a word into the operands of eight codes; the powers of two go into the queries and the result.
//   scores: S^T = K Q^T, m16n8k16, A = 16 tokens, B = the kv head's G <= 8 query heads.  Lane 4 g + c holds
//     words 4c.. of tokens g and g + 8; the k index is a permutation of head elements, the same one in B.
//   outputs: O^T += V^T P^T, A = 16 head elements x 16 tokens from words of tokens 2c, 2c + 1, 2c + 8, 2c + 9
//     (a byte permute pairs two tokens), B = the weights, moved into fragment order with movmatrix.
// Queries are f16, a row scaled by a power of two below 2^15 (bf16 numbers are exact down to 2^-27 of the row's
// largest); f32 queries in two parts (22 bits).  A weight w = p step is f16 relative to a running
// reference, w = 2^(s - R) step <= 2^8, in one part for bf16 outputs (2^-11) and two for f32 ones (2^-22).  The
// weights' sum as the products saw them comes out of a tile of ones, so that the 8 is subtracted as it entered.
// f32 rows take c - 8 as a normal number, one operation more for two codes, for K too (its offset is low + 8 step
// then): the tensor cores' sums were cut off at 2^-18 or so of their largest product with subnormal operands, and sums of c
// are 15 to 20 times as large as the results of 53 keys: 1.5e-5 of the results' norm so, 5e-6 with c - 8 as a subnormal
// number, 3e-7 now.  bf16 rows' outputs are rounded at 2^-8, beside which 2^-18 does not show, not in scores whose two
// terms are large and opposite either: with queries of size 1 beside a common offset of 256 results are off by
// what their rounding makes, to within half a percent.
// (m16n8k32 on e4m3 bytes, where c is c 2^-9 as well, would need fewer operations, but ran as two f16
// products and the conversions, 963 warp instructions for a stage.)
//
// What bounds it: the read of D + 8 bytes per token and kv head at HBM rate; next are the logic
// operations (about 200 of a warp for 32 tokens at D = 128, two to a clock, where HBM takes 186 clocks).
// Measured at D = 128 and 8 kv heads, bf16 queries: 370 us for 64 rows of 30000 to 32768 tokens with 32 query heads (2.19 GB:
// 322 us at the copy rate), 137 us for 512 rows of 64 to 2662 with 16 (763 MB: 112 us); issue slots 60% busy, which
// with 16 warps to an SM (128 registers) and their waits for their own results is near what they hide.
#include "pa_decode_mma.cuh"

namespace pa {

constexpr int kI4Warps = 4;
constexpr int kI4Stages = 3;   // ring slots of a warp
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
  uint64_t stall;              // never completed: the injected-stall test waits here
  int32_t bad;                 // a page id was out of range or a wait gave up
  int32_t last;                // this CTA merges the splits of its (row, kv head)
  uint32_t place[kMaxUnitPages];  // of the unit's pages: (page Hkv + h) P / 16
};

template <int D>
__host__ __device__ constexpr size_t i4_smem() {
  return (sizeof(I4Header) + 127) / 128 * 128 + I4Geom<D>::RING;
}

__device__ __forceinline__ float2 range_of(uint32_t w) {  // (step, low)
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ void copy16(uint32_t dst_smem, const unsigned char* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst_smem), "l"(src) : "memory");
}

// Tokens t0 .. t0 + 31 of a unit into the stage at `st`, in halves of 16 (which lie in one page); halves in pages
// behind the unit's last are left out (their slots are masked).  One group of copies to a call.
template <int D>
__device__ __forceinline__ void i4_issue(const AttnParams& p, const I4Header* hdr, uint32_t st, int t0, int j0, int npg, int lg_p,
                                         int lane) {
  using Geo = I4Geom<D>;
  constexpr int CHUNKS = Geo::ROW / 16, ROWS = 32 / CHUNKS;  // of a token; tokens that one instruction copies
  const int mask = (1 << lg_p) - 1;
  const uint32_t own = static_cast<uint32_t>(lane) * 16u;  // rows of a page follow one another
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = t0 + 16 * h, page = (t >> lg_p) - j0;
    if (page < npg) {
      const uint64_t at = static_cast<uint64_t>(hdr->place[page]) * (16u * Geo::ROW) + (static_cast<uint32_t>(t & mask) * Geo::ROW + own);
      const unsigned char* k = static_cast<const unsigned char*>(p.k_pool) + at;
      const unsigned char* v = static_cast<const unsigned char*>(p.v_pool) + at;
#pragma unroll
      for (int i = 0; i < 16 / ROWS; ++i) {
        copy16(st + Geo::K + (16 * h + i * ROWS) * Geo::ROW + own, k + i * ROWS * Geo::ROW);
        copy16(st + Geo::V + (16 * h + i * ROWS) * Geo::ROW + own, v + i * ROWS * Geo::ROW);
      }
    }
  }
  // ranges: lanes 0-3, 4-7 those of K and V of the first half, 8-11, 12-15 of the second
  const int t = t0 + 16 * ((lane >> 3) & 1), page = (t >> lg_p) - j0;
  if (lane < 16 && page < npg) {
    const unsigned char* base = static_cast<const unsigned char*>((lane & 4) ? p.v_ranges : p.k_ranges);
    const uint64_t at = static_cast<uint64_t>(hdr->place[page]) * 64u + (static_cast<uint32_t>(t & mask) * 4u + (lane & 3) * 16u);
    copy16(st + ((lane & 4) ? Geo::VR : Geo::KR) + (lane >> 3) * 64 + (lane & 3) * 16, base + at);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Codes 2 s and 2 s + 1 (s = 0, 1) of both halves of a word as f16: c 2^-24 and c 2^-20, or, where CENTRED, the normal
// numbers c - 8 and 16 (c - 8), from 1024 + c and 1024 + 16 c (all exact).
template <int S, bool CENTRED>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t x = S == 0 ? w : w >> 8;
  if constexpr (CENTRED) {
    even = sub_f16x2((x & 0x000f000fu) | 0x64006400u, 0x64086408u);
    odd = sub_f16x2((x & 0x00f000f0u) | 0x64006400u, 0x64806480u);
  } else {
    even = x & 0x000f000fu;
    odd = x & 0x00f000f0u;
  }
}

template <int D, bool QF32>
struct I4State {
  static constexpr int PARTS = QF32 ? 2 : 1;
  uint32_t q[PARTS][D / 16][2];       // B of scores: head g
  // of heads 2c, 2c + 1: a score is (step sum + low q_sum) scale (log2 domain), where sum and q_sum are of the scaled
  // query, so that nothing before the last product leaves the finite numbers
  float q_sum[2], scale[2];
  float r[2], l[2], fix[2];           // reference; this lane's parts of sum p and sum p (low + 8 step)
  float o[I4Geom<D>::NW][4][4];       // head elements (2 to a lane's tile) x heads 2c, 2c + 1
  float ones[4];                      // the weights' sums (bf16 rows)
};

// Codes of 16 tokens times their weights into the results.  An MMA cuts its products off below the sum that it adds to;
// for f32 rows 16 tokens are summed apart and added with a rounding.
template <bool QF32>
__device__ __forceinline__ void i4_add(float (&o)[4], const uint32_t (&a)[4], const uint32_t (&b)[QF32 ? 2 : 1][4], int u) {
  if constexpr (QF32) {
    float t[4] = {};
#pragma unroll
    for (int part = 0; part < 2; ++part) mma_f16_16816(t, a, b[part][2 * u], b[part][2 * u + 1]);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] += t[k];
  } else {
    mma_f16_16816(o, a, b[0][2 * u], b[0][2 * u + 1]);
  }
}

constexpr float kI4Top = 8.0f, kI4Start = 6.0f;  // log2 of the largest weight: what it may reach, where the reference puts it

// One stage: scores of 32 tokens, the softmax update, the outputs.
template <int D, bool QF32, bool WHOLE>
__device__ __forceinline__ void i4_stage(I4State<D, QF32>& st, const unsigned char* sm, int n_valid, int lane) {
  using Geo = I4Geom<D>;
  constexpr int PARTS = I4State<D, QF32>::PARTS;
  const int g = lane >> 2, c = lane & 3;
  // e[i][k]: token 8 i + g, head 2c + k
  float e[4][2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {  // 16 tokens
    float s[2][4] = {};  // two sums, so that each product waits for the one before the last
    uint32_t w[2][D / 32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned char* row = sm + Geo::K + (16 * u + 8 * h + g) * Geo::ROW;
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * c);
        w[h][0] = x.x; w[h][1] = x.y; w[h][2] = x.z; w[h][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(row + 8 * c);
        w[h][0] = x.x; w[h][1] = x.y;
      }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t a[4];
      codes_f16<0, QF32>(w[0][i], a[0], a[2]);
      codes_f16<0, QF32>(w[1][i], a[1], a[3]);
#pragma unroll
      for (int part = 0; part < PARTS; ++part) mma_f16_16816(s[0], a, st.q[part][2 * i][0], st.q[part][2 * i][1]);
      codes_f16<1, QF32>(w[0][i], a[0], a[2]);
      codes_f16<1, QF32>(w[1][i], a[1], a[3]);
#pragma unroll
      for (int part = 0; part < PARTS; ++part) mma_f16_16816(s[1], a, st.q[part][2 * i + 1][0], st.q[part][2 * i + 1][1]);
    }
    e[2 * u][0] = s[0][0] + s[1][0];
    e[2 * u][1] = s[0][1] + s[1][1];
    e[2 * u + 1][0] = s[0][2] + s[1][2];
    e[2 * u + 1][1] = s[0][3] + s[1][3];
  }
  float2 v[4];
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t kw = *reinterpret_cast<const uint32_t*>(sm + Geo::KR + (8 * i + g) * 4);
    uint32_t vw = *reinterpret_cast<const uint32_t*>(sm + Geo::VR + (8 * i + g) * 4);
    const bool valid = WHOLE || 8 * i + g < n_valid;
    if (!valid) kw = vw = 0u;  // ranges of unused slots may be anything
    const float2 k = range_of(kw);
    v[i] = range_of(vw);
    float lg;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(fabsf(v[i].x) + 0x1p-24f));  // (rows of one value have step 0)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (codes count in 2^-24, those of f32 rows in 1 and less 8)
      const float x = QF32 ? fmaf(k.x, e[i][h], fmaf(8.0f, k.x, k.y) * st.q_sum[h])
                           : fmaf(k.x * 0x1p24f, e[i][h], k.y * st.q_sum[h]);
      e[i][h] = x * st.scale[h];
      if (!valid) e[i][h] = -INFINITY;
      top[h] = fmaxf(top[h], e[i][h] + lg);
    }
  }
  // the reference is the same in every lane of a head; it is looked at again only when a lane's weight passes the top
  if (__any_sync(0xffffffffu, top[0] - st.r[0] > kI4Top || top[1] - st.r[1] > kI4Top)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int d = 4; d < 32; d *= 2) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], d));
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool move = top[h] - st.r[h] > kI4Top;
      const float r = move ? top[h] - kI4Start : st.r[h];
      f[h] = move ? ex2(st.r[h] - r) : 1.0f;
      st.r[h] = r;
      st.l[h] *= f[h];
      st.fix[h] *= f[h];
      st.ones[h] *= f[h];
    }
#pragma unroll
    for (int i = 0; i < Geo::NW; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[i][j][k] *= f[k & 1];
  }
  // weights of token 8 i + g as (head 2c, head 2c + 1), transposed into (tokens 8 i + 2c, + 1) of head g
  uint32_t b[PARTS][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p0 = ex2(e[i][0] - st.r[0]), p1 = ex2(e[i][1] - st.r[1]);
    const float low8 = fmaf(8.0f, v[i].x, v[i].y);
    st.l[0] += p0;
    st.l[1] += p1;
    st.fix[0] = fmaf(p0, low8, st.fix[0]);
    st.fix[1] = fmaf(p1, low8, st.fix[1]);
    const float w0 = p0 * v[i].x, w1 = p1 * v[i].x;
    const uint32_t hi = pack_f16x2(w0, w1);
    b[0][i] = movmatrix_trans(hi);
    if constexpr (QF32) {
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      b[PARTS - 1][i] = movmatrix_trans(pack_f16x2(w0 - back.x, w1 - back.y));
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {  // 16 tokens
    uint32_t x[4][Geo::NW];      // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const unsigned char* row = sm + Geo::V + (16 * u + 2 * c + (t & 1) + 8 * (t >> 1)) * Geo::ROW;
      if constexpr (D == 128) {
        const uint2 y = *reinterpret_cast<const uint2*>(row + 8 * g);
        x[t][0] = y.x;
        x[t][1] = y.y;
      } else {
        x[t][0] = *reinterpret_cast<const uint32_t*>(row + 4 * g);
      }
    }
    const uint32_t one[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
    if constexpr (!QF32) mma_f16_16816(st.ones, one, b[0][2 * u], b[0][2 * u + 1]);
#pragma unroll
    for (int i = 0; i < Geo::NW; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // codes 4q .. 4q + 3 of the word
        const uint32_t z0 = __byte_perm(x[0][i], x[1][i], q == 0 ? 0x5410 : 0x7632);
        const uint32_t z1 = __byte_perm(x[2][i], x[3][i], q == 0 ? 0x5410 : 0x7632);
        uint32_t a[4];
        codes_f16<0, QF32>(z0, a[0], a[1]);
        codes_f16<0, QF32>(z1, a[2], a[3]);
        i4_add<QF32>(st.o[i][2 * q], a, b, u);
        codes_f16<1, QF32>(z0, a[0], a[1]);
        codes_f16<1, QF32>(z1, a[2], a[3]);
        i4_add<QF32>(st.o[i][2 * q + 1], a, b, u);
      }
  }
}

// The row's query (head g of the group; heads >= G are zero) as B operands, and the scores' factors.
template <int D, bool QF32>
__device__ __forceinline__ void i4_prep(const AttnParams& p, I4State<D, QF32>& st, size_t out_row, int G, int lane) {
  using Geo = I4Geom<D>;
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int i = 0; i < Geo::NW; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) st.o[i][j][0] = st.o[i][j][1] = st.o[i][j][2] = st.o[i][j][3] = 0.0f;
  st.ones[0] = st.ones[1] = st.ones[2] = st.ones[3] = 0.0f;
  float q[D / 4], big = 0.0f;
  bool finite = true;
  const size_t base = (out_row + (g < G ? g : 0)) * D + (D / 4) * c;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float x[8];
    load_q_vec<8>(p.q, !QF32, base + 8 * i, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[8 * i + j] = g < G ? x[j] : 0.0f;
      big = fmaxf(big, fabsf(q[8 * i + j]));
      finite = finite && fabsf(q[8 * i + j]) < INFINITY;
    }
  }
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
    finite = __shfl_xor_sync(0xffffffffu, static_cast<int>(finite), d) != 0 && finite;
  }
  // the largest element into [2^14, 2^15): times 2^(14 - its exponent), a normal number either way
  const int exponent = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100), 127);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - exponent) << 23);
  const float down = __uint_as_float(static_cast<uint32_t>(127 - 14 + exponent) << 23);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 4; ++i) sum = fmaf(q[i], up, sum);
#pragma unroll
  for (int d = 1; d < 4; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  // a query with an infinity or NaN makes its scores NaN
  const float scale = finite ? down * p.qk_scale_log2_h[0] : __uint_as_float(0x7fc00000u);
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // head h2 sits in lanes 4 h2 ..
    st.q_sum[h] = __shfl_sync(0xffffffffu, sum, 4 * (2 * c + h));
    st.scale[h] = __shfl_sync(0xffffffffu, scale, 4 * (2 * c + h));
    st.r[h] = -0x1.fffffep127f;  // (below every finite score, and finite itself, so that differences to it are numbers)
    st.l[h] = st.fix[h] = 0.0f;
  }
  // k-step 2 i + s: elements 2 s, 2 s + 4 and, as codes there count 16 times as much, a sixteenth of 2 s + 1, 2 s + 5
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        const float f = odd ? up * 0.0625f : up;
        const float x = q[8 * i + 2 * s + odd] * f, y = q[8 * i + 2 * s + odd + 4] * f;
        const uint32_t hi = pack_f16x2(x, y);
        st.q[0][2 * i + s][odd] = hi;
        if constexpr (QF32) {
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          st.q[1][2 * i + s][odd] = pack_f16x2(x - back.x, y - back.y);
        }
      }
}

template <int D, bool QF32>
__global__ void __launch_bounds__(32 * kI4Warps, QF32 ? 3 : 4) decode_int4_kernel(const __grid_constant__ AttnParams p) {
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
    mbar_init(&hdr->stall, 1);
    hdr->bad = 0;
    hdr->last = 0;
    fence_barrier_init();
  }
  bool bad_page = false;
  for (int i = tid; i < npg && i < kMaxUnitPages; i += THREADS) {
    const int pid = __ldg(p.block_tables + static_cast<size_t>(seq) * p.max_blocks + j0 + i);
    bad_page |= pid < 0 || pid >= p.num_pages;
    hdr->place[i] = static_cast<uint32_t>((static_cast<uint64_t>(pid) * p.Hkv + h) << (lg_p - 4));  // (32 bits: checked by the host)
  }
  bool bad = __syncthreads_or(bad_page) != 0;
  if (bad && tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
  griddep_wait();  // the rows that a preceding append stores

  // warp w takes stages w, w + kI4Warps, ..
  unsigned char* ring = rings + static_cast<size_t>(warp) * kI4Stages * Geo::STAGE;
  const int mine = bad || warp >= nstage ? 0 : (nstage - warp + kI4Warps - 1) / kI4Warps;
  const uint32_t ring_at = smem_addr(ring);
  auto issue = [&](int n) {
    if (n < mine)
      i4_issue<D>(p, hdr, ring_at + (n % kI4Stages) * Geo::STAGE, t_begin + (warp + n * kI4Warps) * kI4Tokens, j0, npg, lg_p, lane);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");  // (an empty group, so that one more is always newer)
  };
#pragma unroll 1
  for (int n = 0; n < kI4Stages; ++n) issue(n);

  I4State<D, QF32> st;
  i4_prep<D, QF32>(p, st, out_row, G, lane);

  if (p.debug_stall && !mbar_wait(&hdr->stall, 0, p.wait_limit)) {  // runs out by construction
    record_error(p.status, ST_TIMEOUT);
    hdr->bad = 1;
  }
#pragma unroll 1
  for (int n = 0; n < mine; ++n) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kI4Stages - 1) : "memory");
    __syncwarp();
    const unsigned char* stage = ring + (n % kI4Stages) * Geo::STAGE;
    const int left = t_end - (t_begin + (warp + n * kI4Warps) * kI4Tokens);
    if (left >= kI4Tokens)
      i4_stage<D, QF32, true>(st, stage, kI4Tokens, lane);
    else
      i4_stage<D, QF32, false>(st, stage, left, lane);
    __syncwarp();
    issue(n + kI4Stages);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // the lanes' parts of a row's sums, then the warps' states in shared memory
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {
      st.l[h] += __shfl_xor_sync(0xffffffffu, st.l[h], d);
      st.fix[h] += __shfl_xor_sync(0xffffffffu, st.fix[h], d);
    }
  __syncthreads();  // every ring is read
  bad = bad || hdr->bad != 0;
  float* acc = reinterpret_cast<float*>(rings);    // [warps][G][D]
  float* ml = acc + kI4Warps * G * D;              // [warps][G][2]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int head = 2 * c + h;
    if (head >= G) continue;
    const float offset = QF32 ? st.fix[h] : fmaf(-8.0f, st.ones[h], st.fix[h]);
    float* row = acc + (warp * G + head) * D + 8 * Geo::NW * g;
#pragma unroll
    for (int i = 0; i < Geo::NW; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // elements 2j (codes in 2^-24, or 1) and 2j + 1 (16 times that) of word i
        constexpr float even = QF32 ? 1.0f : 0x1p24f, odd = even * 0.0625f;
        const float2 two = make_float2(fmaf(even, st.o[i][j][h], offset), fmaf(odd, st.o[i][j][2 + h], offset));
        *reinterpret_cast<float2*>(row + 8 * i + 2 * j) = two;
      }
    if (g == 0) {
      ml[(warp * G + head) * 2] = st.r[h];
      ml[(warp * G + head) * 2 + 1] = st.l[h];
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
  if (units > 0x7fffffffLL || static_cast<long long>(p.num_pages) * p.Hkv * p.P / 16 > 0xffffffffLL) return cudaErrorInvalidConfiguration;
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
