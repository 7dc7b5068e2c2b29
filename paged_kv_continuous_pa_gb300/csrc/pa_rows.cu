// pa_rows.cu -- a step's rows on their way into the cache and back: rotary positions
// (pa_rope_rows, pa_rope_append), the append to 4-bit pools, and cached tokens as
// dense rows (pa_read_kv).
//
// A pair (a, b) at position p turns by the angle p f_i:
//   (a, b) -> m (a cos - b sin, a sin + b cos)
// The angle is taken in turns: f_i / 2 pi is a 64-bit fraction of a turn, so p f_i modulo
// whole turns is one wrapping integer product, off by 2^-33 of a turn at any position (an
// FP32 product is off by 0.06 rad at position 10^6); sincospi gets its upper 32 bits.  A row's
// sines and cosines are the same for all of its heads, so a CTA computes them once
// for its rows into shared memory.
//
// What bounds it is memory: every element is read and written once; and close behind it
// the instructions, so that what can be is worked out once for several rows.  A warp takes
// one head of a few neighbouring rows at a time: its kind (query, key, value) is the whole
// warp's.  D / 8 lanes share one row, 8 consecutive elements (one or two 16-byte accesses) to
// a lane; the partner octet of the half layout sits in another lane of the same group and comes
// by shuffle.  So a row of a head is in one place when it is rotated, which a 4-bit pool
// needs: its range is a reduction over the group.
//
// Measured: 128 us for 32768 rows of 32 query heads over 8, 64 of 128 elements rotated (806 MB: 119 us at the copy
// rate); 40 us for 16384 rows of 8 heads into a 4-bit pool (85 MB: 13 us), which takes 190 warp instructions for
// 256 elements, two thirds of the issue slots, and 31 us to read them back as f32 (151 MB: 22 us), whose warps wait for
// their row's page and then its codes.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

constexpr int kRowsThreads = 256;
constexpr int kRowsPerCta = 16;  // at a time, at most
constexpr int kRowsCtas = 3;     // to an SM

// 8 consecutive elements of one head, as loaded (plain loads: queries may be rotated in place)
template <bool BF16>
struct Octet {
  uint32_t w[BF16 ? 4 : 8];
};

template <bool BF16>
__device__ __forceinline__ Octet<BF16> load_octet(const void* base, int64_t element) {
  Octet<BF16> o;
  if constexpr (BF16) {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + element);
    o.w[0] = a.x; o.w[1] = a.y; o.w[2] = a.z; o.w[3] = a.w;
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + element);
    const uint4 a = s[0], b = s[1];
    o.w[0] = a.x; o.w[1] = a.y; o.w[2] = a.z; o.w[3] = a.w;
    o.w[4] = b.x; o.w[5] = b.y; o.w[6] = b.z; o.w[7] = b.w;
  }
  return o;
}

template <bool BF16>
__device__ __forceinline__ void widen(const Octet<BF16>& o, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (BF16)
      x[i] = (i & 1) ? bf16hi(o.w[i / 2]) : bf16lo(o.w[i / 2]);
    else
      x[i] = __uint_as_float(o.w[i]);
  }
}

__device__ __forceinline__ void store_f32(void* base, int64_t element, const float (&x)[8]) {
  float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + element);
  d[0] = make_float4(x[0], x[1], x[2], x[3]);
  d[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ void store_bf16(void* base, int64_t element, const float (&x)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + element) = make_uint4(o[0], o[1], o[2], o[3]);
}

// Largest and smallest of two or three numbers; NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two binary32 numbers at a time, each operation rounded once.
__device__ __forceinline__ uint64_t two_of(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void halves_of(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// STEPS tokens of one kv head into a 4-bit pool: L lanes hold 8 elements of each (token[s] < 0: nothing is stored).
// The codes are taken against the range as it is stored, so that a code is off by half a step at most (each
// conversion below rounds once, to nearest even).  The tokens' extremes are joined together: in each exchange a lane
// passes on half of what it holds, until it has one token's, whose range it works out; so all ranges take the
// instructions of one, and the tokens hide each other's latencies (40 us for 16384 rows of 8 heads, token by token 44).
// The format divides in binary32.  With y the rounded reciprocal of the step, one per token, d y corrected once by the
// exact remainder is the rounded quotient (Markstein's theorem: quotients here are below 32 and the
// remainder is a multiple of what binary32 holds): two multiply-adds in place of a division for each element.
template <int L, int STEPS>
__device__ __forceinline__ void store_int4(void* codes, void* ranges, const int64_t (&token)[STEPS], int l, float (&x)[STEPS][8]) {
  float hi[STEPS], down[STEPS];  // largest x and -x; NaN where there is one
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    float lo = min_nan(x[s][0], x[s][1], x[s][2]);
    hi[s] = max_nan(x[s][0], x[s][1], x[s][2]);
#pragma unroll
    for (int i = 3; i < 7; i += 2) {
      lo = min_nan(lo, x[s][i], x[s][i + 1]);
      hi[s] = max_nan(hi[s], x[s][i], x[s][i + 1]);
    }
    down[s] = -min_nan(lo, x[s][7], x[s][7]);
    hi[s] = max_nan(hi[s], x[s][7]);
  }
  auto trade = [&](float give, float keep, int d) { return max_nan(keep, __shfl_xor_sync(0xffffffffu, give, d)); };
  int own = 0, d = 1;  // the token whose extremes this lane ends up with
#pragma unroll
  for (int n = STEPS / 2; n >= 1; n /= 2, d *= 2) {
    const bool upper = (l & d) != 0;
    own += upper ? n : 0;
#pragma unroll
    for (int s = 0; s < n; ++s) {
      hi[s] = trade(upper ? hi[s] : hi[s + n], upper ? hi[s + n] : hi[s], d);
      down[s] = trade(upper ? down[s] : down[s + n], upper ? down[s + n] : down[s], d);
    }
  }
  const bool upper = (l & STEPS) != 0;
  float v = trade(upper ? down[0] : hi[0], upper ? hi[0] : down[0], STEPS);
#pragma unroll
  for (d = 2 * STEPS; d < L; d *= 2) v = trade(v, v, d);
  const float w = __shfl_xor_sync(0xffffffffu, v, STEPS);
  float top = upper ? v : w, bottom = -(upper ? w : v);
  const bool nan = top != top, far = !(top <= 65504.0f && bottom >= -65504.0f);  // the range is held in f16
  if (__any_sync(0xffffffffu, far)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[s][i] = fminf(fmaxf(x[s][i], -65504.0f), 65504.0f);
    top = fminf(fmaxf(top, -65504.0f), 65504.0f);
    bottom = fminf(fmaxf(bottom, -65504.0f), 65504.0f);
  }
  const __half low = __float2half_rn(bottom);
  // a fifteenth of the width, rounded once as below (what is too small for an exact remainder is 0 in f16)
  constexpr float fifteenth = 1.0f / 15.0f;
  const float lf = __half2float(low), width = __fsub_rn(top, lf), part = __fmul_rn(width, fifteenth);
  const __half step = __float2half_rn(fmaxf(fmaf(fmaf(-part, 15.0f, width), fifteenth, part), 0.0f));
  const float sf = __half2float(step);
  const uint32_t range = nan ? 0x7fff7fffu : static_cast<uint32_t>(__half_as_ushort(step)) | static_cast<uint32_t>(__half_as_ushort(low)) << 16;
  const float y = __frcp_rn(sf);
  // A step that is a normal f16 number is off by 2^-11 of it, and low by 2^-11 of low: quotients stay within -1/4
  // and 15 + 1/4 unless low is large beside the step.
  const bool loose = __any_sync(0xffffffffu, !(sf >= 0x1p-14f && fabsf(lf) <= 512.0f * sf));
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    int from = 0;  // a lane with token s
#pragma unroll
    for (int n = STEPS / 2, b = 1; n >= 1; n /= 2, b *= 2) from |= (s & n) ? b : 0;
    const uint32_t r = __shfl_sync(0xffffffffu, range, from, L);
    const float ys = __shfl_sync(0xffffffffu, y, from, L);
    const float2 pair = __half22float2(*reinterpret_cast<const __half2*>(&r));  // (step, low)
    float c[8];
    const uint64_t y2 = two_of(ys, ys), down2 = two_of(-pair.y, -pair.y), minus2 = two_of(-pair.x, -pair.x);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t e = add2(two_of(x[s][i], x[s][i + 1]), down2), q = mul2(e, y2);
      halves_of(fma2(fma2(q, minus2, e), y2, q), c[i], c[i + 1]);
    }
    if (loose) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(c[i], 0.0f), 15.0f);
    }
    // c + 1.5 2^23 rounds to the integer (ties to even) in the lowest bits; the rest goes below
    uint32_t word = 0, rest = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float a, b;
      halves_of(add2(two_of(c[i], c[i + 1]), two_of(12582912.0f, 12582912.0f)), a, b);
      word += (__float_as_uint(a) << (4 * i)) + (__float_as_uint(b) << (4 * i + 4));
      rest += (0x4b400000u << (4 * i)) + (0x4b400000u << (4 * i + 4));
    }
    if (token[s] >= 0) static_cast<uint32_t*>(codes)[token[s] * L + l] = pair.x > 0.0f ? word - rest : 0u;
  }
  int64_t mine = token[0];
#pragma unroll
  for (int s = 1; s < STEPS; ++s) mine = own == s ? token[s] : mine;
  if (l < STEPS && mine >= 0) static_cast<uint32_t*>(ranges)[mine] = range;
}

struct RowsSmem {  // of the rows at hand and of the next ones
  float2 turn[2][kRowsPerCta][64];  // (cos, sin) of the row's pairs
  int32_t page[2][kRowsPerCta];     // of the row's token (-1: a row that is skipped)
  int32_t slot[2][kRowsPerCta];
  float x[kRowsThreads * 8];        // heads whose partners do not sit in one lane
};

// A CTA goes through sets of rows, STEPS to each group of lanes (every gridDim.x-th set), and of their heads takes
// blockIdx.y, + gridDim.y, .. in turns of its warps.  The next set's angles and pages are looked up at the end of a set.
template <int D, bool BF16, int STEPS, bool INT4>
__global__ void __launch_bounds__(kRowsThreads, kRowsCtas) rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int L = D / 8, G = 32 / L, kRows = G * STEPS, kWarps = kRowsThreads / 32;
  static_assert(kRows <= kRowsPerCta, "rows of a CTA");
  __shared__ __align__(16) RowsSmem sm;
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % L, g = lane / L;
  const int64_t sets = (static_cast<int64_t>(p.n_rows) + kRows - 1) / kRows;
  const int H = p.Hq + 2 * p.Hkv, step = kWarps * gridDim.y, first = blockIdx.y * kWarps + warp;

  auto load = [&](int64_t set, int head, Octet<BF16> (&raw)[STEPS]) {
    if (head >= H || set >= sets) return;
    const int64_t row = set * kRows + g;
    const bool is_q = head < p.Hq, is_k = head < p.Hq + p.Hkv;
    const void* base = is_q ? p.q : is_k ? p.k : p.v;
    const int64_t stride = is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride;
    int64_t at = row * stride + (head - (is_q ? 0 : is_k ? p.Hq : p.Hq + p.Hkv)) * D + 8 * l;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (row + s * G < p.n_rows) raw[s] = load_octet<BF16>(base, at);
      at += G * stride;
    }
  };
  const int pairs = p.rot / 2;
  auto look_up = [&](int64_t set, int buf) {
    const int64_t row0 = set * kRows;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), p.n_rows - row0));
    if (p.Hkv > 0 && tid < rows) {
      const int seq = __ldg(p.seq_ids + row0 + tid), pos = __ldg(p.positions + row0 + tid);
      int page = -1;
      if (seq >= 0 && seq < p.num_seqs && pos >= 0 && pos < static_cast<int64_t>(p.max_blocks) * p.P)
        page = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks + pos / p.P);
      if (page < 0 || page >= p.num_pages) {
        page = -1;
        record_error(p.status, ST_OUT_OF_RANGE);
      }
      sm.page[buf][tid] = page;
      sm.slot[buf][tid] = pos & (p.P - 1);
    }
    for (int i = tid; i < rows * pairs; i += kRowsThreads) {
      const int r = i / pairs, j = i - r * pairs;
      const int64_t pos = __ldg(p.positions + row0 + r);
      const uint64_t phase = p.turns[j] * static_cast<uint64_t>(pos) + (1ull << 31);
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s, &c);
      sm.turn[buf][r][j] = make_float2(c * p.magnitude, s * p.magnitude * p.sign);
    }
  };
  // the first head is on its way while the angles are computed
  Octet<BF16> raw[STEPS] = {};
  load(blockIdx.x, first, raw);
  look_up(blockIdx.x, 0);
  __syncthreads();

  const bool half_octets = !p.interleaved && pairs % 8 == 0;
  const int o8 = pairs / 8;
  const int partner = lane - l + (l < o8 ? l + o8 : l < 2 * o8 ? l - o8 : l);
  int buf = 0;
  for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, buf ^= 1) {
    const int64_t row0 = set * kRows;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), p.n_rows - row0));
    for (int h = first; h < H; h += step) {  // the same head for every lane of a warp
      Octet<BF16> next[STEPS] = {};
      const bool last = h + step >= H;
      load(last ? set + gridDim.x : set, last ? first : h + step, next);
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv, turned = !is_v && p.rot > 0;
      const int kvh = h - p.Hq - (is_v ? p.Hkv : 0);
      void* pool = is_v ? p.v_pool : p.k_pool;
      // row s G + g of the set, rotated
      auto take = [&](int s, float (&x)[8]) {
        const int r = s * G + g;
        widen<BF16>(raw[s], x);
        if (turned && p.interleaved) {
          const float2* t = &sm.turn[buf][r][4 * l];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (8 * l + 2 * i >= p.rot) break;
            const float a = x[2 * i], c = x[2 * i + 1];
            x[2 * i] = a * t[i].x - c * t[i].y;
            x[2 * i + 1] = c * t[i].x + a * t[i].y;
          }
        } else if (turned && half_octets) {
          Octet<BF16> other;
#pragma unroll
          for (int i = 0; i < (BF16 ? 4 : 8); ++i) other.w[i] = __shfl_sync(0xffffffffu, raw[s].w[i], partner);
          if (l < 2 * o8) {
            float y[8];
            widen<BF16>(other, y);
            const float4* t = reinterpret_cast<const float4*>(&sm.turn[buf][r][l < o8 ? 8 * l : 8 * (l - o8)]);
            const float way = l < o8 ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 two = t[i];  // (cos, sin) of two pairs
              x[2 * i] = x[2 * i] * two.x + (way * y[2 * i]) * two.y;
              x[2 * i + 1] = x[2 * i + 1] * two.z + (way * y[2 * i + 1]) * two.w;
            }
          }
        } else if (turned) {  // partners across octets: the head through shared memory
          float* head = sm.x + (tid - l) * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) head[8 * l + i] = x[i];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = 8 * l + i;
            if (e >= p.rot) break;
            const float2 t = sm.turn[buf][r][e < pairs ? e : e - pairs];
            x[i] = e < pairs ? x[i] * t.x - head[e + pairs] * t.y : x[i] * t.x + head[e - pairs] * t.y;
          }
          __syncwarp();
        }
      };
      auto token_of = [&](int page, int r) { return (static_cast<int64_t>(page) * p.Hkv + kvh) * p.P + sm.slot[buf][r]; };
      if (INT4 && !is_q) {
        float x[STEPS][8];
        int64_t token[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          take(s, x[s]);
          const int r = s * G + g, page = r < rows ? sm.page[buf][r] : -1;
          token[s] = page < 0 ? -1 : token_of(page, r);
        }
        store_int4<L>(pool, is_v ? p.v_ranges : p.k_ranges, token, l, x);
      } else {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int r = s * G + g;
          float x[8];
          take(s, x);
          const int page = p.Hkv > 0 ? sm.page[buf][r] : 0;
          const bool stored = r < rows && page >= 0;
          if (stored && is_q) {
            const int64_t at = (row0 + r) * p.out_stride + h * D + 8 * l;
            if constexpr (BF16)
              store_bf16(p.q_out, at, x);
            else
              store_f32(p.q_out, at, x);
          } else if (stored) {
            const int64_t at = token_of(page, r) * D + 8 * l;
            if constexpr (INT4) {
            } else if (p.kv_dtype == KV_F32) {
              store_f32(pool, at, x);
            } else if (p.kv_dtype == KV_BF16) {
              if (BF16 && !turned)  // a copy, whatever the bits
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + at) =
                    make_uint4(raw[s].w[0], raw[s].w[1], raw[s].w[2], raw[s].w[3]);
              else
                store_bf16(pool, at, x);
            } else {
              const float scale = is_v ? p.v_scale_h[PA_HEAD(p, kvh)] : p.k_scale_h[PA_HEAD(p, kvh)];
              uint32_t o[2] = {0u, 0u};
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i / 4] |= encode_e4m3(x[i], scale) << (8 * (i % 4));
              *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at) = make_uint2(o[0], o[1]);
            }
          }
        }
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s) raw[s] = next[s];
    }
    if (set + gridDim.x < sets) look_up(set + gridDim.x, buf ^ 1);
    __syncthreads();
  }
}

// A warp per row and 16 bytes of output at a time to a lane (E elements), gridDim.y shares of a row.
template <int KV, bool BF16>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int E = BF16 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.n_rows) return;
  const int seq = __ldg(p.seq_ids + row), pos = __ldg(p.positions + row);
  int page = -1;
  if (seq >= 0 && seq < p.num_seqs && pos >= 0 && pos < static_cast<int64_t>(p.max_blocks) * p.P)
    page = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks + pos / p.P);
  if (page < 0 || page >= p.num_pages) {
    page = -1;
    if (lane == 0 && blockIdx.y == 0) record_error(p.status, ST_OUT_OF_RANGE);
  }
  const int lg_units = (p.D == 128 ? 7 : 6) - (BF16 ? 3 : 2), units = p.Hkv << lg_units;  // of a head; of a row's K or V
  const int64_t token0 = static_cast<int64_t>(page) * p.Hkv * p.P + (pos & (p.P - 1));
  for (int side = p.k_out == nullptr ? 1 : 0; side < (p.v_out == nullptr ? 1 : 2); ++side) {
    const void* pool = side ? p.v_pool : p.k_pool;
    const uint32_t* ranges = static_cast<const uint32_t*>(side ? p.v_ranges : p.k_ranges);
    void* out = side ? p.v_out : p.k_out;
#pragma unroll 4
    for (int o = blockIdx.y * 32 + lane; o < units; o += 32 * gridDim.y) {
      const int h = o >> lg_units;
      float x[E] = {};
      if (page >= 0) {
        const int64_t token = token0 + static_cast<int64_t>(h) * p.P;
        const int64_t at = (token << lg_units) + (o & ((1 << lg_units) - 1));  // in units
        if constexpr (KV == KV_INT4) {
          const uint32_t w = BF16 ? __ldg(static_cast<const uint32_t*>(pool) + at) : __ldg(static_cast<const uint16_t*>(pool) + at);
          const uint32_t range = __ldg(ranges + token);
          const float step = __half2float(__ushort_as_half(static_cast<unsigned short>(range & 0xffffu)));
          const float low = __half2float(__ushort_as_half(static_cast<unsigned short>(range >> 16)));
#pragma unroll
          for (int i = 0; i < E; ++i) x[i] = fmaf(static_cast<float>((w >> (4 * i)) & 15u), step, low);
        } else if constexpr (KV == KV_E4M3) {
          const float scale = side ? p.v_scale_h[PA_HEAD(p, h)] : p.k_scale_h[PA_HEAD(p, h)];
          const uint32_t* src = static_cast<const uint32_t*>(pool) + at * (E / 4);
#pragma unroll
          for (int i = 0; i < E / 4; ++i) {
            const uint32_t w = __ldg(src + i);
            const float2 a = e4m3x2_to_float2(w), b = e4m3x2_to_float2(w >> 16);
            x[4 * i] = a.x * scale;
            x[4 * i + 1] = a.y * scale;
            x[4 * i + 2] = b.x * scale;
            x[4 * i + 3] = b.y * scale;
          }
        } else if constexpr (KV == KV_BF16) {
          const uint2* src = static_cast<const uint2*>(pool) + at * (E / 4);
#pragma unroll
          for (int i = 0; i < E / 4; ++i) {
            const uint2 w = __ldg(src + i);
            x[4 * i] = bf16lo(w.x);
            x[4 * i + 1] = bf16hi(w.x);
            x[4 * i + 2] = bf16lo(w.y);
            x[4 * i + 3] = bf16hi(w.y);
          }
        } else {
          const float4* src = static_cast<const float4*>(pool) + at * (E / 4);
#pragma unroll
          for (int i = 0; i < E / 4; ++i) {
            const float4 w = __ldg(src + i);
            x[4 * i] = w.x;
            x[4 * i + 1] = w.y;
            x[4 * i + 2] = w.z;
            x[4 * i + 3] = w.w;
          }
        }
      }
      const int64_t to = row * units + o;
      if constexpr (BF16)
        store_bf16(out, to * 8, x);
      else
        static_cast<float4*>(out)[to] = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

template <int D, bool BF16, int STEPS, bool INT4>
cudaError_t launch_rows_inst(const RowsParams& p, cudaStream_t stream) {
  constexpr int kRows = 256 / D * STEPS;
  const int64_t sets = (static_cast<int64_t>(p.n_rows) + kRows - 1) / kRows, most = 152 * kRowsCtas;
  // few rows: their heads are shared out to as many CTAs as the GPU holds at once (each computes the angles)
  const int64_t turns = (p.Hq + 2 * p.Hkv + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  const int64_t share = std::max<int64_t>(1, std::min<int64_t>(turns, most / sets));
  rows_kernel<D, BF16, STEPS, INT4><<<dim3(static_cast<unsigned>(std::min(sets, most)), static_cast<unsigned>(share)), kRowsThreads, 0,
                                stream>>>(p);
  count_launch();
  return cudaGetLastError();
}

template <int D, bool BF16, bool INT4>
cudaError_t launch_rows_steps(const RowsParams& p, cudaStream_t stream) {
  // One step to a lane as long as that makes no more CTAs than the GPU holds at once: rotated and appended rows of
  // 16 heads over 8 take 3.1 us for 64 rows (4.7 with four steps), 5.5 for 608 (6.2); 1216 rows 9.7 (8.6), 8192 47.6 (38.8).
  return p.n_rows <= 152 * 2 * (256 / D) ? launch_rows_inst<D, BF16, 1, INT4>(p, stream)
                                         : launch_rows_inst<D, BF16, BF16 ? 4 : 2, INT4>(p, stream);
}

cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream) {
  if (p.n_rows <= 0) return cudaSuccess;
  const bool bf16 = p.in_dtype == KV_BF16;
  // (instances of their own for 4-bit pools: in one kernel with them the other types' rows have fewer registers, 151
  // instead of 128 us for 32768 rotated rows)
  if (p.kv_dtype == KV_INT4 && p.Hkv > 0) {
    if (p.D == 128) return bf16 ? launch_rows_steps<128, true, true>(p, stream) : launch_rows_steps<128, false, true>(p, stream);
    return bf16 ? launch_rows_steps<64, true, true>(p, stream) : launch_rows_steps<64, false, true>(p, stream);
  }
  if (p.D == 128) return bf16 ? launch_rows_steps<128, true, false>(p, stream) : launch_rows_steps<128, false, false>(p, stream);
  return bf16 ? launch_rows_steps<64, true, false>(p, stream) : launch_rows_steps<64, false, false>(p, stream);
}

cudaError_t launch_read(const ReadParams& p, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(p.n_rows) + 7) / 8;
  const int64_t turns = (static_cast<int64_t>(p.Hkv) * p.D / (p.out_bf16 ? 8 : 4) + 31) / 32;
  const int64_t share = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(turns, 64), 152 * 4 / blocks));
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(share));
  auto go = [&](auto kernel) { kernel<<<grid, 256, 0, stream>>>(p); };
  switch (p.kv_dtype) {
    case KV_F32: p.out_bf16 ? go(read_kernel<KV_F32, true>) : go(read_kernel<KV_F32, false>); break;
    case KV_BF16: p.out_bf16 ? go(read_kernel<KV_BF16, true>) : go(read_kernel<KV_BF16, false>); break;
    case KV_E4M3: p.out_bf16 ? go(read_kernel<KV_E4M3, true>) : go(read_kernel<KV_E4M3, false>); break;
    default: p.out_bf16 ? go(read_kernel<KV_INT4, true>) : go(read_kernel<KV_INT4, false>); break;
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace pa

using pa::aligned;
using pa::cuda_fail;
using pa::elt_bytes;
using pa::fail;

struct pa_rope {
  pa_rope_desc desc;
  double frequencies[64];
  double magnitude;
  uint64_t turns[64];
};

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kTwoPiRest = 2.4492935982947064e-16;  // 2 pi - kTwoPi

// f / 2 pi modulo whole turns, in 2^-64 of a turn.  A quotient in binary64 alone is off by 2^-54 of itself, which the
// position multiplies (2^-22 rad at 2^31 for f of 1, 0.01 for 10^5): what it leaves of f is divided, too.
uint64_t turns_of(double f) {
  const double q = f / kTwoPi;
  const double rest = (std::fma(-q, kTwoPi, f) - q * kTwoPiRest) / kTwoPi;
  const double high = std::ldexp(std::fmod(q, 1.0), 32), whole = std::floor(high);
  return (static_cast<uint64_t>(whole) << 32) + static_cast<uint64_t>(std::llrint(std::ldexp(high - whole, 32))) +
         static_cast<uint64_t>(std::llrint(std::ldexp(std::fmod(rest, 1.0), 63))) * 2;  // (either sign: sums wrap)
}

// rows of `elements` elements, `stride` apart, as the kernels read them
pa_status check_stride(const char* name, const void* base, int64_t stride, int64_t elements, pa_dtype dtype) {
  if (base == nullptr) return fail(PA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(base, 16)) return fail(PA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride < elements || stride * static_cast<int64_t>(elt_bytes(dtype)) % 16 != 0)
    return fail(PA_ERR_INVALID_ARG, "%s rows of %lld elements, %lld apart: a multiple of 16 bytes, at least a row", name,
                (long long)elements, (long long)stride);
  if (stride > (1ll << 40)) return fail(PA_ERR_INVALID_ARG, "%s rows %lld elements apart", name, (long long)stride);
  return PA_OK;
}

void set_rope(pa::RowsParams* p, const pa_rope* rope) {
  p->sign = p->magnitude = 1.0f;
  if (rope == nullptr) return;
  p->rot = rope->desc.rotary_dim;
  p->interleaved = rope->desc.layout == PA_ROPE_INTERLEAVED;
  p->magnitude = static_cast<float>(rope->magnitude);
  for (int i = 0; i < p->rot / 2; ++i) p->turns[i] = rope->turns[i];
}

}  // namespace

extern "C" {

pa_status pa_rope_create(const pa_rope_desc* desc, pa_rope** out) {
  if (out == nullptr) return fail(PA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (desc == nullptr) return fail(PA_ERR_INVALID_ARG, "rope descriptor is NULL");
  const pa_rope_desc& d = *desc;
  const int r = d.rotary_dim;
  if (r < 2 || r > 128 || r % 2 != 0) return fail(PA_ERR_INVALID_ARG, "rotary_dim %d is not an even number in [2, 128]", r);
  if (d.layout != PA_ROPE_HALF && d.layout != PA_ROPE_INTERLEAVED) return fail(PA_ERR_INVALID_ARG, "unknown rope layout");
  if (!(std::isfinite(d.base) && d.base > 1.0)) return fail(PA_ERR_INVALID_ARG, "rope base %g must be above 1", d.base);
  if (d.scaling < PA_ROPE_NONE || d.scaling > PA_ROPE_BANDS) return fail(PA_ERR_INVALID_ARG, "unknown rope scaling");
  if (d.scaling != PA_ROPE_NONE && !(std::isfinite(d.factor) && d.factor > 0.0))
    return fail(PA_ERR_INVALID_ARG, "rope factor %g must be positive", d.factor);
  const bool ranged = d.scaling == PA_ROPE_RAMP || d.scaling == PA_ROPE_BANDS;
  if (ranged && (d.original_positions <= 0 || !(std::isfinite(d.high) && d.low > 0.0 && d.high > d.low)))
    return fail(PA_ERR_INVALID_ARG, "rope ranges need original_positions > 0 and 0 < low < high");
  if (d.scaling == PA_ROPE_BASE && r == 2) return fail(PA_ERR_INVALID_ARG, "a changed base needs rotary_dim > 2");
  // (the kernels hold it in binary32)
  if (!(d.magnitude == 0.0 || (d.magnitude > 0.0 && d.magnitude <= FLT_MAX && static_cast<float>(d.magnitude) > 0.0f)))
    return fail(PA_ERR_INVALID_ARG, "rope magnitude %g must be 0 or a positive binary32 number", d.magnitude);
  pa_rope* p = new (std::nothrow) pa_rope;
  if (p == nullptr) return fail(PA_ERR_INVALID_ARG, "out of host memory");
  p->desc = d;
  // (a factor of 1 or less stretches nothing: the logarithm is negative there, and the sum with it from e^-10 on)
  const double own = d.scaling == PA_ROPE_RAMP && d.factor > 1.0 ? 0.1 * std::log(d.factor) + 1.0 : 1.0;
  p->magnitude = d.magnitude > 0.0 ? d.magnitude : own;
  const double base = d.scaling == PA_ROPE_BASE ? d.base * std::pow(d.factor, static_cast<double>(r) / (r - 2)) : d.base;
  // PA_ROPE_RAMP: the pair index at which a pair turns t times over the original positions
  auto index_of = [&](double t) { return r * std::log(d.original_positions / (kTwoPi * t)) / (2.0 * std::log(d.base)); };
  double from = 0.0, to = 0.0;
  if (d.scaling == PA_ROPE_RAMP) {
    from = std::max(std::floor(index_of(d.high)), 0.0);
    to = std::min(std::ceil(index_of(d.low)), r - 1.0);
  }
  for (int i = 0; i < r / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    double keep = 1.0;  // the weight of the unchanged frequency
    if (d.scaling == PA_ROPE_LINEAR) keep = 0.0;
    if (d.scaling == PA_ROPE_RAMP) keep = 1.0 - std::min(std::max((i - from) / std::max(to - from, 0.001), 0.0), 1.0);
    if (d.scaling == PA_ROPE_BANDS)
      keep = std::min(std::max((d.original_positions * f / kTwoPi - d.low) / (d.high - d.low), 0.0), 1.0);
    const double g = keep == 1.0 ? f : f / d.factor * (1.0 - keep) + f * keep;
    if (!std::isfinite(base) || !std::isfinite(g)) {
      delete p;
      return fail(PA_ERR_INVALID_ARG, "rope base %g and factor %g give no finite frequencies", d.base, d.factor);
    }
    p->frequencies[i] = g;
    p->turns[i] = turns_of(g);
  }
  *out = p;
  return PA_OK;
}

void pa_rope_destroy(pa_rope* rope) { delete rope; }

pa_status pa_rope_frequencies(const pa_rope* rope, double* frequencies, double* magnitude) {
  if (rope == nullptr) return fail(PA_ERR_INVALID_ARG, "rope is NULL");
  for (int i = 0; frequencies != nullptr && i < rope->desc.rotary_dim / 2; ++i) frequencies[i] = rope->frequencies[i];
  if (magnitude != nullptr) *magnitude = rope->magnitude;
  return PA_OK;
}

pa_status pa_rope_rows(const pa_rope* rope, int32_t n_rows, const void* x, int64_t x_stride, void* out,
                       int64_t out_stride, pa_dtype dtype, int32_t n_heads, int32_t head_dim, const int32_t* positions,
                       int32_t inverse, void* stream) {
  if (rope == nullptr) return fail(PA_ERR_INVALID_ARG, "rope is NULL");
  if (n_rows < 0) return fail(PA_ERR_INVALID_ARG, "n_rows %d < 0", n_rows);
  if (dtype != PA_F32 && dtype != PA_BF16) return fail(PA_ERR_INVALID_ARG, "rope rows are f32 or bf16");
  if (head_dim != 64 && head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", head_dim);
  if (rope->desc.rotary_dim > head_dim)
    return fail(PA_ERR_INVALID_ARG, "rotary_dim %d of head_dim %d", rope->desc.rotary_dim, head_dim);
  if (n_heads <= 0 || n_heads > (1 << 16)) return fail(PA_ERR_INVALID_ARG, "n_heads %d not in [1, 65536]", n_heads);
  if (n_rows == 0) return PA_OK;
  const int64_t row = static_cast<int64_t>(n_heads) * head_dim;
  pa_status st = check_stride("x", x, x_stride, row, dtype);
  if (st == PA_OK) st = check_stride("out", out, out_stride, row, dtype);
  if (st != PA_OK) return st;
  if (positions == nullptr) return fail(PA_ERR_INVALID_ARG, "positions is NULL");
  if (out == x && out_stride != x_stride) return fail(PA_ERR_INVALID_ARG, "in place the two strides are the same");
  pa::RowsParams p{};
  p.q = x;
  p.q_out = out;
  p.q_stride = x_stride;
  p.out_stride = out_stride;
  p.positions = positions;
  p.n_rows = n_rows;
  p.Hq = n_heads;
  p.D = head_dim;
  p.P = 16;  // (no page is looked up)
  p.in_dtype = dtype == PA_F32 ? pa::KV_F32 : pa::KV_BF16;
  set_rope(&p, rope);
  if (inverse != 0) p.sign = -1.0f;
  const cudaError_t e = pa::launch_rows(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "rope launch");
}

pa_status pa_rope_append(const pa_pool* pool, const pa_rope* rope, int32_t n_rows, const void* q, int64_t q_stride,
                         int32_t num_q_heads, void* q_out, const void* k, int64_t k_stride, const void* v,
                         int64_t v_stride, pa_dtype dtype, const int32_t* seq_ids, const int32_t* positions,
                         const int32_t* block_tables, int32_t num_seqs, int32_t max_blocks_per_seq, int32_t* status_dev,
                         void* stream) {
  if (pool == nullptr) return fail(PA_ERR_INVALID_ARG, "pool is NULL");
  const pa_pool_desc& d = pool->desc;
  if (n_rows < 0) return fail(PA_ERR_INVALID_ARG, "n_rows %d < 0", n_rows);
  if (dtype != PA_F32 && dtype != PA_BF16) return fail(PA_ERR_INVALID_ARG, "rope rows are f32 or bf16");
  if (num_q_heads < 0 || num_q_heads > (1 << 16))
    return fail(PA_ERR_INVALID_ARG, "num_q_heads %d not in [0, 65536]", num_q_heads);
  if (rope != nullptr && rope->desc.rotary_dim > d.head_dim)
    return fail(PA_ERR_INVALID_ARG, "rotary_dim %d of head_dim %d", rope->desc.rotary_dim, d.head_dim);
  if (num_seqs <= 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID_ARG, "num_seqs and max_blocks_per_seq must be positive");
  if (d.num_kv_heads > (1 << 16)) return fail(PA_ERR_UNSUPPORTED, "%d kv heads", d.num_kv_heads);
  if (n_rows == 0) return PA_OK;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * d.head_dim, kv_row = static_cast<int64_t>(d.num_kv_heads) * d.head_dim;
  pa_status st = PA_OK;
  if (num_q_heads > 0) {
    st = check_stride("q", q, q_stride, q_row, dtype);
    if (st == PA_OK) st = check_stride("q_out", q_out, q_row, q_row, dtype);
    if (st == PA_OK && q_out == q && q_stride != q_row)
      return fail(PA_ERR_INVALID_ARG, "q_out is contiguous; in place q has to be, too");
  }
  if (st == PA_OK) st = check_stride("k", k, k_stride, kv_row, dtype);
  if (st == PA_OK) st = check_stride("v", v, v_stride, kv_row, dtype);
  if (st != PA_OK) return st;
  if (!seq_ids || !positions || !block_tables) return fail(PA_ERR_INVALID_ARG, "rope append: a device pointer is NULL");
  pa::RowsParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.out_stride = q_row;
  p.k_pool = pool->k;
  p.v_pool = pool->v;
  p.k_ranges = pool->k_ranges;
  p.v_ranges = pool->v_ranges;
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.block_tables = block_tables;
  p.n_rows = n_rows;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.num_pages = d.num_pages;
  p.P = d.page_size;
  p.Hq = num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.D = d.head_dim;
  p.in_dtype = dtype == PA_F32 ? pa::KV_F32 : pa::KV_BF16;
  p.kv_dtype = static_cast<int32_t>(d.kv_dtype);
  p.head_scales = pool->head_scales ? 1 : 0;
  for (int h = 0; h < (pool->head_scales ? d.num_kv_heads : 1); ++h) {
    p.k_scale_h[h] = pool->head_scales ? pool->k_scale_h[h] : d.k_scale;
    p.v_scale_h[h] = pool->head_scales ? pool->v_scale_h[h] : d.v_scale;
  }
  p.status = status_dev;
  set_rope(&p, rope);
  const cudaError_t e = pa::launch_rows(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "rope append launch");
}

pa_status pa_read_kv(const pa_pool* pool, int32_t n_rows, const int32_t* seq_ids, const int32_t* positions,
                     const int32_t* block_tables, int32_t num_seqs, int32_t max_blocks_per_seq, void* k_out,
                     void* v_out, pa_dtype out_dtype, int32_t* status_dev, void* stream) {
  if (pool == nullptr) return fail(PA_ERR_INVALID_ARG, "pool is NULL");
  const pa_pool_desc& d = pool->desc;
  if (n_rows < 0) return fail(PA_ERR_INVALID_ARG, "n_rows %d < 0", n_rows);
  if (out_dtype != PA_F32 && out_dtype != PA_BF16) return fail(PA_ERR_INVALID_ARG, "read output dtype must be f32 or bf16");
  if (num_seqs <= 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID_ARG, "num_seqs and max_blocks_per_seq must be positive");
  if (n_rows == 0 || (k_out == nullptr && v_out == nullptr)) return PA_OK;
  if (!seq_ids || !positions || !block_tables) return fail(PA_ERR_INVALID_ARG, "read: a device pointer is NULL");
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(PA_ERR_INVALID_ARG, "k_out / v_out must be 16-byte aligned");
  if (static_cast<int64_t>(d.num_kv_heads) * d.head_dim > (1 << 28)) return fail(PA_ERR_UNSUPPORTED, "%d kv heads", d.num_kv_heads);
  pa::ReadParams p{};
  p.k_pool = pool->k;
  p.v_pool = pool->v;
  p.k_ranges = pool->k_ranges;
  p.v_ranges = pool->v_ranges;
  p.k_out = k_out;
  p.v_out = v_out;
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.block_tables = block_tables;
  p.n_rows = n_rows;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.num_pages = d.num_pages;
  p.P = d.page_size;
  p.Hkv = d.num_kv_heads;
  p.D = d.head_dim;
  p.out_bf16 = out_dtype == PA_BF16;
  p.kv_dtype = static_cast<int32_t>(d.kv_dtype);
  p.head_scales = pool->head_scales ? 1 : 0;
  for (int h = 0; h < (pool->head_scales ? d.num_kv_heads : 1); ++h) {
    p.k_scale_h[h] = pool->head_scales ? pool->k_scale_h[h] : d.k_scale;
    p.v_scale_h[h] = pool->head_scales ? pool->v_scale_h[h] : d.v_scale;
  }
  p.status = status_dev;
  const cudaError_t e = pa::launch_read(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "read launch");
}

}  // extern "C"
