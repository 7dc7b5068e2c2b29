// pa_tables.cu -- block tables, the rows of a step and its slot map from request
// lengths, on the GPU (pa_tables_grow, pa_tables_release).
//
// Request i with l tokens cached and w new ones needs ceil((l + w) / P) - ceil(l / P) pages
// and w rows.  Everything follows from the two exclusive sums over the requests: page k
// of the call is free_pages[count - 1 - k], and row r belongs to the request whose
// range holds r.  One CTA takes the sums (and, for a decode step's few rows, writes
// the rest as well); the rows of prompts are written by a dependent launch over all
// SMs, four consecutive rows to a thread, found by binary search.
//
// What bounds it is latency: the chain of one load, two scans and a store for a decode step (4.2 us for 8
// requests, 5.3 for 512; the launch alone takes 2 to 3), and the second launch's behind it for
// prompts (10.4 us for 698000 rows of 512 requests, 11.5 MB, which HBM takes in 1.7).
#include <algorithm>

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

constexpr int kTablesThreads = 1024;
constexpr int kTablesMaxSlots = 1 << 19;  // two bits to a slot in shared memory
// Up to here one CTA writes the rows as well (1024 rows 4.5 us, with a second launch 5.3; 2048 rows 6.0 and 6.5; 4032
// rows 8.2 and 7.6; 8192 rows 12.7 and 6.8).
constexpr int kTablesOneCtaRows = 2048;
constexpr int kTablesRowThreads = 256;
constexpr int kTablesRowsPerThread = 4;
constexpr int kTablesStaged = 4096;  // requests whose row starts a CTA copies
enum { ST_NO_PAGES = 6 };

struct TablesParams {
  const int32_t* seq_ids;
  const int32_t* lengths;
  const int32_t* new_tokens;  // release: the tokens that stay (null: none)
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_left;
  int32_t* block_tables;
  int32_t* row_starts;
  int32_t* page_starts;
  int32_t* row_seqs;
  int32_t* row_positions;
  int64_t* row_slots;
  int32_t* status;
  int32_t n, num_pages, lg_p, num_seqs, max_blocks, max_rows;
  int32_t rows_aligned;  // the rows' arrays start on 16 bytes
};

struct ScanSmem {
  long long rows[32], pages[32];  // the warps' sums
  long long last_rows, last_pages;  // the sums up to the last request served
};

// Slots that a call lists twice: a bit for "seen" and one for "again" to each slot.
__device__ __forceinline__ void mark_slots(const TablesParams& p, uint32_t* bits, int words) {
  for (int i = threadIdx.x; i < 2 * words; i += kTablesThreads) bits[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kTablesThreads) {
    const int s = p.seq_ids[i];
    if (s < 0 || s >= p.num_seqs) continue;
    const uint32_t bit = 1u << (s & 31);
    if (atomicOr(bits + (s >> 5), bit) & bit) atomicOr(bits + words + (s >> 5), bit);
  }
  __syncthreads();
}

__device__ __forceinline__ bool listed_once(const TablesParams& p, const uint32_t* bits, int words, int s) {
  return s >= 0 && s < p.num_seqs && ((bits[words + (s >> 5)] >> (s & 31)) & 1u) == 0u;
}

// Inclusive sums of two numbers over the CTA's threads.
__device__ __forceinline__ void scan2(ScanSmem& sm, long long& a, long long& b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sm.rows[warp] = a;
    sm.pages[warp] = b;
  }
  __syncthreads();
  if (warp == 0) {
    long long x = sm.rows[lane], y = sm.pages[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) {
        x += u;
        y += v;
      }
    }
    sm.rows[lane] = x;
    sm.pages[lane] = y;
  }
  __syncthreads();
  if (warp > 0) {
    a += sm.rows[warp - 1];
    b += sm.pages[warp - 1];
  }
}

// The last index i of starts[0 .. n] (ascending) with starts[i] <= x; i < n where x < starts[n].
__device__ __forceinline__ int find_start(const int32_t* starts, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (starts[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Page k of the call goes to the table, for k = first, first + step, ..
__device__ __forceinline__ void write_pages(const TablesParams& p, int before, int total, int first, int step) {
  for (int k = first; k < total; k += step) {
    const int i = find_start(p.page_starts, p.n, k);
    const int held = (p.lengths[i] + (1 << p.lg_p) - 1) >> p.lg_p;
    const int column = held + k - p.page_starts[i];
    int page = p.free_pages[before - 1 - k];
    if (page < 0 || page >= p.num_pages) {
      page = -1;
      record_error(p.status, ST_OUT_OF_RANGE);
    }
    p.block_tables[static_cast<int64_t>(p.seq_ids[i]) * p.max_blocks + column] = page;
  }
}

// Rows r0 .. r0 + count - 1; starts and their requests may be a copy of p.row_starts in shared memory.
__device__ __forceinline__ void write_rows(const TablesParams& p, const int32_t* starts, int before, int total, int r0, int count) {
  if (r0 >= total) return;
  int i = find_start(starts, p.n, r0);
  const int mask = (1 << p.lg_p) - 1;
  for (int r = r0, end = min(r0 + count, total); r < end;) {
    while (starts[i + 1] <= r) ++i;
    const int seq = p.seq_ids[i], length = p.lengths[i];
    const int pos = length + r - starts[i];
    // rows of one request in one page: one lookup for all of them
    const int run = min(min(end, starts[i + 1]) - r, mask + 1 - (pos & mask));
    int64_t slot = -1;
    if (p.row_slots != nullptr) {
      const int column = pos >> p.lg_p, held = (length + mask) >> p.lg_p;
      // a new page by its place on the stack: the table's entry may not be written yet
      const int page = column < held ? p.block_tables[static_cast<int64_t>(seq) * p.max_blocks + column]
                                     : p.free_pages[before - 1 - (p.page_starts[i] + column - held)];
      if (page >= 0 && page < p.num_pages)
        slot = (static_cast<int64_t>(page) << p.lg_p) + (pos & mask);
      else
        record_error(p.status, ST_OUT_OF_RANGE);
    }
    if (run == 4 && (r & 3) == 0 && p.rows_aligned) {
      *reinterpret_cast<int4*>(p.row_seqs + r) = make_int4(seq, seq, seq, seq);
      *reinterpret_cast<int4*>(p.row_positions + r) = make_int4(pos, pos + 1, pos + 2, pos + 3);
      if (p.row_slots != nullptr) {
        const int64_t one = slot < 0 ? 0 : 1;
        longlong2* s = reinterpret_cast<longlong2*>(p.row_slots + r);
        s[0] = make_longlong2(slot, slot + one);
        s[1] = make_longlong2(slot + 2 * one, slot + 3 * one);
      }
    } else {
      for (int k = 0; k < run; ++k) {
        p.row_seqs[r + k] = seq;
        p.row_positions[r + k] = pos + k;
        if (p.row_slots != nullptr) p.row_slots[r + k] = slot < 0 ? -1 : slot + k;
      }
    }
    r += run;
  }
}

template <bool ROWS>
__global__ void __launch_bounds__(kTablesThreads) tables_grow_kernel(const __grid_constant__ TablesParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ ScanSmem sm;
  griddep_launch_dependents();  // (they wait for the sums)
  const int tid = threadIdx.x, words = (p.num_seqs + 31) / 32;
  int count = p.free_count[0];
  const bool bad_count = count < 0 || count > p.num_pages;
  if (bad_count) {
    count = 0;
    if (tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
  }
  if (tid == 0) sm.last_rows = sm.last_pages = 0;
  mark_slots(p, bits, words);
  const int64_t room = static_cast<int64_t>(p.max_blocks) << p.lg_p;
  long long rows_before = 0, pages_before = 0;  // all requests so far, served or not
  for (int i0 = 0; i0 < p.n; i0 += kTablesThreads) {
    const int i = i0 + tid;
    long long rows = 0, pages = 0;
    if (i < p.n) {
      const int s = p.seq_ids[i];
      const int64_t length = p.lengths[i], more = p.new_tokens[i];
      if (listed_once(p, bits, words, s) && length >= 0 && more >= 0 && length + more <= room) {
        rows = more;
        pages = ((length + more + (1 << p.lg_p) - 1) >> p.lg_p) - ((length + (1 << p.lg_p) - 1) >> p.lg_p);
      } else {
        record_error(p.status, ST_OUT_OF_RANGE);
      }
    }
    const bool asks = rows > 0;
    scan2(sm, rows, pages);
    rows += rows_before;
    pages += pages_before;
    // sums never fall, so the requests served are the first ones
    const bool served = rows <= p.max_rows && pages <= count;
    if (!served && asks) record_error(p.status, ST_NO_PAGES);
    if (tid == __syncthreads_count(served) - 1) {
      sm.last_rows = rows;
      sm.last_pages = pages;
    }
    __syncthreads();
    if (i < p.n) {
      p.row_starts[i + 1] = static_cast<int32_t>(served ? rows : sm.last_rows);
      p.page_starts[i + 1] = static_cast<int32_t>(served ? pages : sm.last_pages);
    }
    rows_before += sm.rows[31];
    pages_before += sm.pages[31];
    __syncthreads();
  }
  const int total_rows = static_cast<int>(sm.last_rows), total_pages = static_cast<int>(sm.last_pages);
  if (tid == 0) {
    p.row_starts[0] = p.page_starts[0] = 0;
    p.free_left[0] = bad_count ? p.free_count[0] : count - total_pages;
  }
  if constexpr (ROWS) {
    __syncthreads();
    write_pages(p, count, total_pages, tid, kTablesThreads);
    for (int r = tid; r < total_rows; r += kTablesThreads) write_rows(p, p.row_starts, count, total_rows, r, 1);
  }
}

__global__ void __launch_bounds__(kTablesRowThreads) tables_rows_kernel(const __grid_constant__ TablesParams p) {
  __shared__ int32_t staged[kTablesStaged + 1];
  griddep_wait();  // the sums are another launch's
  const int total_pages = p.page_starts[p.n], total_rows = p.row_starts[p.n];
  const int before = p.free_left[0] + total_pages;
  const int thread = blockIdx.x * kTablesRowThreads + threadIdx.x, threads = gridDim.x * kTablesRowThreads;
  const int32_t* starts = p.row_starts;
  if (p.n <= kTablesStaged) {  // a search of dependent loads is short in shared memory
    for (int i = threadIdx.x; i <= p.n; i += kTablesRowThreads) staged[i] = p.row_starts[i];
    __syncthreads();
    starts = staged;
  }
  for (int64_t r = static_cast<int64_t>(thread) * kTablesRowsPerThread; r < total_rows;
       r += static_cast<int64_t>(threads) * kTablesRowsPerThread)
    write_rows(p, starts, before, total_rows, static_cast<int>(r), kTablesRowsPerThread);
  write_pages(p, before, total_pages, thread, threads);
}

// One CTA: which requests are sound (a warp each looks over its pages), their place
// on the stack, then the pages themselves.
__global__ void __launch_bounds__(kTablesThreads) tables_release_kernel(const __grid_constant__ TablesParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ int32_t bad_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, words = (p.num_seqs + 31) / 32;
  const int P1 = (1 << p.lg_p) - 1;
  const int count = p.free_count[0];
  mark_slots(p, bits, words);
  const int64_t room = static_cast<int64_t>(p.max_blocks) << p.lg_p;
  // the pages of request i: columns first .. last - 1 (none of a request that is refused)
  auto range = [&](int i, int& first, int& last) -> bool {
    first = last = 0;
    const int s = p.seq_ids[i], length = p.lengths[i], keep = p.new_tokens == nullptr ? 0 : p.new_tokens[i];
    if (!listed_once(p, bits, words, s) || length < 0 || length > room || keep < 0) return false;
    last = static_cast<int>((static_cast<int64_t>(length) + P1) >> p.lg_p);
    first = min(last, static_cast<int>((static_cast<int64_t>(keep) + P1) >> p.lg_p));
    return true;
  };
  // two passes over the requests, 32 at a time, each its warp's: the sum of sound pages, then their moves
  long long total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long before = 0;
    if (pass == 1) {
      const bool fits = count >= 0 && total <= p.num_pages - static_cast<long long>(count);
      if (!fits) {
        if (tid == 0) record_error(p.status, ST_OUT_OF_RANGE);
        return;
      }
    }
    for (int i0 = 0; i0 < p.n; i0 += 32) {
      const int i = i0 + warp;
      int first = 0, last = 0;
      bool good = i < p.n && range(i, first, last);
      const int32_t* row = good ? p.block_tables + static_cast<int64_t>(p.seq_ids[i]) * p.max_blocks : nullptr;
      bool bad = false;
      for (int c = first + lane; c < last; c += 32) {
        const int page = row[c];
        bad |= page < 0 || page >= p.num_pages;
      }
      good = good && !__any_sync(0xffffffffu, bad);
      if (pass == 0 && !good && i < p.n && lane == 0) record_error(p.status, ST_OUT_OF_RANGE);
      if (lane == 0) bad_warp[warp] = good ? last - first : 0;
      __syncthreads();
      long long mine = before;
      for (int w = 0; w < warp; ++w) mine += bad_warp[w];
      for (int w = 0; w < 32; ++w) before += bad_warp[w];
      if (pass == 1 && good) {
        int32_t* out = p.block_tables + static_cast<int64_t>(p.seq_ids[i]) * p.max_blocks;
        for (int c = first + lane; c < last; c += 32) {
          p.free_pages[count + total - 1 - (mine + c - first)] = out[c];
          out[c] = -1;
        }
      }
      __syncthreads();
    }
    if (pass == 0) total = before;
  }
  if (tid == 0) p.free_left[0] = count + static_cast<int>(total);
}

}  // namespace pa

using pa::cuda_fail;
using pa::fail;

namespace {

pa_status check_tables(int32_t n, int32_t num_pages, int32_t page_size, int32_t num_seqs, int32_t max_blocks) {
  if (n < 0) return fail(PA_ERR_INVALID_ARG, "n %d < 0", n);
  if (num_pages <= 0 || num_seqs <= 0 || max_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "num_pages, num_seqs and max_blocks_per_seq must be positive");
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
    return fail(PA_ERR_UNSUPPORTED, "page_size %d not in {16, 32, 64, 128, 256}", page_size);
  if (num_seqs > pa::kTablesMaxSlots) return fail(PA_ERR_UNSUPPORTED, "%d slots (at most %d)", num_seqs, pa::kTablesMaxSlots);
  if (static_cast<int64_t>(max_blocks) * page_size > 0x7fffffff)  // (positions stay int32)
    return fail(PA_ERR_UNSUPPORTED, "a block-table row of %d pages of %d tokens", max_blocks, page_size);
  return PA_OK;
}

int log2_of(int32_t p) {
  int lg = 0;
  while ((1 << lg) < p) ++lg;
  return lg;
}

size_t slot_bits(int32_t num_seqs) { return static_cast<size_t>((num_seqs + 31) / 32) * 2 * sizeof(uint32_t); }

}  // namespace

extern "C" {

pa_status pa_tables_grow(int32_t n, const int32_t* seq_ids, const int32_t* lengths, const int32_t* new_tokens,
                         const int32_t* free_pages, const int32_t* free_count, int32_t* free_left, int32_t num_pages,
                         int32_t page_size, int32_t* block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                         int32_t* row_starts, int32_t* page_starts, int32_t max_rows, int32_t* row_seqs,
                         int32_t* row_positions, int64_t* row_slots, int32_t* status_dev, void* stream) {
  const pa_status st = check_tables(n, num_pages, page_size, num_seqs, max_blocks_per_seq);
  if (st != PA_OK) return st;
  if (max_rows < 0) return fail(PA_ERR_INVALID_ARG, "max_rows %d < 0", max_rows);
  if ((n > 0 && (!seq_ids || !lengths || !new_tokens)) || !free_pages || !free_count || !free_left || !block_tables ||
      !row_starts || !page_starts || (max_rows > 0 && (!row_seqs || !row_positions)))
    return fail(PA_ERR_INVALID_ARG, "tables: a device pointer is NULL");
  pa::TablesParams p{};
  p.seq_ids = seq_ids;
  p.lengths = lengths;
  p.new_tokens = new_tokens;
  p.free_pages = const_cast<int32_t*>(free_pages);
  p.free_count = free_count;
  p.free_left = free_left;
  p.block_tables = block_tables;
  p.row_starts = row_starts;
  p.page_starts = page_starts;
  p.row_seqs = row_seqs;
  p.row_positions = row_positions;
  p.row_slots = row_slots;
  p.status = status_dev;
  p.n = n;
  p.num_pages = num_pages;
  p.lg_p = log2_of(page_size);
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.max_rows = max_rows;
  p.rows_aligned = pa::aligned(row_seqs, 16) && pa::aligned(row_positions, 16) && pa::aligned(row_slots, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool one = max_rows <= pa::kTablesOneCtaRows;
  static std::atomic<unsigned long long> done_one{0}, done_two{0};
  constexpr size_t most = static_cast<size_t>(pa::kTablesMaxSlots) / 4;
  cudaError_t e = one ? pa::allow_dynamic_smem(pa::tables_grow_kernel<true>, done_one, most)
                      : pa::allow_dynamic_smem(pa::tables_grow_kernel<false>, done_two, most);
  if (e != cudaSuccess) return cuda_fail(e, "tables shared memory");
  e = one ? pa::launch_kernel(pa::tables_grow_kernel<true>, dim3(1), dim3(pa::kTablesThreads), slot_bits(num_seqs), s, false, p)
          : pa::launch_kernel(pa::tables_grow_kernel<false>, dim3(1), dim3(pa::kTablesThreads), slot_bits(num_seqs), s, false, p);
  pa::count_launch();
  if (e == cudaSuccess && !one) {
    const int64_t per_cta = pa::kTablesRowThreads * pa::kTablesRowsPerThread;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((max_rows + per_cta - 1) / per_cta, 152 * 8));
    e = pa::launch_kernel(pa::tables_rows_kernel, dim3(grid), dim3(pa::kTablesRowThreads), 0, s, true, p);
    pa::count_launch();
  }
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "tables launch");
}

pa_status pa_tables_release(int32_t n, const int32_t* seq_ids, const int32_t* lengths, const int32_t* keep_tokens,
                            int32_t* free_pages, int32_t* free_count, int32_t num_pages, int32_t page_size,
                            int32_t* block_tables, int32_t num_seqs, int32_t max_blocks_per_seq, int32_t* status_dev,
                            void* stream) {
  const pa_status st = check_tables(n, num_pages, page_size, num_seqs, max_blocks_per_seq);
  if (st != PA_OK) return st;
  if (n == 0) return PA_OK;
  if (!seq_ids || !lengths || !free_pages || !free_count || !block_tables)
    return fail(PA_ERR_INVALID_ARG, "tables: a device pointer is NULL");
  pa::TablesParams p{};
  p.seq_ids = seq_ids;
  p.lengths = lengths;
  p.new_tokens = keep_tokens;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.free_left = free_count;
  p.block_tables = block_tables;
  p.status = status_dev;
  p.n = n;
  p.num_pages = num_pages;
  p.lg_p = log2_of(page_size);
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = pa::allow_dynamic_smem(pa::tables_release_kernel, done, static_cast<size_t>(pa::kTablesMaxSlots) / 4);
  if (e != cudaSuccess) return cuda_fail(e, "tables shared memory");
  e = pa::launch_kernel(pa::tables_release_kernel, dim3(1), dim3(pa::kTablesThreads), slot_bits(num_seqs),
                        static_cast<cudaStream_t>(stream), false, p);
  pa::count_launch();
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "tables launch");
}

}  // extern "C"
