// diffragged_step: lengths, pages, table, q_start, positions and slots of a
// packed batch's step.
//
// Everything follows from three prefix sums over the sequences (pages given back,
// pages taken, rows), and pages given back may be taken again, so a block of 1024
// threads does it, 1024 sequences at a time: it adds everything up first and
// touches nothing where that does not fit, gives back, takes, and writes q_start
// and the rows.  Pages and rows are moved flat, a thread each, whichever sequence
// they belong to (found in the prefix sums in shared memory), so that one long
// prompt does not wait for one thread.  For many of them a cluster of eight
// blocks shares the moves, every block with sums of its own.
//
// Bound: latency.  Some ten dependent steps (loads, block scans) of half a
// microsecond at most; the bytes are nothing.  Measured on GB300: 64 sequences
// with a token each 4.3 us; 768 sequences, 46703 rows, 17000 pages moved 11 us (a
// single block, its rows by a second kernel, 16 us).
#include <cuda_runtime.h>

#include <cstdint>

#include "debug_check.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "ragged.h"

namespace diffattn {
namespace {

constexpr int kThreads = 1024;
// A cluster of eight blocks from this many rows or sequences on, which may move many pages.
constexpr int64_t kFewRows = 4096, kFewSequences = 256;
constexpr int kBlocks = 8;

struct StepParams {
  int32_t *kv_len, *held, *page_table, *free_pages, *free_count;
  const int32_t *new_len;
  int32_t *q_start, *positions;
  int64_t *slots;
  int32_t *status;
  int32_t B, max_pages, page_size;
  bool rows;  // positions or slots are wanted
  int64_t capacity, N;
  FastDiv by_page;
};

// One sequence before and after the step.
struct Change {
  int32_t len, rows, held, need;  // len: after
  bool bad;
};
__device__ __forceinline__ Change change_of(const StepParams &p, int32_t b) {
  const int32_t n = p.new_len[b], len = p.kv_len[b], held = p.held[b];
  const int32_t most = p.max_pages * p.page_size;
  Change c = {0, 0, held, 0, false};
  c.bad = n < -1 || len < 0 || len > most || held < 0 || held > p.max_pages || n > most - len;
  if (c.bad) return c;
  c.bad = p.by_page.div(len + p.page_size - 1) > held;
  if (n >= 0) {
    c.len = len + n;
    c.rows = n;
  }
  c.need = p.by_page.div(c.len + p.page_size - 1);
  return c;
}

struct Scan {
  int32_t before, total;
};
// Sum over the threads before this one, and over all.
__device__ __forceinline__ Scan block_scan(int32_t x, int32_t *sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int32_t w = sums[lane], all = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += y;
  }
  const Scan s = {incl - x + (warp ? __shfl_sync(0xffffffffu, all, warp - 1) : 0),
                  __shfl_sync(0xffffffffu, all, 31)};
  __syncthreads();
  return s;
}

// The last k with at[k] <= x, of kThreads (at[0] = 0; equal ones: the last).
__device__ __forceinline__ int find(const int32_t *at, int32_t x) {
  int k = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step /= 2)
    if (at[k + step] <= x) k += step;
  return k;
}

__device__ __forceinline__ void write_row(const StepParams &p, int64_t row, int32_t b, int32_t pos) {
  if (!dbg_ok(row >= 0 && row < p.N && pos >= 0 && p.by_page.div(pos) < p.max_pages, p.status, 91))
    return;
  if (p.positions != nullptr) p.positions[row] = pos;
  if (p.slots != nullptr) {
    const int32_t k = p.by_page.div(pos);
    const int64_t page = p.page_table[static_cast<int64_t>(b) * p.max_pages + k];
    p.slots[row] = page * p.page_size + (pos - k * p.page_size);
  }
}
__device__ __forceinline__ void write_none(const StepParams &p, int64_t row) {
  if (p.positions != nullptr) p.positions[row] = -1;
  if (p.slots != nullptr) p.slots[row] = -1;
}

// A barrier over the cluster's blocks, and what they wrote before it seen behind it.
__device__ __forceinline__ void all_blocks(uint32_t blocks) {
  if (blocks == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

// The block's and the other blocks' share of `total` pieces of work, a thread each: first, step.
struct Flat {
  int32_t first, step;
};

// (No early launch of the kernel behind: page tables and lengths are read through the read-only path
// by kernels that may follow, which must not be resident while this one writes them.)
__global__ void __launch_bounds__(kThreads, 1) diffragged_step_kernel(const StepParams p) {
  __shared__ int32_t sums[32];
  __shared__ int32_t at[kThreads], first[kThreads];
  __shared__ unsigned long long total[3];
  __shared__ int32_t any_bad;
  const int tid = threadIdx.x;
  uint32_t rank, blocks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(blocks));
  const Flat flat = {static_cast<int32_t>(rank * kThreads + tid),
                     static_cast<int32_t>(blocks * kThreads)};
  if (tid < 3) total[tid] = 0;
  if (tid == 0) any_bad = 0;
  __syncthreads();
  grid_dependency_wait();

  // What the step comes to (every block for itself).
  const int32_t count0 = *p.free_count;
  Change mine = {0, 0, 0, 0, false};  // of the first 1024 sequences
  {
    int64_t sum[3] = {0, 0, 0};  // given back, taken, rows
    bool bad = false;
    for (int32_t b = tid; b < p.B; b += kThreads) {
      const Change c = change_of(p, b);
      if (b == tid) mine = c;
      bad |= c.bad;
      if (c.held > c.need)
        sum[0] += c.held - c.need;
      else
        sum[1] += c.need - c.held;
      sum[2] += c.rows;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
      if (tid % 32 == 0 && sum[k] != 0)
        atomicAdd(&total[k], static_cast<unsigned long long>(sum[k]));
    }
    if (bad) any_bad = 1;
  }
  __syncthreads();
  const int64_t given = total[0], taken = total[1], rows = total[2];
  if (any_bad || count0 < 0 || count0 + given > p.capacity || taken > count0 + given ||
      rows > p.N) {
    for (int32_t b = flat.first; b <= p.B; b += flat.step) p.q_start[b] = 0;
    if (p.rows)  // (N may be anything where no rows are wanted)
      for (int64_t r = flat.first; r < p.N; r += flat.step) write_none(p, r);
    if (tid == 0 && rank == 0) report_bad_page(p.status);
    return;
  }
  const int32_t count1 = count0 + static_cast<int32_t>(given);
  const auto change = [&](int32_t b0) {
    return b0 == 0 ? mine : b0 + tid < p.B ? change_of(p, b0 + tid) : Change{0, 0, 0, 0, false};
  };
  // `move(x, k)` for all pieces k of sequence b0 + x, `count` each from the chunk's `base` on: the
  // place of a piece among all is base + k, in its sequence k - at[x].
  const auto spread = [&](int32_t sum, const auto &move) {
#pragma unroll 4
    for (int32_t k = flat.first; k < sum; k += flat.step) move(find(at, k), k);
  };

  // Pages given back.
  if (given > 0) {
    int32_t base = 0;
    for (int32_t b0 = 0; b0 < p.B; b0 += kThreads) {
      const Change c = change(b0);
      const Scan s = block_scan(max(0, c.held - c.need), sums);
      at[tid] = s.before;
      first[tid] = c.need;
      __syncthreads();
      spread(s.total, [&](int x, int32_t k) {
        p.free_pages[count0 + base + k] =
            p.page_table[static_cast<int64_t>(b0 + x) * p.max_pages + first[x] + (k - at[x])];
      });
      base += s.total;
      __syncthreads();
    }
  }
  all_blocks(blocks);

  // Pages taken.
  if (taken > 0) {
    int32_t base = 0;
    for (int32_t b0 = 0; b0 < p.B; b0 += kThreads) {
      const Change c = change(b0);
      const Scan s = block_scan(max(0, c.need - c.held), sums);
      at[tid] = s.before;
      first[tid] = c.held;
      __syncthreads();
      spread(s.total, [&](int x, int32_t k) {
        p.page_table[static_cast<int64_t>(b0 + x) * p.max_pages + first[x] + (k - at[x])] =
            p.free_pages[count1 - 1 - base - k];
      });
      base += s.total;
      __syncthreads();
    }
    all_blocks(blocks);
  }

  // q_start and the rows.
  int32_t row0 = 0;
  for (int32_t b0 = 0; b0 < p.B; b0 += kThreads) {
    const Change c = change(b0);
    const Scan r = block_scan(c.rows, sums);
    at[tid] = r.before;
    first[tid] = c.len - c.rows;
    if (rank == 0 && b0 + tid < p.B) p.q_start[b0 + tid] = row0 + r.before;
    if (p.rows) {
      __syncthreads();
      spread(r.total, [&](int x, int32_t k) {
        write_row(p, row0 + k, b0 + x, first[x] + (k - at[x]));
      });
      __syncthreads();
    }
    row0 += r.total;
  }
  if (p.rows)
    for (int64_t r = rows + flat.first; r < p.N; r += flat.step) write_none(p, r);

  // The lengths and counts, once no block reads them again.
  if (p.B > kThreads) all_blocks(blocks);
  if (rank != 0) return;
  for (int32_t b0 = 0; b0 < p.B; b0 += kThreads) {
    const Change c = change(b0);
    if (b0 + tid < p.B) {
      p.kv_len[b0 + tid] = c.len;
      p.held[b0 + tid] = c.need;
    }
  }
  if (tid == 0) {
    p.q_start[p.B] = static_cast<int32_t>(rows);
    *p.free_count = count1 - static_cast<int32_t>(taken);
  }
}

}  // namespace

diffattn_status launch_ragged_step(const diffragged_book &book, const int32_t *new_len, int64_t N,
                                   int32_t *q_start, int32_t *positions, int64_t *slots,
                                   int32_t *status, cudaStream_t stream) {
  StepParams p = {};
  p.kv_len = book.kv_len;
  p.held = book.held;
  p.page_table = book.page_table;
  p.free_pages = book.free_pages;
  p.free_count = book.free_count;
  p.new_len = new_len;
  p.q_start = q_start;
  p.positions = positions;
  p.slots = slots;
  p.status = status;
  p.B = static_cast<int32_t>(book.B);
  p.max_pages = static_cast<int32_t>(book.max_pages);
  p.page_size = book.page_size;
  p.capacity = book.capacity;
  p.N = N;
  p.by_page = fast_div(static_cast<uint32_t>(book.page_size));
  p.rows = positions != nullptr || slots != nullptr;
  cudaLaunchConfig_t cfg = {};
  const unsigned blocks = (p.rows && N > kFewRows) || p.B > kFewSequences ? kBlocks : 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, diffragged_step_kernel, p) == cudaSuccess ? DIFFATTN_OK
                                                                            : DIFFATTN_ERR_CUDA;
}

}  // namespace diffattn
