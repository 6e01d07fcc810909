// gdn_tables.cu -- the tables of one engine step, built on the GPU from the
// request lengths and state slots: packed row offsets, state pointers, and the
// maps row -> sequence, row -> slot and chunk -> sequence.
//
// Row offsets are an exclusive sum of the lengths, chunk offsets one of
// ceil(len / 64).  Both sums saturate at one above their buffer's capacity
// (min(x + y, cap + 1) is associative over non-negative numbers), so no input
// makes them overflow, and offsets are written clamped to the capacity: a
// later call never reads behind the rows.
//
// Bound: latency (a few KB to a few MB): 4.6 us for 64 sequences of one row, 8.4 us for
// 300 of up to 512 rows, 14.3 us for 4096 (1.8 MB of tables).  One launch, no CTA waits on another:
// every CTA sums all the lengths itself, a tile of kTile at a time, and writes
// its own share of the outputs -- tiles in turn for the per-sequence tables,
// and for the maps the positions of its own range, each found by a binary
// search in the tile's offsets.
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr int kTabThreads = 256;
constexpr int kPer = 4;                      // lengths per thread and tile
constexpr int kTile = kTabThreads * kPer;    // lengths per tile
constexpr int kTabChunk = 64;
constexpr uint32_t kTabFlagError = 2u;       // GDN_FLAG_ERROR

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t top) {
  return min(a + b, top);  // a, b <= 2^31
}

// Exclusive saturating sum over the CTA of one value per thread; *total gets
// the sum of all.  `warp_sums` holds one word per warp.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t top, uint32_t* warp_sums,
                                               uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc = sat_add(inc, y, top);
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w < warp) before = sat_add(before, warp_sums[w], top);
    all = sat_add(all, warp_sums[w], top);
  }
  *total = all;
  // exclusive within the warp: the inclusive sum of the lane before
  const uint32_t prev = __shfl_up_sync(0xffffffffu, inc, 1);
  return lane == 0 ? before : sat_add(before, prev, top);
}

// The sequence of position `x`: the largest i in [0, n) with off[i] <= x
// (off is nondecreasing and off[0] <= x).
__device__ __forceinline__ int find_seq(const uint32_t* off, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) tables_kernel(TablesCall c) {
  __shared__ uint32_t rows[kTile + 1], chunks[kTile + 1];  // offsets of the tile's sequences
  __shared__ int32_t slot_of[kTile];
  __shared__ uint32_t sums[2][kTabThreads / 32];
  const int tid = threadIdx.x;
  grid_launch_next();
  const uint32_t row_top = uint32_t(c.row_capacity) + 1u;
  const uint32_t chunk_top = uint32_t(c.chunk_capacity) + 1u;
  // this CTA's range of map positions
  const uint32_t row_share = uint32_t((c.row_capacity + gridDim.x - 1) / gridDim.x);
  const uint32_t chunk_share = uint32_t((c.chunk_capacity + gridDim.x - 1) / gridDim.x);
  const uint32_t row_lo = min(blockIdx.x * row_share, uint32_t(c.row_capacity));
  const uint32_t row_hi = min(row_lo + row_share, uint32_t(c.row_capacity));
  const uint32_t chunk_lo = min(blockIdx.x * chunk_share, uint32_t(c.chunk_capacity));
  const uint32_t chunk_hi = min(chunk_lo + chunk_share, uint32_t(c.chunk_capacity));
  uint32_t row_at = 0, chunk_at = 0;  // sums before the tile
  bool bad = false;
  for (int t0 = 0, tile = 0; t0 < c.num_seqs; t0 += kTile, ++tile) {
    const int n = min(kTile, c.num_seqs - t0);
    const bool mine = tile % int(gridDim.x) == int(blockIdx.x);
    uint32_t len[kPer], nch[kPer], rsum = 0, csum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = kPer * tid + i;
      int x = 0;
      if (j < n) {
        x = c.lens != nullptr ? c.lens[t0 + j] : c.cu_in[t0 + j + 1] - c.cu_in[t0 + j];
        if (x < 0) {
          x = 0;
          bad = true;
        }
      }
      len[i] = min(uint32_t(x), row_top);
      nch[i] = min((uint32_t(x) + kTabChunk - 1) / kTabChunk, chunk_top);
      rsum = sat_add(rsum, len[i], row_top);
      csum = sat_add(csum, nch[i], chunk_top);
    }
    uint32_t rtot, ctot;
    uint32_t r = sat_add(row_at, block_scan(rsum, row_top, sums[0], &rtot), row_top);
    uint32_t k = sat_add(chunk_at, block_scan(csum, chunk_top, sums[1], &ctot), chunk_top);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = kPer * tid + i;
      if (j < n) {
        rows[j] = r;
        chunks[j] = k;
        if (c.slots != nullptr) {
          int sl = c.slots[t0 + j];
          if (sl >= c.num_slots) {
            bad = true;
            sl = -1;
          }
          slot_of[j] = max(sl, -1);
          if (mine)
            c.h_table[t0 + j] = sl < 0 ? nullptr : c.pool + size_t(sl) * size_t(c.slot_floats);
        }
        if (mine) {
          if (c.cu_seqlens != nullptr) c.cu_seqlens[t0 + j] = int(min(r, row_top - 1));
          if (c.cu_chunks != nullptr) c.cu_chunks[t0 + j] = int(min(k, chunk_top - 1));
        }
      }
      r = sat_add(r, len[i], row_top);
      k = sat_add(k, nch[i], chunk_top);
    }
    const uint32_t row_end = sat_add(row_at, rtot, row_top);
    const uint32_t chunk_end = sat_add(chunk_at, ctot, chunk_top);
    __syncthreads();
    // the maps: this CTA's positions that fall into the tile
    if (c.row_seq != nullptr || c.row_slot != nullptr) {
      const uint32_t hi = min(row_hi, row_end);
      for (uint32_t x = max(row_lo, row_at) + tid; x < hi; x += kTabThreads) {
        const int j = find_seq(rows, n, x);
        if (c.row_seq != nullptr) c.row_seq[x] = t0 + j;
        if (c.row_slot != nullptr) c.row_slot[x] = slot_of[j];
      }
    }
    if (c.chunk_seq != nullptr) {
      const uint32_t hi = min(chunk_hi, chunk_end);
      for (uint32_t x = max(chunk_lo, chunk_at) + tid; x < hi; x += kTabThreads)
        c.chunk_seq[x] = t0 + find_seq(chunks, n, x);
    }
    __syncthreads();  // the tile's offsets are rewritten next
    row_at = row_end;
    chunk_at = chunk_end;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (c.cu_seqlens != nullptr) c.cu_seqlens[c.num_seqs] = int(min(row_at, row_top - 1));
    if (c.cu_chunks != nullptr) c.cu_chunks[c.num_seqs] = int(min(chunk_at, chunk_top - 1));
    if (row_at >= row_top || (c.chunk_seq != nullptr && chunk_at >= chunk_top)) bad = true;
  }
  if (bad && c.flag != nullptr) atomicOr(c.flag, kTabFlagError);
}

cudaError_t launch_tables(const TablesCall& c, cudaStream_t s) {
  // One CTA per 2048 positions of the maps that are made and per tile of lengths, at most one
  // per SM: more would only repeat the sums.
  const long long rows = c.row_seq != nullptr || c.row_slot != nullptr ? c.row_capacity : 0;
  const long long chunks = c.chunk_seq != nullptr ? c.chunk_capacity : 0;
  const long long tiles = (c.num_seqs + (long long)kTile - 1) / kTile;
  long long grid = ((rows > chunks ? rows : chunks) + 2047) / 2048;
  if (grid < tiles) grid = tiles;
  if (grid > sm_count()) grid = sm_count();
  if (grid < 1) grid = 1;
  tables_kernel<<<unsigned(grid), kTabThreads, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace gdn
