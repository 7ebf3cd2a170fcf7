// Block operations of the paged cache: copy, reserve, fork, release, compact.
//
// State (caller-owned): page_table [rows, max_blocks] physical block ids (-1: none), seq_lens
// [rows], ref_counts [num_blocks] (0: free). There is no free list: an allocation takes the
// lowest free ids in the order of the requests, and reference counts only see commuting integer
// atomics, so every result is the same whatever order the GPU runs in.
//
// Planning kernels (alloc_kernel, compact_plan_kernel) are one CTA of 1024 threads: their work is
// a scan over ref_counts (4 ids per thread and step, 4 KiB of counts per 16 KiB step), bound by the
// latency of a few block-wide scans; one CTA needs no grid barrier. The bytes move in apply
// kernels that fill the GPU: HBM-bound copies, kUnroll 16-byte loads in flight per thread.
// Measured: 629 MB of listed blocks 104 us a call (89 % of the copy rate); compaction of a pool of
// 2048 blocks, 515 MB, 5 + 76 us on the device (the copy 99 %), 96 us a call; a fork of 64 children
// 6 + 30 us, their release 4 us.
#include "pbs_device.cuh"
#include "pbs_internal.h"
#include "pdl.cuh"

namespace pbs {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kIdsPerThread = 4;
constexpr int kIdsPerStep = kPlanThreads * kIdsPerThread;
constexpr int kCopyThreads = 256;
constexpr int kUnroll = 8;
constexpr int64_t kPiece = int64_t(kCopyThreads) * kUnroll * 16;  // bytes a CTA moves per step

// Exclusive prefix sum of v over the block's threads, and the total. All threads must call it.
__device__ __forceinline__ int block_scan(int v, int* total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int before = warp > 0 ? warp_sums[warp - 1] : 0;
  *total = warp_sums[31];
  __syncthreads();  // warp_sums may be written again
  return before + x - v;
}

// ids id0 .. id0 + 3 of ref_counts; out-of-range ids read as -1 (neither free nor live).
__device__ __forceinline__ void load_refs(const int32_t* refs, int num_blocks, int id0, int (&r)[kIdsPerThread]) {
#pragma unroll
  for (int i = 0; i < kIdsPerThread; ++i) r[i] = id0 + i < num_blocks ? __ldcg(refs + id0 + i) : -1;
}

// Hands the lowest free ids at or after *cursor to the threads that ask (want), in thread order: the
// thread's id, or -1 when the pool has run out. Sets ref_counts of the ids it hands out to 1 and
// moves *cursor behind the last. All threads must call it.
__device__ int take_free(bool want, int32_t* refs, int num_blocks, int* cursor, int* list, int* warp_sums) {
  int need;
  const int rank = block_scan(want ? 1 : 0, &need, warp_sums);
  int found = 0, at = *cursor;  // every thread keeps its own copy
  if (need > 0) {
    __shared__ int s_next;
    while (found < need && at < num_blocks) {
      const int id0 = at + static_cast<int>(threadIdx.x) * kIdsPerThread;
      int r[kIdsPerThread];
      load_refs(refs, num_blocks, id0, r);
      int mine = 0;
#pragma unroll
      for (int i = 0; i < kIdsPerThread; ++i) mine += r[i] == 0;
      int total;
      int pos = found + block_scan(mine, &total, warp_sums);
#pragma unroll
      for (int i = 0; i < kIdsPerThread; ++i) {
        if (r[i] != 0) continue;
        if (pos < need) {
          list[pos] = id0 + i;
          if (pos == need - 1) s_next = id0 + i + 1;
        }
        ++pos;
      }
      found += total;
      at += kIdsPerStep;
      __syncthreads();
    }
    if (found >= need) at = s_next;
    __syncthreads();
  }
  *cursor = at;
  int id = -1;
  if (want && rank < found) {
    id = list[rank];
    refs[id] = 1;
  }
  __syncthreads();  // list may be written again
  return id;
}

// Fork: child i's tail block and the copy pair; reserve: the blocks behind each row's tokens.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const BlockArgs a) {
  __shared__ int list[kPlanThreads];
  __shared__ int warp_sums[32];
  pdl_release();
  int cursor = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    bool want = false;
    int src_block = -1;
    int state = -1;  // copy_dst of a child without a tail block of its own
    if (i < a.n) {
      const int s = __ldg(a.src_rows + i), d = __ldg(a.dst_rows + i);
      if (s < 0 || s >= a.num_rows || d < 0 || d >= a.num_rows || s == d) {
        set_err(a.err_word, PBS_DEVERR_TABLE);
        state = -2;  // skipped
      } else {
        const int len = a.seq_lens[s];
        const int full = len / kSparseBlock;
        if (len > 0 && len % kSparseBlock != 0 && full < a.max_blocks) {
          src_block = a.page_table[s * a.pt_row_stride + full];
          if (src_block >= a.num_blocks) set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
          want = src_block >= 0 && src_block < a.num_blocks;
        }
      }
    }
    const int id = take_free(want, a.ref_counts, a.num_blocks, &cursor, list, warp_sums);
    if (i < a.n) {
      if (want && id < 0) {
        set_err(a.err_word, PBS_DEVERR_NO_BLOCK);
        state = -3;  // the child becomes an empty row
      }
      a.copy_src[i] = want && id >= 0 ? src_block : -1;
      a.copy_dst[i] = want && id >= 0 ? id : state;
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const BlockArgs a) {
  __shared__ int list[kPlanThreads];
  __shared__ int warp_sums[32];
  __shared__ int start[kPlanThreads + 1];  // first flat entry of each row of the batch
  __shared__ int missing[kPlanThreads];
  int cursor = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int t = static_cast<int>(threadIdx.x), i = i0 + t;
    int row = -1, first = 0, count = 0, add = 0;
    bool bad = false;
    if (i < a.n) {
      row = __ldg(a.dst_rows + i);
      add = __ldg(a.new_tokens + i);
      if (row < 0 || row >= a.num_rows || add < 0) {
        bad = true;
      } else if (add > 0) {
        const int64_t len = a.seq_lens[row];
        const int64_t end = (len + add + kSparseBlock - 1) / kSparseBlock;
        if (len < 0 || end > a.max_blocks) bad = true;
        else {
          first = static_cast<int>(len / kSparseBlock);
          count = static_cast<int>(end) - first;
        }
      }
      if (bad) set_err(a.err_word, PBS_DEVERR_TABLE);
    }
    int total;
    start[t] = block_scan(count, &total, warp_sums);
    missing[t] = 0;
    if (t == 0) start[kPlanThreads] = total;
    __syncthreads();
    for (int f0 = 0; f0 < total; f0 += kPlanThreads) {
      const int f = f0 + t;
      bool want = false;
      int owner = 0;
      int32_t* entry = nullptr;
      if (f < total) {
        // last row whose first entry is <= f (rows without entries share their successor's start)
        int lo = 0, hi = kPlanThreads;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (start[mid] <= f) lo = mid; else hi = mid;
        }
        owner = lo;
        const int r = __ldg(a.dst_rows + i0 + owner);
        const int b = a.seq_lens[r] / kSparseBlock + (f - start[owner]);
        entry = a.page_table + r * a.pt_row_stride + b;
        want = *entry < 0;
      }
      const int id = take_free(want, a.ref_counts, a.num_blocks, &cursor, list, warp_sums);
      if (want) {
        if (id >= 0) *entry = id;
        else {
          set_err(a.err_word, PBS_DEVERR_NO_BLOCK);
          missing[owner] = 1;
        }
      }
    }
    __syncthreads();
    // lengths move only now: the loop above reads the old ones
    if (row >= 0 && !bad && add > 0 && missing[t] == 0) a.seq_lens[row] += add;
    __syncthreads();
  }
}

// One block of every layer per pair (src, dst), in pieces of kPiece bytes.
__device__ __forceinline__ void copy_pairs(const BlockArgs& a, const int32_t* src, const int32_t* dst, int count) {
  const int64_t units = static_cast<int64_t>(a.block_page_stride) / a.pages_per_unit;  // contiguous runs of a block
  const int64_t pieces = (a.unit_bytes + kPiece - 1) / kPiece;
  const int64_t items = static_cast<int64_t>(count) * a.num_layers * units * pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    int64_t x = it;
    const int64_t piece = x % pieces;
    x /= pieces;
    const int64_t unit = x % units;
    x /= units;
    const int64_t layer = x % a.num_layers;
    const int p = static_cast<int>(x / a.num_layers);
    const int s = src[p], d = dst[p];
    if (s < 0 || d < 0 || s == d) continue;
    if (s >= a.num_blocks || d >= a.num_blocks) {
      if (threadIdx.x == 0) set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
      continue;
    }
    const int64_t in_unit = unit * a.pages_per_unit * a.page_stride_bytes + piece * kPiece;
    const int64_t block_bytes = static_cast<int64_t>(a.block_page_stride) * a.page_stride_bytes;
    const uint8_t* from = a.kv_cache + layer * a.layer_stride_bytes + s * block_bytes + in_unit;
    uint8_t* to = a.kv_cache + layer * a.layer_stride_bytes + d * block_bytes + in_unit;
    const int64_t left = a.unit_bytes - piece * kPiece;
    const int n16 = static_cast<int>((left < kPiece ? left : kPiece) / 16);
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int c = u * kCopyThreads + static_cast<int>(threadIdx.x);
      if (c < n16) v[u] = __ldcs(reinterpret_cast<const uint4*>(from) + c);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int c = u * kCopyThreads + static_cast<int>(threadIdx.x);
      if (c < n16) __stcs(reinterpret_cast<uint4*>(to) + c, v[u]);
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const BlockArgs a) {
  copy_pairs(a, a.src_rows, a.dst_rows, a.n);
}

// Fork, second launch: the children's table rows, the shared blocks' counts, the tails' bytes.
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const BlockArgs a) {
  pdl_wait();
  const int64_t entries = static_cast<int64_t>(a.n) * a.max_blocks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries; e += step) {
    const int i = static_cast<int>(e / a.max_blocks), b = static_cast<int>(e % a.max_blocks);
    const int tail = a.copy_dst[i];
    if (tail == -2) continue;  // not rows of the table
    const int s = __ldg(a.src_rows + i), d = __ldg(a.dst_rows + i);
    const int len = tail == -3 ? 0 : a.seq_lens[s];
    const int full = len / kSparseBlock;
    int id = -1;
    if (b < full) {
      id = a.page_table[s * a.pt_row_stride + b];
      if (id >= a.num_blocks) {
        set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
        id = -1;
      }
      if (id >= 0) atomicAdd(a.ref_counts + id, 1);
      else id = -1;
    } else if (b == full) {
      id = tail >= 0 ? tail : -1;
    }
    a.page_table[d * a.pt_row_stride + b] = id;
    if (b == 0) a.seq_lens[d] = len;
  }
  copy_pairs(a, a.copy_src, a.copy_dst, a.n);
}

__global__ void __launch_bounds__(kCopyThreads) release_kernel(const BlockArgs a) {
  const int64_t entries = static_cast<int64_t>(a.n) * a.max_blocks;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  if (e >= entries) return;
  const int i = static_cast<int>(e / a.max_blocks), b = static_cast<int>(e % a.max_blocks);
  const int row = __ldg(a.dst_rows + i);
  if (row < 0 || row >= a.num_rows) {
    if (b == 0) set_err(a.err_word, PBS_DEVERR_TABLE);
    return;
  }
  if (a.window > 0) {
    // only blocks that no query at position seq_len or later sees: its keys n have
    // num_sinks <= n <= seq_len - window
    const int64_t key0 = static_cast<int64_t>(b) * kSparseBlock;
    if (key0 < a.num_sinks || key0 + kSparseBlock - 1 > static_cast<int64_t>(a.seq_lens[row]) - a.window) return;
  }
  // an exchange: a row listed twice gives each block back once
  const int id = atomicExch(a.page_table + row * a.pt_row_stride + b, -1);
  if (a.window <= 0 && b == 0) a.seq_lens[row] = 0;
  if (id < 0) return;
  if (id >= a.num_blocks) {
    set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
    return;
  }
  if (atomicSub(a.ref_counts + id, 1) <= 0) {
    atomicAdd(a.ref_counts + id, 1);
    set_err(a.err_word, PBS_DEVERR_TABLE);
  }
}

// Compact, first launch. Live blocks at ids >= n_live (movers, ascending) take the free ids below
// n_live (holes, ascending); there are as many of the one as of the other. copy_src / copy_dst: the
// pairs; remap: every block's new id (-1: free).
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const BlockArgs a) {
  pdl_release();
  __shared__ int warp_sums[32];
  const int t = static_cast<int>(threadIdx.x);
  int mine = 0;
  for (int id0 = t * kIdsPerThread; id0 < a.num_blocks; id0 += kIdsPerStep) {
    int r[kIdsPerThread];
    load_refs(a.ref_counts, a.num_blocks, id0, r);
#pragma unroll
    for (int i = 0; i < kIdsPerThread; ++i) mine += r[i] > 0;
  }
  int n_live;
  block_scan(mine, &n_live, warp_sums);
  int holes = 0, movers = 0;
  for (int base = 0; base < a.num_blocks; base += kIdsPerStep) {
    const int id0 = base + t * kIdsPerThread;
    int r[kIdsPerThread];
    load_refs(a.ref_counts, a.num_blocks, id0, r);
    int nh = 0, nm = 0;
#pragma unroll
    for (int i = 0; i < kIdsPerThread; ++i) {
      if (id0 + i >= a.num_blocks) continue;
      nh += r[i] <= 0 && id0 + i < n_live;
      nm += r[i] > 0 && id0 + i >= n_live;
    }
    // a step has at most 4096 of each: both counts in one scan
    int both;
    const int before = block_scan(nh | (nm << 16), &both, warp_sums);
    int h = holes + (before & 0xffff), m = movers + (before >> 16);
#pragma unroll
    for (int i = 0; i < kIdsPerThread; ++i) {
      const int id = id0 + i;
      if (id >= a.num_blocks) continue;
      if (r[i] <= 0 && id < n_live) a.copy_dst[h++] = id;
      if (r[i] > 0 && id >= n_live) a.copy_src[m++] = id;
      a.remap[id] = r[i] > 0 ? id : -1;
    }
    holes += both & 0xffff;
    movers += both >> 16;
  }
  __syncthreads();
  for (int p = t; p < movers; p += kPlanThreads) a.remap[a.copy_src[p]] = a.copy_dst[p];
  if (t == 0) {
    a.counts[0] = n_live;
    a.counts[1] = movers;
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const BlockArgs a) {
  pdl_wait();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  const int moves = a.counts[1];
  for (int64_t p = t0; p < moves; p += step) {
    const int s = a.copy_src[p], d = a.copy_dst[p];
    a.ref_counts[d] = a.ref_counts[s];
    a.ref_counts[s] = 0;
  }
  const int64_t entries = static_cast<int64_t>(a.num_rows) * a.max_blocks;
  for (int64_t e = t0; e < entries; e += step) {
    int32_t* entry = a.page_table + (e / a.max_blocks) * a.pt_row_stride + e % a.max_blocks;
    const int id = *entry;
    if (id < 0) continue;
    if (id >= a.num_blocks) {
      set_err(a.err_word, PBS_DEVERR_BLOCK_OOB);
      continue;
    }
    const int to = a.remap[id];
    if (to < 0) set_err(a.err_word, PBS_DEVERR_TABLE);  // the row names a free block
    if (to != id) *entry = to;
  }
  copy_pairs(a, a.copy_src, a.copy_dst, moves);
}

// CTAs of an apply kernel: enough to hold ~64 KiB of loads per SM in flight.
unsigned copy_grid(const BlockArgs& a, int64_t max_pairs) {
  const int64_t units = a.block_page_stride / a.pages_per_unit;
  const int64_t items = max_pairs * a.num_layers * units * ((a.unit_bytes + kPiece - 1) / kPiece);
  const int64_t most = 152 * 6;
  return static_cast<unsigned>(items < 1 ? 1 : items < most ? items : most);
}

}  // namespace

cudaError_t launch_copy_blocks(const BlockArgs& a, cudaStream_t stream) {
  copy_kernel<<<copy_grid(a, a.n), kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_reserve_blocks(const BlockArgs& a, cudaStream_t stream) {
  reserve_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_fork(const BlockArgs& a, cudaStream_t stream) {
  fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_second(fork_apply_kernel, copy_grid(a, a.n), kCopyThreads, 0, stream, a);
}

cudaError_t launch_release(const BlockArgs& a, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(a.n) * a.max_blocks;
  release_kernel<<<static_cast<unsigned>((entries + kCopyThreads - 1) / kCopyThreads), kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_compact(const BlockArgs& a, cudaStream_t stream) {
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_second(compact_apply_kernel, copy_grid(a, a.num_blocks / 2 + 1), kCopyThreads, 0, stream, a);
}

}  // namespace pbs
