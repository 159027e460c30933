// Block tables, slot maps and positions built on the GPU from request
// lengths, with the free blocks on a device-resident stack.
//
// "GPU 学习日报 Day 28" §二 (KV Cache Manager: block tables and a free list)
// and §4.2 (blocks are taken on demand, one when the previous one is full):
// the arithmetic of the host pool for sequences that share no partly filled
// block, done where the decode step runs, so that a step needs no upload.
//
// For row s holding L_s tokens and getting n_s more, with exclusive sums
// over the rows
//     old_s = ceil(L_s / 16),  need_s = ceil((L_s + n_s) / 16) - old_s,
//     Q_s = sum n,             B_s = sum need,
// the row's i-th new block is free[count - 1 - (B_s + i)] (the top of the
// stack first), and its token t (Q_s <= t < Q_s + n_s) stands at position
// p = L_s + t - Q_s in slot table[s][p / 16] * 16 + p % 16.
//
// What bounds it: latency. A decode step reads and writes a few KB; the two
// exclusive sums over the rows are the only dependence. Every CTA of one
// cluster scans all the rows itself (two integers a row, from L2), so no
// partial sums travel between CTAs; a cluster barrier stands between the
// last read and the first write of the lengths and the count, which the
// caller may update in place.
#pragma once

#include "decode.cuh"

namespace pa {

constexpr int kTabThreads = 1024;
constexpr int kTabCluster = 8;            // CTAs of the (one) cluster
constexpr int kTabMaxSeqs = 16384;        // rows whose sums one CTA's shared memory holds
constexpr int kTokThreads = 256;
constexpr int kTokPerThread = 4;

constexpr uint32_t kErrOutOfBlocks = 0x20u;
constexpr uint32_t kErrLengthRange = 0x40u;
constexpr uint32_t kErrFreeRange = 0x80u;

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Exclusive sums over the block's threads of two 64-bit counts (tokens of
// up to 16384 rows can pass 32 bits); the totals go to every thread.
struct Two {
  int64_t a, b;
};
__device__ __forceinline__ Two block_exclusive_sum(Two v, Two &total) {
  __shared__ Two s_warp[kTabThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Two x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, x.a, o), b = __shfl_up_sync(0xffffffffu, x.b, o);
    if (lane >= o) {
      x.a += a;
      x.b += b;
    }
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Two w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, w.a, o), b = __shfl_up_sync(0xffffffffu, w.b, o);
      if (lane >= o) {
        w.a += a;
        w.b += b;
      }
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  total = s_warp[kTabThreads / 32 - 1];
  const Two before = warp ? s_warp[warp - 1] : Two{0, 0};
  return Two{before.a + x.a - v.a, before.b + x.b - v.b};
}

// Largest index i in [lo, hi) with start[i] <= v (start ascending,
// start[lo] <= v).
template <typename P>
__device__ __forceinline__ int last_not_above(P start, int lo, int hi, int v) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct ExtendParams {
  int32_t *block_tables;        // [S][W], new entries written
  const int32_t *context_lens;  // [S]; may be context_lens_out
  const int32_t *new_lens;      // [S]
  const int32_t *free_blocks;   // [free_capacity]
  const int32_t *free_count;    // [1]; may be free_count_out
  int32_t *context_lens_out;
  int32_t *free_count_out;
  int64_t *slot_mapping;        // [num_tokens]
  int32_t *positions;           // [num_tokens]
  int32_t *query_start;         // [S + 1]
  int max_blocks_per_seq;
  int num_seqs;
  int num_tokens;
  int num_blocks;               // pool size: ids are checked against it
  int free_capacity;
};

// Lengths, count and new table entries: one cluster. Shared memory holds
// the rows' exclusive block sums.
__global__ void __launch_bounds__(kTabThreads) extend_rows_kernel(const ExtendParams p) {
  extern __shared__ int32_t s_first[];  // [S + 1] blocks needed by earlier rows
  const int S = p.num_seqs;
  const int per = (S + kTabThreads - 1) / kTabThreads;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  const int64_t row_cap = static_cast<int64_t>(p.max_blocks_per_seq) * kBS;
  Two mine{0, 0};
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    const int64_t L = p.context_lens[s], n = p.new_lens[s];
    bad |= L < 0 || n < 0 || L + n > row_cap;
    mine.a += n;
    mine.b += (L + n + kBS - 1) / kBS - (L + kBS - 1) / kBS;
  }
  const int count = *p.free_count;
  Two total;
  const Two first = block_exclusive_sum(mine, total);
  const bool length_bad = __syncthreads_or(bad) || total.a > p.num_tokens;
  const bool count_bad = count < 0 || count > p.free_capacity;
  const bool short_of = !length_bad && !count_bad && total.b > count;
  const bool ok = !length_bad && !count_bad && !short_of;
  const uint32_t rank = cluster_rank();
  if (!ok && rank == 0 && threadIdx.x == 0)
    raise_error((length_bad ? kErrLengthRange : 0u) | (count_bad ? kErrFreeRange : 0u) |
                (short_of ? kErrOutOfBlocks : 0u));
  // the rows' sums; with nothing to do every sum is zero
  int64_t q = first.a, b = first.b;
  for (int s = s0; s < s1; ++s) {
    s_first[s] = ok ? static_cast<int>(b) : 0;
    if (rank == 0) p.query_start[s] = ok ? static_cast<int>(q) : 0;
    const int64_t L = p.context_lens[s], n = p.new_lens[s];
    q += n;
    b += (L + n + kBS - 1) / kBS - (L + kBS - 1) / kBS;
  }
  const int blocks = ok ? static_cast<int>(total.b) : 0;
  if (threadIdx.x == 0) {
    s_first[S] = blocks;
    if (rank == 0) p.query_start[S] = ok ? static_cast<int>(total.a) : 0;
  }
  __syncthreads();
  // new table entries, the cluster's threads side by side over the blocks
  for (int k = rank * kTabThreads + threadIdx.x; k < blocks; k += kTabCluster * kTabThreads) {
    const int s = last_not_above(s_first, 0, S, k);
    const int old = (p.context_lens[s] + kBS - 1) / kBS;
    p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq + old + k - s_first[s]] =
        p.free_blocks[count - 1 - k];
  }
  cluster_sync_all();  // every CTA has read the lengths and the count
  if (rank == 0) {
    for (int s = threadIdx.x; s < S; s += kTabThreads)
      p.context_lens_out[s] = p.context_lens[s] + (ok ? p.new_lens[s] : 0);
    if (threadIdx.x == 0) *p.free_count_out = count - blocks;
  }
}

// Slots and positions, four consecutive tokens a thread.
__global__ void __launch_bounds__(kTokThreads) extend_tokens_kernel(const ExtendParams p) {
  const int S = p.num_seqs;
  const int total = p.query_start[S];
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kTokThreads + threadIdx.x) * kTokPerThread;
  int s = -1, end = -1;
  for (int64_t t64 = t0; t64 < min(t0 + kTokPerThread, static_cast<int64_t>(p.num_tokens)); ++t64) {
    const int t = static_cast<int>(t64);
    int64_t slot = -1;
    int pos = 0;
    if (t < total) {
      if (t >= end) {
        s = last_not_above(p.query_start, 0, S, t);
        end = p.query_start[s + 1];
      }
      pos = p.context_lens_out[s] - (end - t);
      const int id = p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq + pos / kBS];
      if (id >= 0 && id < p.num_blocks)
        slot = static_cast<int64_t>(id) * kBS + pos % kBS;
      else
        raise_error(kErrBlockRange);
    }
    p.slot_mapping[t] = slot;
    p.positions[t] = pos;
  }
}

struct ReleaseParams {
  const int32_t *block_tables;  // [S][W]
  const int32_t *context_lens;  // [S]; may be context_lens_out
  const int32_t *release;       // [S], non-zero: the row ends
  int32_t *free_blocks;         // [free_capacity], pushed to
  const int32_t *free_count;    // [1]; may be free_count_out
  int32_t *context_lens_out;
  int32_t *free_count_out;
  int max_blocks_per_seq;
  int num_seqs;
  int num_blocks;
  int free_capacity;
  int keep_blocks;
};

__device__ __forceinline__ int64_t released_blocks(const ReleaseParams &p, int s) {
  if (p.release[s] == 0) return 0;
  const int64_t held = (static_cast<int64_t>(p.context_lens[s]) + kBS - 1) / kBS;
  return held > p.keep_blocks ? held - p.keep_blocks : 0;
}

// Ended rows give back the blocks behind their first keep_blocks, row by
// row, in table order.
__global__ void __launch_bounds__(kTabThreads) release_rows_kernel(const ReleaseParams p) {
  extern __shared__ int32_t s_first[];  // [S + 1] blocks pushed by earlier rows
  const int S = p.num_seqs;
  const int per = (S + kTabThreads - 1) / kTabThreads;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  Two mine{0, 0};
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    const int64_t L = p.context_lens[s];
    bad |= p.release[s] != 0 && (L < 0 || L > static_cast<int64_t>(p.max_blocks_per_seq) * kBS);
    mine.b += released_blocks(p, s);
  }
  const int count = *p.free_count;
  Two total;
  const Two first = block_exclusive_sum(mine, total);
  const bool length_bad = __syncthreads_or(bad);
  const bool count_bad =
      count < 0 || count > p.free_capacity || (!length_bad && count + total.b > p.free_capacity);
  const bool ok = !length_bad && !count_bad;
  const uint32_t rank = cluster_rank();
  if (!ok && rank == 0 && threadIdx.x == 0)
    raise_error((length_bad ? kErrLengthRange : 0u) | (count_bad ? kErrFreeRange : 0u));
  int64_t b = first.b;
  for (int s = s0; s < s1; ++s) {
    s_first[s] = ok ? static_cast<int>(b) : 0;
    b += released_blocks(p, s);
  }
  const int blocks = ok ? static_cast<int>(total.b) : 0;
  if (threadIdx.x == 0) s_first[S] = blocks;
  __syncthreads();
  // one warp a row, the cluster's warps side by side
  const int lane = threadIdx.x & 31;
  bool bad_id = false;
  for (int s = rank * (kTabThreads / 32) + (threadIdx.x >> 5); s < S;
       s += kTabCluster * (kTabThreads / 32)) {
    const int n = s_first[s + 1] - s_first[s];
    const int32_t *row = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + p.keep_blocks;
    for (int i = lane; i < n; i += 32) {
      const int id = row[i];
      bad_id |= id < 0 || id >= p.num_blocks;
      p.free_blocks[count + s_first[s] + i] = id;
    }
  }
  if (bad_id) raise_error(kErrBlockRange);
  cluster_sync_all();  // every CTA has read the lengths and the count
  if (rank == 0) {
    for (int s = threadIdx.x; s < S; s += kTabThreads) {
      const int L = p.context_lens[s];
      p.context_lens_out[s] =
          (ok && p.release[s] != 0)
              ? static_cast<int>(min(static_cast<int64_t>(L), static_cast<int64_t>(p.keep_blocks) * kBS))
              : L;
    }
    if (threadIdx.x == 0) *p.free_count_out = count + blocks;
  }
}

}  // namespace pa
