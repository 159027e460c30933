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
// What bounds it: latency for a decode step (a few KB), the slots' and
// positions' 12 bytes a token for large admissions. The two exclusive sums
// over the rows are the only dependence: every CTA scans all the rows itself
// (two integers a row, from L2) into shared memory, where the row of a token
// or a block is then found by bisection, so no partial sums travel between
// CTAs. The lengths and the count may be updated in place, so they are
// written only when no CTA reads them any more: a small call is one CTA with
// a barrier between, a large one a launch over the GPU for the tokens and a
// one-CTA launch for the lengths and the count (TablePhase).
#pragma once

#include "decode.cuh"
#include "ptx_step.cuh"

namespace pa {

constexpr int kTabThreads = 1024;
constexpr int kTabMaxSeqs = 16384;        // rows whose sums one CTA's shared memory holds
constexpr int kTabBatch = 4;              // tokens or blocks of a thread in flight
constexpr int kTabPerCta = kTabThreads * kTabBatch;   // of a CTA of kTabThreads
constexpr int kTabSmallTokens = 2 * kTabPerCta;   // extend: one CTA up to here
constexpr int kTabSmallBlocks = 8 * kTabPerCta;   // release: one CTA up to this bound of its pushes

constexpr uint32_t kErrOutOfBlocks = 0x20u;
constexpr uint32_t kErrLengthRange = 0x40u;
constexpr uint32_t kErrFreeRange = 0x80u;

enum class TablePhase {
  kAll,     // one CTA
  kWork,    // any number of CTAs: everything but the lengths and the count
  kFinish,  // one CTA, after kWork: the lengths and the count
};

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
    Two w = lane < blockDim.x / 32 ? s_warp[lane] : Two{0, 0};
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
  total = s_warp[blockDim.x / 32 - 1];
  const Two before = warp ? s_warp[warp - 1] : Two{0, 0};
  return Two{before.a + x.a - v.a, before.b + x.b - v.b};
}

// For each v[i]: the largest index k in [0, n) with start[k] <= v[i] (start
// ascending, start[0] <= v[i]). A fixed number of halvings, the searches side
// by side.
template <int N>
__device__ __forceinline__ void last_not_above(const int32_t *start, int n, const int (&v)[N], int (&k)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) k[i] = 0;
  for (int step = n <= 1 ? 0 : 1 << (31 - __clz(n - 1)); step > 0; step >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = k[i] + step;
      if (c < n && start[c] <= v[i]) k[i] = c;
    }
  }
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
  bool wide;                    // slot_mapping is 32-byte, positions 16-byte aligned
};

template <TablePhase PHASE>
__global__ void __launch_bounds__(kTabThreads) extend_kernel(const ExtendParams p) {
  extern __shared__ int32_t s_rows[];
  const int S = p.num_seqs;
  int32_t *s_query = s_rows;           // [S + 1] tokens of earlier rows
  int32_t *s_first = s_query + S + 1;  // [S] blocks needed by earlier rows
  int32_t *s_len = s_first + S;        // [S]
  const int per = (S + blockDim.x - 1) / blockDim.x;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  const int64_t row_cap = static_cast<int64_t>(p.max_blocks_per_seq) * kBS;
  const int count = *p.free_count;
  auto need = [](int64_t L, int64_t n) { return (L + n + kBS - 1) / kBS - (L + kBS - 1) / kBS; };
  Two mine{0, 0};
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    const int64_t L = p.context_lens[s], n = p.new_lens[s];
    bad |= L < 0 || n < 0 || L + n > row_cap;
    mine.a += n;
    mine.b += need(L, n);
  }
  Two total;
  const Two first = block_exclusive_sum(mine, total);
  const bool length_bad = __syncthreads_or(bad) || total.a > p.num_tokens;
  const bool count_bad = count < 0 || count > p.free_capacity;
  const bool short_of = !length_bad && !count_bad && total.b > count;
  const bool ok = !length_bad && !count_bad && !short_of;
  if (PHASE != TablePhase::kWork) {
    if (!ok && threadIdx.x == 0)
      raise_error((length_bad ? kErrLengthRange : 0u) | (count_bad ? kErrFreeRange : 0u) |
                  (short_of ? kErrOutOfBlocks : 0u));
  }
  if (PHASE != TablePhase::kFinish) {
    // the rows' sums; where nothing is to be done no token is live
    const int tokens = ok ? static_cast<int>(total.a) : 0;
    int64_t q = first.a, b = first.b;
    for (int s = s0; s < s1; ++s) {
      const int64_t L = p.context_lens[s], n = p.new_lens[s];
      s_query[s] = ok ? static_cast<int>(q) : 0;
      s_first[s] = static_cast<int>(b);
      s_len[s] = static_cast<int>(L);
      if (blockIdx.x == 0) p.query_start[s] = ok ? static_cast<int>(q) : 0;
      q += n;
      b += need(L, n);
    }
    if (threadIdx.x == 0) {
      s_query[S] = tokens;
      if (blockIdx.x == 0) p.query_start[S] = tokens;
    }
    __syncthreads();
    bool bad_id = false;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x * kTabBatch;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * kTabBatch;
         t0 < p.num_tokens; t0 += stride) {
      // four consecutive tokens: their rows, then their block ids, then the stores
      int pos[kTabBatch], id[kTabBatch];
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i) {
        pos[i] = 0;
        id[i] = -1;
      }
      const int live = static_cast<int>(min(static_cast<int64_t>(kTabBatch), tokens - t0));  // <= 0: padding
      // the id of block j of row s, from its table or the stack; a new
      // block's entry is written by the thread of its first token
      auto block_id = [&](int s, int j, int old, bool starts) {
        int32_t *entry = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + j;
        if (j < old) return *entry;
        const int b = p.free_blocks[count - 1 - (s_first[s] + j - old)];
        if (starts) *entry = b;
        return b;
      };
      if (live > 0) {
        const int v[1] = {static_cast<int>(t0)};
        int k[1] = {-1};
        // rows of few tokens are looked up one token at a time
        if (p.num_tokens > kTabBatch * S) last_not_above(s_query, S, v, k);
        if (k[0] >= 0 && v[0] + live <= s_query[k[0] + 1]) {  // one row: its positions follow one another, in two blocks at most
          const int s = k[0], L = s_len[s], old = (L + kBS - 1) / kBS;
          const int p0 = L + v[0] - s_query[s], off = p0 % kBS, next = (p0 + live - 1) / kBS;
          const int id0 = block_id(s, p0 / kBS, old, off == 0);
          const int id1 = next != p0 / kBS ? block_id(s, next, old, true) : id0;
#pragma unroll
          for (int i = 0; i < kTabBatch; ++i)
            if (i < live) {
              pos[i] = p0 + i;
              id[i] = off + i < kBS ? id0 : id1;
            }
        } else {
          int t[kTabBatch], s[kTabBatch];
#pragma unroll
          for (int i = 0; i < kTabBatch; ++i) t[i] = v[0] + min(i, live - 1);
          last_not_above(s_query, S, t, s);
#pragma unroll
          for (int i = 0; i < kTabBatch; ++i)
            if (i < live) {
              const int L = s_len[s[i]];
              pos[i] = L + t[i] - s_query[s[i]];
              id[i] = block_id(s[i], pos[i] / kBS, (L + kBS - 1) / kBS, pos[i] % kBS == 0);
            }
        }
      }
      int64_t slot[kTabBatch];
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i) {
        const bool in_pool = id[i] >= 0 && id[i] < p.num_blocks;
        bad_id |= i < live && !in_pool;
        slot[i] = in_pool ? static_cast<int64_t>(id[i]) * kBS + pos[i] % kBS : -1;
      }
      if (p.wide && t0 + kTabBatch <= p.num_tokens) {  // whole sectors
        uint32_t w[2 * kTabBatch];
#pragma unroll
        for (int i = 0; i < kTabBatch; ++i) {
          w[2 * i] = static_cast<uint32_t>(slot[i]);
          w[2 * i + 1] = static_cast<uint32_t>(slot[i] >> 32);
        }
        st_global_v8(p.slot_mapping + t0, w);
        *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int i = 0; i < kTabBatch; ++i)
          if (t0 + i < p.num_tokens) {
            p.slot_mapping[t0 + i] = slot[i];
            p.positions[t0 + i] = pos[i];
          }
      }
    }
    if (bad_id) raise_error(kErrBlockRange);
  }
  if (PHASE != TablePhase::kWork) {
    if (PHASE == TablePhase::kAll) __syncthreads();
    if (PHASE == TablePhase::kFinish) wait_for_primary();
    for (int s = s0; s < s1; ++s)  // the rows this thread alone has read
      p.context_lens_out[s] = p.context_lens[s] + (ok ? p.new_lens[s] : 0);
    if (threadIdx.x == 0) *p.free_count_out = count - (ok ? static_cast<int>(total.b) : 0);
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
template <TablePhase PHASE>
__global__ void __launch_bounds__(kTabThreads) release_kernel(const ReleaseParams p) {
  extern __shared__ int32_t s_first[];  // [S] blocks pushed by earlier rows
  const int S = p.num_seqs;
  const int per = (S + blockDim.x - 1) / blockDim.x;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  const int count = *p.free_count;
  Two mine{0, 0};
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    const int64_t L = p.context_lens[s];
    bad |= p.release[s] != 0 && (L < 0 || L > static_cast<int64_t>(p.max_blocks_per_seq) * kBS);
    mine.b += released_blocks(p, s);
  }
  Two total;
  const Two first = block_exclusive_sum(mine, total);
  const bool length_bad = __syncthreads_or(bad);
  const bool count_bad =
      count < 0 || count > p.free_capacity || (!length_bad && count + total.b > p.free_capacity);
  const bool ok = !length_bad && !count_bad;
  const int blocks = ok ? static_cast<int>(total.b) : 0;
  if (PHASE != TablePhase::kFinish) {
    int64_t b = first.b;
    for (int s = s0; s < s1; ++s) {
      s_first[s] = static_cast<int>(b);
      b += released_blocks(p, s);
    }
    __syncthreads();
    const int stride = gridDim.x * blockDim.x;
    bool bad_id = false;
    for (int64_t k0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; k0 < blocks; k0 += kTabBatch * stride) {
      int k[kTabBatch], s[kTabBatch], id[kTabBatch];
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i) k[i] = static_cast<int>(min(k0 + i * stride, static_cast<int64_t>(blocks - 1)));
      last_not_above(s_first, S, k, s);
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i)
        id[i] = p.block_tables[static_cast<int64_t>(s[i]) * p.max_blocks_per_seq + p.keep_blocks + k[i] - s_first[s[i]]];
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i)
        if (k0 + i * stride < blocks) {
          bad_id |= id[i] < 0 || id[i] >= p.num_blocks;
          p.free_blocks[count + k[i]] = id[i];
        }
    }
    if (bad_id) raise_error(kErrBlockRange);
  }
  if (PHASE != TablePhase::kWork) {
    if (!ok && threadIdx.x == 0)
      raise_error((length_bad ? kErrLengthRange : 0u) | (count_bad ? kErrFreeRange : 0u));
    if (PHASE == TablePhase::kAll) __syncthreads();
    if (PHASE == TablePhase::kFinish) wait_for_primary();
    for (int s = s0; s < s1; ++s) {  // the rows this thread alone has read
      const int64_t L = p.context_lens[s];
      p.context_lens_out[s] = static_cast<int>(
          (ok && p.release[s] != 0) ? min(L, static_cast<int64_t>(p.keep_blocks) * kBS) : L);
    }
    if (threadIdx.x == 0) *p.free_count_out = count + blocks;
  }
}

}  // namespace pa
