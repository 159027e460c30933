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
// What bounds it. A decode step moves a few KB: the chain launch, lengths,
// sums, ids, stores (3.2 us for 128 rows of one token, in a graph). A large
// admission writes 12 bytes a token (4.7 us at the copy rate for 2.6 million
// tokens of 2000 rows), but spends its time on issuing instructions, about
// 100 a token: 16 us, of which the sums take 4. The two exclusive sums over the rows are
// the only dependence: every CTA scans all the rows itself (two integers a
// row, from L2) into shared memory, where the row of a token or a block is
// then found by bisection, so no partial sums travel between CTAs. A thread
// takes four neighbours, which mostly are of one row: one search, one or two
// ids (all read before an entry is stored, since a store between them would
// hold the next read back), whole sectors out.
//
// The lengths and the count may be updated in place, so they are written
// only when no CTA reads them any more (TablePhase): a small call is one CTA
// with a barrier between, a large one a launch over the GPU for the tokens
// and a one-CTA launch that sums the rows beside it on an SM left free and
// writes the lengths and the count when it has ended. One CTA against two
// launches, in a graph, 128 rows: extend 3.5 us against 3.7 at 2048 tokens,
// 4.4 against 3.9 at 4096; release at a bound of 8192 blocks 3.7 against 3.9
// with few rows ended and 6.6 against 3.9 with all of them, at 16384 3.9 and
// 9.9 against 4.0. The second launch costs the host 2 us, so one CTA is kept
// to 2048 tokens and 8192 blocks.
#pragma once

#include "decode.cuh"
#include "ptx_step.cuh"

namespace pa {

constexpr int kTabThreads = 1024;
constexpr int kTabMaxSeqs = 16384;        // rows whose sums one CTA's shared memory holds
constexpr int kTabBatch = 4;              // tokens or blocks of a thread in flight
constexpr int kTabSmallTokens = 2048;     // extend: one CTA up to here
constexpr int kTabSmallBlocks = 8192;    // release: one CTA up to this bound of its pushes

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
  if (PHASE == TablePhase::kWork) launch_dependents();
  const int S = p.num_seqs;
  int32_t *s_query = s_rows;           // [S + 1] tokens of earlier rows
  int32_t *s_first = s_query + S + 1;  // [S] blocks needed by earlier rows
  int32_t *s_len = s_first + S;        // [S]
  const int per = (S + blockDim.x - 1) / blockDim.x;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  const int64_t row_cap = static_cast<int64_t>(p.max_blocks_per_seq) * kBS;
  const int count = *p.free_count;
  // (of lengths out of range, whose sums are not used, anything)
  auto need = [](uint32_t L, uint32_t n) { return (L + n + kBS - 1) / kBS - (L + kBS - 1) / kBS; };
  Two mine{0, 0};
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    const int L = p.context_lens[s], n = p.new_lens[s];
    bad |= L < 0 || n < 0 || static_cast<int64_t>(L) + n > row_cap;
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
      const int L = p.context_lens[s], n = p.new_lens[s];
      s_query[s] = ok ? static_cast<int>(q) : 0;
      s_first[s] = static_cast<int>(b);
      s_len[s] = L;
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
    const uint32_t total_tokens = p.num_tokens, stride = gridDim.x * blockDim.x * kTabBatch;
    // where the id of block j of row s is read: its table or, behind the
    // row's `old` blocks, the stack
    auto source = [&](int s, uint32_t j, uint32_t old) -> const int32_t * {
      return j < old ? p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + j
                     : p.free_blocks + (count - 1 - s_first[s] - static_cast<int>(j - old));
    };
    auto put_entry = [&](int s, uint32_t j, int id) {
      p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq + j] = id;
    };
    // slot of position x in block id, as two words
    auto put_slot = [&](uint32_t *w, int id, uint32_t x) {
      const bool in_pool = static_cast<uint32_t>(id) < static_cast<uint32_t>(p.num_blocks);
      const uint64_t slot = in_pool ? static_cast<uint64_t>(id) * kBS + x % kBS : ~0ull;
      w[0] = static_cast<uint32_t>(slot);
      w[1] = static_cast<uint32_t>(slot >> 32);
      bad_id |= !in_pool;
    };
    for (uint32_t t0 = (blockIdx.x * blockDim.x + threadIdx.x) * kTabBatch; t0 < total_tokens; t0 += stride) {
      // four consecutive tokens: their rows, then their block ids, then the stores
      uint32_t pos[kTabBatch] = {}, w[2 * kTabBatch];
#pragma unroll
      for (int i = 0; i < 2 * kTabBatch; ++i) w[i] = 0xffffffffu;
      const int live = min(kTabBatch, tokens - static_cast<int>(t0));  // <= 0: padding
      if (live > 0) {
        const int v[1] = {static_cast<int>(t0)};
        int k[1] = {-1};
        // rows of few tokens are looked up one token at a time
        if (total_tokens > static_cast<uint32_t>(kTabBatch) * S) last_not_above(s_query, S, v, k);
        if (k[0] >= 0 && v[0] + live <= s_query[k[0] + 1]) {  // one row: its positions follow one another, in two blocks at most
          const int s = k[0];
          const uint32_t L = s_len[s], old = (L + kBS - 1) / kBS, p0 = L + (t0 - s_query[s]), last = p0 + live - 1;
          const uint32_t j0 = p0 / kBS, j1 = last / kBS;
          // both ids are on their way before an entry is stored
          const int id0 = *source(s, j0, old);
          const int id1 = j1 != j0 ? *source(s, j1, old) : id0;
          // a new block's entry is written by the thread of its first token
          if (p0 % kBS == 0 && j0 >= old) put_entry(s, j0, id0);
          if (j1 != j0 && j1 >= old) put_entry(s, j1, id1);
#pragma unroll
          for (int i = 0; i < kTabBatch; ++i)
            if (i < live) {
              pos[i] = p0 + i;
              put_slot(w + 2 * i, pos[i] / kBS == j0 ? id0 : id1, pos[i]);
            }
        } else {
          int t[kTabBatch], s[kTabBatch], id[kTabBatch];
          uint32_t old[kTabBatch];
#pragma unroll
          for (int i = 0; i < kTabBatch; ++i) t[i] = v[0] + min(i, live - 1);
          if (k[0] >= 0 && v[0] + live <= s_query[min(k[0] + 2, S)]) {  // this row and the next
#pragma unroll
            for (int i = 0; i < kTabBatch; ++i) s[i] = k[0] + (t[i] >= s_query[k[0] + 1]);
          } else {
            last_not_above(s_query, S, t, s);
          }
#pragma unroll
          for (int i = 0; i < kTabBatch; ++i) {
            const uint32_t L = s_len[s[i]];
            old[i] = (L + kBS - 1) / kBS;
            pos[i] = L + (t[i] - s_query[s[i]]);
            id[i] = *source(s[i], pos[i] / kBS, old[i]);
          }
#pragma unroll
          for (int i = 0; i < kTabBatch; ++i)
            if (i < live) {
              const uint32_t j = pos[i] / kBS;
              if (pos[i] % kBS == 0 && j >= old[i]) put_entry(s[i], j, id[i]);
              put_slot(w + 2 * i, id[i], pos[i]);
            } else {
              pos[i] = 0;
            }
        }
      }
      if (p.wide && t0 + kTabBatch <= total_tokens) {  // whole sectors
        st_global_v8(p.slot_mapping + t0, w);
        *reinterpret_cast<uint4 *>(p.positions + t0) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int i = 0; i < kTabBatch; ++i)
          if (t0 + i < total_tokens) {
            p.slot_mapping[t0 + i] = static_cast<int64_t>(static_cast<uint64_t>(w[2 * i + 1]) << 32 | w[2 * i]);
            p.positions[t0 + i] = static_cast<int>(pos[i]);
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
  if (PHASE == TablePhase::kWork) launch_dependents();
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
    const uint32_t stride = gridDim.x * blockDim.x * kTabBatch;
    bool bad_id = false;
    for (uint32_t k0 = (blockIdx.x * blockDim.x + threadIdx.x) * kTabBatch; k0 < static_cast<uint32_t>(blocks); k0 += stride) {
      // four consecutive pushes, mostly of one row or of two neighbours
      const int k = k0, more = min(kTabBatch, blocks - k) - 1;
      const int first_k[1] = {k};
      int r[1];
      last_not_above(s_first, S, first_k, r);
      const int next = r[0] + 1 < S ? s_first[r[0] + 1] : blocks, after = r[0] + 2 < S ? s_first[r[0] + 2] : blocks;
      int s[kTabBatch], id[kTabBatch], kk[kTabBatch];
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i) {
        kk[i] = k + min(i, more);
        s[i] = r[0] + (kk[i] >= next);
      }
      if (k + more >= after) last_not_above(s_first, S, kk, s);
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i)
        id[i] = p.block_tables[static_cast<int64_t>(s[i]) * p.max_blocks_per_seq + p.keep_blocks + kk[i] - s_first[s[i]]];
#pragma unroll
      for (int i = 0; i < kTabBatch; ++i)
        if (i <= more) {
          bad_id |= id[i] < 0 || id[i] >= p.num_blocks;
          p.free_blocks[count + kk[i]] = id[i];
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
