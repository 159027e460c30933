// Decode attention for groups of sequences that share a prefix.
//
// "第 7 章推理框架" §7.1 (前缀共享) and "GPU 学习日报 Day 28" §4.2, §七: the
// sequences behind one system prompt or document hold the same physical
// blocks at the head of their tables. Group g is the sequences
// group_start[g] .. group_start[g+1] - 1; their first prefix_blocks[g] table
// entries agree (the first sequence's are read). For sequence s with
// L = context_lens[s] and P = 16 prefix_blocks[g],
//     out = v_scale (sum_{t<min(L,P)} e_t V_t + sum_{P<=t<L} e_t V_t) / sum e_t,
// e_t = exp(sm_scale k_scale q . K_t): what pa_decode computes.
//
// The prefix kernel (tensor core) takes the rows of a KV head — its group's
// query heads times the group's sequences — as one matrix against a stretch
// of the prefix and leaves records
//     m (log2 units), l = sum 2^(z - m), o = sum 2^(z - m) V
// in the workspace. The suffix kernel streams each sequence's own blocks as
// the plain decode does, launched so that it fills the SMs as the prefix
// kernel leaves them; its parts are records too. The join kernel adds up each
// row's records. A sequence that ends inside its prefix takes its whole context as its own
// part, so that no masked product ever meets a value it must not see (0 * NaN).
//
// Precision. The output is fp32, so the weights 2^(z - m) enter the value
// product as two 16-bit halves (hi = round(p), lo = round(p - hi)): bf16
// against bf16 caches (16 significant bits), f16 against E4M3 widened to f16
// (22 bits). One half alone would leave 2^-9 or 2^-12 of every weight.
#pragma once

#include "decode.cuh"
#include "prefill.cuh"

namespace pa {

constexpr uint32_t kErrGroupRange = 0x100u;

struct SharedParams {
  float *out;                    // [S][Hq][D]
  const uint16_t *q;             // bf16 [S][Hq][D]
  const int32_t *block_tables;   // [S][max_blocks_per_seq]
  const int32_t *context_lens;   // [S]
  const int32_t *group_start;    // [G + 1]
  const int32_t *prefix_blocks;  // [G]
  int max_blocks_per_seq;
  int max_context_len;
  int max_prefix_blocks;
  int max_suffix_len;
  int num_groups;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int group;                     // query heads per KV head
  int num_blocks;
  int tokens_per_tile;           // sequences of a 128-row query tile (128 / group, floor)
  int prefix_parts;              // CTAs along the longest prefix
  int part_records;              // records of a part (kSpRecordTiles)
  int suffix_parts;              // suffix parts, part_len tokens each (the last one to the end)
  int part_len;
  float score_scale;             // sm_scale * log2(e) [* k_scale for fp8]
  float out_scale;               // v_scale for fp8, 1 for bf16
  int row_tiles;                 // CTAs along the prefix rows, two 128-row query tiles each
  // Prefix records, o as 16-byte chunks in the order the tensor memory's
  // rows lie in (thread r writes chunk c at [c][r], whole lines a warp):
  float *pre_o;                  // [prefix_parts * part_records][Hkv][2 row_tiles][D / 4][128][4]
  float2 *pre_ml;                // the same without chunks
  int32_t *row_of;               // [S] a sequence's place among the tiles: tile * tokens_per_tile + place
  // Suffix parts:
  float *suf_o;                  // [suffix_parts][S * Hq][D]
  float2 *suf_ml;                // [suffix_parts][S * Hq]
};

// Flags groups that are not ascending inside the batch, and prefixes outside
// their bound or the table (clamped where they are used). One CTA's threads.
__device__ __forceinline__ void check_groups(const SharedParams &p) {
  bool bad = false;
  for (int g = threadIdx.x; g < p.num_groups; g += blockDim.x) {
    const int a = p.group_start[g], b = p.group_start[g + 1], n = p.prefix_blocks[g];
    bad |= a < 0 || b < a || b > p.num_seqs || n < 0 || n > min(p.max_prefix_blocks, p.max_blocks_per_seq);
  }
  if (bad) raise_error(kErrGroupRange);
}

// The prefix of sequence s's group in blocks (clamped; 0 for a sequence of
// no group).
__device__ __forceinline__ int shared_blocks_of(const SharedParams &p, int s) {
  int lo = 0, hi = p.num_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.group_start[mid] <= s)
      lo = mid;
    else
      hi = mid;
  }
  if (p.num_groups == 0 || s < p.group_start[lo] || s >= p.group_start[lo + 1]) return 0;
  return min(max(p.prefix_blocks[lo], 0), min(p.max_prefix_blocks, p.max_blocks_per_seq));
}

constexpr int kSpRows = 128;                // rows of a query tile (MMA M)
constexpr int kSpKeys = 128;                // keys of a prefix tile (score MMA N)
constexpr int kSpBlocks = kSpKeys / kBS;
// Most key tiles that add into one record. The tensor core's accumulator
// truncates, so a sum over n tiles shrinks by about n * 2.6e-7 of itself
// (measured: 8.3e-6 at 32 tiles); records are added up in fp32 by the join.
constexpr int kSpRecordTiles = 16;

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// How a prefix of `blocks` blocks is cut: parts (CTAs) of `tiles` key tiles,
// each of `records` records of `record_tiles` tiles.
struct PrefixCut {
  int parts, tiles, records, record_tiles;
};
__device__ __forceinline__ PrefixCut cut_prefix(int blocks, int max_parts) {
  PrefixCut c;
  const int all = ceil_div(blocks, kSpBlocks);
  c.tiles = ceil_div(all, max_parts);
  c.parts = ceil_div(all, c.tiles);
  c.records = ceil_div(c.tiles, kSpRecordTiles);
  c.record_tiles = ceil_div(c.tiles, c.records);
  return c;
}

// A sequence's share of the work.
struct SharedRow {
  int shared_blocks;  // its group's prefix; 0 where it takes its whole context itself
  int own_tokens;     // behind them
  int prefix_parts;   // the prefix's parts
  int own_parts;
  bool bad_len;
};

__device__ __forceinline__ SharedRow shared_row(const SharedParams &p, int s) {
  SharedRow r;
  const int L = clamped_len(p.context_lens, s, p.max_context_len, p.max_blocks_per_seq, &r.bad_len);
  int nb = shared_blocks_of(p, s);
  const bool inside = L < nb * kBS;  // ends inside its group's prefix
  if (inside) nb = 0;
  r.shared_blocks = nb;
  r.own_tokens = L - nb * kBS;
  if (!inside && r.own_tokens > p.max_suffix_len) {
    r.own_tokens = p.max_suffix_len;
    r.bad_len = true;
  }
  r.prefix_parts = nb > 0 ? cut_prefix(nb, p.prefix_parts).parts : 0;
  r.own_parts = min(ceil_div(r.own_tokens, p.part_len), p.suffix_parts);
  return r;
}

// Programmatic dependent launch: let the next kernel of the stream start
// beside this one, and wait until the one before has finished (its writes
// visible). Without the launch attribute neither does anything.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------ prefix parts

constexpr int kSpSoftmaxWarps = 8;  // two warpgroups
// Largest sum of 64 weights against an older reference: bf16 halves have
// fp32's range, f16 ones reach 2^16.
constexpr float kSpSumMaxBf16 = 1.0e18f;
constexpr float kSpSumMaxF16 = 32768.f;
constexpr float kSpF16Log2 = 8.f;          // f16 weights are 2^(z - m + 8): small ones keep bits

template <int D, bool FP8>
struct SpPlan {
  static constexpr int kThreads = FP8 ? 512 : 384;
  // setmaxnreg shares, adding up to what the block launches with (128 and
  // 168 registers a thread, four and three warpgroups)
  static constexpr int kSoftmaxRegs = FP8 ? 192 : 208;
  static constexpr int kIssueRegs = 88;
  static constexpr int kConvertRegs = 40;
  static_assert(FP8 ? 2 * kSoftmaxRegs + kIssueRegs + kConvertRegs <= 4 * 128
                    : 2 * kSoftmaxRegs + kIssueRegs <= 3 * 168,
                "register split");
  static constexpr int kIssueWarp0 = kThreads / 32 - 4;  // K (and Q) loads, V loads, two MMA warps
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kSpRows * 128;       // [128 rows][64 elements of 16 bits]
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // a Q, K or V operand tile
  static constexpr int kByteTile = kSpKeys * D;          // a K or V tile of E4M3 bytes
  static constexpr int kNK = 2;
  static constexpr int kNV = FP8 ? 1 : 2;
  static constexpr int kNB = FP8 ? 2 : 0;                // byte stages of K, and of V
  static constexpr int kKOff = 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kNK * kTileBytes;
  static constexpr int kKbOff = kVOff + kNV * kTileBytes;
  static constexpr int kVbOff = kKbOff + kNB * kByteTile;
  static constexpr int kBarOff = kVbOff + kNB * kByteTile;
  // q_full[2] q_conv[2] k_full[NK] k_empty[NK] v_full[NV] v_empty[NV]
  // kb_full[2] kb_empty[2] vb_full[2] vb_empty[2] s_full[2] p_full[2][2] o_half[2] o_done[2] drain[2]
  static constexpr int kNumBars = 4 + 2 * kNK + 2 * kNV + 8 + 10 + 2;
  static constexpr int kSmemBytes = 1024 + kBarOff + 8 * kNumBars + 16;
  static constexpr int kTmemCols = 512;
  static constexpr int kOCol = 2 * kSpKeys;
  static_assert(kOCol + 2 * D <= kTmemCols, "tensor-memory plan");
  static_assert(kSmemBytes <= 227 * 1024, "shared-memory plan");
  static_assert(kNK * kTileBytes >= kSpRows * D * 4, "the K ring holds a tile's output");
};

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// Arrive at named barrier `id` without waiting (its other threads sync).
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Byte of 16-byte chunk c (0..7) of row r in one 64-element half of an
// operand tile (128-byte swizzle).
__device__ __forceinline__ uint32_t op_chunk(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(SpPlan<D, FP8>::kThreads, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap tmap_q,
                         const __grid_constant__ CUtensorMap tmap_k,
                         const __grid_constant__ CUtensorMap tmap_v, const SharedParams p) {
  using PL = SpPlan<D, FP8>;
  constexpr int H = PL::kHalves, NK = PL::kNK, NV = PL::kNV, NB = PL::kNB;
  // K and V loads; the MMAs of slot 0 and of slot 1
  constexpr int kKWarp = PL::kIssueWarp0, kVWarp = kKWarp + 1, kMmaWarp = kKWarp + 2;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;
  uint8_t *base_ptr = smem_raw + (base - raw_u32);
  const uint32_t sq = base, sk = base + PL::kKOff, sv = base + PL::kVOff;
  const uint32_t skb = base + PL::kKbOff, svb = base + PL::kVbOff;
  const uint32_t bar_q = base + PL::kBarOff;          // [tile]
  const uint32_t bar_qc = bar_q + 16;                 // [tile]
  const uint32_t bar_k_full = bar_qc + 16;
  const uint32_t bar_k_empty = bar_k_full + 8 * NK;
  const uint32_t bar_v_full = bar_k_empty + 8 * NK;
  const uint32_t bar_v_empty = bar_v_full + 8 * NV;
  const uint32_t bar_kb_full = bar_v_empty + 8 * NV;
  const uint32_t bar_kb_empty = bar_kb_full + 16;
  const uint32_t bar_vb_full = bar_kb_empty + 16;
  const uint32_t bar_vb_empty = bar_vb_full + 16;
  const uint32_t bar_s_full = bar_vb_empty + 16;      // [tile]
  const uint32_t bar_p_full = bar_s_full + 16;        // [tile][half of the keys]
  const uint32_t bar_o_half = bar_p_full + 32;        // [tile] the first half's product
  const uint32_t bar_o_done = bar_o_half + 16;        // [tile]
  const uint32_t bar_drain = bar_o_done + 16;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(base_ptr + PL::kBarOff + 8 * PL::kNumBars);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);

  const int h = blockIdx.y, part = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpt = p.tokens_per_tile;
  launch_dependents();  // the suffix kernel reads nothing of this one before its end

  // The row pair-tile blockIdx.x of the groups with a prefix, in order:
  // 32 groups at a time, each warp for itself.
  int seq0 = 0, nseq = 0, blocks = 0, first = 0;
  {
    const int cap = min(p.max_prefix_blocks, p.max_blocks_per_seq);
    int before = 0;
    const int x = blockIdx.x;
    for (int gb = 0; gb < p.num_groups; gb += 32) {
      const int g = gb + lane;
      int a = 0, b = 0, nb = 0;
      if (g < p.num_groups) {
        a = min(max(p.group_start[g], 0), p.num_seqs);
        b = min(max(p.group_start[g + 1], a), p.num_seqs);
        nb = min(max(p.prefix_blocks[g], 0), cap);
      }
      const int tiles = nb > 0 ? (b - a + 2 * tpt - 1) / (2 * tpt) : 0;
      int incl = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, x < before + incl);
      if (here) {
        const int src = __ffs(here) - 1;
        const int skip = x - before - __shfl_sync(0xffffffffu, incl - tiles, src);
        first = __shfl_sync(0xffffffffu, a, src);
        blocks = __shfl_sync(0xffffffffu, nb, src);
        seq0 = first + skip * 2 * tpt;
        nseq = min(2 * tpt, __shfl_sync(0xffffffffu, b, src) - seq0);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (nseq <= 0) return;  // no such tile
  const PrefixCut cut = cut_prefix(blocks, p.prefix_parts);
  const int blk0 = part * cut.tiles * kSpBlocks;
  const int nblk = min(blocks - blk0, cut.tiles * kSpBlocks);
  if (nblk <= 0) return;  // no such part of this prefix
  const int nt = ceil_div(nblk, kSpBlocks);
  if (h == 0 && part == 0)
    for (int i = threadIdx.x; i < nseq; i += PL::kThreads) p.row_of[seq0 + i] = blockIdx.x * 2 * tpt + i;
  // One query tile only: both softmax warpgroups take it, with alternate key
  // tiles, and their results are joined at the end.
  const bool alternate = nseq <= tpt;
  const int my_tiles0 = alternate ? (nt + 1) / 2 : nt, my_tiles1 = alternate ? nt / 2 : nt;

  if (threadIdx.x == 0) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar_q + 8u * g, 1);
      mbar_init(bar_qc + 8u * g, 128);
      mbar_init(bar_s_full + 8u * g, 1);
      mbar_init(bar_p_full + 16u * g, 4);  // a warp each
      mbar_init(bar_p_full + 16u * g + 8u, 4);
      mbar_init(bar_drain + 8u * g, 1);
      mbar_init(bar_o_half + 8u * g, 1);
      mbar_init(bar_o_done + 8u * g, 1);
      mbar_init(bar_kb_full + 8u * g, 1);
      mbar_init(bar_kb_empty + 8u * g, 128);
      mbar_init(bar_vb_full + 8u * g, 1);
      mbar_init(bar_vb_empty + 8u * g, 128);
    }
    for (int i = 0; i < NK; ++i) {
      mbar_init(bar_k_full + 8u * i, FP8 ? 128 : 1);
      mbar_init(bar_k_empty + 8u * i, alternate ? 1 : 2);  // both slots read a tile
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(bar_v_full + 8u * i, FP8 ? 128 : 1);
      mbar_init(bar_v_empty + 8u * i, alternate ? 1 : 2);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(s_tmem), PL::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *s_tmem;

  if (warp >= PL::kIssueWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PL::kIssueRegs));
    if (warp == kKWarp || warp == kVWarp) {
      // ------------------------------------------------------- producers
      const bool is_k = warp == kKWarp;
      const int nst = FP8 ? NB : (is_k ? NK : NV);
      const uint32_t ring = FP8 ? (is_k ? skb : svb) : (is_k ? sk : sv);
      const uint32_t stage_bytes = FP8 ? PL::kByteTile : PL::kTileBytes;
      const uint32_t bar_full = FP8 ? (is_k ? bar_kb_full : bar_vb_full) : (is_k ? bar_k_full : bar_v_full);
      const uint32_t bar_empty = FP8 ? (is_k ? bar_kb_empty : bar_vb_empty) : (is_k ? bar_k_empty : bar_v_empty);
      const CUtensorMap *tmap = is_k ? &tmap_k : &tmap_v;
      if (lane == 0) {
        prefetch_tmap(tmap);
        if (is_k) {
          prefetch_tmap(&tmap_q);
          for (int g = 0; g < (alternate ? 1 : 2); ++g) {
            mbar_arrive_expect_tx(bar_q + 8u * g, H * 128 * p.group * tpt);
#pragma unroll
            for (int x = 0; x < H; ++x)
              tma_load_3d(sq + g * PL::kTileBytes + x * PL::kHalfBytes, &tmap_q, bar_q + 8u * g, 64 * x,
                          h * p.group, seq0 + g * tpt);
          }
        }
      }
      const int32_t *bt = p.block_tables + static_cast<int64_t>(first) * p.max_blocks_per_seq + blk0;
      const int total_rows = p.num_blocks * p.num_kv_heads * kBS;
      bool ok = true, bad_id = false;
      int issued = 0, mine = -1;
      for (int j = 0; j < nt && ok; ++j) {
        if ((j & 3) == 0) {  // 32 table entries, four tiles, a load
          const int jb = j * kSpBlocks + lane;
          mine = jb < nblk ? bt[jb] : -1;
        }
        int phys[kSpBlocks];
#pragma unroll
        for (int b = 0; b < kSpBlocks; ++b) phys[b] = __shfl_sync(0xffffffffu, mine, (j & 3) * kSpBlocks + b);
        if (lane == 0) {
          const int st = j % nst;
          if (j >= nst) ok = tc_wait(bar_empty + 8u * st, ((j / nst) - 1) & 1, s_abort);
          if (ok) {
            const uint32_t full = bar_full + 8u * st, dst = ring + st * stage_bytes;
            mbar_arrive_expect_tx(full, stage_bytes);
#pragma unroll
            for (int b = 0; b < kSpBlocks; ++b) {
              const bool real = j * kSpBlocks + b < nblk;
              int y;
              if (!real || phys[b] < 0 || phys[b] >= p.num_blocks) {
                y = total_rows;  // past the tensor's end: TMA fills zeros
                bad_id |= real;
              } else {
                y = (phys[b] * p.num_kv_heads + h) * kBS;
              }
              if constexpr (FP8) {
                tma_load_2d(dst + b * kBS * D, tmap, full, 0, y);
              } else {
#pragma unroll
                for (int x = 0; x < H; ++x)
                  tma_load_2d(dst + x * PL::kHalfBytes + b * 2048, tmap, full, 64 * x, y);
              }
            }
            issued = j + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (lane == 0) {
        if (bad_id && is_k) raise_error(kErrBlockRange);
        // no bulk copy may still be landing when the CTA exits
        if (is_k)
          for (int g = 0; g < (alternate ? 1 : 2); ++g) mbar_wait_bounded(bar_q + 8u * g, 0, kWaitLimitNs);
        for (int j = max(0, issued - nst); j < issued; ++j)
          mbar_wait_bounded(bar_full + 8u * (j % nst), (j / nst) & 1, kWaitLimitNs);
      }
    } else {
      // ------------------------------------------------------------- MMA
      // A thread for each slot g, so that neither waits for the other's
      // softmax: S_g(0), then PV_g(n), S_g(n+1). S_g(n+1) overwrites the
      // columns PV_g(n) reads and is issued behind it (one thread's MMAs run
      // in issue order).
      const int g = warp - kMmaWarp;
      const int ntg = g == 0 ? my_tiles0 : my_tiles1;
      if (lane == 0 && ntg > 0) {
        constexpr uint32_t id_s = FP8 ? tc_idesc_f16(kSpRows, kSpKeys, false) : tc_idesc_bf16(kSpRows, kSpKeys, false);
        constexpr uint32_t id_pv = FP8 ? tc_idesc_f16(kSpRows, D, true) : tc_idesc_bf16(kSpRows, D, true);
        const int qt = alternate ? 0 : g;
        const uint32_t qst = sq + qt * PL::kTileBytes;
        const uint32_t st = tmem + g * kSpKeys, o = tmem + PL::kOCol + g * D;
        auto tile_of = [&](int n) { return alternate ? 2 * n + g : n; };
        bool ok = tc_wait((FP8 ? bar_qc : bar_q) + 8u * qt, 0, s_abort);
        // scores of the n-th key tile into the slot's columns
        auto issue_s = [&](int n) {
          const int j = tile_of(n);
          ok = ok && tc_wait(bar_k_full + 8u * (j % NK), (j / NK) & 1, s_abort);
          if (!ok) return;
          tc_fence_after_sync();
          const uint32_t kst = sk + (j % NK) * PL::kTileBytes;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks >> 2) * PL::kHalfBytes + (ks & 3) * 32;
            tc_mma_ss(st, tc_desc_sw128(qst + off, 16, 1024), tc_desc_sw128(kst + off, 16, 1024), id_s, ks > 0);
          }
          tc_commit(bar_s_full + 8u * g);
          tc_commit(bar_k_empty + 8u * (j % NK));
        };
        issue_s(0);
        for (int n = 0; n < ntg && ok; ++n) {
          const int j = tile_of(n);
          const uint32_t vst = sv + (j % NV) * PL::kTileBytes;
          // O += (hi + lo) V, the first 64 keys as soon as their weights are
          // there; a record's first tile overwrites
          const bool fresh = n % cut.record_tiles == 0;
          // one stage and two readers: the other slot's phase first (a parity
          // wait cannot tell a phase from the one two before)
          if (NV == 1 && alternate && j > 0) ok = tc_wait(bar_v_full, (j - 1) & 1, s_abort);
          ok = ok && tc_wait(bar_v_full + 8u * (j % NV), (j / NV) & 1, s_abort);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && tc_wait(bar_p_full + 16u * g + 8u * half, n & 1, s_abort);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < kSpBlocks; ++kk) {
              const int k16 = kk % (kSpBlocks / 2), lo = kk / (kSpBlocks / 2);
              tc_mma_ts(o, st + half * 64 + lo * 32 + k16 * 8,
                        tc_desc_sw128(vst + (half * (kSpBlocks / 2) + k16) * 2048, PL::kHalfBytes, 1024), id_pv,
                        !fresh || half > 0 || kk > 0);
            }
            if (half == 0) tc_commit(bar_o_half + 8u * g);
          }
          if (!ok) break;
          tc_commit(bar_v_empty + 8u * (j % NV));
          if (n + 1 < ntg)
            issue_s(n + 1);
          else
            tc_commit(bar_o_done + 8u * g);
        }
        // every MMA issued here has completed before tensor memory is freed
        tc_commit(bar_drain + 8u * g);
        mbar_wait_bounded(bar_drain + 8u * g, 0, kWaitLimitNs);
      }
      __syncwarp();
    }
  } else if (warp >= kSpSoftmaxWarps) {
    if constexpr (FP8) {
      // --------------------------------------------- widening, E4M3 -> f16
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PL::kConvertRegs));
      const int c = threadIdx.x - kSpSoftmaxWarps * 32;
      bool ok = true;
      // 16 codes a step: eight neighbouring lanes take four chunks of two
      // rows, whose f16 chunks then fall into different banks
      auto widen = [&](uint32_t src, uint32_t dst) {
#pragma unroll 4
        for (int i = 0; i < D / 16; ++i) {
          const int n = i * 128 + c;
          const int ch = n & 3, row = (n >> 2) & 127, half = n >> 9;
          const uint4 x = ld_shared_v4(src + swz<D, true>(row, half * 64 + ch * 16));
          uint4 a, b;
          e4m3x4_to_f16x2x2(x.x, a.x, a.y);
          e4m3x4_to_f16x2x2(x.y, a.z, a.w);
          e4m3x4_to_f16x2x2(x.z, b.x, b.y);
          e4m3x4_to_f16x2x2(x.w, b.z, b.w);
          st_shared_v4(dst + half * PL::kHalfBytes + op_chunk(row, 2 * ch), a);
          st_shared_v4(dst + half * PL::kHalfBytes + op_chunk(row, 2 * ch + 1), b);
        }
        fence_proxy_async_smem();
      };
      auto take_k = [&](int j) {
        if (j >= nt) return;
        ok = ok && tc_wait(bar_kb_full + 8u * (j % NB), (j / NB) & 1, s_abort) &&
             (j < NK || tc_wait(bar_k_empty + 8u * (j % NK), ((j / NK) - 1) & 1, s_abort));
        if (!ok) return;
        widen(skb + (j % NB) * PL::kByteTile, sk + (j % NK) * PL::kTileBytes);
        mbar_arrive(bar_kb_empty + 8u * (j % NB));
        mbar_arrive(bar_k_full + 8u * (j % NK));
      };
      // in the order the MMA warp asks for them: K0 K1 V0 K2 V1 K3 ...
      take_k(0);
      for (int j = 0; j < nt && ok; ++j) {
        take_k(j + 1);
        ok = ok && tc_wait(bar_vb_full + 8u * (j % NB), (j / NB) & 1, s_abort) &&
             (j < NV || tc_wait(bar_v_empty + 8u * (j % NV), ((j / NV) - 1) & 1, s_abort));
        if (!ok) break;
        widen(svb + (j % NB) * PL::kByteTile, sv + (j % NV) * PL::kTileBytes);
        mbar_arrive(bar_vb_empty + 8u * (j % NB));
        mbar_arrive(bar_v_full + 8u * (j % NV));
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PL::kSoftmaxRegs));
    // ------------------------------------------------------------- softmax
    const int g = warp >> 2;                       // slot of this warpgroup
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;             // row = tensor-memory lane
    const int tl = r / p.group;
    const int sl = (alternate ? 0 : g * tpt) + tl; // sequence of the CTA's stretch
    const bool valid = tl < tpt && sl < nseq;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t scol = g * kSpKeys, ocol = PL::kOCol + g * D;
    const int ntg = g == 0 ? my_tiles0 : my_tiles1;
    float scale = p.score_scale;
    bool ok = true;
    if constexpr (FP8) {
      // Q to f16 in place, each row times a power of two that puts its
      // largest element in [2^14, 2^15): exact; divided out of the scores
      if (!alternate || g == 0) {
        ok = __all_sync(0xffffffffu, tc_wait(bar_q + 8u * g, 0, s_abort));
      } else {  // the other warpgroup converts; the scale is needed here too
        ok = __all_sync(0xffffffffu, tc_wait(bar_q, 0, s_abort));
      }
      const uint32_t qrow = sq + (alternate ? 0 : g * PL::kTileBytes);
      float amax = 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 8 && ok; ++c) {
        const uint4 x = ld_shared_v4(qrow + (c >> 3) * PL::kHalfBytes + op_chunk(r, c & 7));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
      }
      int ex = 0;
      if (amax > 0.f && amax <= 3.0e38f) {
        int E;
        frexpf(amax, &E);
        ex = min(max(15 - E, -126), 126);
      }
      const float up = __int_as_float((127 + ex) << 23);
      scale *= __int_as_float((127 - ex) << 23);
      // every reader of the bf16 rows is done before they are overwritten
      if (alternate) named_bar_sync(3, 256);
      if (!alternate || g == 0) {
#pragma unroll 1
        for (int c = 0; c < D / 8 && ok; ++c) {
          const uint32_t at = qrow + (c >> 3) * PL::kHalfBytes + op_chunk(r, c & 7);
          uint4 x = ld_shared_v4(at);
          uint32_t *w = &x.x;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack2<true>(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
          st_shared_v4(at, x);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar_qc + 8u * g);
      }
    }
    // record `rec` of this part, this warpgroup's rows (tile 0's, where both take it)
    auto record_at = [&](int rec) {
      return ((static_cast<int64_t>(part) * p.part_records + rec) * p.num_kv_heads + h) * (2 * p.row_tiles) +
             2 * blockIdx.x + (alternate ? 0 : g);
    };
    constexpr float kSumMax = FP8 ? kSpSumMaxF16 : kSpSumMaxBf16;
    float m_used = -INFINITY, l = 0.f;
    // slot g's sums so far as record `rec`
    auto write_record = [&](int rec) {
      const int64_t at = record_at(rec);
      float4 *dst = reinterpret_cast<float4 *>(p.pre_o) + at * (D / 4) * kSpRows + r;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tc_ld_32x32b_x32(trow + ocol + cc * 32, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          dst[(cc * 8 + e / 4) * kSpRows] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                        __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
      }
      p.pre_ml[at * kSpRows + r] = make_float2(m_used, l);
    };
    // Records in the order they are written: with alternate key tiles the
    // first warpgroup's, the second's, and last the joined rest of both.
    int rec = (alternate && g == 1) ? (my_tiles0 - 1) / cut.record_tiles : 0;
    // The two warpgroups take turns at the exponentials (named barriers 4 and
    // 5, a turn of slot 0 and of slot 1): left alone they fall into step,
    // because they share the key tiles, and the tensor core idles while both
    // compute. Every turn is passed on, whatever was aborted.
    const int other_tiles = g == 0 ? my_tiles1 : my_tiles0;
    if (g == 1 && my_tiles0 > 0) named_bar_arrive(4, 256);
    for (int n = 0; n < ntg; ++n) {
      const int j = alternate ? 2 * n + g : n;     // key tile
      if (ok) ok = __all_sync(0xffffffffu, tc_wait(bar_s_full + 8u * g, n & 1, s_abort));
      tc_fence_after_sync();
      const bool fresh = n % cut.record_tiles == 0;
      if (ok && fresh && n > 0) {  // the earlier tiles' products completed before these scores
        write_record(rec++);
        l = 0.f;
      }
      uint32_t sr[2][64];
      if (ok) {
        tc_ld_cols<64>(trow + scol, sr[0]);
        tc_ld_cols<64>(trow + scol + 64, sr[1]);
        tc_wait_ld();
      }
      named_bar_sync(4 + g, 256);
      const int keys = nblk * kBS - j * kSpKeys;   // keys past the part's last block: loaded as zeros
      // A softmax is the same for any reference m, and the halves keep their
      // relative precision as long as the weights stay in the type's range. A
      // row's first 64 keys take their maximum first; any later 64 are formed
      // against the reference in use, without a maximum, and only where their
      // sum leaves the range formed again against a raised one. 64 keys go to
      // the MMA warp while the next are formed; P overwrites their scores:
      // hi in the first 32 columns, lo in the last 32.
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!ok) break;
        const uint32_t col = trow + scol + 64 * half;
        float mul = scale;
        if (keys < 64 * half + 64) {  // scaled here: a masked key is -inf whatever the scale's sign
#pragma unroll
          for (int c = 0; c < 64; ++c)
            sr[half][c] = __float_as_uint(64 * half + c < keys ? __uint_as_float(sr[half][c]) * scale : -INFINITY);
          mul = 1.f;
        }
        float sum = 0.f;
        auto form = [&]() {
          const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
          const uint64_t sc2 = f2(mul, mul), nm2 = f2(neg_m, neg_m);
          uint64_t lsum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
          for (int qq = 0; qq < 2; ++qq) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int c = 32 * qq + 2 * e;
              float x0, x1, u0, u1;
              f2_split(f2_fma(f2(__uint_as_float(sr[half][c]), __uint_as_float(sr[half][c + 1])), sc2, nm2), x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              hi[e] = pack2<FP8>(p0, p1);
              unpack2<FP8>(hi[e], u0, u1);
              lo[e] = pack2<FP8>(p0 - u0, p1 - u1);
              lsum[e & 1] = f2_add(lsum[e & 1], f2(p0, p1));
            }
            tc_st_32x32b_x16(col + 16 * qq, hi);
            tc_st_32x32b_x16(col + 32 + 16 * qq, lo);
          }
          float a0, a1, b0, b1;
          f2_split(lsum[0], a0, a1);
          f2_split(lsum[1], b0, b1);
          sum = (a0 + b0) + (a1 + b1);
        };
        bool redo = !__all_sync(0xffffffffu, !valid || m_used != -INFINITY);
        if (!redo) {
          form();
          redo = __any_sync(0xffffffffu, valid && !(sum <= kSumMax));
        }
        if (redo) {
          tc_wait_st();  // the same columns are written again
          float mx = __uint_as_float(sr[half][0]);  // the largest argument is that of an end of the scores
#pragma unroll
          for (int c = 1; c < 64; ++c)
            mx = mul >= 0.f ? fmaxf(mx, __uint_as_float(sr[half][c])) : fminf(mx, __uint_as_float(sr[half][c]));
          const float m_new = fmaxf(m_used, mx * mul - (FP8 ? kSpF16Log2 : 0.f));
          const float alpha = m_new == m_used ? 1.f : ex2_approx(m_used - m_new);
          m_used = m_new;
          l *= alpha;
          // Earlier tiles' products completed before these scores; that of
          // this tile's first half has a barrier of its own.
          if (half == 1) ok = __all_sync(0xffffffffu, tc_wait(bar_o_half + 8u * g, n & 1, s_abort));
          if ((half == 1 || !fresh) && __any_sync(0xffffffffu, alpha != 1.f)) {
            tc_fence_after_sync();
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tc_ld_32x32b_x32(trow + ocol + cc * 32, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc_st_32x32b_x32(trow + ocol + cc * 32, o);
            }
          }
          form();
        }
        l += sum;
        tc_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full + 16u * g + 8u * half);
      }
      // slot 1 follows slot 0's n-th turn, slot 0's (n+1)-th slot 1's n-th
      if (g == 0 ? n < other_tiles : n + 1 < other_tiles) named_bar_arrive(5 - g, 256);
    }
    // ------------------------------------------------------------ epilogue
    if (ok && ntg > 0) ok = __all_sync(0xffffffffu, tc_wait(bar_o_done + 8u * g, 0, s_abort));
    tc_fence_after_sync();
    if (!alternate || nt == 1) {
      if (ok && ntg > 0) write_record(rec);
    } else {
      // Both warpgroups hold a share of the same rows. Every MMA and copy has
      // completed once both have seen their last product, so the second
      // leaves its share in the K ring and the first joins it.
      ok = named_bar_and(3, 256, ok);
      float4 *so = reinterpret_cast<float4 *>(base_ptr + PL::kKOff);    // [D / 4][128]
      float2 *sml = reinterpret_cast<float2 *>(base_ptr + PL::kTileBytes);  // query tile 1's place
      rec = (my_tiles0 - 1) / cut.record_tiles + (my_tiles1 - 1) / cut.record_tiles;
      if (ok && g == 1) {
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tc_ld_32x32b_x32(trow + ocol + cc * 32, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            so[(cc * 8 + e / 4) * kSpRows + r] =
                make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                            __uint_as_float(o[e + 3]));
        }
        sml[r] = make_float2(m_used, l);
      }
      named_bar_sync(3, 256);
      if (ok && g == 0) {
        const int64_t at = record_at(rec);
        float4 *dst = reinterpret_cast<float4 *>(p.pre_o) + at * (D / 4) * kSpRows + r;
        const float2 other = sml[r];
        const float M = fmaxf(m_used, other.x);
        const float wa = M == -INFINITY ? 0.f : ex2_approx(m_used - M);
        const float wb = M == -INFINITY ? 0.f : ex2_approx(other.x - M);
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tc_ld_32x32b_x32(trow + ocol + cc * 32, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 x = so[(cc * 8 + e / 4) * kSpRows + r];
            dst[(cc * 8 + e / 4) * kSpRows] =
                make_float4(wa * __uint_as_float(o[e]) + wb * x.x, wa * __uint_as_float(o[e + 1]) + wb * x.y,
                            wa * __uint_as_float(o[e + 2]) + wb * x.z, wa * __uint_as_float(o[e + 3]) + wb * x.w);
          }
        }
        p.pre_ml[at * kSpRows + r] = make_float2(M, wa * l + wb * other.y);
      }
    }
    // records of this part that no tile fell into
    if (g == 0 || !alternate)
      for (int i = rec + 1; i < p.part_records; ++i) p.pre_ml[record_at(i) * kSpRows + r] = make_float2(-INFINITY, 0.f);
    tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, PL::kTmemCols);
  }
}

// ------------------------------------------------------------ suffix parts

// attend_blocks of decode.cuh for E4M3 tiles with the weights in two f16
// halves (one half leaves 2^-12 of each).
template <int D, int NT, int NB, bool TAIL>
__device__ __forceinline__ void attend_e4m3_halves(const uint32_t (&kt)[NB], const uint32_t (&vt)[NB], int valid,
                                                   int lane, const uint32_t (&qf)[NT][D / 16][2],
                                                   const float (&cs)[NT][2], WarpState<D, NT> &ws) {
  constexpr int KS = D / 16;
  const int mi = lane >> 3, mrow = lane & 7, gq = lane >> 2, qd = lane & 3;
  float sc[NB][NT][2][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) sc[b][nt][c][0] = sc[b][nt][c][1] = sc[b][nt][c][2] = sc[b][nt][c][3] = 0.f;
#pragma unroll
  for (int kk = 0; kk < KS / 2; ++kk)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t r0, r1, r2, r3, a0, a1, a2, a3, c0, c1, c2, c3;
      ldsm_x4(kt[b] + swz<D, true>((mi & 1) * 8 + mrow, 32 * kk + (mi >> 1) * 16), r0, r1, r2, r3);
      e4m3x4_to_f16x2x2(r0, a0, a2);
      e4m3x4_to_f16x2x2(r1, a1, a3);
      e4m3x4_to_f16x2x2(r2, c0, c2);
      e4m3x4_to_f16x2x2(r3, c1, c3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816<true>(sc[b][nt][0], a0, a1, a2, a3, qf[nt][2 * kk][0], qf[nt][2 * kk][1]);
        mma_16816<true>(sc[b][nt][1], c0, c1, c2, c3, qf[nt][2 * kk + 1][0], qf[nt][2 * kk + 1][1]);
      }
    }
  uint32_t ph[NB][NT][2], pl[NB][NT][2];
  float alpha[NT][2];
  bool rescale = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float z[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[b][e] = (sc[b][nt][0][e] + sc[b][nt][1][e]) * cs[nt][e & 1];
        if (TAIL && gq + (e >> 1) * 8 >= valid - kBS * b) z[b][e] = -INFINITY;
      }
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      mx0 = fmaxf(mx0, fmaxf(z[b][0], z[b][2]));
      mx1 = fmaxf(mx1, fmaxf(z[b][1], z[b][3]));
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
    }
    const float mn0 = fmaxf(ws.m[nt][0], mx0), mn1 = fmaxf(ws.m[nt][1], mx1);
    alpha[nt][0] = exp2f(ws.m[nt][0] - mn0);
    alpha[nt][1] = exp2f(ws.m[nt][1] - mn1);
    rescale |= (ws.m[nt][0] != mn0) || (ws.m[nt][1] != mn1);
    ws.m[nt][0] = mn0;
    ws.m[nt][1] = mn1;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float p0 = exp2f(z[b][0] - mn0), p1 = exp2f(z[b][1] - mn1);
      const float p2 = exp2f(z[b][2] - mn0), p3 = exp2f(z[b][3] - mn1);
      s0 += p0 + p2;
      s1 += p1 + p3;
      // weights times 2^8 (kSpF16Log2), so that small ones keep their bits in f16
      const float w0 = p0 * 256.f, w1 = p1 * 256.f, w2 = p2 * 256.f, w3 = p3 * 256.f;
      const uint32_t h01 = pack2<true>(w0, w1), h23 = pack2<true>(w2, w3);
      float u0, u1, u2, u3;
      unpack2<true>(h01, u0, u1);
      unpack2<true>(h23, u2, u3);
      ph[b][nt][0] = movmatrix_trans(h01);
      ph[b][nt][1] = movmatrix_trans(h23);
      pl[b][nt][0] = movmatrix_trans(pack2<true>(w0 - u0, w1 - u1));
      pl[b][nt][1] = movmatrix_trans(pack2<true>(w2 - u2, w3 - u3));
    }
    ws.l[nt][0] = ws.l[nt][0] * alpha[nt][0] + s0 * 256.f;
    ws.l[nt][1] = ws.l[nt][1] * alpha[nt][1] + s1 * 256.f;
  }
  if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) ws.acc[nt][mt][e] *= alpha[nt][e & 1];
  }
  uint32_t mlo[NB], mhi[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int vb = valid - kBS * b;
    mlo[b] = (2 * qd < vb ? 0x0000ffffu : 0u) | (2 * qd + 1 < vb ? 0xffff0000u : 0u);
    mhi[b] = (2 * qd + 8 < vb ? 0x0000ffffu : 0u) | (2 * qd + 9 < vb ? 0xffff0000u : 0u);
  }
#pragma unroll
  for (int cc = 0; cc < KS / 2; ++cc)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // bytes of r: (t, 2g) (t, 2g+1) (t+1, 2g) (t+1, 2g+1), t = 2qd, g = gq
      uint32_t r0, r1, r2, r3, a0, a1, a2, a3, c0, c1, c2, c3;
      ldsm_x4_trans(vt[b] + swz<D, true>((mi & 1) * 8 + mrow, 32 * cc + (mi >> 1) * 16), r0, r1, r2, r3);
      e4m3x4_to_f16x2x2(prmt(r0, 0x3120), a0, a1);
      e4m3x4_to_f16x2x2(prmt(r1, 0x3120), a2, a3);
      e4m3x4_to_f16x2x2(prmt(r2, 0x3120), c0, c1);
      e4m3x4_to_f16x2x2(prmt(r3, 0x3120), c2, c3);
      if constexpr (TAIL) {
        a0 &= mlo[b]; a1 &= mlo[b]; a2 &= mhi[b]; a3 &= mhi[b];
        c0 &= mlo[b]; c1 &= mlo[b]; c2 &= mhi[b]; c3 &= mhi[b];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816<true>(ws.acc[nt][2 * cc], a0, a1, a2, a3, ph[b][nt][0], ph[b][nt][1]);
        mma_16816<true>(ws.acc[nt][2 * cc + 1], c0, c1, c2, c3, ph[b][nt][0], ph[b][nt][1]);
        mma_16816<true>(ws.acc[nt][2 * cc], a0, a1, a2, a3, pl[b][nt][0], pl[b][nt][1]);
        mma_16816<true>(ws.acc[nt][2 * cc + 1], c0, c1, c2, c3, pl[b][nt][0], pl[b][nt][1]);
      }
    }
}

// One CTA a (part, KV head, sequence): the blocks of the part through the
// ring of the plain decode (decode.cuh: one producer warp, four consumer
// warps, 8 KB stages), the warps' states merged at the end.
template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kDecodeThreads, NT == 1 ? 3 : 2)
    shared_suffix_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                         const SharedParams p) {
  using G = Geo<D, FP8>;
  using PL = Plan<D, FP8, NT, false>;
  constexpr int NS = PL::kStages, KS = G::kKSteps, BPS = G::kBPS;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t ring = (raw_u32 + 1023u) & ~1023u;
  uint8_t *base_ptr = smem_raw + (ring - raw_u32);
  uint64_t *bars = reinterpret_cast<uint64_t *>(base_ptr + PL::kBarOffset);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * NS;
  volatile int *s_abort = reinterpret_cast<volatile int *>(bars + 2 * NS);

  const int part = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  const SharedRow row = shared_row(p, s);
  if (part == 0 && h == 0) {
    if (threadIdx.x == 0 && row.bad_len) raise_error(kErrContextClamp);
    if (s == 0) check_groups(p);
  }
  if (part >= row.own_parts) {
    wait_for_primary();  // this grid ends after the prefix kernel
    return;
  }
  const int tok0 = part * p.part_len;   // of the own part; the last takes what is left
  const int toks = part + 1 == p.suffix_parts ? row.own_tokens - tok0 : min(p.part_len, row.own_tokens - tok0);
  const int j0 = row.shared_blocks + tok0 / kBS;
  const int nblk = (toks + kBS - 1) / kBS;
  const int nst = (nblk + BPS - 1) / BPS;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full0 + 8u * i, 1);
      mbar_init(empty0 + 8u * i, 1);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
    const int32_t *bt = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + j0;
    const int total_rows = p.num_blocks * p.num_kv_heads * kBS;
    int issued = 0;
    bool ok = true, bad_id = false;
    for (int jb = 0; jb < nst * BPS && ok; jb += 32) {
      const int mine = jb + lane < nblk ? bt[jb + lane] : -1;
      const int i_end = min(nst, (jb + 32) / BPS);
      for (int i = jb / BPS; i < i_end; ++i) {
        int phys[BPS];
#pragma unroll
        for (int b = 0; b < BPS; ++b) phys[b] = __shfl_sync(0xffffffffu, mine, i * BPS + b - jb);
        if (lane == 0) {
          const int st = i % NS;
          if (i >= NS) ok = tc_wait(empty0 + 8u * st, ((i / NS) - 1) & 1, s_abort);
          if (ok) {
            const uint32_t fb = full0 + 8u * st;
            const uint32_t kdst = ring + st * G::kStageBytes, vdst = kdst + BPS * G::kTileBytes;
            mbar_arrive_expect_tx(fb, G::kStageBytes);
#pragma unroll
            for (int b = 0; b < BPS; ++b) {
              const bool real = i * BPS + b < nblk;
              int y;
              if (!real || phys[b] < 0 || phys[b] >= p.num_blocks) {
                y = total_rows;  // whole box out of range: TMA fills zeros
                bad_id |= real;
              } else {
                y = (phys[b] * p.num_kv_heads + h) * kBS;
              }
#pragma unroll
              for (int x = 0; x < G::kBoxes; ++x) {
                tma_load_2d(kdst + b * G::kTileBytes + x * G::kBoxBytes, &tmap_k, fb, x * (G::kBoxRow / G::kEB), y);
                tma_load_2d(vdst + b * G::kTileBytes + x * G::kBoxBytes, &tmap_v, fb, x * (G::kBoxRow / G::kEB), y);
              }
            }
            issued = i + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
    }
    wait_for_primary();
    if (lane == 0) {
      if (bad_id) raise_error(kErrBlockRange);
      for (int i = max(0, issued - NS); i < issued; ++i)
        mbar_wait_bounded(full0 + 8u * (i % NS), (i / NS) & 1, kWaitLimitNs);
    }
    __syncthreads();  // the merge reuses the ring
    return;
  }

  // ------------------------------------------------------------ consumers
  const int gq = lane >> 2, qd = lane & 3;
  WarpState<D, NT> ws;
  ws.reset();
  uint32_t qf[NT][KS][2];
  float cs[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = nt * 8 + gq;
    const bool live = n < p.group;
    const uint16_t *qrow = p.q + (static_cast<int64_t>(s) * p.num_q_heads + h * p.group + (live ? n : 0)) * D;
    if constexpr (!FP8) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[nt][ks][0] = live ? *reinterpret_cast<const uint32_t *>(qrow + 16 * ks + 2 * qd) : 0u;
        qf[nt][ks][1] = live ? *reinterpret_cast<const uint32_t *>(qrow + 16 * ks + 8 + 2 * qd) : 0u;
      }
      cs[nt][0] = cs[nt][1] = p.score_scale;
    } else {
      // dims (4qd, 4qd+1) and (4qd+2, 4qd+3) of each 16, as the K fragments
      // hold them; a power of two puts the head's largest element in [2^14, 2^15)
      float v[KS][4];
      float amax = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 w = live ? *reinterpret_cast<const uint2 *>(qrow + 16 * ks + 4 * qd) : make_uint2(0u, 0u);
        unpack2<false>(w.x, v[ks][0], v[ks][1]);
        unpack2<false>(w.y, v[ks][2], v[ks][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(v[ks][e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int ex = 0;
      if (amax > 0.f && amax <= 3.0e38f) {
        int E;
        frexpf(amax, &E);
        ex = min(max(15 - E, -126), 126);
      }
      const float up = __int_as_float((127 + ex) << 23), down = __int_as_float((127 - ex) << 23);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[nt][ks][0] = pack2<true>(v[ks][0] * up, v[ks][1] * up);
        qf[nt][ks][1] = pack2<true>(v[ks][2] * up, v[ks][3] * up);
      }
      cs[nt][0] = p.score_scale * __shfl_sync(0xffffffffu, down, 8 * qd);
      cs[nt][1] = p.score_scale * __shfl_sync(0xffffffffu, down, 8 * qd + 4);
    }
  }
  for (int i = warp; i < nst; i += kConsumerWarps) {
    const int st = i % NS;
    if (!__all_sync(0xffffffffu, tc_wait(full0 + 8u * st, (i / NS) & 1, s_abort))) break;
    const uint32_t k0 = ring + st * G::kStageBytes;
    uint32_t kt[BPS], vt[BPS];
#pragma unroll
    for (int b = 0; b < BPS; ++b) {
      kt[b] = k0 + b * G::kTileBytes;
      vt[b] = k0 + (BPS + b) * G::kTileBytes;
    }
    const int valid = toks - i * BPS * kBS;
    if constexpr (FP8) {
      if (valid >= BPS * kBS)
        attend_e4m3_halves<D, NT, BPS, false>(kt, vt, BPS * kBS, lane, qf, cs, ws);
      else
        attend_e4m3_halves<D, NT, BPS, true>(kt, vt, valid, lane, qf, cs, ws);
    } else {
      if (valid >= BPS * kBS)
        attend_blocks<D, FP8, NT, BPS, false>(kt, vt, BPS * kBS, lane, qf, cs, ws);
      else
        attend_blocks<D, FP8, NT, BPS, true>(kt, vt, valid, lane, qf, cs, ws);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8u * st);
  }
  __syncthreads();  // all loads consumed: the ring is idle
  // ------------------------------------------------- merge (as decode.cuh)
  float *mbuf = reinterpret_cast<float *>(base_ptr);
  constexpr int LF = PL::kLaneFloats;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) ws.l[nt][c] += __shfl_xor_sync(0xffffffffu, ws.l[nt][c], o);
  if (warp >= 2) store_record<D, NT>(ws, mbuf + ((warp - 2) * 32 + lane) * LF);
  consumer_bar_sync();
  if (warp >= 2) return;
  combine_record<D, NT>(ws, mbuf + (warp * 32 + lane) * LF);
  pair_bar_sync();  // both have read their records
  if (warp == 1) store_record<D, NT>(ws, mbuf + lane * LF);
  pair_bar_sync();
  if (warp == 1) return;
  combine_record<D, NT>(ws, mbuf + lane * LF);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = nt * 8 + 2 * qd + c;
      if (n >= p.group) continue;
      const int64_t at = (static_cast<int64_t>(part) * p.num_seqs + s) * p.num_q_heads + h * p.group + n;
      float *dst = p.suf_o + at * D;
      if (gq == 0)  // weights of E4M3 tiles are 2^(z - m + 8)
        p.suf_ml[at] = make_float2(ws.m[nt][c] - (FP8 ? kSpF16Log2 : 0.f), ws.l[nt][c]);
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int d0 = FP8 ? 16 * mt + 2 * gq : 16 * mt + gq, d1 = FP8 ? d0 + 1 : d0 + 8;
        dst[d0] = ws.acc[nt][mt][c];
        dst[d1] = ws.acc[nt][mt][2 + c];
      }
    }
}

// ------------------------------------------------------------------- join

// 32 rows (sequence, head of KV head h) and 32 of their elements a CTA:
//     out = out_scale sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i
// over a row's prefix records and its own parts. First a thread takes one
// 16-byte chunk of a row of the prefix records as they lie (a warp reads one
// chunk of 32 rows, whole lines), then, through shared memory, a warp takes
// a row. Small CTAs: the records of a few thousand rows fill the GPU's loads.
constexpr int kJoinRows = 32;
constexpr int kJoinCols = 32;

template <int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const SharedParams p) {
  constexpr int U = 4;  // records in flight
  __shared__ float s_o[kJoinRows][kJoinCols + 4];
  __shared__ float2 s_ml[kJoinRows];
  __shared__ int s_parts[kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, all = p.num_seqs * p.group;
  const int idx = blockIdx.x * kJoinRows + lane;  // this lane's row
  SharedRow r{};
  if (idx < all) r = shared_row(p, idx / p.group);
  wait_for_primary();
  // all records of the row's parts; unused ones are empty
  const int records = r.prefix_parts * p.part_records;
  const int64_t stride = static_cast<int64_t>(p.num_kv_heads) * (2 * p.row_tiles) * kSpRows;
  int64_t at = 0;
  if (records > 0) {
    const int s = idx / p.group;
    // groups that overlap leave places unwritten: kept inside the records
    const int slot = min(max(p.row_of[s], 0), 2 * p.row_tiles * p.tokens_per_tile - 1);
    const int tile = slot / p.tokens_per_tile;
    at = (static_cast<int64_t>(h) * (2 * p.row_tiles) + tile) * kSpRows + (slot - tile * p.tokens_per_tile) * p.group +
         (idx - s * p.group);
  }
  const float2 *pre_ml = p.pre_ml + at;
  // rows are the fastest index of a chunk: record i's chunk c of tile-row `at`
  const float4 *pre_o = reinterpret_cast<const float4 *>(p.pre_o) + (at / kSpRows * (D / 4) + blockIdx.z * 8 + warp) * kSpRows +
                        at % kSpRows;
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < records; i0 += U) {
    float2 ml[U];
    float4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + u < records) {
        ml[u] = pre_ml[(i0 + u) * stride];
        x[u] = pre_o[(i0 + u) * stride * (D / 4)];
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
    const float a = M == -INFINITY ? 0.f : exp2f(M - top);
    l *= a;
    acc.x *= a;
    acc.y *= a;
    acc.z *= a;
    acc.w *= a;
    M = top;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ml[u].x == -INFINITY) continue;  // an empty record holds no o
      const float w = exp2f(ml[u].x - M);
      l += w * ml[u].y;
      acc.x += w * x[u].x;
      acc.y += w * x[u].y;
      acc.z += w * x[u].z;
      acc.w += w * x[u].w;
    }
  }
  *reinterpret_cast<float4 *>(&s_o[lane][4 * warp]) = acc;
  if (warp == 0) {
    s_ml[lane] = make_float2(M, l);
    s_parts[lane] = idx < all ? r.own_parts + (records > 0 ? 65536 : 0) : -1;
  }
  __syncthreads();
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_q_heads;
#pragma unroll
  for (int k = warp; k < kJoinRows; k += 8) {
    const int parts = s_parts[k] & 65535;
    if (s_parts[k] < 0) continue;
    const int i0 = blockIdx.x * kJoinRows + k, s = i0 / p.group;
    const int64_t row = static_cast<int64_t>(s) * p.num_q_heads + h * p.group + (i0 - s * p.group);
    const float2 pre = s_ml[k];
    float top = pre.x, sum = pre.y, x = s_o[k][lane];
    const float *o = p.suf_o + row * D + blockIdx.z * kJoinCols + lane;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float2 ml = p.suf_ml[i * rows + row];
      const float y = o[i * rows * D];
      const float t = fmaxf(top, ml.x);
      const float a = top == -INFINITY ? 0.f : exp2f(top - t), w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - t);
      top = t;
      sum = sum * a + w * ml.y;
      x = x * a + w * y;
    }
    // no token at all: zeros
    p.out[row * D + blockIdx.z * kJoinCols + lane] = s_parts[k] > 0 ? x / sum * p.out_scale : 0.f;
  }
}

}  // namespace pa
