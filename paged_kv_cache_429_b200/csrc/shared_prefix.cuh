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
// the plain decode does, its CTAs started on the SMs as the prefix kernel
// leaves them (each waits for that kernel's end before it merges, so an SM
// takes one set of them until then); its parts are records too. The join
// kernel adds up each row's records. A sequence that ends inside its prefix
// takes its whole context as its own part, so that no masked product ever
// meets a value it must not see (0 * NaN).
//
// The prefix kernel's CTA: two query tiles of 128 rows against at most 16
// key tiles of 128, K and V by TMA (E4M3 bytes widened to f16 by a warpgroup
// of their own), scores and outputs in tensor memory, a softmax warpgroup a
// query tile with a thread a row, and one thread that issues PV_0, S_0,
// PV_1, S_1 in turn, so that one tile's softmax runs beside the other's
// products. What bounds it: 48 products of 75 to 85 cycles a key tile, 3780
// cycles of the tensor core for both query tiles, against 5000 (bf16) and
// 6100 (E4M3) measured, in which the two softmaxes and the hand-overs are
// not all covered; and about 10 us of a CTA's start and end, since shared
// memory holds one CTA an SM. 64 sequences of 64 heads over 8 KV heads and
// 32768 shared tokens: 104 us, 660 TFLOP/s of the formula's, 990 with the
// second halves of the weights. The suffix kernel is bound by DRAM where
// there is enough of it (256 sequences of 40 heads, 992 shared and up to 2048
// own tokens: the whole call 2.58 GB in 400 to 417 us, 0.95 to 0.985 of the
// copy bandwidth); short suffixes of few heads (130 sequences of 250 tokens,
// 8 heads, E4M3) take 24 us against 10, the latency of a part's start and of
// its merge.
//
// Precision. The output is fp32, so the weights 2^(z - m) enter the value
// product as two 16-bit halves (hi = round(p), lo = round(p - hi)): bf16
// against bf16 caches (16 significant bits), f16 against E4M3 widened to f16
// (22 bits). One half alone would leave 2^-9 or 2^-12 of every weight.
#pragma once

#include "decode.cuh"
#include "prefill.cuh"
#include "ptx_step.cuh"

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
  int prefix_parts;              // parts of the longest prefix, a CTA (and a record) each
  int suffix_parts;              // suffix parts, part_len tokens each (the last one to the end)
  int part_len;
  float score_scale;             // sm_scale * log2(e) [* k_scale for fp8]
  float out_scale;               // v_scale for fp8, 1 for bf16
  int row_tiles;                 // CTAs along the prefix rows, two 128-row query tiles each
  // Records, [prefix_parts + suffix_parts][S * Hq], the prefix's first: o
  // [D] of each, and (m, l).
  float *rec_o;
  float2 *rec_ml;
};

// (unsigned: with bounds near 2^31, a + b passes a signed 32-bit sum)
__host__ __device__ constexpr int ceil_div(int a, int b) {
  return static_cast<int>((static_cast<uint32_t>(a) + static_cast<uint32_t>(b) - 1u) / static_cast<uint32_t>(b));
}

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
// no group). All lanes of the warp with the same s: 32 groups a load, so that
// up to 32 groups cost one load's latency and 65535 four.
__device__ __forceinline__ int shared_blocks_of(const SharedParams &p, int s) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.num_groups;
  while (n > 32) {  // the last of 32 stretches that starts at s or before
    const int step = ceil_div(n, 32), g = lane * step;
    const uint32_t at = __ballot_sync(0xffffffffu, g < n && p.group_start[lo + min(g, n - 1)] <= s);
    const int k = max(__popc(at) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  bool here = false;
  int blocks = 0;
  if (lane < n) {
    here = p.group_start[lo + lane] <= s && s < p.group_start[lo + lane + 1];
    blocks = p.prefix_blocks[lo + lane];
  }
  const uint32_t in = __ballot_sync(0xffffffffu, here);
  blocks = __shfl_sync(0xffffffffu, blocks, in ? __ffs(in) - 1 : 0);
  return in ? min(max(blocks, 0), min(p.max_prefix_blocks, p.max_blocks_per_seq)) : 0;
}

constexpr int kSpRows = 128;                // rows of a query tile (MMA M)
constexpr int kSpKeys = 128;                // keys of a prefix tile (score MMA N)
constexpr int kSpBlocks = kSpKeys / kBS;
// Most key tiles of a part. The tensor core's accumulator truncates, so a sum
// over n tiles shrinks by about n * 2.6e-7 of itself (measured: 8.3e-6 at 32
// tiles, and 1.35e-5 where all values have the same sign); the parts are
// added up in fp32 by the join.
constexpr int kSpPartTiles = 16;

// A prefix of `blocks` blocks cut into at most max_parts parts of `tiles` key tiles.
struct PrefixCut {
  int parts, tiles;
};
__device__ __forceinline__ PrefixCut cut_prefix(int blocks, int max_parts) {
  PrefixCut c;
  const int all = ceil_div(blocks, kSpBlocks);
  c.tiles = ceil_div(all, max_parts);
  c.parts = ceil_div(all, c.tiles);
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

// ------------------------------------------------------------ prefix parts

constexpr int kSpSoftmaxWarps = 8;  // two warpgroups
constexpr float kSpSumMaxBf16 = 1.0e18f;   // a tile's weights against an older maximum
constexpr float kSpSumMaxF16 = 32768.f;    // f16 halves: every weight <= 2^15
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
  static constexpr int kIssueWarp0 = kThreads / 32 - 4;  // K (and Q) loads, V loads, MMA, idle
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
  // kb_full[2] kb_empty[2] vb_full[2] vb_empty[2] s_full[2] p_full[2] o_done[2] drain
  static constexpr int kNumBars = 4 + 2 * kNK + 2 * kNV + 8 + 6 + 1;
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
  const uint32_t bar_p_full = bar_s_full + 16;        // [tile]
  const uint32_t bar_o_done = bar_p_full + 16;        // [tile]
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
  // One query tile only: both softmax warpgroups take it, with alternate key
  // tiles, and their results are joined at the end. Whole calls against the
  // second query tile left empty: 8 sequences of 32 heads over 8, 16384
  // shared tokens, 26 us against 34 (E4M3 29 against 38); 16 of 64 over 8,
  // 32768 tokens, 43 against 57 (44 against 63).
  const bool alternate = nseq <= tpt;
  const int my_tiles0 = alternate ? (nt + 1) / 2 : nt, my_tiles1 = alternate ? nt / 2 : nt;

  // the producers' first table entries, on their way during the set-up
  const int32_t *bt = p.block_tables + static_cast<int64_t>(first) * p.max_blocks_per_seq + blk0;
  int first_ids = -1;
  if ((warp == kKWarp || warp == kVWarp) && lane < nblk) first_ids = bt[lane];
  if (threadIdx.x == 0) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar_q + 8u * g, 1);
      mbar_init(bar_qc + 8u * g, 128);
      mbar_init(bar_s_full + 8u * g, 1);
      mbar_init(bar_p_full + 8u * g, 128);
      mbar_init(bar_o_done + 8u * g, 1);
      mbar_init(bar_kb_full + 8u * g, 1);
      mbar_init(bar_kb_empty + 8u * g, 128);
      mbar_init(bar_vb_full + 8u * g, 1);
      mbar_init(bar_vb_empty + 8u * g, 128);
    }
    for (int i = 0; i < NK; ++i) {
      mbar_init(bar_k_full + 8u * i, FP8 ? 128 : 1);
      mbar_init(bar_k_empty + 8u * i, 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(bar_v_full + 8u * i, FP8 ? 128 : 1);
      mbar_init(bar_v_empty + 8u * i, 1);
    }
    mbar_init(bar_drain, 1);
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
      const int total_rows = p.num_blocks * p.num_kv_heads * kBS;
      bool ok = true, bad_id = false;
      int issued = 0, mine = -1;
      for (int j = 0; j < nt && ok; ++j) {
        if ((j & 3) == 0) {  // 32 table entries, four tiles, a load
          const int jb = j * kSpBlocks + lane;
          mine = j == 0 ? first_ids : (jb < nblk ? bt[jb] : -1);
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
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------- MMA
      if (lane == 0) {
        constexpr uint32_t id_s = FP8 ? tc_idesc_f16(kSpRows, kSpKeys, false) : tc_idesc_bf16(kSpRows, kSpKeys, false);
        constexpr uint32_t id_pv = FP8 ? tc_idesc_f16(kSpRows, D, true) : tc_idesc_bf16(kSpRows, D, true);
        bool ok = true;
        auto wait_k = [&](int j) {
          ok = ok && tc_wait(bar_k_full + 8u * (j % NK), (j / NK) & 1, s_abort);
          tc_fence_after_sync();
        };
        auto wait_q = [&](int g) {
          ok = ok && tc_wait((FP8 ? bar_qc : bar_q) + 8u * g, 0, s_abort);
          tc_fence_after_sync();
        };
        // P of tile slot g's n-th key tile, and V of key tile j
        auto wait_pv = [&](int g, int n, int j) {
          ok = ok && tc_wait(bar_p_full + 8u * g, n & 1, s_abort) &&
               tc_wait(bar_v_full + 8u * (j % NV), (j / NV) & 1, s_abort);
          tc_fence_after_sync();
        };
        // scores of query tile qt against key tile j, into slot g's columns
        auto issue_s = [&](int g, int qt, int j) {
          const uint32_t kst = sk + (j % NK) * PL::kTileBytes;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks >> 2) * PL::kHalfBytes + (ks & 3) * 32;
            tc_mma_ss(tmem + g * kSpKeys, tc_desc_sw128(sq + qt * PL::kTileBytes + off, 16, 1024),
                      tc_desc_sw128(kst + off, 16, 1024), id_s, ks > 0);
          }
          tc_commit(bar_s_full + 8u * g);
        };
        // O_g += (hi + lo) V: the halves of P in slot g's columns, hi first
        auto issue_pv = [&](int g, int j, bool accumulate) {
          const uint32_t vst = sv + (j % NV) * PL::kTileBytes;
          const uint32_t pt = tmem + g * kSpKeys, o = tmem + PL::kOCol + g * D;
#pragma unroll
          for (int kk = 0; kk < 2 * kSpBlocks; ++kk)
            tc_mma_ts(o, pt + kk * 8, tc_desc_sw128(vst + (kk % kSpBlocks) * 2048, PL::kHalfBytes, 1024), id_pv,
                      accumulate || kk > 0);
        };
        if (!alternate) {
          wait_q(0);
          wait_q(1);
          wait_k(0);
          if (ok) {
            issue_s(0, 0, 0);
            issue_s(1, 1, 0);
            tc_commit(bar_k_empty);
          }
          // PV_0(j), S_0(j+1), PV_1(j), S_1(j+1): S_g(j+1) overwrites the
          // columns PV_g(j) reads and is issued behind it
          for (int j = 0; j < nt && ok; ++j) {
            const bool next = j + 1 < nt;
            wait_pv(0, j, j);
            if (!ok) break;
            issue_pv(0, j, j > 0);
            if (!next) tc_commit(bar_o_done);
            if (next) {
              wait_k(j + 1);
              if (!ok) break;
              issue_s(0, 0, j + 1);
            }
            wait_pv(1, j, j);
            if (!ok) break;
            issue_pv(1, j, j > 0);
            if (!next) tc_commit(bar_o_done + 8u);
            tc_commit(bar_v_empty + 8u * (j % NV));
            if (next) {
              issue_s(1, 1, j + 1);
              tc_commit(bar_k_empty + 8u * ((j + 1) % NK));
            }
          }
        } else {
          wait_q(0);
          for (int j = 0; j < min(nt, 2) && ok; ++j) {
            wait_k(j);
            if (!ok) break;
            issue_s(j, 0, j);
            tc_commit(bar_k_empty + 8u * (j % NK));
          }
          for (int j = 0; j < nt && ok; ++j) {
            const int g = j & 1;
            wait_pv(g, j >> 1, j);
            if (!ok) break;
            issue_pv(g, j, j > 1);
            tc_commit(bar_v_empty + 8u * (j % NV));
            if (j + 2 >= nt) {
              tc_commit(bar_o_done + 8u * g);
            } else {
              wait_k(j + 2);
              if (!ok) break;
              issue_s(g, 0, j + 2);
              tc_commit(bar_k_empty + 8u * (j % NK));
            }
          }
        }
        // every MMA issued here has completed before tensor memory is freed
        tc_commit(bar_drain);
        mbar_wait_bounded(bar_drain, 0, kWaitLimitNs);
      }
      __syncwarp();
    }
  } else if (warp >= kSpSoftmaxWarps) {
    if constexpr (FP8) {
      // --------------------------------------------- widening, E4M3 -> f16
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PL::kConvertRegs));
      const int c = threadIdx.x - kSpSoftmaxWarps * 32;
      bool ok = true;
      // A thread takes chunk c & 3 (16 codes) of rows c / 4, c / 4 + 32, ... of
      // each 64-element half: eight neighbouring lanes then hold four chunks
      // of two rows, whose f16 chunks fall into different banks, and a row's
      // place under the swizzle is the same in every step.
      const int ch = c & 3, row = c >> 2;
      const uint32_t from = swz<D, true>(row, ch * 16);
      const uint32_t to0 = op_chunk(row, 2 * ch), to1 = op_chunk(row, 2 * ch + 1);
      auto widen = [&](uint32_t src, uint32_t dst) {
#pragma unroll
        for (int half = 0; half < H; ++half) {
          uint4 x[4];
          // bytes 64 .. 127 of a row: chunk index + 4, under the swizzle chunk ^ 4
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = ld_shared_v4(src + (from ^ (half * 64)) + i * 32 * D);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 a, b;
            e4m3x4_to_f16x2x2(x[i].x, a.x, a.y);
            e4m3x4_to_f16x2x2(x[i].y, a.z, a.w);
            e4m3x4_to_f16x2x2(x[i].z, b.x, b.y);
            e4m3x4_to_f16x2x2(x[i].w, b.z, b.w);
            st_shared_v4(dst + half * PL::kHalfBytes + to0 + i * 32 * 128, a);
            st_shared_v4(dst + half * PL::kHalfBytes + to1 + i * 32 * 128, b);
          }
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
    const int tl = r / p.group, nh = r - tl * p.group;
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
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
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
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
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
    float m_used = -INFINITY, l = 0.f;
    for (int n = 0; n < ntg && ok; ++n) {
      const int j = alternate ? 2 * n + g : n;     // key tile
      ok = __all_sync(0xffffffffu, tc_wait(bar_s_full + 8u * g, n & 1, s_abort));
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t sr[4][32];
#pragma unroll
      for (int x = 0; x < 4; ++x) tc_ld_32x32b_x32(trow + scol + 32 * x, sr[x]);
      tc_wait_ld();
      float z[kSpKeys];
#pragma unroll
      for (int c = 0; c < kSpKeys; ++c) z[c] = __uint_as_float(sr[c >> 5][c & 31]);
      // keys past the part's last block (the last tile's, loaded as zeros)
      const int keys = nblk * kBS - j * kSpKeys;
      float mul = scale;
      if (keys < kSpKeys) {  // scaled here: a masked key is -inf whatever the scale's sign
#pragma unroll
        for (int c = 0; c < kSpKeys; ++c) z[c] = c < keys ? z[c] * scale : -INFINITY;
        mul = 1.f;
      }
      uint64_t lsum[2];
      // P = 2^(z mul - m) in two 16-bit halves over the score columns: hi
      // in the first 64, lo in the last 64; l sums P in fp32
      auto form_p = [&](float neg_m) {
        const uint64_t sc2 = f2(mul, mul), nm2 = f2(neg_m, neg_m);
        lsum[0] = lsum[1] = f2(0.f, 0.f);
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c = 32 * qq + 2 * e;
            float x0, x1, u0, u1;
            f2_split(f2_fma(f2(z[c], z[c + 1]), sc2, nm2), x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            hi[e] = pack2<FP8>(p0, p1);
            unpack2<FP8>(hi[e], u0, u1);
            lo[e] = pack2<FP8>(p0 - u0, p1 - u1);
            lsum[e & 1] = f2_add(lsum[e & 1], f2(p0, p1));
          }
          tc_st_32x32b_x16(trow + scol + 16 * qq, hi);
          tc_st_32x32b_x16(trow + scol + 64 + 16 * qq, lo);
        }
      };
      auto tile_sum = [&]() {
        float a0, a1, b0, b1;
        f2_split(lsum[0], a0, a1);
        f2_split(lsum[1], b0, b1);
        return (a0 + b0) + (a1 + b1);
      };
      // A row's first tile takes its maximum first. Any later one is formed
      // against the reference in use: a softmax is the same for any
      // reference, and the halves keep their relative precision as long as
      // the weights stay in the type's range, which the tile's sum tells.
      constexpr float kSumMax = FP8 ? kSpSumMaxF16 : kSpSumMaxBf16;
      bool redo = true;
      if (__all_sync(0xffffffffu, !valid || m_used != -INFINITY)) {
        form_p(m_used == -INFINITY ? 0.f : -m_used);
        redo = __any_sync(0xffffffffu, valid && !(tile_sum() <= kSumMax));
        if (redo) tc_wait_st();  // the second pass rewrites the same columns
      }
      if (redo) {
        float mx = z[0];
#pragma unroll
        for (int c = 1; c + 1 < kSpKeys; c += 2) mx = fmax3(mx, z[c], z[c + 1]);
        mx = fmaxf(mx, z[kSpKeys - 1]);
        if (mul < 0.f) {  // then the largest argument is the smallest score's
          mx = z[0];
#pragma unroll
          for (int c = 1; c < kSpKeys; ++c) mx = fminf(mx, z[c]);
        }
        const float m_new = fmaxf(m_used, mx * mul - (FP8 ? kSpF16Log2 : 0.f));
        const float alpha = m_new == m_used ? 1.f : ex2_approx(m_used - m_new);
        m_used = m_new;
        l *= alpha;
        form_p(m_used == -INFINITY ? 0.f : -m_used);
        if (n > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O_g holds the earlier products: they completed before these scores
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tc_ld_32x32b_x32(trow + ocol + cc * 32, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc_st_32x32b_x32(trow + ocol + cc * 32, o);
          }
        }
      }
      l += tile_sum();
      tc_wait_st();
      tc_fence_before_sync();
      mbar_arrive(bar_p_full + 8u * g);
    }
    // ------------------------------------------------------------ epilogue
    if (ok && ntg > 0) ok = __all_sync(0xffffffffu, tc_wait(bar_o_done + 8u * g, 0, s_abort));
    tc_fence_after_sync();
    const int64_t at = (static_cast<int64_t>(part) * p.num_seqs + seq0 + sl) * p.num_q_heads + h * p.group + nh;
    float *dst = p.rec_o + at * D;
    if (!alternate || nt == 1) {
      if (ok && ntg > 0) {
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tc_ld_32x32b_x32(trow + ocol + cc * 32, o);
          tc_wait_ld();
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_global_v8(dst + cc * 32 + e, o + e);
          }
        }
        if (valid) p.rec_ml[at] = make_float2(m_used, l);
      }
    } else {
      // Both warpgroups hold a share of the same rows. Every MMA and copy has
      // completed once both have seen their last product, so the second
      // leaves its share in the K ring and the first joins it.
      ok = named_bar_and(3, 256, ok);
      float4 *so = reinterpret_cast<float4 *>(base_ptr + PL::kKOff);    // [D / 4][128]
      float2 *sml = reinterpret_cast<float2 *>(base_ptr + PL::kTileBytes);  // query tile 1's place
      if (ok && g == 1) {
#pragma unroll 1
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
        const float2 other = sml[r];
        const float M = fmaxf(m_used, other.x);
        const float wa = M == -INFINITY ? 0.f : ex2_approx(m_used - M);
        const float wb = M == -INFINITY ? 0.f : ex2_approx(other.x - M);
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tc_ld_32x32b_x32(trow + ocol + cc * 32, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 y = so[(cc * 8 + e / 4) * kSpRows + r];
            o[e] = __float_as_uint(wa * __uint_as_float(o[e]) + wb * y.x);
            o[e + 1] = __float_as_uint(wa * __uint_as_float(o[e + 1]) + wb * y.y);
            o[e + 2] = __float_as_uint(wa * __uint_as_float(o[e + 2]) + wb * y.z);
            o[e + 3] = __float_as_uint(wa * __uint_as_float(o[e + 3]) + wb * y.w);
          }
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_global_v8(dst + cc * 32 + e, o + e);
          }
        }
        if (valid) p.rec_ml[at] = make_float2(M, wa * l + wb * other.y);
      }
    }
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
      const int64_t at = (static_cast<int64_t>(p.prefix_parts + part) * p.num_seqs + s) * p.num_q_heads + h * p.group + n;
      float *dst = p.rec_o + at * D;
      if (gq == 0)  // weights of E4M3 tiles are 2^(z - m + 8)
        p.rec_ml[at] = make_float2(ws.m[nt][c] - (FP8 ? kSpF16Log2 : 0.f), ws.l[nt][c]);
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int d0 = FP8 ? 16 * mt + 2 * gq : 16 * mt + gq, d1 = FP8 ? d0 + 1 : d0 + 8;
        dst[d0] = ws.acc[nt][mt][c];
        dst[d1] = ws.acc[nt][mt][2 + c];
      }
    }
}

// ------------------------------------------------------------------- join

// One warp a row (sequence, query head), its prefix records and its own parts:
//     out = out_scale sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i,
// kJoinBatch records in flight, M the maximum so far. Bound by L2: the long
// prefix's 19 records a row are 41 MB. Whole calls with two, four and eight
// in flight: 10.0, 9.4, 9.6 us (4 sequences), 152, 150, 150 (64 sequences
// behind 32768 tokens).
constexpr int kJoinBatch = 4;

template <int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const SharedParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_q_heads;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= rows) return;
  const SharedRow r = shared_row(p, static_cast<int>(w / p.num_q_heads));
  const int n = r.prefix_parts + r.own_parts;
  wait_for_primary();
  float acc[V], M = -INFINITY, l = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int i0 = 0; i0 < n; i0 += kJoinBatch) {
    float2 ml[kJoinBatch];
    float x[kJoinBatch][V];
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      const int i = min(i0 + u, n - 1);
      const int64_t at = (i < r.prefix_parts ? i : p.prefix_parts + i - r.prefix_parts) * rows + w;
      ml[u] = p.rec_ml[at];
      const float *o = p.rec_o + at * D + lane * V;
      if constexpr (V == 4) {
        const float4 y = *reinterpret_cast<const float4 *>(o);
        x[u][0] = y.x;
        x[u][1] = y.y;
        x[u][2] = y.z;
        x[u][3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2 *>(o);
        x[u][0] = y.x;
        x[u][1] = y.y;
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) top = fmaxf(top, ml[u].x);
    const float a = M == -INFINITY ? 0.f : exp2f(M - top);
    M = top;
    l *= a;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= a;
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      if (i0 + u >= n || ml[u].x == -INFINITY) continue;
      const float wt = exp2f(ml[u].x - M);
      l += wt * ml[u].y;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += wt * x[u][v];
    }
  }
  float *out = p.out + w * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = n > 0 ? acc[v] / l * p.out_scale : 0.f;  // no token: zeros
  if constexpr (V == 4)
    *reinterpret_cast<float4 *>(out) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  else
    *reinterpret_cast<float2 *>(out) = make_float2(acc[0], acc[1]);
}

}  // namespace pa
