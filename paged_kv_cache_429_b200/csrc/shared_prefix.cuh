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
#pragma once

#include "decode.cuh"

namespace pa {

constexpr uint32_t kErrGroupRange = 0x100u;

struct SharedParams {
  float *out;                    // [S][Hq][D]
  const uint16_t *q;             // bf16 [S][Hq][D]
  const void *k_cache;
  const void *v_cache;
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
  float score_scale;             // sm_scale * log2(e) [* k_scale for fp8]
  float out_scale;               // v_scale for fp8, 1 for bf16
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

// The group of sequence s: its prefix in blocks (clamped; 0 for a sequence
// of no group) and its first sequence, whose table holds the prefix.
__device__ __forceinline__ int shared_blocks_of(const SharedParams &p, int s, int *first) {
  int lo = 0, hi = p.num_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.group_start[mid] <= s)
      lo = mid;
    else
      hi = mid;
  }
  *first = s;
  if (p.num_groups == 0 || s < p.group_start[lo] || s >= p.group_start[lo + 1]) return 0;
  *first = max(p.group_start[lo], 0);
  return min(max(p.prefix_blocks[lo], 0), min(p.max_prefix_blocks, p.max_blocks_per_seq));
}

// Element e of a cache row of 16-bit or E4M3 elements.
template <bool FP8>
__device__ __forceinline__ float cache_value(const void *cache, int64_t i) {
  if constexpr (FP8) {
    float lo, hi;
    e4m3x2_to_f32x2(static_cast<const uint8_t *>(cache)[i], lo, hi);
    return lo;
  } else {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(cache)[i]) << 16);
  }
}

// One warp a (sequence, query head): the running maximum and sum of the
// softmax over the tokens one by one, each lane a head_dim / 32 slice.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) shared_prefix_simple_kernel(const SharedParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int s = static_cast<int>(w / p.num_q_heads), hq = static_cast<int>(w % p.num_q_heads);
  if (blockIdx.x == 0) check_groups(p);
  if (s >= p.num_seqs) return;
  const int h = hq / p.group;
  bool bad_len;
  int L = clamped_len(p.context_lens, s, p.max_context_len, p.max_blocks_per_seq, &bad_len);
  int first;
  const int nb = shared_blocks_of(p, s, &first);
  if (L - nb * kBS > p.max_suffix_len) {
    bad_len = true;
    L = nb * kBS + p.max_suffix_len;
  }
  if (lane == 0 && hq == 0 && bad_len) raise_error(kErrContextClamp);
  float q[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    q[v] = cache_value<false>(p.q, w * D + v * 32 + lane);
    acc[v] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  bool bad_id = false;
  for (int t = 0; t < L; ++t) {
    const int j = t / kBS;
    const int row = j < nb ? first : s;
    const int id = p.block_tables[static_cast<int64_t>(row) * p.max_blocks_per_seq + j];
    const bool in_pool = id >= 0 && id < p.num_blocks;
    bad_id |= !in_pool;
    const int64_t at = ((static_cast<int64_t>(id) * p.num_kv_heads + h) * kBS + t % kBS) * D + lane;
    float z = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) z += in_pool ? q[v] * cache_value<FP8>(p.k_cache, at + v * 32) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z *= p.score_scale;
    const float mn = fmaxf(m, z);
    const float a = m == mn ? 1.f : exp2f(m - mn), e = exp2f(z - mn);
    l = l * a + e;
#pragma unroll
    for (int v = 0; v < V; ++v)
      acc[v] = acc[v] * a + e * (in_pool ? cache_value<FP8>(p.v_cache, at + v * 32) : 0.f);
    m = mn;
  }
  if (bad_id && lane == 0) raise_error(kErrBlockRange);
#pragma unroll
  for (int v = 0; v < V; ++v) p.out[w * D + v * 32 + lane] = L > 0 ? acc[v] / l * p.out_scale : 0.f;
}

}  // namespace pa
