// Rotary positions of a step's queries and keys, with the keys and values
// written to their cache slots in the same pass.
//
// The key rows that reshape_and_cache ("第 7 章推理框架：vLLM 与
// PagedAttention" §7.1 "Block 与 Block Table"; "GPU 学习日报 Day 28" §4.2)
// stores are already rotated; this kernel takes the projections' output
// instead. For pair i of a head (elements (i, i + r/2), or (2i, 2i + 1)
// interleaved, of its first r) of the token at position t:
//     theta = t * inv_freq[i],
//     (a, b) -> rope_scale * (a cos theta - b sin theta, b cos theta + a sin theta),
// in fp32, rounded once to what is stored (bf16, or E4M3 of y / scale).
//
// The angle. t * inv_freq in fp32 is off by up to 2^-25 of the angle: 4e-3
// radians at position 131072, more than bf16 resolves. Only the fraction of
// a turn matters, so inv_freq / 2 pi is held as a 64-bit fixed-point
// fraction of a turn, F = round(2^64 frac(inv_freq / 2 pi)), and
// t * F mod 2^64 is one integer product that wraps; its high word as a float
// (2^-25 of a half turn) goes to sincospi. The product multiplies F's own
// error by t, so F is formed from inv_freq / 2 pi in two doubles (off by
// 2^-105 of it) and is off by one unit of 2^-64 turns: at 2^31, 2^-33 turns.
// One double would leave 2^-53 of the angle, 2e-5 radians for 100 at 2^31.
// Together below 2^-23 radians + 2^-104 |t inv_freq|.
//
// What bounds it: DRAM for prompts (32768 tokens of 32 query and 8 KV heads
// of 128, 806 MB, in 132 to 137 us: 0.90 to 0.93 of the copy bandwidth), the
// latency of a launch, a load and a sincospi for a decode step (64 tokens of
// 32 and 32 heads 2.5 us, in a graph). Layout: a CTA takes a few tokens,
// computes each (token, pair)'s cosine and sine once into shared memory,
// then moves units of 16 elements (two 16-byte loads, two stores): a pair
// of partner chunks in the half layout, two neighbouring chunks in the
// interleaved one, so every unit needs eight consecutive frequencies.
#pragma once

#include "cache_ops.cuh"

namespace pa {

constexpr int kRopeThreads = 128;
constexpr int kRopeTokens = 4;     // most tokens of a CTA
constexpr int kRopeBatch = 3;      // units of a thread in flight
constexpr int kRopeMaxPairs = 64;  // rotary_dim <= 128

struct RopeParams {
  const uint16_t *q;          // bf16, token stride q_stride, heads contiguous
  const uint16_t *key;
  const uint16_t *value;
  uint16_t *q_out;            // bf16 [T][Hq][D]
  void *k_cache;
  void *v_cache;
  const int64_t *slots;       // [T]
  const int32_t *positions;   // [T]
  const double *inv_freq;     // [rotary_dim / 2]
  int64_t q_stride, k_stride, v_stride;  // elements
  int64_t num_slots;
  int num_tokens;
  int tokens_per_cta;         // <= kRopeTokens
  int units_per_cta;          // grid.y slices of the tokens' units
  int num_q_heads;
  int num_kv_heads;
  int rotary_dim;
  float rope_scale;
  float k_scale, v_scale;
};

// cosine and sine of position * inv_freq (see the head comment), times scale
__device__ __forceinline__ float2 rope_cos_sin(int position, double inv_freq, float scale) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / 2 pi
  double hi = inv_freq * kHi;
  double lo = fma(inv_freq, kLo, fma(inv_freq, kHi, -hi));
  hi -= rint(hi);
  lo -= rint(lo);
  constexpr double kUnits = 18446744073709551616.0;
  const uint64_t f = static_cast<uint64_t>(__double2ll_rn(hi * kUnits)) + static_cast<uint64_t>(__double2ll_rn(lo * kUnits));
  const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(position)) * f;
  const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ void unpack8(const uint4 x, float (&f)[8]) {
  unpack2<false>(x.x, f[0], f[1]);
  unpack2<false>(x.y, f[2], f[3]);
  unpack2<false>(x.z, f[4], f[5]);
  unpack2<false>(x.w, f[6], f[7]);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<false>(f[0], f[1]), pack2<false>(f[2], f[3]), pack2<false>(f[4], f[5]),
                    pack2<false>(f[6], f[7]));
}
// eight floats -> E4M3(f / scale), rounded once from fp32
__device__ __forceinline__ uint2 e4m3_of8(const float (&f)[8], float scale) {
  uint32_t o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(f[4 * j], scale), __fdiv_rn(f[4 * j + 1], scale)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(f[4 * j + 2], scale), __fdiv_rn(f[4 * j + 3], scale)), __NV_SATFINITE, __NV_E4M3);
    o[j] = (lo & 0xFFFFu) | (hi << 16);
  }
  return make_uint2(o[0], o[1]);
}

template <int D, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_and_cache_kernel(const RopeParams p) {
  constexpr int UNITS = D / 16;  // units of a head row
  constexpr int U = kRopeBatch;
  __shared__ float2 s_cs[kRopeTokens][kRopeMaxPairs];
  __shared__ int64_t s_slot[kRopeTokens];
  const int pairs = p.rotary_dim / 2;
  const int t0 = blockIdx.x * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, p.num_tokens - t0);
  const int per_token = (p.num_q_heads + 2 * p.num_kv_heads) * UNITS;
  // this CTA's slice of its tokens' units
  const int first = blockIdx.y * p.units_per_cta, last = min(first + p.units_per_cta, nt * per_token);

  struct Unit {
    const uint16_t *src;
    int tl, h, e0, e1;
    bool is_q, is_v, turned;
  };
  auto unit = [&](int i) {
    Unit n;
    n.tl = 0;
#pragma unroll
    for (int k = 1; k < kRopeTokens; ++k) n.tl += i >= k * per_token;
    const int r = (i - n.tl * per_token) / UNITS, u = i % UNITS;
    n.is_q = r < p.num_q_heads;
    n.is_v = r >= p.num_q_heads + p.num_kv_heads;
    n.h = n.is_q ? r : (n.is_v ? r - p.num_q_heads - p.num_kv_heads : r - p.num_q_heads);
    n.turned = !n.is_v && 16 * u < p.rotary_dim;
    const bool apart = n.turned && !INTERLEAVED;
    n.e0 = apart ? 8 * u : 16 * u;
    n.e1 = apart ? p.rotary_dim / 2 + 8 * u : 16 * u + 8;
    const int64_t t = t0 + n.tl;
    n.src = (n.is_q ? p.q + t * p.q_stride : (n.is_v ? p.value + t * p.v_stride : p.key + t * p.k_stride)) + n.h * D;
    return n;
  };

  bool ready = false;
  for (int base = first; base < last; base += U * kRopeThreads) {
    // the batch's loads first: they are in flight while the angles are formed
    uint4 x0[U], x1[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = base + k * kRopeThreads + threadIdx.x;
      if (i < last) {
        const Unit n = unit(i);
        x0[k] = *reinterpret_cast<const uint4 *>(n.src + n.e0);
        x1[k] = *reinterpret_cast<const uint4 *>(n.src + n.e1);
      }
    }
    if (!ready) {
      for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
        const int t = i / pairs, f = i - t * pairs;
        s_cs[t][f] = rope_cos_sin(p.positions[t0 + t], p.inv_freq[f], p.rope_scale);
      }
      if (static_cast<int>(threadIdx.x) < nt) {
        int64_t slot = p.slots[t0 + threadIdx.x];
        if (slot >= p.num_slots) {
          if (blockIdx.y == 0) raise_error(kErrSlotRange);
          slot = -1;
        }
        s_slot[threadIdx.x] = slot;
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = base + k * kRopeThreads + threadIdx.x;
      if (i >= last) continue;
      const Unit n = unit(i);
      const int64_t slot = s_slot[n.tl];
      if (!n.is_q && slot < 0) continue;
      float a[8], b[8];
      unpack8(x0[k], a);
      unpack8(x1[k], b);
      if (n.turned) {
        const float2 *cs = &s_cs[n.tl][8 * (i % UNITS)];
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float2 w = cs[j / 2], z = cs[4 + j / 2];
            const float a0 = a[j], a1 = a[j + 1], b0 = b[j], b1 = b[j + 1];
            a[j] = a0 * w.x - a1 * w.y;
            a[j + 1] = a1 * w.x + a0 * w.y;
            b[j] = b0 * z.x - b1 * z.y;
            b[j + 1] = b1 * z.x + b0 * z.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 w = cs[j];
            const float a0 = a[j], b0 = b[j];
            a[j] = a0 * w.x - b0 * w.y;
            b[j] = b0 * w.x + a0 * w.y;
          }
        }
      }
      if (n.is_q) {
        uint16_t *dst = p.q_out + (static_cast<int64_t>(t0 + n.tl) * p.num_q_heads + n.h) * D;
        *reinterpret_cast<uint4 *>(dst + n.e0) = n.turned ? pack8(a) : x0[k];
        *reinterpret_cast<uint4 *>(dst + n.e1) = n.turned ? pack8(b) : x1[k];
      } else {
        const int64_t row = ((slot / kBS * p.num_kv_heads + n.h) * kBS + slot % kBS) * D;
        void *cache = n.is_v ? p.v_cache : p.k_cache;
        if constexpr (FP8) {
          const float scale = n.is_v ? p.v_scale : p.k_scale;
          uint8_t *dst = static_cast<uint8_t *>(cache) + row;
          *reinterpret_cast<uint2 *>(dst + n.e0) = e4m3_of8(a, scale);
          *reinterpret_cast<uint2 *>(dst + n.e1) = e4m3_of8(b, scale);
        } else {
          uint16_t *dst = static_cast<uint16_t *>(cache) + row;
          *reinterpret_cast<uint4 *>(dst + n.e0) = n.turned ? pack8(a) : x0[k];
          *reinterpret_cast<uint4 *>(dst + n.e1) = n.turned ? pack8(b) : x1[k];
        }
      }
    }
  }
}

}  // namespace pa
