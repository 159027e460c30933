// C ABI of libpa.so: argument checks, TMA descriptor set-up and launches.
// Declarations and the contract of every entry point: include/pa.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pa.h"
#include "cache_ops.cuh"
#include "decode.cuh"
#include "decode_tc.cuh"
#include "prefill.cuh"
#include "rope.cuh"
#include "shared_prefix.cuh"
#include "tables.cuh"

namespace {

using pa::DecodeParams;
using pa::Geo;
using pa::ReduceParams;

constexpr int kMaxDevices = 64;
constexpr int kDefaultPartition = 512;   // automatic split, contexts up to kLongContext
constexpr int kLongPartition = 2048;     // automatic split above kLongContext tokens
constexpr int kLongContext = 16384;

bool aligned(const void *ptr, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) % a) == 0;
}

// --- driver entry point for tensor-map encoding (no link against libcuda)
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  std::call_once(g_encode_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault,
                                &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

int device_sm_count(int dev) {
  static std::atomic<int> cache[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return 148;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
    v = 148;
  cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Tensor map over one cache viewed as a 2-D array [num_blocks*Hkv*16][D].
template <int D, bool FP8>
bool make_cache_tmap(CUtensorMap *map, const void *base, int rows) {
  using G = Geo<D, FP8>;
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(G::kRowBytes)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(G::kBoxRow / G::kEB), static_cast<cuuint32_t>(pa::kBS)};
  cuuint32_t estr[2] = {1, 1};
  const CUtensorMapSwizzle sw =
      G::kBoxRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  CUresult r = enc(map, FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   2, const_cast<void *>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Q rows of a prefill tile: a 3-D view [tokens][query heads][head_dim] of
// the bf16 queries, box (64 dims, the GQA group's heads, tokens of the tile)
// with the 128-byte swizzle, so a tile lands as 128-byte rows ordered
// (token, head) — the K-major operand layout of the tensor core.
bool make_q_tmap(CUtensorMap *map, const void *q, int num_tokens, int num_q_heads,
                 int head_dim, int group, int tokens_per_tile) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(num_q_heads),
                        static_cast<cuuint64_t>(num_tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2,
                           static_cast<cuuint64_t>(num_q_heads) * head_dim * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group),
                       static_cast<cuuint32_t>(tokens_per_tile)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Prefill output rows: a 3-D view [tokens][query heads][head_dim] of the
// fp32 output, box (16 columns = 64 bytes, the GQA group's heads, tokens
// of a tile) with the 64-byte swizzle, the layout the kernel stages O in.
bool make_out_tmap(CUtensorMap *map, float *out, int num_tokens, int num_q_heads, int head_dim,
                   int group, int tokens_per_tile) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(num_q_heads),
                        static_cast<cuuint64_t>(num_tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 4,
                           static_cast<cuuint64_t>(num_q_heads) * head_dim * 4};
  cuuint32_t box[3] = {16, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tokens_per_tile)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, out, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <typename Kern>
bool ensure_smem_attr(Kern kern, size_t bytes, std::atomic<uint64_t> &done, int dev) {
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) != cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

template <int D, bool FP8, int NT, bool CHUNKED, bool APPEND>
pa_status launch_decode(const void *k_cache, const void *v_cache, int rows,
                        const DecodeParams &p, int num_seqs, int grid_x,
                        cudaStream_t stream, int dev) {
  CUtensorMap tk, tv;
  if (!make_cache_tmap<D, FP8>(&tk, k_cache, rows) ||
      !make_cache_tmap<D, FP8>(&tv, v_cache, rows))
    return PA_ERR_CUDA;
  auto kern = NT == 1 ? pa::paged_decode_kernel<D, FP8, CHUNKED, APPEND>
                      : pa::paged_decode_kernel_wide<D, FP8, CHUNKED, APPEND>;
  static std::atomic<uint64_t> attr_done{0};
  const size_t smem = pa::Plan<D, FP8, NT, CHUNKED>::kSmemBytes;
  if (!ensure_smem_attr(kern, smem, attr_done, dev)) return PA_ERR_CUDA;
  dim3 grid(grid_x, p.num_kv_heads, num_seqs);
  kern<<<grid, pa::kDecodeThreads, smem, stream>>>(tk, tv, p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// The fp8 decode on the 5th-generation tensor core (decode_tc.cuh): head_dim
// 128, single-pass, one CTA per (sequence, KV head).
template <int GMAX, bool APPEND>
pa_status launch_decode_tc(const void *k_cache, const void *v_cache, int rows,
                           const DecodeParams &p, int num_seqs, cudaStream_t stream, int dev) {
  CUtensorMap tk, tv;
  if (!make_cache_tmap<128, true>(&tk, k_cache, rows) ||
      !make_cache_tmap<128, true>(&tv, v_cache, rows))
    return PA_ERR_CUDA;
  auto kern = pa::paged_decode_tc_kernel<GMAX, APPEND>;
  static std::atomic<uint64_t> attr_done{0};
  const size_t smem = pa::TdPlan<GMAX>::kSmemBytes;
  if (!ensure_smem_attr(kern, smem, attr_done, dev)) return PA_ERR_CUDA;
  dim3 grid(1, p.num_kv_heads, num_seqs);
  kern<<<grid, pa::kTdThreads, smem, stream>>>(tk, tv, p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D>
pa_status launch_reduce(const ReduceParams &r, int num_seqs, cudaStream_t stream) {
  dim3 grid(r.num_q_heads, num_seqs);
  pa::paged_decode_reduce_kernel<D><<<grid, pa::kReduceWarps * 32, 0, stream>>>(r);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool FP8>
pa_status dispatch_nt(int nt, bool chunked, const void *kc, const void *vc, int rows,
                      const DecodeParams &p, int num_seqs, int grid_x, cudaStream_t st,
                      int dev) {
  if (p.new_k) {
    if (chunked)
      return nt == 1 ? launch_decode<D, FP8, 1, true, true>(kc, vc, rows, p, num_seqs, grid_x, st, dev)
                     : launch_decode<D, FP8, 2, true, true>(kc, vc, rows, p, num_seqs, grid_x, st, dev);
    return nt == 1 ? launch_decode<D, FP8, 1, false, true>(kc, vc, rows, p, num_seqs, grid_x, st, dev)
                   : launch_decode<D, FP8, 2, false, true>(kc, vc, rows, p, num_seqs, grid_x, st, dev);
  }
  if (chunked)
    return nt == 1 ? launch_decode<D, FP8, 1, true, false>(kc, vc, rows, p, num_seqs, grid_x, st, dev)
                   : launch_decode<D, FP8, 2, true, false>(kc, vc, rows, p, num_seqs, grid_x, st, dev);
  return nt == 1 ? launch_decode<D, FP8, 1, false, false>(kc, vc, rows, p, num_seqs, grid_x, st, dev)
                 : launch_decode<D, FP8, 2, false, false>(kc, vc, rows, p, num_seqs, grid_x, st, dev);
}

// Consecutive partitions per CTA in the split path: about 1 MB of K/V per
// CTA, while keeping at least four CTAs per SM in the grid. Chunks of more
// than one partition need partitions of a whole number of ring rounds
// (4 consumer warps x `bps` blocks per stage).
int partitions_per_cta(int64_t units, int64_t P, int psize, int head_dim, int eb, int bps,
                       int sms) {
  const int pb = psize / pa::kBS;
  if (pb % (pa::kConsumerWarps * bps) != 0) return 1;
  const int64_t part_bytes = static_cast<int64_t>(psize) * head_dim * eb * 2;
  int64_t ppc = std::max<int64_t>(1, (int64_t{1} << 20) / std::max<int64_t>(part_bytes, 1));
  ppc = std::min<int64_t>(ppc, P);
  while (ppc > 1 && units * ((P + ppc - 1) / ppc) < 4LL * sms) ppc = (ppc + 1) / 2;
  return static_cast<int>(ppc);
}

size_t workspace_bytes_for(int num_seqs, int num_q_heads, int head_dim, int max_context_len,
                           int psize) {
  const int64_t P = (static_cast<int64_t>(max_context_len) + psize - 1) / psize;
  const int64_t floats = static_cast<int64_t>(num_seqs) * num_q_heads * P * (head_dim + 2);
  const int64_t bytes = floats * 4 + 2 * 256;  // two sub-array alignments
  return static_cast<size_t>((bytes + 255) / 256 * 256);
}

// How pa_decode_shared_prefix cuts its work, from the host-known bounds alone
// (the workspace size must not depend on the device).
struct SharedPlan {
  int row_tiles;      // CTAs along the rows: pairs of 128-row query tiles over all groups
  int prefix_parts;   // parts of the longest prefix
  int suffix_parts;   // parts of the longest suffix
  int part_len;
  size_t o_bytes, bytes;  // of the records' o, and of the whole workspace
};

SharedPlan shared_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int num_groups,
                       int max_prefix_blocks, int max_suffix_len) {
  constexpr int kSms = 148;
  SharedPlan s{};
  const int per_cta = 2 * (pa::kSpRows / (num_q_heads / num_kv_heads));
  const int64_t groups = std::min(num_groups, num_seqs);
  s.row_tiles = groups > 0 && max_prefix_blocks > 0
                    ? static_cast<int>((num_seqs + groups * (per_cta - 1)) / per_cta)
                    : 0;
  // Prefix parts, of at most kSpPartTiles key tiles: the number that makes
  // waves x (key tiles of a part + 2) smallest; two tiles stand for a CTA's
  // start and its output (four in their place chose the same parts).
  if (s.row_tiles > 0) {
    const int64_t tiles = pa::ceil_div(max_prefix_blocks, pa::kSpBlocks);
    const int64_t units = static_cast<int64_t>(s.row_tiles) * num_kv_heads;
    const int64_t least = (tiles + pa::kSpPartTiles - 1) / pa::kSpPartTiles;
    int64_t best = INT64_MAX;
    for (int64_t n = least; n <= std::max<int64_t>(std::min<int64_t>(tiles, 128), least); ++n) {
      const int64_t per = (tiles + n - 1) / n, used = (tiles + per - 1) / per;
      const int64_t cost = (units * used + kSms - 1) / kSms * (per + 2);
      if (cost < best) {
        best = cost;
        s.prefix_parts = static_cast<int>(used);
      }
    }
  }
  // Suffix parts: about three waves of resident CTAs (3 per SM), at least 256
  // tokens each. Suffixes alone, bf16, 32 query and 8 KV heads: 16 sequences
  // of up to 4096 tokens 33.3 us (two waves 34.8, four 35.8), 64 of up to
  // 1024 33.3 (37.0, 35.8), 4 of up to 8192 16.0 (15.5, 16.0); 4 of up to
  // 1000 with 32 KV heads 11.6 (13.5 with parts of 128 tokens, 15.5 of 512).
  const int64_t units = std::max<int64_t>(static_cast<int64_t>(num_seqs) * num_kv_heads, 1);
  const int64_t wanted = std::max<int64_t>(1, 3 * 3 * kSms / units);
  int64_t len = (max_suffix_len + wanted - 1) / wanted;
  len = std::max<int64_t>((len + 127) / 128 * 128, 256);
  s.part_len = static_cast<int>(std::min<int64_t>(len, INT32_MAX / 128 * 128));
  s.suffix_parts = static_cast<int>(
      std::max<int64_t>((static_cast<int64_t>(max_suffix_len) + s.part_len - 1) / s.part_len, 1));
  const size_t rows = (static_cast<size_t>(s.prefix_parts) + s.suffix_parts) * num_seqs * num_q_heads;
  s.o_bytes = (rows * head_dim * 4 + 255) / 256 * 256;
  s.bytes = s.o_bytes + (rows * 8 + 255) / 256 * 256;
  return s;
}

// A prefix part is a CTA along grid.z: bounds above 134 million tokens have too many.
constexpr int kSharedMaxPrefixBlocks = 65535 * pa::kSpPartTiles * pa::kSpBlocks;

// A launch that may start before the stream's kernel in front has finished
// (the kernel itself waits for it before it reads what that one writes).
template <typename... Params, typename... Args>
pa_status launch_beside(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool FP8, int NT>
pa_status launch_shared_suffix(const CUtensorMap &tk, const CUtensorMap &tv, const pa::SharedParams &p,
                               cudaStream_t st, int dev) {
  auto kern = pa::shared_suffix_kernel<D, FP8, NT>;
  static std::atomic<uint64_t> attr_done{0};
  constexpr size_t smem = pa::Plan<D, FP8, NT, false>::kSmemBytes;
  if (!ensure_smem_attr(kern, smem, attr_done, dev)) return PA_ERR_CUDA;
  const dim3 grid(p.suffix_parts, p.num_kv_heads, p.num_seqs);
  if (p.row_tiles > 0) return launch_beside(kern, grid, pa::kDecodeThreads, smem, st, tk, tv, p);
  kern<<<grid, pa::kDecodeThreads, smem, st>>>(tk, tv, p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool FP8>
pa_status launch_shared(const pa::SharedParams &p, const void *k_cache, const void *v_cache, int rows,
                        cudaStream_t st, int dev) {
  CUtensorMap tq, tk, tv;
  if (!make_q_tmap(&tq, p.q, p.num_seqs, p.num_q_heads, D, p.group, p.tokens_per_tile) ||
      !make_cache_tmap<D, FP8>(&tk, k_cache, rows) || !make_cache_tmap<D, FP8>(&tv, v_cache, rows))
    return PA_ERR_CUDA;
  if (p.row_tiles > 0) {
    auto kern = pa::shared_prefix_kernel<D, FP8>;
    static std::atomic<uint64_t> attr_done{0};
    using PL = pa::SpPlan<D, FP8>;
    if (!ensure_smem_attr(kern, PL::kSmemBytes, attr_done, dev)) return PA_ERR_CUDA;
    kern<<<dim3(p.row_tiles, p.num_kv_heads, p.prefix_parts), PL::kThreads, PL::kSmemBytes, st>>>(tq, tk, tv, p);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  }
  const pa_status rc = p.group <= 8 ? launch_shared_suffix<D, FP8, 1>(tk, tv, p, st, dev)
                                    : launch_shared_suffix<D, FP8, 2>(tk, tv, p, st, dev);
  if (rc != PA_OK) return rc;
  const int64_t warps = static_cast<int64_t>(p.num_seqs) * p.num_q_heads;
  return launch_beside(pa::shared_join_kernel<D>, dim3(static_cast<unsigned>((warps + 7) / 8)), 256, 0, st, p);
}

template <int D, bool FP8>
pa_status launch_rope(pa::RopeParams p, bool interleaved, cudaStream_t st, int dev) {
  // Few tokens: one a CTA and its units cut into slices of one a thread, so
  // that a decode step fills the GPU; from 10 tokens an SM on, a CTA takes
  // four tokens whole and their angles are formed once. Slices against whole
  // tokens, 32 query and 32 KV heads of 128: 3.5 us against 12.6 at 128
  // tokens, 13.2 against 14.4 at 1024, 26.5 against 22.9 at 2048, 102 against
  // 70 at 8192; 32 and 8 heads, E4M3: 8.3 against 10.7 at 1024, 14.5 against
  // 13.3 at 2048; 8 and 8 heads of 64: 3.2 against 3.5, 5.0 against 4.0.
  const bool few = p.num_tokens < 10 * device_sm_count(dev);
  p.tokens_per_cta = few ? 1 : pa::kRopeTokens;
  const int units = p.tokens_per_cta * (p.num_q_heads + 2 * p.num_kv_heads) * (D / 16);
  p.units_per_cta = few ? pa::kRopeThreads : units;
  const int64_t ctas = (static_cast<int64_t>(p.num_tokens) + p.tokens_per_cta - 1) / p.tokens_per_cta;
  const dim3 grid(static_cast<unsigned>(ctas), (units + p.units_per_cta - 1) / p.units_per_cta);
  if (grid.y > 65535) return PA_ERR_UNSUPPORTED;
  if (interleaved)
    pa::rope_and_cache_kernel<D, FP8, true><<<grid, pa::kRopeThreads, 0, st>>>(p);
  else
    pa::rope_and_cache_kernel<D, FP8, false><<<grid, pa::kRopeThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// One phase of a table kernel, with `ints` integers of dynamic shared memory
// (at most max_ints for any call).
template <typename Params>
pa_status launch_table_kernel(void (*kern)(Params), const Params &p, int64_t ctas, int threads, size_t ints,
                              size_t max_ints, std::atomic<uint64_t> &attr_done, cudaStream_t st, int dev) {
  if (!ensure_smem_attr(kern, max_ints * sizeof(int32_t), attr_done, dev)) return PA_ERR_CUDA;
  kern<<<static_cast<unsigned>(ctas), threads, ints * sizeof(int32_t), st>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Threads of a one-CTA call: as many as its rows, or its tokens four a
// thread, keep busy (a small CTA starts and synchronises sooner).
int table_threads(int64_t rows, int64_t items) {
  const int64_t want = std::max(rows, (items + pa::kTabBatch - 1) / pa::kTabBatch);
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>((want + 31) / 32 * 32, 64), pa::kTabThreads));
}

// The first launch of a large call: at most a CTA on every SM but one, which
// is left to the second launch (it sums the rows meanwhile). CTAs are as
// small as their share of the items lets them be, of 256 threads or more and
// two rows a thread at most.
struct TableGrid {
  int64_t ctas;
  int threads;
};
TableGrid table_grid(int64_t rows, int64_t items, int dev) {
  const int64_t most = std::max(device_sm_count(dev) - 1, 1);
  const int threads = std::max(table_threads((rows + 1) / 2, (items + most - 1) / most), 256);
  const int64_t per_cta = static_cast<int64_t>(threads) * pa::kTabBatch;
  return {std::min((items + per_cta - 1) / per_cta, most), threads};
}

}  // namespace

extern "C" {

const char *pa_status_string(pa_status status) {
  switch (status) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
    case PA_ERR_CUDA: return "PA_ERR_CUDA";
    case PA_ERR_OUT_OF_BLOCKS: return "PA_ERR_OUT_OF_BLOCKS";
    case PA_ERR_NOT_FOUND: return "PA_ERR_NOT_FOUND";
    case PA_ERR_DEVICE: return "PA_ERR_DEVICE";
  }
  return "PA_ERR_UNKNOWN";
}

size_t pa_decode_workspace_size(int num_seqs, int num_q_heads, int head_dim,
                                int max_context_len, int partition_size) {
  if (num_seqs < 0 || num_q_heads <= 0 || head_dim <= 0 || max_context_len < 0)
    return 0;
  if (partition_size == 0) return 0;
  const int psize = partition_size < 0 ? kDefaultPartition : partition_size;
  if (psize % pa::kBS != 0) return 0;
  return workspace_bytes_for(num_seqs, num_q_heads, head_dim, max_context_len, psize);
}

// pa_decode, and with new_k / new_v set pa_decode_append (the step's new
// tokens written by the decode kernel itself).
static pa_status decode_common(float *out, const void *q, const void *k_cache,
                               const void *v_cache, pa_kv_dtype kv_dtype, float k_scale,
                               float v_scale, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *context_lens,
                               int max_context_len, int num_seqs, int num_q_heads,
                               int num_kv_heads, int head_dim, int block_size, int num_blocks,
                               float sm_scale, int partition_size, void *workspace,
                               size_t workspace_bytes, void *stream, const void *new_k,
                               const void *new_v) {
  // ---- shape and pointer checks (host only; nothing launched on error)
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_blocks_per_seq < 0 || max_context_len < 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (block_size != pa::kBS) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  if (group > 16) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale)) return PA_ERR_INVALID_ARG;
  if (kv_dtype == PA_KV_FP8_E4M3 &&
      !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARG;
  if (partition_size < -1 || (partition_size > 0 && partition_size % pa::kBS != 0))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PA_ERR_INVALID_ARG;
  if ((new_k || new_v) && !(new_k && new_v && aligned(new_k, 16) && aligned(new_v, 16)))
    return PA_ERR_INVALID_ARG;
  const int64_t rows64 = static_cast<int64_t>(num_blocks) * num_kv_heads * pa::kBS;
  if (rows64 + pa::kBS >= INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_seqs) > 65535) return PA_ERR_UNSUPPORTED;  // grid.z
  if (num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;                     // grid.y

  const int ctx_cap = static_cast<int>(
      std::min<int64_t>(max_context_len, static_cast<int64_t>(max_blocks_per_seq) * pa::kBS));
  if (partition_size > 0) {  // forced split: the workspace must fit (host check)
    const int64_t P = (static_cast<int64_t>(ctx_cap) + partition_size - 1) / partition_size;
    if (P > 65535) return PA_ERR_UNSUPPORTED;
    const size_t need = workspace_bytes_for(num_seqs, num_q_heads, head_dim, ctx_cap,
                                            partition_size);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need)
      return PA_ERR_WORKSPACE;
  }

  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);

  // ---- path choice
  int psize = partition_size;
  if (psize < 0) {
    // Single-pass when the (sequence, KV head) pairs fill at least two full
    // waves of resident CTAs (3 per SM) and contexts are not long enough for
    // the last wave's imbalance to matter; otherwise split the contexts.
    // Above kLongContext tokens the partitions are 2048 tokens long: a
    // quarter of the partial records to write and combine, and the grid
    // still holds the same number of CTAs (each streams about 1 MB).
    const int64_t units = static_cast<int64_t>(num_seqs) * num_kv_heads;
    const bool wide = units >= 2LL * 3 * device_sm_count(dev);
    const int auto_ps = ctx_cap > kLongContext ? kLongPartition : kDefaultPartition;
    const size_t need = workspace_bytes_for(num_seqs, num_q_heads, head_dim, ctx_cap, auto_ps);
    const bool have_ws = workspace && aligned(workspace, 256) && workspace_bytes >= need;
    psize = (!wide || ctx_cap > kLongContext) && have_ws && ctx_cap > kDefaultPartition
                ? auto_ps
                : 0;
  }

  DecodeParams p{};
  p.out = out;
  p.q = static_cast<const uint16_t *>(q);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.num_blocks = num_blocks;
  if (new_k) {  // selects the APPEND kernels
    p.new_k = static_cast<const uint16_t *>(new_k);
    p.new_v = static_cast<const uint16_t *>(new_v);
    p.k_cache = const_cast<void *>(k_cache);
    p.v_cache = const_cast<void *>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
  }
  const float log2e = 1.4426950408889634f;
  if (kv_dtype == PA_KV_BF16) {
    p.score_scale = sm_scale * log2e;
    p.out_scale = 1.f;
  } else {
    p.score_scale = sm_scale * k_scale * log2e;
    p.out_scale = v_scale;
  }
  int grid_x = 1;
  int64_t P = 1;
  if (psize > 0) {
    P = (static_cast<int64_t>(ctx_cap) + psize - 1) / psize;
    if (P == 0) P = 1;
    if (P > 65535) return PA_ERR_UNSUPPORTED;
    const size_t need = workspace_bytes_for(num_seqs, num_q_heads, head_dim, ctx_cap, psize);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need)
      return PA_ERR_WORKSPACE;
    const int64_t rows = static_cast<int64_t>(num_seqs) * num_q_heads * P;
    char *ws = static_cast<char *>(workspace);
    const size_t o_bytes = (static_cast<size_t>(rows) * head_dim * 4 + 255) / 256 * 256;
    const size_t m_bytes = (static_cast<size_t>(rows) * 4 + 255) / 256 * 256;
    p.ws_o = reinterpret_cast<float *>(ws);
    p.ws_m = reinterpret_cast<float *>(ws + o_bytes);
    p.ws_l = reinterpret_cast<float *>(ws + o_bytes + m_bytes);
    p.partition_blocks = psize / pa::kBS;
    p.max_partitions = static_cast<int>(P);
    const int eb = kv_dtype == PA_KV_BF16 ? 2 : 1;
    const int bps = (pa::kBS * head_dim * eb) >= 4096 ? 1 : 4096 / (pa::kBS * head_dim * eb);
    p.partitions_per_cta = partitions_per_cta(static_cast<int64_t>(num_seqs) * num_kv_heads, P,
                                              psize, head_dim, eb, bps, device_sm_count(dev));
    grid_x = static_cast<int>((P + p.partitions_per_cta - 1) / p.partitions_per_cta);
  }

  const int nt = group <= 8 ? 1 : 2;
  const bool chunked = psize > 0;
  const int rows = static_cast<int>(rows64);
  pa_status rc;
  if (kv_dtype == PA_KV_FP8_E4M3 && head_dim == 128 && !chunked && group <= 8) {
    if (new_k)
      return group <= 4 ? launch_decode_tc<4, true>(k_cache, v_cache, rows, p, num_seqs, st, dev)
                        : launch_decode_tc<8, true>(k_cache, v_cache, rows, p, num_seqs, st, dev);
    return group <= 4 ? launch_decode_tc<4, false>(k_cache, v_cache, rows, p, num_seqs, st, dev)
                      : launch_decode_tc<8, false>(k_cache, v_cache, rows, p, num_seqs, st, dev);
  }
  if (kv_dtype == PA_KV_BF16)
    rc = head_dim == 128
             ? dispatch_nt<128, false>(nt, chunked, k_cache, v_cache, rows, p, num_seqs, grid_x, st, dev)
             : dispatch_nt<64, false>(nt, chunked, k_cache, v_cache, rows, p, num_seqs, grid_x, st, dev);
  else
    rc = head_dim == 128
             ? dispatch_nt<128, true>(nt, chunked, k_cache, v_cache, rows, p, num_seqs, grid_x, st, dev)
             : dispatch_nt<64, true>(nt, chunked, k_cache, v_cache, rows, p, num_seqs, grid_x, st, dev);
  if (rc != PA_OK || psize == 0) return rc;

  ReduceParams r{};
  r.out = out;
  r.ws_o = p.ws_o;
  r.ws_m = p.ws_m;
  r.ws_l = p.ws_l;
  r.context_lens = context_lens;
  r.max_context_len = max_context_len;
  r.max_blocks_per_seq = max_blocks_per_seq;
  r.num_q_heads = num_q_heads;
  r.partition_tokens = psize;
  r.max_partitions = static_cast<int>(P);
  return head_dim == 128 ? launch_reduce<128>(r, num_seqs, st)
                         : launch_reduce<64>(r, num_seqs, st);
}

pa_status pa_decode(float *out, const void *q, const void *k_cache, const void *v_cache,
                    pa_kv_dtype kv_dtype, float k_scale, float v_scale,
                    const int32_t *block_tables, int max_blocks_per_seq,
                    const int32_t *context_lens, int max_context_len, int num_seqs,
                    int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                    int num_blocks, float sm_scale, int partition_size, void *workspace,
                    size_t workspace_bytes, void *stream) {
  return decode_common(out, q, k_cache, v_cache, kv_dtype, k_scale, v_scale, block_tables,
                       max_blocks_per_seq, context_lens, max_context_len, num_seqs, num_q_heads,
                       num_kv_heads, head_dim, block_size, num_blocks, sm_scale, partition_size,
                       workspace, workspace_bytes, stream, nullptr, nullptr);
}

pa_status pa_decode_append(float *out, const void *q, const void *key, const void *value,
                           void *k_cache, void *v_cache, pa_kv_dtype kv_dtype, float k_scale,
                           float v_scale, const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int max_context_len, int num_seqs,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, float sm_scale, int partition_size, void *workspace,
                           size_t workspace_bytes, void *stream) {
  if (num_seqs > 0 && (!key || !value)) return PA_ERR_INVALID_ARG;
  return decode_common(out, q, k_cache, v_cache, kv_dtype, k_scale, v_scale, block_tables,
                       max_blocks_per_seq, context_lens, max_context_len, num_seqs, num_q_heads,
                       num_kv_heads, head_dim, block_size, num_blocks, sm_scale, partition_size,
                       workspace, workspace_bytes, stream, num_seqs > 0 ? key : nullptr,
                       num_seqs > 0 ? value : nullptr);
}

size_t pa_decode_shared_prefix_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                              int head_dim, int num_groups, int max_prefix_blocks,
                                              int max_suffix_len) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_groups < 0 ||
      max_prefix_blocks < 0 || (num_groups > 0 && max_prefix_blocks > kSharedMaxPrefixBlocks) ||
      max_suffix_len < 0 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > 16)
    return 0;
  return shared_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, num_groups, max_prefix_blocks,
                     max_suffix_len)
      .bytes;
}

pa_status pa_decode_shared_prefix(float *out, const void *q, const void *k_cache,
                                  const void *v_cache, pa_kv_dtype kv_dtype, float k_scale,
                                  float v_scale, const int32_t *block_tables,
                                  int max_blocks_per_seq, const int32_t *context_lens,
                                  int max_context_len, const int32_t *group_start,
                                  const int32_t *prefix_blocks, int num_groups,
                                  int max_prefix_blocks, int max_suffix_len, int num_seqs,
                                  int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                  int num_blocks, float sm_scale, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_blocks_per_seq < 0 || max_context_len < 0 || num_blocks <= 0 || num_groups < 0 ||
      max_prefix_blocks < 0 || max_suffix_len < 0)
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (block_size != pa::kBS) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  if (group > 16) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale)) return PA_ERR_INVALID_ARG;
  if (kv_dtype == PA_KV_FP8_E4M3 &&
      !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARG;
  if (num_groups > 65535) return PA_ERR_UNSUPPORTED;
  if (max_blocks_per_seq > INT32_MAX / pa::kBS) return PA_ERR_UNSUPPORTED;  // token counts are 32-bit
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
    return PA_ERR_INVALID_ARG;
  if (num_groups > 0 && max_prefix_blocks > kSharedMaxPrefixBlocks) return PA_ERR_UNSUPPORTED;
  if (num_groups > 0 && (!group_start || !prefix_blocks)) return PA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(group_start, 4) ||
      !aligned(prefix_blocks, 4))
    return PA_ERR_INVALID_ARG;
  const int64_t rows64 = static_cast<int64_t>(num_blocks) * num_kv_heads * pa::kBS;
  if (rows64 + pa::kBS >= INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  pa::SharedParams p{};
  p.out = out;
  p.q = static_cast<const uint16_t *>(q);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.group_start = group_start;
  p.prefix_blocks = prefix_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.max_prefix_blocks = max_prefix_blocks;
  p.max_suffix_len = max_suffix_len;
  p.num_groups = num_groups;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.num_blocks = num_blocks;
  const float log2e = 1.4426950408889634f;
  const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
  p.score_scale = fp8 ? sm_scale * k_scale * log2e : sm_scale * log2e;
  p.out_scale = fp8 ? v_scale : 1.f;
  const SharedPlan plan = shared_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, num_groups,
                                      max_prefix_blocks, max_suffix_len);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < plan.bytes) return PA_ERR_WORKSPACE;
  p.tokens_per_tile = pa::kSpRows / group;
  p.prefix_parts = plan.prefix_parts;
  p.suffix_parts = plan.suffix_parts;
  p.part_len = plan.part_len;
  p.row_tiles = plan.row_tiles;
  char *ws = static_cast<char *>(workspace);
  p.rec_o = reinterpret_cast<float *>(ws);
  p.rec_ml = reinterpret_cast<float2 *>(ws + plan.o_bytes);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rows = static_cast<int>(rows64);
  if (head_dim == 128)
    return fp8 ? launch_shared<128, true>(p, k_cache, v_cache, rows, st, dev)
               : launch_shared<128, false>(p, k_cache, v_cache, rows, st, dev);
  return fp8 ? launch_shared<64, true>(p, k_cache, v_cache, rows, st, dev)
             : launch_shared<64, false>(p, k_cache, v_cache, rows, st, dev);
}

pa_status pa_prefill(float *out, const void *q, const void *k_cache, const void *v_cache,
                     pa_kv_dtype kv_dtype, const int32_t *block_tables, int max_blocks_per_seq,
                     const int32_t *query_start, const int32_t *context_lens, int max_query_len,
                     int max_context_len, int num_seqs, int num_tokens, int num_q_heads,
                     int num_kv_heads, int head_dim, int block_size, int num_blocks,
                     float sm_scale, void *stream) {
  if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      max_blocks_per_seq < 0 || max_context_len < 0 || max_query_len < 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16) return PA_ERR_UNSUPPORTED;
  if (block_size != pa::kBS) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  if (group > 16) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(sm_scale)) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PA_ERR_INVALID_ARG;
  const int64_t rows64 = static_cast<int64_t>(num_blocks) * num_kv_heads * pa::kBS;
  if (rows64 + pa::kBS >= INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  pa::PrefillParams p{};
  p.out = out;
  p.q = static_cast<const uint16_t *>(q);
  p.block_tables = block_tables;
  p.query_start = query_start;
  p.context_lens = context_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.tokens_per_tile = pa::kPfRows / group;
  p.num_blocks = num_blocks;
  p.score_scale = sm_scale * 1.4426950408889634f;
  const int rows = static_cast<int>(rows64);
  const int64_t cta_tokens = static_cast<int64_t>(pa::kPfQTiles) * p.tokens_per_tile;
  const int64_t tiles = (static_cast<int64_t>(max_query_len) + cta_tokens - 1) / cta_tokens;
  if (tiles > INT32_MAX) return PA_ERR_UNSUPPORTED;
  // each CTA takes two tile pairs of a chunk, a heavy and a light one
  dim3 grid(static_cast<unsigned>((tiles + 1) / 2), num_kv_heads, num_seqs);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tq, tk, tv, to;
  if (!make_q_tmap(&tq, q, num_tokens, num_q_heads, head_dim, group, p.tokens_per_tile) ||
      !make_out_tmap(&to, out, num_tokens, num_q_heads, head_dim, group, p.tokens_per_tile))
    return PA_ERR_CUDA;
  if (head_dim == 128) {
    if (!make_cache_tmap<128, false>(&tk, k_cache, rows) ||
        !make_cache_tmap<128, false>(&tv, v_cache, rows))
      return PA_ERR_CUDA;
    auto kern = pa::paged_prefill_kernel<128>;
    const size_t smem = pa::PfPlan<128>::kSmemBytes;
    static std::atomic<uint64_t> attr_done{0};
    if (!ensure_smem_attr(kern, smem, attr_done, dev)) return PA_ERR_CUDA;
    kern<<<grid, pa::kPfThreads, smem, st>>>(tq, tk, tv, to, p);
  } else {
    if (!make_cache_tmap<64, false>(&tk, k_cache, rows) ||
        !make_cache_tmap<64, false>(&tv, v_cache, rows))
      return PA_ERR_CUDA;
    auto kern = pa::paged_prefill_kernel<64>;
    const size_t smem = pa::PfPlan<64>::kSmemBytes;
    static std::atomic<uint64_t> attr_done{0};
    if (!ensure_smem_attr(kern, smem, attr_done, dev)) return PA_ERR_CUDA;
    kern<<<grid, pa::kPfThreads, smem, st>>>(tq, tk, tv, to, p);
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_reshape_and_cache(const void *key, const void *value, void *k_cache,
                               void *v_cache, const int64_t *slot_mapping, int num_tokens,
                               int num_kv_heads, int head_dim, int block_size, int num_blocks,
                               pa_kv_dtype kv_dtype, float k_scale, float v_scale,
                               void *stream) {
  if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (block_size != pa::kBS) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (kv_dtype == PA_KV_FP8_E4M3 &&
      !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PA_ERR_INVALID_ARG;
  const int chunks_per_row = head_dim / 8;
  const int chunks_per_token = chunks_per_row * num_kv_heads;
  const int64_t total = static_cast<int64_t>(num_tokens) * chunks_per_token;
  const int64_t num_slots = static_cast<int64_t>(num_blocks) * pa::kBS;
  int64_t blocks = (total + pa::kCacheThreads - 1) / pa::kCacheThreads;
  if (blocks > 1 << 20) blocks = 1 << 20;  // grid-stride beyond this
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (kv_dtype == PA_KV_BF16)
    pa::reshape_and_cache_kernel<false><<<static_cast<unsigned>(blocks), pa::kCacheThreads, 0, st>>>(
        static_cast<const uint4 *>(key), static_cast<const uint4 *>(value), k_cache, v_cache,
        slot_mapping, total, chunks_per_token, chunks_per_row, num_kv_heads, head_dim, num_slots,
        1.f, 1.f);
  else
    pa::reshape_and_cache_kernel<true><<<static_cast<unsigned>(blocks), pa::kCacheThreads, 0, st>>>(
        static_cast<const uint4 *>(key), static_cast<const uint4 *>(value), k_cache, v_cache,
        slot_mapping, total, chunks_per_token, chunks_per_row, num_kv_heads, head_dim, num_slots,
        k_scale, v_scale);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_rope_frequencies(double *inv_freq_out, float *rope_scale_out, int rotary_dim,
                              double base, pa_rope_scaling scaling, double factor,
                              double original_max_position, double low, double high) {
  if (!inv_freq_out || !rope_scale_out || rotary_dim <= 0 || rotary_dim % 2 != 0 ||
      !(std::isfinite(base) && base > 1.0))
    return PA_ERR_INVALID_ARG;
  if (scaling < PA_ROPE_NONE || scaling > PA_ROPE_YARN) return PA_ERR_INVALID_ARG;
  if (scaling != PA_ROPE_NONE && !(std::isfinite(factor) && factor >= 1.0)) return PA_ERR_INVALID_ARG;
  if (scaling == PA_ROPE_BASE && rotary_dim <= 2) return PA_ERR_INVALID_ARG;
  const bool ramped = scaling == PA_ROPE_BANDS || scaling == PA_ROPE_YARN;
  if (ramped && !(std::isfinite(original_max_position) && original_max_position > 0.0 && low > 0.0 &&
                  std::isfinite(high) && high > low))
    return PA_ERR_INVALID_ARG;
  const double r = rotary_dim, two_pi = 2.0 * std::acos(-1.0);
  if (scaling == PA_ROPE_BASE) base *= std::pow(factor, r / (r - 2.0));
  if (!std::isfinite(base)) return PA_ERR_INVALID_ARG;
  // YaRN's ramp: the (real-valued) component that turns `turns` times in the
  // original context, N base^(-2i/r) / 2 pi = turns
  double lo = 0.0, hi = 1.0;
  if (scaling == PA_ROPE_YARN) {
    const auto component = [&](double turns) {
      return r * std::log(original_max_position / (turns * two_pi)) / (2.0 * std::log(base));
    };
    lo = std::max(std::floor(component(high)), 0.0);
    hi = std::min(std::ceil(component(low)), r - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == PA_ROPE_LINEAR) keep = 0.0;
    if (scaling == PA_ROPE_BANDS)
      keep = (original_max_position * f / two_pi - low) / (high - low);
    if (scaling == PA_ROPE_YARN) keep = 1.0 - (i - lo) / std::max(hi - lo, 1e-3);
    keep = std::min(std::max(keep, 0.0), 1.0);
    inv_freq_out[i] = keep == 1.0 ? f : f * (keep + (1.0 - keep) / factor);
  }
  *rope_scale_out = scaling == PA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return PA_OK;
}

pa_status pa_rope_and_cache(void *q_out, const void *q, const void *key, const void *value,
                            void *k_cache, void *v_cache, const int64_t *slot_mapping,
                            const int32_t *positions, const double *inv_freq, int rotary_dim,
                            int interleaved, float rope_scale, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int num_tokens, int num_q_heads, int num_kv_heads,
                            int head_dim, int block_size, int num_blocks, pa_kv_dtype kv_dtype,
                            float k_scale, float v_scale, void *stream) {
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 ||
      rotary_dim <= 0)
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (block_size != pa::kBS) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (rotary_dim > head_dim || rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  // unit counts of a CTA's tokens stay inside 32 bits
  if (num_q_heads > 65535 || num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(rope_scale)) return PA_ERR_INVALID_ARG;
  if (kv_dtype == PA_KV_FP8_E4M3 &&
      !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride % 8 != 0 ||
      k_stride % 8 != 0 || v_stride % 8 != 0)
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (!q_out || !q || !key || !value || !k_cache || !v_cache || !slot_mapping || !positions || !inv_freq)
    return PA_ERR_INVALID_ARG;
  if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(key, 16) || !aligned(value, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_mapping, 8) ||
      !aligned(positions, 4) || !aligned(inv_freq, 8))
    return PA_ERR_INVALID_ARG;
  if (q_out == q && q_stride != q_row) return PA_ERR_INVALID_ARG;
  pa::RopeParams p{};
  p.q = static_cast<const uint16_t *>(q);
  p.key = static_cast<const uint16_t *>(key);
  p.value = static_cast<const uint16_t *>(value);
  p.q_out = static_cast<uint16_t *>(q_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slots = slot_mapping;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.num_slots = static_cast<int64_t>(num_blocks) * pa::kBS;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.rotary_dim = rotary_dim;
  p.rope_scale = rope_scale;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool il = interleaved != 0, fp8 = kv_dtype == PA_KV_FP8_E4M3;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  if (head_dim == 128)
    return fp8 ? launch_rope<128, true>(p, il, st, dev) : launch_rope<128, false>(p, il, st, dev);
  return fp8 ? launch_rope<64, true>(p, il, st, dev) : launch_rope<64, false>(p, il, st, dev);
}

pa_status pa_extend_tables(int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                           const int32_t *new_lens, const int32_t *free_blocks, int free_capacity,
                           const int32_t *free_count, int32_t *context_lens_out,
                           int32_t *free_count_out, int64_t *slot_mapping, int32_t *positions,
                           int32_t *query_start, int num_seqs, int num_tokens, int block_size,
                           int num_blocks, void *stream) {
  if (num_seqs < 0 || num_tokens < 0 || max_blocks_per_seq < 0 || free_capacity < 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (block_size != pa::kBS) return PA_ERR_UNSUPPORTED;
  if (num_seqs > pa::kTabMaxSeqs || max_blocks_per_seq > INT32_MAX / pa::kBS) return PA_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !query_start) return PA_ERR_INVALID_ARG;
  if (free_capacity > 0 && !free_blocks) return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!context_lens || !new_lens || !context_lens_out)) return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables) return PA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!slot_mapping || !positions)) return PA_ERR_INVALID_ARG;
  if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(new_lens, 4) ||
      !aligned(free_blocks, 4) || !aligned(free_count, 4) || !aligned(context_lens_out, 4) ||
      !aligned(free_count_out, 4) || !aligned(slot_mapping, 8) || !aligned(positions, 4) ||
      !aligned(query_start, 4))
    return PA_ERR_INVALID_ARG;
  pa::ExtendParams p{};
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.new_lens = new_lens;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.context_lens_out = context_lens_out;
  p.free_count_out = free_count_out;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.query_start = query_start;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.num_blocks = num_blocks;
  p.free_capacity = free_capacity;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  p.wide = aligned(slot_mapping, 32) && aligned(positions, 16);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  using pa::TablePhase;
  const size_t ints = 3 * static_cast<size_t>(num_seqs) + 1, most = 3 * pa::kTabMaxSeqs + 1;
  static std::atomic<uint64_t> attr_all{0}, attr_work{0};
  if (num_tokens <= pa::kTabSmallTokens)
    return launch_table_kernel(pa::extend_kernel<TablePhase::kAll>, p, 1, table_threads(num_seqs, num_tokens), ints, most,
                               attr_all, st, dev);
  const TableGrid grid = table_grid(num_seqs, num_tokens, dev);
  const pa_status rc = launch_table_kernel(pa::extend_kernel<TablePhase::kWork>, p, grid.ctas, grid.threads, ints, most,
                                           attr_work, st, dev);
  if (rc != PA_OK) return rc;
  return launch_beside(pa::extend_kernel<TablePhase::kFinish>, dim3(1), pa::kTabThreads, 0, st, p);
}

pa_status pa_release_tables(const int32_t *block_tables, int max_blocks_per_seq,
                            const int32_t *context_lens, const int32_t *release,
                            int32_t *free_blocks, int free_capacity, const int32_t *free_count,
                            int32_t *context_lens_out, int32_t *free_count_out, int keep_blocks,
                            int num_seqs, int block_size, int num_blocks, void *stream) {
  if (num_seqs < 0 || max_blocks_per_seq < 0 || free_capacity < 0 || keep_blocks < 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (block_size != pa::kBS) return PA_ERR_UNSUPPORTED;
  if (num_seqs > pa::kTabMaxSeqs || max_blocks_per_seq > INT32_MAX / pa::kBS) return PA_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out) return PA_ERR_INVALID_ARG;
  if (free_capacity > 0 && !free_blocks) return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!context_lens || !release || !context_lens_out)) return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables) return PA_ERR_INVALID_ARG;
  if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(release, 4) ||
      !aligned(free_blocks, 4) || !aligned(free_count, 4) || !aligned(context_lens_out, 4) ||
      !aligned(free_count_out, 4))
    return PA_ERR_INVALID_ARG;
  pa::ReleaseParams p{};
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.release = release;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.context_lens_out = context_lens_out;
  p.free_count_out = free_count_out;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_blocks = num_blocks;
  p.free_capacity = free_capacity;
  p.keep_blocks = keep_blocks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  using pa::TablePhase;
  static std::atomic<uint64_t> attr_all{0}, attr_work{0};
  const int64_t pushes = static_cast<int64_t>(num_seqs) * std::max(max_blocks_per_seq - keep_blocks, 0);  // at most
  if (pushes <= pa::kTabSmallBlocks)
    return launch_table_kernel(pa::release_kernel<TablePhase::kAll>, p, 1, table_threads(num_seqs, pushes / 4), num_seqs,
                               pa::kTabMaxSeqs, attr_all, st, dev);
  const TableGrid grid = table_grid(num_seqs, pushes, dev);
  const pa_status rc = launch_table_kernel(pa::release_kernel<TablePhase::kWork>, p, grid.ctas, grid.threads, num_seqs,
                                           pa::kTabMaxSeqs, attr_work, st, dev);
  if (rc != PA_OK) return rc;
  return launch_beside(pa::release_kernel<TablePhase::kFinish>, dim3(1), pa::kTabThreads, 0, st, p);
}

pa_status pa_copy_blocks(void *k_cache, void *v_cache, const int64_t *block_pairs, int num_pairs,
                         size_t block_bytes, int num_blocks, void *stream) {
  if (num_pairs < 0 || num_blocks <= 0 || block_bytes == 0 || block_bytes % 16 != 0)
    return PA_ERR_INVALID_ARG;
  if (num_pairs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_pairs) return PA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return PA_ERR_INVALID_ARG;
  if (num_pairs > (1 << 30)) return PA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  pa::copy_blocks_kernel<<<2 * num_pairs, pa::kCacheThreads, 0, st>>>(
      static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache),
      static_cast<const uint4 *>(k_cache), static_cast<const uint4 *>(v_cache), block_pairs,
      static_cast<int64_t>(block_bytes / 16), num_blocks, num_blocks);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Device-accessible address of `p` on the current device: device memory of
// this device, managed memory, or page-locked host memory registered with
// CUDA (through its device mapping). nullptr for anything else, e.g.
// pageable host memory, which a kernel must never be given.
static const void *device_view(const void *p, int dev) {
  cudaPointerAttributes a{};
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();  // clear the (non-sticky) error the query left
    return nullptr;
  }
  switch (a.type) {
    case cudaMemoryTypeDevice:
      return a.device == dev ? p : nullptr;
    case cudaMemoryTypeManaged:
      return p;
    case cudaMemoryTypeHost: {
      if (!a.devicePointer) return nullptr;
      // keep the byte offset of p inside its registered range
      return static_cast<const char *>(a.devicePointer) +
             (static_cast<const char *>(p) - static_cast<const char *>(a.hostPointer));
    }
    default:
      return nullptr;
  }
}

pa_status pa_swap_blocks(void *dst_k_cache, void *dst_v_cache, const void *src_k_cache,
                         const void *src_v_cache, const int64_t *block_pairs, int num_pairs,
                         size_t block_bytes, int src_num_blocks, int dst_num_blocks,
                         void *stream) {
  if (num_pairs < 0 || src_num_blocks <= 0 || dst_num_blocks <= 0 || block_bytes == 0 ||
      block_bytes % 16 != 0)
    return PA_ERR_INVALID_ARG;
  if (num_pairs == 0) return PA_OK;
  if (!dst_k_cache || !dst_v_cache || !src_k_cache || !src_v_cache || !block_pairs)
    return PA_ERR_INVALID_ARG;
  if (!aligned(dst_k_cache, 16) || !aligned(dst_v_cache, 16) || !aligned(src_k_cache, 16) ||
      !aligned(src_v_cache, 16) || !aligned(block_pairs, 8))
    return PA_ERR_INVALID_ARG;
  if (num_pairs > (1 << 30)) return PA_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  const void *dk = device_view(dst_k_cache, dev), *dv = device_view(dst_v_cache, dev);
  const void *sk = device_view(src_k_cache, dev), *sv = device_view(src_v_cache, dev);
  const void *pr = device_view(block_pairs, dev);
  if (!dk || !dv || !sk || !sv || !pr) return PA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  pa::copy_blocks_kernel<<<2 * num_pairs, pa::kCacheThreads, 0, st>>>(
      static_cast<uint4 *>(const_cast<void *>(dk)), static_cast<uint4 *>(const_cast<void *>(dv)),
      static_cast<const uint4 *>(sk), static_cast<const uint4 *>(sv),
      static_cast<const int64_t *>(pr), static_cast<int64_t>(block_bytes / 16), src_num_blocks,
      dst_num_blocks);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_get_device_error(uint32_t *code_out) {
  if (!code_out) return PA_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return PA_ERR_CUDA;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, pa::g_pa_error, sizeof v) != cudaSuccess) return PA_ERR_CUDA;
  if (cudaMemcpyToSymbol(pa::g_pa_error, &zero, sizeof zero) != cudaSuccess) return PA_ERR_CUDA;
  *code_out = v;
  return v ? PA_ERR_DEVICE : PA_OK;
}

}  // extern "C"
