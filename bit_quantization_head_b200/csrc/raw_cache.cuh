// Shared by the calls around the cache and on the uncompressed pages: argument checks, the
// current device's SM count and launches with programmatic stream serialization.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "kvtc_internal.h"

namespace kvtc {
namespace raw {

constexpr int kRowElems = kD;                              // elements of one K or V row
constexpr long long kKindElems = static_cast<long long>(kPage) * kD;  // K or V of one page and head

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether two buffers share memory (null or empty ones do not).
inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

// The sizes and pointers every call on the uncompressed pages needs.
inline kvtc_status check_cache(const kvtc_raw_cache* c, int layer) {
  if (!c || !c->pool) return fail(KVTC_EINVAL, "cache is incomplete");
  if (c->dtype != KVTC_BF16 && c->dtype != KVTC_F16) return fail(KVTC_EINVAL, "the pages' dtype must be BF16 or F16");
  if (c->n_layers < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->n_pages < 1)
    return fail(KVTC_EINVAL, "bad cache sizes");
  // rows of all layers are counted in 31 bits (tensor map coordinates, page ids); the row
  // count is bounded step by step, so no product overflows
  const uint64_t row_limit = 1ull << 31;
  const uint64_t per_page = 2ull * kPage * static_cast<uint64_t>(c->n_kv_heads);
  if (c->n_pages >= row_limit / per_page || static_cast<uint64_t>(c->n_layers) > row_limit / (per_page * c->n_pages))
    return fail(KVTC_EINVAL, "the pool has more than 2^31 rows");
  if (layer < 0 || layer >= c->n_layers) return fail(KVTC_EINVAL, "layer out of range");
  if (reinterpret_cast<uintptr_t>(c->pool) & 127) return fail(KVTC_EINVAL, "pool must be 128-byte aligned");
  return KVTC_OK;
}

// The factor from a score to the exponent of 2 of its weight (scale 0 means 1 / sqrt(128)).
inline float exp2_scale(float scale) {
  return (scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(kD))) * 1.4426950408889634f;
}

// What both attention calls need beyond that.
inline kvtc_status check_attention(const kvtc_raw_cache* c, int layer, int n_q_heads, int max_group, int max_seq_len,
                                   float scale) {
  kvtc_status st = check_cache(c, layer);
  if (st != KVTC_OK) return st;
  if (!c->block_table) return fail(KVTC_EINVAL, "cache is incomplete");
  if (c->n_seq < 1 || c->max_pages < 1 || c->max_pages >= (1 << 24)) return fail(KVTC_EINVAL, "bad sizes");
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads != 0)
    return fail(KVTC_EINVAL, "n_q_heads must be a positive multiple of n_kv_heads");
  if (n_q_heads / c->n_kv_heads > max_group) return fail(KVTC_EINVAL, "too many query heads per KV head");
  if (max_seq_len < 0 || max_seq_len > static_cast<long long>(c->max_pages) * kPage)
    return fail(KVTC_EINVAL, "max_seq_len exceeds the block table");
  if (!std::isfinite(scale) || scale < 0.0f) return fail(KVTC_EINVAL, "softmax_scale must be finite and >= 0");
  if (!std::isfinite(exp2_scale(scale))) return fail(KVTC_EINVAL, "softmax_scale is too large");
  return KVTC_OK;
}

inline uint64_t pool_bytes(const kvtc_raw_cache* c) {
  return static_cast<uint64_t>(c->n_layers) * c->n_pages * static_cast<uint64_t>(c->n_kv_heads) * 2 * kKindElems * 2;
}

struct Range {
  const void* p;
  uint64_t bytes;
};
inline bool overlaps_any(const void* p, uint64_t bytes, std::initializer_list<Range> others) {
  for (const Range& r : others)
    if (overlap(p, bytes, r.p, r.bytes)) return true;
  return false;
}

// What an attention call writes shares memory with nothing else that it touches (cu_q: null
// without query offsets).
inline kvtc_status check_overlap(const kvtc_raw_cache* c, const void* q, const void* out, uint64_t rows, const void* ws,
                                 uint64_t ws_bytes, const int32_t* seq_lens, const int32_t* cu_q) {
  const uint64_t n = static_cast<uint64_t>(c->n_seq);
  const std::initializer_list<Range> lists = {{seq_lens, 4 * n},
                                              {cu_q, 4 * (n + 1)},
                                              {c->block_table, 4 * n * static_cast<uint64_t>(c->max_pages)}};
  if (overlaps_any(out, rows, lists) || overlaps_any(ws, ws_bytes, lists))
    return fail(KVTC_EINVAL, "out or the workspace overlaps the lengths, the row offsets or the block table");
  if (overlaps_any(c->status, 4, lists) ||
      overlaps_any(c->status, 4, {{out, rows}, {ws, ws_bytes}, {q, rows}, {c->pool, pool_bytes(c)}}))
    return fail(KVTC_EINVAL, "the status word overlaps another buffer");
  if (overlap(q, rows, out, rows)) return fail(KVTC_EINVAL, "out overlaps q");
  if (overlap(out, rows, c->pool, pool_bytes(c)) || overlap(out, rows, ws, ws_bytes))
    return fail(KVTC_EINVAL, "out overlaps the pool or the workspace");
  if (overlap(ws, ws_bytes, c->pool, pool_bytes(c)) || overlap(ws, ws_bytes, q, rows))
    return fail(KVTC_EINVAL, "the workspace overlaps the pool or q");
  return KVTC_OK;
}

// SM count of the current device (a constant of the device, read once for each).
inline kvtc_status sm_count(int* out) {
  static std::atomic<int> known[64];
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev >= 0 && dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return KVTC_OK;
  int n = 0;
  e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess || n < 1) return cuda_fail(e, "device query");
  if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  *out = n;
  return KVTC_OK;
}

// Lets a kernel use `bytes` of dynamic shared memory on the current device (set once for
// each device).
template <auto Kernel>
inline kvtc_status allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return KVTC_OK;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  done.fetch_or(bit, std::memory_order_relaxed);
  return KVTC_OK;
}

// The pool as a 2-D tensor of rows (128 elements), loaded in 128-byte-swizzled boxes of 64
// elements x box_rows rows; row of (layer, page, head, kind, token) = (((layer * n_pages +
// page) * n_kv_heads + head) * 2 + kind) * 128 + token (raw_decode.cu).
kvtc_status pool_map(CUtensorMap* m, const kvtc_raw_cache* c, int box_rows);
// [n_tok][n_q_heads][128] queries as (element, head of the group, KV head, token), in
// swizzled boxes of 64 elements x box_heads x 1 x box_tok.
kvtc_status query_map(CUtensorMap* m, const void* q, kvtc_dtype dtype, int n_tok, int n_kv_heads, int group,
                      int box_heads, int box_tok);

// Launch that may start while the previous kernel of the stream finishes; the kernel calls
// griddepcontrol.wait before it touches memory.
template <typename... KArgs, typename... Args>
inline cudaError_t launch(void (*fn)(KArgs...), dim3 grid, int block, size_t smem, void* stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fn, std::forward<Args>(args)...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace raw
}  // namespace kvtc
