// kvtc_raw_cross_attention, plainly: a warp per query row and
// head walks its sequence's tokens with the running maximum and sum of the softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "raw_cache.cuh"

namespace kvtc {
namespace {

struct AttnArgs {
  const char* pages;
  long long n_pages;
  int H, G, f16;
  const int32_t* table;
  int n_seq, max_pages, max_len;
  int32_t* status;
  const void* q;
  const int32_t* cu_q;  // null: one row per sequence
  int n_tok;
  const int32_t* seq_lens;
  float scale;
  void* out;
};

__device__ __forceinline__ float4 load4(const void* p, int f16) {
  const uint2 w = *static_cast<const uint2*>(p);
  if (f16) {
    const float2 a = half2_to_float2(w.x), b = half2_to_float2(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

__global__ void __launch_bounds__(128) attention_kernel(const __grid_constant__ AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int hq = a.H * a.G;
  const int row = static_cast<int>(w / hq), head = static_cast<int>(w % hq), h = head / a.G;
  if (row >= a.n_tok) return;
  int s = row;
  if (a.cu_q) {
    for (s = 0; s < a.n_seq; ++s) {
      const int b = a.cu_q[s], e = a.cu_q[s + 1];
      if (b < 0 || e < b || e > a.n_tok) {
        if (lane == 0 && a.status) atomicOr(a.status, static_cast<int>(KVTC_STATUS_BAD_POS));
        continue;
      }
      if (row >= b && row < e) break;
    }
    if (s == a.n_seq) return;
  }
  const size_t at = (static_cast<size_t>(row) * hq + head) * kD + 4 * lane;
  const float4 q = load4(static_cast<const uint16_t*>(a.q) + at, a.f16);
  int len = a.seq_lens[s];
  uint32_t flags = 0;
  if (len < 0 || len > a.max_len) flags = KVTC_STATUS_BAD_POS, len = 0;
  float m = -INFINITY, l = 0.0f;
  float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p = 0; p * kPage < len; ++p) {
    const int id = a.table[static_cast<size_t>(s) * a.max_pages + p];
    if (id < 0 || id >= a.n_pages) {
      flags = KVTC_STATUS_BAD_PAGE;
      z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      l = 0.0f;
      break;
    }
    const uint16_t* k = reinterpret_cast<const uint16_t*>(a.pages) + (static_cast<long long>(id) * a.H + h) * 2 * raw::kKindElems;
    const int n = min(kPage, len - p * kPage);
    for (int t = 0; t < n; ++t) {
      const float4 x = load4(k + t * kD + 4 * lane, a.f16);
      float sc = q.x * x.x + q.y * x.y + q.z * x.z + q.w * x.w;
#pragma unroll
      for (int o = 16; o; o >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, o);
      sc *= a.scale;
      const float mn = fmaxf(m, sc), f = __expf(m - mn), e = __expf(sc - mn);
      const float4 y = load4(k + raw::kKindElems + t * kD + 4 * lane, a.f16);
      m = mn;
      l = l * f + e;
      z.x = z.x * f + e * y.x;
      z.y = z.y * f + e * y.y;
      z.z = z.z * f + e * y.z;
      z.w = z.w * f + e * y.w;
    }
  }
  if (flags && lane == 0 && a.status) atomicOr(a.status, static_cast<int>(flags));
  const float r = l > 0.0f ? 1.0f / l : 0.0f;
  const float o[4] = {z.x * r, z.y * r, z.z * r, z.w * r};
  uint16_t b[4];
  for (int i = 0; i < 4; ++i)
    b[i] = a.f16 ? __half_as_ushort(__float2half_rn(o[i])) : __bfloat16_as_ushort(__float2bfloat16_rn(o[i]));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
      make_uint2(b[0] | static_cast<uint32_t>(b[1]) << 16, b[2] | static_cast<uint32_t>(b[3]) << 16);
}

kvtc_status run(const kvtc_raw_cache* c, int layer, const void* q, int n_q_heads, const int32_t* cu_q, int n_tok,
                const int32_t* seq_lens, int max_seq_len, float scale, void* out, void* stream) {
  AttnArgs a;
  a.H = c->n_kv_heads;
  a.G = n_q_heads / c->n_kv_heads;
  a.pages = static_cast<const char*>(c->pool) + static_cast<uint64_t>(layer) * c->n_pages * a.H * 4 * raw::kKindElems;
  a.n_pages = static_cast<long long>(c->n_pages);
  a.f16 = c->dtype == KVTC_F16;
  a.table = c->block_table;
  a.n_seq = c->n_seq;
  a.max_pages = c->max_pages;
  a.max_len = max_seq_len;
  a.status = c->status;
  a.q = q;
  a.cu_q = cu_q;
  a.n_tok = n_tok;
  a.seq_lens = seq_lens;
  a.scale = scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(kD));
  a.out = out;
  const long long warps = static_cast<long long>(n_tok) * n_q_heads;
  const cudaError_t e = raw::launch(attention_kernel, dim3(static_cast<unsigned>((warps + 3) / 4)), 128, 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e, "raw attention launch");
  return KVTC_OK;
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" uint64_t kvtc_raw_cross_workspace_bytes(int n_seq, int n_tok, int n_q_heads, int n_kv_heads,
                                                   int max_seq_len) {
  if (n_seq < 1 || n_tok < 0 || n_kv_heads < 1 || n_q_heads < n_kv_heads || max_seq_len < 0) return 0;
  return 16;
}

extern "C" kvtc_status kvtc_raw_cross_attention(const kvtc_raw_cache* cache, int layer, const void* q, int n_q_heads,
                                                const int32_t* cu_q, int n_tok, const int32_t* seq_lens,
                                                int max_seq_len, float softmax_scale, void* out, void* workspace,
                                                uint64_t workspace_bytes, void* stream) {
  kvtc_status st = raw::check_attention(cache, layer, n_q_heads, 128, max_seq_len, softmax_scale);
  if (st != KVTC_OK) return st;
  if (n_tok < 0) return fail(KVTC_EINVAL, "n_tok must be >= 0");
  if (n_tok == 0) return KVTC_OK;
  if (!q || !cu_q || !seq_lens || !out || !workspace) return fail(KVTC_EINVAL, "null device pointer");
  if (!raw::aligned16(q) || !raw::aligned16(out) || !raw::aligned16(workspace))
    return fail(KVTC_EINVAL, "q, out and workspace must be 16-byte aligned");
  if (workspace_bytes < kvtc_raw_cross_workspace_bytes(cache->n_seq, n_tok, n_q_heads, cache->n_kv_heads, max_seq_len))
    return fail(KVTC_ECAPACITY, "cross attention workspace too small");
  if (raw::overlap(q, out, static_cast<uint64_t>(n_tok) * n_q_heads * kD * 2))
    return fail(KVTC_EINVAL, "out overlaps q");
  return run(cache, layer, q, n_q_heads, cu_q, n_tok, seq_lens, max_seq_len, softmax_scale, out, stream);
}
