// kvtc_rope and kvtc_raw_append: multi-axis rotary positions of q and k rows, and the
// write of K and V rows into uncompressed pages.
//
// Pair i of a head, (x_i, x_{i+64}), turns by a = p * base^(-2i/128) with p the row's
// position on the pair's axis: y_i = x_i cos a - x_{i+64} sin a, y_{i+64} = x_{i+64} cos a
// + x_i sin a.  The angle is formed and reduced in fp64 as turns, t = p * (f_i / 2 pi),
// t - rint(t) (at p = 1e5 an fp32 angle is off by about 1e-2 rad), its cosine and sine and
// the rotation are fp32, rounded once to the rows' type.
//
// Bound: memory, each row read and written once.  One kernel serves both calls: a CTA takes
// a few tokens with all their heads, so the 64 (cos, sin) pairs of a token are made once in
// shared memory for its q and k heads; a thread moves 16 bytes at i and 16 at i + 64, so a
// rotation needs no exchange between threads.  The loads of a batch of rows are issued
// before the sines are made.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "ptx.cuh"
#include "raw_cache.cuh"

namespace kvtc {
namespace {

constexpr int kThreads = 256;
constexpr int kHalf = kD / 2;
constexpr int kMaxTok = 16;  // tokens of one CTA

struct RopeArgs {
  const void* x[3];        // q, k, v (null: absent)
  long long stride[3];     // elements between tokens
  int heads[3];
  void* q_out;
  void* k_out;             // kvtc_rope
  const int64_t* slots;    // kvtc_raw_append: k and v go to the pages
  void* pages;             // first element of the layer's pages
  long long n_slots;
  int page_heads;
  const int32_t* positions;
  int n_tok;
  int tok_per_cta;
  int rotate;
  int32_t* status;
  double turns[kHalf];     // +-f_i / 2 pi
  uint8_t axis[kHalf];
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // elements of a 16-byte chunk
  constexpr int kLanes = kHalf / kVec;                     // threads of a row
  constexpr int kRows = kThreads / kLanes;                 // rows moved at a time
  constexpr int kBatch = 4;                                // rows of a thread in flight
  __shared__ float2 cs[kMaxTok][kHalf];
  __shared__ long long slot_of[kMaxTok];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, ch = tid % kLanes;
  const int tok0 = static_cast<int>(blockIdx.x) * a.tok_per_cta;
  const int n_tok = min(a.tok_per_cta, a.n_tok - tok0);
  const int per_tok = a.heads[0] + a.heads[1] + a.heads[2];
  const int n_rows = n_tok * per_tok;
  for (int first = 0; first < n_rows; first += kRows * kBatch) {
    uint4 lo[kBatch], hi[kBatch];
    int tk[kBatch], hd[kBatch], kind[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int row = first + b * kRows + tid / kLanes;
      kind[b] = -1;
      if (row < n_rows) {
        tk[b] = row / per_tok;
        int h = row - tk[b] * per_tok, kd = 0;
        if (h >= a.heads[0]) h -= a.heads[0], kd = 1;
        if (kd == 1 && h >= a.heads[1]) h -= a.heads[1], kd = 2;
        hd[b] = h;
        kind[b] = kd;
        const T* src = static_cast<const T*>(a.x[kd]) + static_cast<long long>(tok0 + tk[b]) * a.stride[kd] +
                       static_cast<long long>(h) * kD + ch * kVec;
        lo[b] = *reinterpret_cast<const uint4*>(src);
        hi[b] = *reinterpret_cast<const uint4*>(src + kHalf);
      }
    }
    if (first == 0) {
      if (a.rotate)
        for (int e = tid; e < n_tok * kHalf; e += kThreads) {
          const int t = e / kHalf, i = e % kHalf;
          const double turn = static_cast<double>(a.positions[static_cast<long long>(a.axis[i]) * a.n_tok + tok0 + t]) * a.turns[i];
          float sn, cn;
          sincospif(static_cast<float>(2.0 * (turn - rint(turn))), &sn, &cn);
          cs[t][i] = make_float2(cn, sn);
        }
      if (a.slots && tid < n_tok) {
        const long long sl = a.slots[tok0 + tid];
        slot_of[tid] = sl < a.n_slots ? sl : -1;
        if (sl >= a.n_slots && a.status) atomicOr(a.status, static_cast<int>(KVTC_STATUS_BAD_PAGE));
      }
      __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (kind[b] < 0) continue;
      T* dst;
      if (kind[b] == 0) {
        dst = static_cast<T*>(a.q_out) + (static_cast<long long>(tok0 + tk[b]) * a.heads[0] + hd[b]) * kD;
      } else if (a.slots) {
        const long long sl = slot_of[tk[b]];
        if (sl < 0) continue;
        dst = static_cast<T*>(a.pages) + (((sl / kPage) * a.page_heads + hd[b]) * 2 + (kind[b] - 1)) * raw::kKindElems +
              (sl % kPage) * kD;
      } else {
        dst = static_cast<T*>(a.k_out) + (static_cast<long long>(tok0 + tk[b]) * a.heads[1] + hd[b]) * kD;
      }
      dst += ch * kVec;
      if (a.rotate && kind[b] < 2) {
        T* l = reinterpret_cast<T*>(&lo[b]);
        T* h = reinterpret_cast<T*>(&hi[b]);
        const float4* c4 = reinterpret_cast<const float4*>(&cs[tk[b]][ch * kVec]);
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
          const float4 v = c4[i / 2];
          const float c[2] = {v.x, v.z}, s[2] = {v.y, v.w};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = to_f<T>(l[i + j]), y = to_f<T>(h[i + j]);
            l[i + j] = from_f<T>(x * c[j] - y * s[j]);
            h[i + j] = from_f<T>(y * c[j] + x * s[j]);
          }
        }
      }
      *reinterpret_cast<uint4*>(dst) = lo[b];
      *reinterpret_cast<uint4*>(dst + kHalf) = hi[b];
    }
  }
}

// Checks a rotary description and fills the frequencies (turns per position) and axes.
kvtc_status set_rope(const kvtc_rope_desc* r, bool inverse, RopeArgs& a) {
  if (r->n_axes < 1 || r->n_axes > KVTC_ROPE_MAX_AXES) return fail(KVTC_EINVAL, "n_axes out of range");
  int left[KVTC_ROPE_MAX_AXES], sum = 0;
  for (int i = 0; i < r->n_axes; ++i) {
    left[i] = r->section[i];
    if (left[i] < 0 || left[i] > kHalf) return fail(KVTC_EINVAL, "section out of range");
    sum += left[i];
  }
  if (sum != kHalf) return fail(KVTC_EINVAL, "the sections must sum to 64 pairs");
  const double base = r->base == 0.0 ? 500000.0 : r->base;
  if (!(base > 1.0) || !std::isfinite(base)) return fail(KVTC_EINVAL, "rope base must be 0 or > 1");
  const double l2 = std::log2(base), two_pi = 6.283185307179586476925;
  int ax = 0;
  for (int i = 0; i < kHalf; ++i) {
    while (left[ax] == 0) ax = (ax + 1) % r->n_axes;
    a.axis[i] = static_cast<uint8_t>(ax);
    --left[ax];
    if (r->interleaved) ax = (ax + 1) % r->n_axes;
    const double f = std::exp2(-l2 * i / kHalf) / two_pi;
    a.turns[i] = inverse ? -f : f;
  }
  a.rotate = 1;
  return KVTC_OK;
}

// Rows of one input: alignment and stride.
kvtc_status check_rows(const void* x, int64_t stride, int heads, size_t es, const void* out) {
  if (heads < 1 || heads > 1024) return fail(KVTC_EINVAL, "number of heads out of range");
  if (!x) return fail(KVTC_EINVAL, "null device pointer");
  if (stride < static_cast<int64_t>(heads) * kD || stride > (1ll << 32) || (stride * static_cast<int64_t>(es)) % 16 != 0)
    return fail(KVTC_EINVAL, "row stride must be a multiple of 16 bytes and at least heads * 128");
  if (!raw::aligned16(x) || !raw::aligned16(out)) return fail(KVTC_EINVAL, "rows must be 16-byte aligned");
  return KVTC_OK;
}

// No output may share memory with an input or the other output, but for rows rotated in
// place (the same contiguous rows).
kvtc_status check_overlap(const RopeArgs& a, size_t es) {
  const void* out[2] = {a.q_out, a.k_out};
  uint64_t span[3], dense[3];
  for (int i = 0; i < 3; ++i) {
    dense[i] = static_cast<uint64_t>(a.n_tok) * static_cast<uint64_t>(a.heads[i]) * kD * es;
    span[i] = static_cast<uint64_t>(a.n_tok - 1) * static_cast<uint64_t>(a.stride[i]) * es +
              static_cast<uint64_t>(a.heads[i]) * kD * es;
  }
  auto meet = [](const void* p, uint64_t np, const void* q, uint64_t nq) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return p && q && x < y + nq && y < x + np;
  };
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < 3; ++i) {
      const bool same = o == i && out[o] == a.x[i] && a.stride[i] == static_cast<long long>(a.heads[i]) * kD;
      if (!same && meet(out[o], dense[o], a.x[i], span[i])) return fail(KVTC_EINVAL, "an output overlaps an input");
    }
  }
  if (meet(out[0], dense[0], out[1], dense[1])) return fail(KVTC_EINVAL, "the outputs overlap");
  return KVTC_OK;
}

kvtc_status launch_rope(RopeArgs& a, kvtc_dtype dtype, void* stream) {
  // tokens of a CTA: about 128 rows (one batch of 4 rows per thread in 16-bit types), so a
  // few tokens share a launch slot and their sines are spread over the threads
  const int per_tok = a.heads[0] + a.heads[1] + a.heads[2];
  a.tok_per_cta = std::min(kMaxTok, std::max(1, 128 / per_tok));
  const unsigned grid = static_cast<unsigned>((a.n_tok + a.tok_per_cta - 1) / a.tok_per_cta);
  cudaError_t e;
  if (dtype == KVTC_F32)
    e = raw::launch(rope_kernel<float>, dim3(grid), kThreads, 0, stream, a);
  else if (dtype == KVTC_BF16)
    e = raw::launch(rope_kernel<__nv_bfloat16>, dim3(grid), kThreads, 0, stream, a);
  else
    e = raw::launch(rope_kernel<__half>, dim3(grid), kThreads, 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  return KVTC_OK;
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" kvtc_status kvtc_rope(const kvtc_rope_desc* rope, const void* q, int64_t q_stride, int n_q_heads,
                                 const void* k, int64_t k_stride, int n_kv_heads, kvtc_dtype dtype,
                                 const int32_t* positions, int n_tok, int inverse, void* q_out, void* k_out,
                                 void* stream) {
  if (!rope) return fail(KVTC_EINVAL, "null argument");
  if (dtype != KVTC_F32 && dtype != KVTC_BF16 && dtype != KVTC_F16)
    return fail(KVTC_EINVAL, "dtype must be F32, BF16 or F16");
  if (n_tok < 0) return fail(KVTC_EINVAL, "n_tok must be >= 0");
  RopeArgs a = {};
  kvtc_status st = set_rope(rope, inverse != 0, a);
  if (st != KVTC_OK) return st;
  if (n_tok == 0) return KVTC_OK;
  if ((!q && n_q_heads != 0) || (!k && n_kv_heads != 0) || (!q && !k) || (q && !q_out) || (k && !k_out) || !positions)
    return fail(KVTC_EINVAL, "null device pointer");
  const size_t es = dtype == KVTC_F32 ? 4 : 2;
  if (q) {
    st = check_rows(q, q_stride, n_q_heads, es, q_out);
    if (st != KVTC_OK) return st;
  }
  if (k) {
    st = check_rows(k, k_stride, n_kv_heads, es, k_out);
    if (st != KVTC_OK) return st;
  }
  a.x[0] = q;
  a.x[1] = k;
  a.stride[0] = q_stride;
  a.stride[1] = k_stride;
  a.heads[0] = q ? n_q_heads : 0;
  a.heads[1] = k ? n_kv_heads : 0;
  a.q_out = q_out;
  a.k_out = k_out;
  a.positions = positions;
  a.n_tok = n_tok;
  st = check_overlap(a, es);
  if (st != KVTC_OK) return st;
  return launch_rope(a, dtype, stream);
}

extern "C" uint64_t kvtc_raw_cache_bytes(int n_layers, uint64_t n_pages, int n_kv_heads) {
  if (n_layers < 1 || n_pages < 1 || n_kv_heads < 1) return 0;
  return static_cast<uint64_t>(n_layers) * n_pages * static_cast<uint64_t>(n_kv_heads) * 2 * raw::kKindElems * 2;
}

extern "C" kvtc_status kvtc_raw_append(const kvtc_raw_cache* cache, int layer, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const int64_t* slot_map, int n_tok,
                                       const kvtc_rope_desc* rope, const int32_t* positions, const void* q,
                                       int64_t q_stride, int n_q_heads, void* q_out, void* stream) {
  kvtc_status st = raw::check_cache(cache, layer);
  if (st != KVTC_OK) return st;
  if (n_tok < 0) return fail(KVTC_EINVAL, "n_tok must be >= 0");
  RopeArgs a = {};
  if (rope) {
    st = set_rope(rope, false, a);
    if (st != KVTC_OK) return st;
  }
  if (q && !rope) return fail(KVTC_EINVAL, "q is rotated: it needs a rope description");
  if (!q && n_q_heads != 0) return fail(KVTC_EINVAL, "null device pointer");
  if (n_tok == 0) return KVTC_OK;
  if (!slot_map || (rope && !positions) || (q && !q_out)) return fail(KVTC_EINVAL, "null device pointer");
  st = check_rows(k, k_stride, cache->n_kv_heads, 2, nullptr);
  if (st == KVTC_OK) st = check_rows(v, v_stride, cache->n_kv_heads, 2, nullptr);
  if (st == KVTC_OK && q) st = check_rows(q, q_stride, n_q_heads, 2, q_out);
  if (st != KVTC_OK) return st;
  a.x[0] = q;
  a.x[1] = k;
  a.x[2] = v;
  a.stride[0] = q_stride;
  a.stride[1] = k_stride;
  a.stride[2] = v_stride;
  a.heads[0] = q ? n_q_heads : 0;
  a.heads[1] = a.heads[2] = cache->n_kv_heads;
  a.q_out = q_out;
  a.slots = slot_map;
  a.pages = static_cast<char*>(cache->pool) +
            static_cast<uint64_t>(layer) * cache->n_pages * static_cast<uint64_t>(cache->n_kv_heads) * 2 * raw::kKindElems * 2;
  a.n_slots = static_cast<long long>(cache->n_pages) * kPage;
  a.page_heads = cache->n_kv_heads;
  a.positions = positions;
  a.n_tok = n_tok;
  a.status = cache->status;
  st = check_overlap(a, 2);
  if (st != KVTC_OK) return st;
  return launch_rope(a, cache->dtype, stream);
}
