// kvtc_rope and kvtc_raw_append: multi-axis rotary positions of q and k rows, and the
// write of K and V rows into uncompressed pages.
//
// Pair i of a head, (x_i, x_{i+64}), turns by a = p * base^(-2i/128) with p the row's
// position on the pair's axis: y_i = x_i cos a - x_{i+64} sin a, y_{i+64} = x_{i+64} cos a
// + x_i sin a.  The angle is formed and reduced in fp64 as turns, t = p * (f_i / 2 pi),
// t - rint(t) (at p = 1e5 an fp32 angle is off by about 1e-2 rad), its cosine and sine and
// the rotation are fp32, rounded once to the rows' type.
//
// Bound: memory, each row read and written once.  One kernel serves both calls: a warp takes
// a token's rows, 16 bytes at i and 16 at i + 64 of a row per lane, so a rotation needs no
// exchange and a lane meets the same pairs in every row: it keeps their cosines and sines in
// registers.  The token's 64 are made once, two (cos, sin) per lane, and dealt through the
// warp's shared memory, after the loads of the first rows have been issued; warps never wait
// for one another (a block of a few tokens that shared them behind a barrier reached 3.3 TB/s,
// at two blocks per SM).  Few tokens: a token's rows are dealt over several warps.  Measured on
// inputs that change from call to call: 32768 bf16 tokens of 40 heads in 105 us (6.4 TB/s, the
// rate of a copy), 16411 tokens into pages in 66 us (6.1 TB/s), 4097 fp32 tokens of 32 heads in
// 26 us (5.2 TB/s; replayed on the same rows, half of them still in L2, 20.9), 16 tokens in
// 3.9 us (3.2 replayed).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ptx.cuh"
#include "raw_cache.cuh"
#include "raw_device.cuh"

namespace kvtc {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kHalf = kD / 2;
// Rows of a lane in flight, and blocks per SM, replayed on the same rows: 4 and 3 in 16 bits
// (32768 tokens 102.5 us, 104.3 with 2 and 4), 2 and 4 in fp32 (4097 tokens of 32 heads, with two
// warps a token: 21.6 us, 23.9 with 4 and 3; one warp a token, as they have now, 20.9).
template <typename T>
constexpr int kBatchOf = sizeof(T) == 4 ? 2 : 4;
template <typename T>
constexpr int kBlocksOf = sizeof(T) == 4 ? 4 : 3;
// Warps per SM from which a token has no more than one: every further warp of a token makes
// its sines again (2000 tokens of 40 heads 9.8 us with 12 or less, 10.0 with 24, 12.8 with 48;
// 300 tokens 4.6 with 12, 5.5 with 24).
constexpr int kBusyWarpsPerSm = 12;

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
  int parts, part_rows;    // warps of a token, rows of each
  int rotate;
  int32_t* status;
  double turns[kHalf];     // +-f_i / 2 pi
  uint8_t axis[kHalf];
};

// Two elements of a 32-bit word (one for fp32, whose second is not used).
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w), 0.0f);
  if constexpr (std::is_same_v<T, __half>) return half2_to_float2(w);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float x, float y) {
  if constexpr (sizeof(T) == 4) return __float_as_uint(x);
  return raw::pack2<std::is_same_v<T, __half>>(x, y);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kBlocksOf<T>) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // elements of a 16-byte chunk
  constexpr int kPer = kVec / 4;                           // elements of a 32-bit word
  constexpr int kLanes = kHalf / kVec;                     // lanes of a row
  constexpr int kRows = 32 / kLanes;                       // rows moved at a time
  constexpr int kBatch = kBatchOf<T>;
  __shared__ float2 cs[kWarps][kHalf];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = lane % kLanes;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int tok = static_cast<int>(a.parts == 1 ? w : w / a.parts);
  if (w >= static_cast<long long>(a.n_tok) * a.parts) return;  // the whole warp
  const int part = static_cast<int>(w - static_cast<long long>(tok) * a.parts);
  const int nq = a.heads[0], nqk = nq + a.heads[1], n_all = nqk + a.heads[2];
  const int r0 = part * a.part_rows, r1 = min(n_all, r0 + a.part_rows);
  long long slot = 0;
  if (a.slots) {
    slot = a.slots[tok];
    if (slot >= a.n_slots) {
      if (lane == 0 && part == 0 && a.status) atomicOr(a.status, static_cast<int>(KVTC_STATUS_BAD_PAGE));
      slot = -1;
    }
  }
  const int end = slot < 0 ? min(r1, nq) : r1;  // rows of k and v without a slot are skipped
  float cn[kVec], sn[kVec];
  for (int first = r0; first < end || first == r0; first += kRows * kBatch) {
    uint4 lo[kBatch], hi[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = first + b * kRows + lane / kLanes;
      if (r < end) {
        const int kd = r < nq ? 0 : r < nqk ? 1 : 2, h = r - (kd == 0 ? 0 : kd == 1 ? nq : nqk);
        const char* src = static_cast<const char*>(kd == 0 ? a.x[0] : kd == 1 ? a.x[1] : a.x[2]) +
                          (static_cast<long long>(tok) * (kd == 0 ? a.stride[0] : kd == 1 ? a.stride[1] : a.stride[2]) +
                           h * kD) * static_cast<long long>(sizeof(T)) + ch * 16;
        lo[b] = *reinterpret_cast<const uint4*>(src);
        hi[b] = *reinterpret_cast<const uint4*>(src + kHalf * sizeof(T));
      }
    }
    if (first == r0 && a.rotate) {
#pragma unroll
      for (int i = lane; i < kHalf; i += 32) {
        const double turn = static_cast<double>(a.positions[static_cast<long long>(a.axis[i]) * a.n_tok + tok]) * a.turns[i];
        float s, c;
        sincospif(static_cast<float>(2.0 * (turn - rint(turn))), &s, &c);
        cs[warp][i] = make_float2(c, s);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float4 v = *reinterpret_cast<const float4*>(&cs[warp][ch * kVec + i]);
        cn[i] = v.x, sn[i] = v.y, cn[i + 1] = v.z, sn[i + 1] = v.w;
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = first + b * kRows + lane / kLanes;
      if (r >= end) continue;
      const int kd = r < nq ? 0 : r < nqk ? 1 : 2, h = r - (kd == 0 ? 0 : kd == 1 ? nq : nqk);
      char* dst;
      if (kd == 0)
        dst = static_cast<char*>(a.q_out) + (static_cast<long long>(tok) * nq + h) * kD * static_cast<long long>(sizeof(T));
      else if (a.slots)
        dst = static_cast<char*>(a.pages) + ((((slot / kPage) * a.page_heads + h) * 2 + (kd - 1)) * raw::kKindElems +
                                             (slot % kPage) * kD) * static_cast<long long>(sizeof(T));
      else
        dst = static_cast<char*>(a.k_out) + (static_cast<long long>(tok) * a.heads[1] + h) * kD * static_cast<long long>(sizeof(T));
      if (a.rotate && kd < 2) {
        uint32_t* l = reinterpret_cast<uint32_t*>(&lo[b]);
        uint32_t* u = reinterpret_cast<uint32_t*>(&hi[b]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack<T>(l[i]), y = unpack<T>(u[i]);
          const int j = kPer * i, k = kPer * i + kPer - 1;
          l[i] = pack<T>(x.x * cn[j] - y.x * sn[j], x.y * cn[k] - y.y * sn[k]);
          u[i] = pack<T>(y.x * cn[j] + x.x * sn[j], y.y * cn[k] + x.y * sn[k]);
        }
      }
      *reinterpret_cast<uint4*>(dst + ch * 16) = lo[b];
      *reinterpret_cast<uint4*>(dst + kHalf * sizeof(T) + ch * 16) = hi[b];
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
  const double two_pi = 6.283185307179586476925;
  // f_i = base^(-i/64): the powers of two by exp2, the others as products of at most six of
  // them (a relative error of a few 2^-53, as exp2's own)
  double f[kHalf];
  f[0] = 1.0;
  for (int i = 1; i < kHalf; ++i) f[i] = i & (i - 1) ? f[i & (i - 1)] * f[i & -i] : std::exp2(-std::log2(base) * i / kHalf);
  int ax = 0;
  for (int i = 0; i < kHalf; ++i) {
    while (left[ax] == 0) ax = (ax + 1) % r->n_axes;
    a.axis[i] = static_cast<uint8_t>(ax);
    --left[ax];
    if (r->interleaved) ax = (ax + 1) % r->n_axes;
    a.turns[i] = (inverse ? -f[i] : f[i]) / two_pi;
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

// No output may share memory with an input, with the positions (of n_axes axes) and slots, or
// with the other output, but for rows rotated in place (the same contiguous rows).
kvtc_status check_rope_overlap(const RopeArgs& a, size_t es, int n_axes, const kvtc_raw_cache* cache) {
  const void* out[2] = {a.q_out, a.k_out};
  uint64_t span[3], dense[3];
  for (int i = 0; i < 3; ++i) {
    dense[i] = static_cast<uint64_t>(a.n_tok) * static_cast<uint64_t>(a.heads[i]) * kD * es;
    span[i] = static_cast<uint64_t>(a.n_tok - 1) * static_cast<uint64_t>(a.stride[i]) * es +
              static_cast<uint64_t>(a.heads[i]) * kD * es;
  }
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < 3; ++i) {
      const bool same = o == i && out[o] == a.x[i] && a.stride[i] == static_cast<long long>(a.heads[i]) * kD;
      if (!same && raw::overlap(out[o], dense[o], a.x[i], span[i])) return fail(KVTC_EINVAL, "an output overlaps an input");
    }
  }
  if (raw::overlap(out[0], dense[0], out[1], dense[1])) return fail(KVTC_EINVAL, "the outputs overlap");
  const uint64_t n = static_cast<uint64_t>(a.n_tok);
  const std::initializer_list<raw::Range> lists = {{a.positions, 4 * n * static_cast<uint64_t>(n_axes)}, {a.slots, 8 * n}};
  if (raw::overlaps_any(out[0], dense[0], lists) || raw::overlaps_any(out[1], dense[1], lists))
    return fail(KVTC_EINVAL, "an output overlaps the positions or the slots");
  if (cache) {
    if (raw::overlaps_any(cache->pool, raw::pool_bytes(cache), lists))
      return fail(KVTC_EINVAL, "the positions or the slots overlap the pool");
    if (raw::overlaps_any(cache->status, 4, lists) ||
        raw::overlaps_any(cache->status, 4, {{cache->pool, raw::pool_bytes(cache)}, {out[0], dense[0]},
                                             {a.x[0], span[0]}, {a.x[1], span[1]}, {a.x[2], span[2]}}))
      return fail(KVTC_EINVAL, "the status word overlaps another buffer");
    bool pool = raw::overlap(out[0], dense[0], cache->pool, raw::pool_bytes(cache));
    for (int i = 0; i < 3; ++i) pool |= raw::overlap(a.x[i], span[i], cache->pool, raw::pool_bytes(cache));
    if (pool) return fail(KVTC_EINVAL, "rows overlap the pool");
  }
  return KVTC_OK;
}

kvtc_status launch_rope(RopeArgs& a, kvtc_dtype dtype, void* stream) {
  // as many warps of a token as keep the chip busy, each with some rows at least
  const int at_once = dtype == KVTC_F32 ? 2 : 4;  // rows a warp moves at a time
  const int n_all = a.heads[0] + a.heads[1] + a.heads[2];
  const int most = (n_all + at_once - 1) / at_once;
  int sms = 0;
  const kvtc_status st = raw::sm_count(&sms);
  if (st != KVTC_OK) return st;
  const long long busy = static_cast<long long>(kBusyWarpsPerSm) * sms;
  const int want = static_cast<int>(std::min<long long>(most, (busy + a.n_tok - 1) / a.n_tok));
  a.part_rows = (most + want - 1) / want * at_once;
  a.parts = (n_all + a.part_rows - 1) / a.part_rows;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.n_tok) * a.parts + kWarps - 1) / kWarps);
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
  st = check_rope_overlap(a, es, rope->n_axes, nullptr);
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
  if (n_tok == 0) return KVTC_OK;  // (empty tensors have null pointers)
  if (!q && n_q_heads != 0) return fail(KVTC_EINVAL, "null device pointer");
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
  st = check_rope_overlap(a, 2, rope ? rope->n_axes : 0, cache);
  if (st != KVTC_OK) return st;
  return launch_rope(a, cache->dtype, stream);
}
