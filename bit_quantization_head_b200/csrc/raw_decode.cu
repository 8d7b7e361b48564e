// kvtc_raw_decode_attention: one new token per sequence over uncompressed pages.
//
// o = sum_t p_t v_t / sum_t p_t with p_t = 2^(c (q . k_t - m)), c = scale * log2(e), in one
// pass with the running maximum m and sum of every query head; the query heads of a KV head
// share each K and V tile.
//
// Bound: HBM, 512 bytes per token and KV head for 4 * 128 flops per query head; the arithmetic
// runs as m16n8k16 MMAs (scores: 16 tokens x 8 heads; values: 16 dims x 8 heads).  Measured
// with up to 8 query heads per KV head: 16 x 32768 tokens of 8 KV heads in 330 us (6.5 TB/s,
// the rate of a copy), one sequence of 131072 tokens and 4 KV heads in 55 us (41 at that rate:
// about 4 us until the first tiles are there, 6 to join 74 parts of a head), 4096 tokens in
// 10.4 us and three chats of up to 1000 tokens in 8.6 us (launch, two dependent reads, a tile,
// and the join of its parts).  With 9 to 16 query heads the consumers are the bound: 446 us for
// the same 16 x 32768 tokens (12 or 16 heads; 4.8 TB/s), 15.6 us for the three chats, 71 us for
// 131072 tokens of 4 KV heads; above 16 heads K and V are read again for every further 16 (17
// or 32 heads 883 us).
//
// Work split.  A unit is (sequence, KV head, group of up to 8 or 16 query heads), its tiles 64
// tokens.  All tiles of all units in a row are cut into one equal run per CTA, whatever the
// lengths are, found on the device from seq_lens: a ragged batch and a single long sequence
// load every SM alike, and the workspace does not grow with the batch.  Up to 8 heads: two CTAs
// per SM with rings of three tiles (one with twice the ring: 440 us for 16 x 32768, its four
// warps do not keep up).  9 to 16: one CTA per SM with a ring of five (two rings of three do not
// fit in shared memory while every stage has room for the queries; neither that nor more
// consumer warps were tried).  A run
// covers whole units but for its first and last; those leave a partial (m, l, z) and the
// last CTA of the unit to arrive (a counter kept by the unit's first CTA) joins them in
// order, so results do not depend on timing.
//
// CTA: 4 consumer warps (16 tokens of each tile each) and a producer warp that walks the run
// and keeps a ring of tiles in flight with TMA (128-byte swizzle: ldmatrix without bank
// conflicts); the queries of a unit arrive with its first tile.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "ptx.cuh"
#include "raw_cache.cuh"
#include "raw_device.cuh"

namespace kvtc {
namespace raw {
namespace {

constexpr int kTile = 64;                          // tokens of a tile
constexpr int kConsumers = 4;                      // warps, 16 tokens each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr uint32_t kBoxBytes = kTile * 128;        // 64 tokens x 64 elements
constexpr uint32_t kTileBytes = 4 * kBoxBytes;     // K, V x two halves
constexpr int kMaxCtas = 320;                      // partial slots in the workspace
constexpr int kRowPad = 132;                       // floats of a scratch row (conflict-free)
// Reference of a head that has met no score above -inf: a weight is then 2^(-inf - it) = 0
// where 2^(-inf - -inf) would be NaN, and its sums are 0, so any factor serves a join.
constexpr float kLowest = -3.402823466e38f;

__host__ __device__ constexpr int stages(int nt) { return nt == 1 ? 3 : 5; }
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 2 : 1; }

// What the producer tells the consumers about a tile.
struct TileDesc {
  int n;       // tokens of the sequence in it (0: none, or not loaded)
  int flags;   // kFirst ..
  int seq, head;  // head: h * groups + group
  int c0, c1;  // CTAs that share the unit
};
enum { kFirst = 1, kLast = 2, kBad = 4, kBegins = 8, kEnds = 16, kRunEnds = 32, kNothing = 64 };

template <int NT>
struct __align__(1024) Smem {
  unsigned char kv[stages(NT)][kTileBytes];
  unsigned char q[stages(NT)][NT * 8 * 256];
  float z[2][8 * kRowPad];  // sums of warps 0 + 2 and of warps 1 + 3
  float m[kConsumers][NT * 8], l[kConsumers][NT * 8];
  TileDesc desc[stages(NT)];
  uint64_t full[stages(NT)], empty[stages(NT)];
  int dead;
  int last;
};

struct DecodeArgs {
  const int32_t* table;
  const int32_t* seq_lens;
  int n_seq, max_pages, max_len;
  long long n_pages;
  int H, G, groups, group_heads;  // query heads per KV head; groups of at most group_heads
  int row0;                       // first pool row of the layer
  const uint16_t* q;
  uint16_t* out;
  float c;                        // scale * log2(e)
  int* tickets;
  float* parts;
  int32_t* status;
};

// Length of sequence s as the kernel uses it, and whether it is out of range.
__device__ __forceinline__ int seq_len(const DecodeArgs& a, int s, bool& bad) {
  const int n = a.seq_lens[s];
  bad = n < 0 || n > a.max_len;
  return bad ? 0 : n;
}
__device__ __forceinline__ int n_tiles(int len) { return max(1, (len + kTile - 1) / kTile); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    mma_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// ------------------------------------------------------------------ producer warp
template <int NT>
__device__ void produce(const DecodeArgs& a, Smem<NT>& s, const CUtensorMap* map) {
  const int lane = threadIdx.x & 31;
  const int units = a.H * a.groups;
  volatile int* dead = &s.dead;
  bool bad_len;
  // the run: tiles f .. f1 - 1 of all units' in a row
  int longest = 0;
  auto tiles = [&](int i) {
    const int n = n_tiles(seq_len(a, i, bad_len));
    longest = max(longest, n);
    return static_cast<long long>(n) * units;
  };
  SlotScan<decltype(tiles)> scan(a.n_seq, tiles);
  const long long total = scan.total;
  // Runs of at least 1 to 4 tiles: fewer parts to join where one sequence has the chip (4096
  // tokens of 8 heads: 10.4 us with 4, 11.8 with 1; 1000 tokens: 7.8 with 1, 8.5 with 2).
  const int shortest = min(4, max(1, __reduce_max_sync(0xffffffffu, longest) / 16));
  const int n_cta = static_cast<int>(min(static_cast<long long>(gridDim.x), divide(total + shortest - 1, shortest)));
  long long f = 0, f1 = 0, base = 0;  // base: first tile of the sequence's units
  if (static_cast<int>(blockIdx.x) < n_cta) {
    f = run_start(blockIdx.x, n_cta, total);
    f1 = run_start(blockIdx.x + 1, n_cta, total);
  } else if (lane == 0) {
    s.desc[0].flags = kNothing;
    mbar_arrive(&s.full[0]);
  }
  int seq = f < f1 ? scan.find(f, base) : 0, it = 0;
  int len = seq_len(a, seq, bad_len), nt = n_tiles(len);
  int page0 = -1, page_id = -1, page_seq = -1;  // 32 page ids from page0 on, one per lane
  bool ok = true;
  uint32_t flags_seen = 0;
  while (f < f1 && ok) {
    while (f >= base + static_cast<long long>(nt) * units) {
      base += static_cast<long long>(nt) * units;
      ++seq;
      len = seq_len(a, seq, bad_len);
      nt = n_tiles(len);
    }
    if (bad_len) flags_seen |= KVTC_STATUS_BAD_POS;
    const int u = static_cast<int>(divide(f - base, nt));
    const int i0 = static_cast<int>(f - base - static_cast<long long>(u) * nt);
    const int i1 = static_cast<int>(min(static_cast<long long>(nt), i0 + (f1 - f)));
    const long long begin = base + static_cast<long long>(u) * nt;
    int c0 = 0, c1 = 0;
    const int h = u / a.groups, grp = u - h * a.groups;
    const int heads = min(a.group_heads, a.G - grp * a.group_heads);
    for (int i = i0; i < i1 && ok; ++i, ++it) {
      const int st = it % stages(NT);
      const int page = i * kTile / kPage;
      if (len > 0 && (page_seq != seq || page < page0 || page >= page0 + 32)) {
        page_seq = seq;
        page0 = page;
        const int p = page + lane;
        // (in pages: p * 128 passes 31 bits behind the last page of the longest table)
        page_id = p < (len + kPage - 1) / kPage ? a.table[static_cast<size_t>(seq) * a.max_pages + p] : -1;
      }
      const int id = __shfl_sync(0xffffffffu, page_id, len > 0 ? page - page0 : 0);
      const bool have = len > 0, good = have && id >= 0 && id < a.n_pages;
      if (have && !good) flags_seen |= KVTC_STATUS_BAD_PAGE;
      if (lane == 0) {
        if (it >= stages(NT)) ok = wait_phase(&s.empty[st], (it / stages(NT) - 1) & 1, dead);
        if (ok) {
          // The copies first, what the consumers read beside them while they fly: the phase
          // cannot end before the arrival below (4096 tokens of 8 heads: 10.7 -> 10.4 us).
          if (good) {
            const int row = a.row0 + (id * a.H + h) * 2 * kPage + (i * kTile) % kPage;
            unsigned char* dst = s.kv[st];
            tma_load_2d(dst, map, 0, row, &s.full[st]);
            tma_load_2d(dst + kBoxBytes, map, 64, row, &s.full[st]);
            tma_load_2d(dst + 2 * kBoxBytes, map, 0, row + kPage, &s.full[st]);
            tma_load_2d(dst + 3 * kBoxBytes, map, 64, row + kPage, &s.full[st]);
          }
          const uint32_t q_bytes = i == i0 ? static_cast<uint32_t>(heads) * 256u : 0u;
          if (q_bytes) {
            bulk_copy_g2s(s.q[st], a.q + (static_cast<size_t>(seq) * a.H * a.G + static_cast<size_t>(h) * a.G + grp * a.group_heads) * kD,
                          q_bytes, &s.full[st]);
            c0 = run_owner(begin, n_cta, total);
            c1 = run_owner(begin + nt - 1, n_cta, total);
          }
          TileDesc& d = s.desc[st];
          d.n = good ? min(kTile, len - i * kTile) : 0;
          d.flags = (i == i0 ? kFirst : 0) | (i == i1 - 1 ? kLast : 0) | (have && !good ? kBad : 0) |
                    (i0 == 0 ? kBegins : 0) | (i1 == nt ? kEnds : 0) |
                    (i == i1 - 1 && f + (i1 - i0) == f1 ? kRunEnds : 0);
          d.seq = seq;
          d.head = u;
          d.c0 = c0;
          d.c1 = c1;
          mbar_arrive_expect_tx(&s.full[st], (good ? kTileBytes : 0u) + q_bytes);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
    }
    f += i1 - i0;
  }
  if (!ok && lane == 0) {
    *dead = 1;
    flags_seen |= KVTC_STATUS_TIMEOUT;
  }
  if (lane == 0 && flags_seen && a.status) atomicOr(a.status, static_cast<int>(flags_seen));
  // drain: every copy in flight lands before the CTA may exit (bounded)
  if (lane == 0) {
    volatile int never = 0;
    for (int k = max(0, it - stages(NT)); k < it; ++k) (void)wait_phase(&s.full[k % stages(NT)], (k / stages(NT)) & 1, &never);
  }
}

// ------------------------------------------------------------------ consumer warps
// One query head's 8 dims of a finished sum (r: 1 / l; where every score is -inf that makes
// 0 / 0, a row without a softmax, and 0 where there is nothing to attend to).
template <bool F16>
__device__ __forceinline__ void store_out(uint16_t* dst, const float (&z)[8], float r) {
  uint4 w;
  w.x = pack2<F16>(z[0] * r, z[1] * r);
  w.y = pack2<F16>(z[2] * r, z[3] * r);
  w.z = pack2<F16>(z[4] * r, z[5] * r);
  w.w = pack2<F16>(z[6] * r, z[7] * r);
  *reinterpret_cast<uint4*>(dst) = w;
}

// Partial slot of CTA c: [NT * 8 heads][128] z, then [NT * 8][2] (m, l).  Slot 1 holds the
// unit that begins in the CTA, slot 0 the one that came from an earlier CTA.
template <int NT>
__device__ __forceinline__ float* part_of(const DecodeArgs& a, int c, int slot) {
  return a.parts + (static_cast<size_t>(c) * 2 + slot) * (NT * 8 * (kD + 2));
}

// Arrives at `ticket` for this CTA's part; the last of n_part CTAs joins their parts (CTAs
// first, first + step, ..; c0: the one where the unit begins) into the output, or into the
// place of the first one's.  False if the CTA gave up; s.last: whether this CTA joined.
template <int NT, bool F16, bool kFinal>
__device__ __forceinline__ bool join_parts(const DecodeArgs& a, Smem<NT>& s, int* ticket, int c0, int first, int step,
                                           int n_part, int heads, size_t out0) {
  const int tid = threadIdx.x;
  auto sync = [&]() -> bool { return consumers_sync(1, 32 * kConsumers, &s.dead); };
  __threadfence();
  if (!sync()) return false;
  if (tid == 0) s.last = atomicAdd(ticket, 1) == n_part - 1;
  if (!sync()) return false;
  if (!s.last) return true;
  __threadfence();
  if (tid == 0) *ticket = 0;
  for (int n = 0; n < NT && n * 8 < heads; ++n) {
    // a head's 16 chunks of 8 dims by 16 threads; with at most 4 heads the parts are dealt
    // over the threads left (their sums are added in order).  The reference moves on from
    // part to part, so that a part's reads are all under way at once.
    const int live = min(8, heads - n * 8), deal = live <= 1 ? 8 : live <= 2 ? 4 : live <= 4 ? 2 : 1, own = 8 / deal;
    const int slot = tid >> 4, hd = slot % own, sub = slot / own, row = n * 8 + hd, dim = (tid & 15) * 8;
    float v[8] = {}, sum = 0.0f, top = kLowest;
    bool any_bad = false;
    auto add = [&](float m, float l, const float (&x)[8]) {
      const float to = fmaxf(top, m);
      const float f0 = ex2((top - to) * a.c), f1 = ex2((m - to) * a.c);
      any_bad |= l < 0.0f;
      sum = sum * f0 + l * f1;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * f0 + x[e] * f1;
      top = to;
    };
    if (hd < live) {
#pragma unroll 8
      for (int i = sub; i < n_part; i += deal) {
        const int c = first + i * step;
        const float* p = part_of<NT>(a, c, c == c0);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + NT * 8 * kD + 2 * row));
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p + row * kD + dim));
        const float4 y = __ldcg(reinterpret_cast<const float4*>(p + row * kD + dim) + 1);
        const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        add(ml.x, ml.y, z);
      }
    }
    if (deal > 1) {
      float* mine = s.z[0] + slot * kRowPad + dim;
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[e] = v[e];
      if ((tid & 15) == 0) {
        s.z[1][2 * slot] = top;
        s.z[1][2 * slot + 1] = any_bad ? -1.0f : sum;
      }
      if (!sync()) return false;
      if (sub == 0) {
        for (int k = 1; k < deal; ++k) {
          const int from = hd + k * own;
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = s.z[0][from * kRowPad + dim + e];
          add(s.z[1][2 * from], s.z[1][2 * from + 1], z);
        }
      }
    }
    // a part's result may go to the place of the first part: all of a head's threads, which are
    // of one warp, have read that one's (m, l) by then
    __syncwarp();
    if (sub == 0 && hd < live) {
      if (any_bad) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
      }
      if (kFinal) {
        store_out<F16>(a.out + (out0 + row) * kD + dim, v, any_bad ? 0.0f : 1.0f / sum);
      } else {
        float* p = part_of<NT>(a, first, first == c0);
        reinterpret_cast<float4*>(p + row * kD + dim)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p + row * kD + dim)[1] = make_float4(v[4], v[5], v[6], v[7]);
        if (dim == 0) {
          p[NT * 8 * kD + 2 * row] = top;
          p[NT * 8 * kD + 2 * row + 1] = any_bad ? -1.0f : sum;
        }
      }
    }
    if (!sync()) return false;
  }
  return true;
}

// The same in two levels: groups of CTAs, then the groups' parts.
template <int NT, bool F16>
__device__ __noinline__ bool join_groups(const DecodeArgs& a, Smem<NT>& s, int c0, int shares, int heads, size_t out0) {
  // Groups of 8 up to 128 parts, of 16 above (74 parts of 7 heads over 131072 tokens 54.3 us
  // with 8, 56.8 with 16; 128 parts of 8 heads 17.9 and 19.1; 148 parts of 4 heads 33.1 and
  // 33.8; 296 parts of 8 heads 26.1 and 24.7).
  const int group = shares <= 128 ? 8 : 16;
  const int begin = (static_cast<int>(blockIdx.x) - c0) / group * group, first = c0 + begin;
  if (!join_parts<NT, F16, false>(a, s, a.tickets + 2 * first + (begin == 0), c0, first, 1, min(group, shares - begin),
                                  heads, out0))
    return false;
  if (!s.last) return true;
  return join_parts<NT, F16, true>(a, s, a.tickets + 2 * kMaxCtas + c0, c0, c0, group, (shares + group - 1) / group, heads,
                                   out0);
}

template <int NT, bool F16>
__device__ void consume(const DecodeArgs& a, Smem<NT>& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  volatile int* dead = &s.dead;
  // ldmatrix addresses inside a stage: K rows (token 16 warp + (lane / 8 % 2) * 8 + lane % 8,
  // dims + lane / 16 * 8), V rows transposed (token + lane / 16 * 8, dims + (lane / 8 % 2) * 8)
  const int krow = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7);
  const int vrow = 16 * warp + (lane >> 4) * 8 + (lane & 7);
  const uint32_t kbase = static_cast<uint32_t>(krow) * 128u, vbase = 2 * kBoxBytes + static_cast<uint32_t>(vrow) * 128u;
  const int kch = lane >> 4, vch = (lane >> 3) & 1;
  uint32_t qf[NT][8][2];
  float z[NT][8][4], m[NT][2], l[NT][2];
  bool bad = false, some = false;  // of the unit's tiles so far: a bad page, tokens
  auto consumer_sync = [&]() -> bool { return consumers_sync(1, 32 * kConsumers, dead); };
  for (int it = 0;; ++it) {
    const int st = it % stages(NT);
    if (!wait_warp(&s.full[st], (it / stages(NT)) & 1, dead)) {
      if (lane == 0) {
        *dead = 1;
        if (a.status) atomicOr(a.status, static_cast<int>(KVTC_STATUS_TIMEOUT));
      }
      __syncwarp();
      leave_barrier(1, 32 * kConsumers);
      return;
    }
    const TileDesc d = s.desc[st];
    if (d.flags & kNothing) return;
    const int h = d.head / a.groups, grp = d.head - h * a.groups;
    const int heads = min(a.group_heads, a.G - grp * a.group_heads);
    if (d.flags & kFirst) {
      bad = some = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool live = n * 8 + g < heads;
        const uint32_t* row = reinterpret_cast<const uint32_t*>(s.q[st] + (n * 8 + g) * 256);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qf[n][ks][0] = live ? row[8 * ks + t] : 0u;
          qf[n][ks][1] = live ? row[8 * ks + 4 + t] : 0u;
          z[n][ks][0] = z[n][ks][1] = z[n][ks][2] = z[n][ks][3] = 0.0f;
        }
        m[n][0] = m[n][1] = kLowest;
        l[n][0] = l[n][1] = 0.0f;
      }
    }
    bad |= (d.flags & kBad) != 0;
    some |= d.n > 0;
    const int nv = d.n - 16 * warp;
    if (nv > 0) {
      const uint32_t tile = smem_u32(s.kv[st]);
      if (nv < 16) {
        // tokens past the end: their V rows may hold anything (0 * NaN is NaN)
        for (int r = nv + (lane >> 4); r < 16; r += 2) {
          unsigned char* row = s.kv[st] + 2 * kBoxBytes + ((lane >> 3) & 1) * kBoxBytes + (16 * warp + r) * 128 + (lane & 7) * 16;
          *reinterpret_cast<uint4*>(row) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // before a later copy into this stage
        __syncwarp();
      }
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t af[4];
        const int chunk = (2 * ks + kch) & 7;
        ldsm4(af, tile + (ks >> 2) * kBoxBytes + kbase + (static_cast<uint32_t>(chunk ^ (krow & 7)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) mma<F16>(sc[n], af, qf[n][ks][0], qf[n][ks][1]);
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (g >= nv) sc[n][0] = sc[n][1] = -INFINITY;
        if (g + 8 >= nv) sc[n][2] = sc[n][3] = -INFINITY;
        float top[2] = {fmaxf(sc[n][0], sc[n][2]), fmaxf(sc[n][1], sc[n][3])};
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
          top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
          top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
        }
        if (__any_sync(0xffffffffu, top[0] > m[n][0] || top[1] > m[n][1])) {
          const float m0 = fmaxf(m[n][0], top[0]), m1 = fmaxf(m[n][1], top[1]);
          const float f0 = ex2((m[n][0] - m0) * a.c), f1 = ex2((m[n][1] - m1) * a.c);
          l[n][0] *= f0;
          l[n][1] *= f1;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            z[n][k][0] *= f0;
            z[n][k][1] *= f1;
            z[n][k][2] *= f0;
            z[n][k][3] *= f1;
          }
          m[n][0] = m0;
          m[n][1] = m1;
        }
        // fp16 weights are 2^15 at the maximum, so those far below it keep clear of the
        // subnormals
        constexpr float kBias = F16 ? 15.0f : 0.0f;
        const float p0 = ex2(fmaf(sc[n][0] - m[n][0], a.c, kBias)), p1 = ex2(fmaf(sc[n][1] - m[n][1], a.c, kBias));
        const float p2 = ex2(fmaf(sc[n][2] - m[n][0], a.c, kBias)), p3 = ex2(fmaf(sc[n][3] - m[n][1], a.c, kBias));
        l[n][0] += p0 + p2;
        l[n][1] += p1 + p3;
        // P enters the value MMA in the pages' type (half a step of relative error on each
        // weight, as for the output; the sum l stays fp32)
        pf[n][0] = movmatrix_trans(pack2<F16>(p0, p1));
        pf[n][1] = movmatrix_trans(pack2<F16>(p2, p3));
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        uint32_t af[4];
        const int chunk = (2 * mt + vch) & 7;
        ldsm4_t(af, tile + (mt >> 2) * kBoxBytes + vbase + (static_cast<uint32_t>(chunk ^ (vrow & 7)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) mma<F16>(z[n][mt], af, pf[n][0], pf[n][1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.empty[st]);
    if (!(d.flags & kLast)) continue;

    // ---- the unit's tiles in this CTA are done: join the four warps
    const bool whole = (d.flags & (kBegins | kEnds)) == (kBegins | kEnds);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) {
        l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], o);
        l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], o);
      }
      if (g == 0) {
        s.m[warp][n * 8 + 2 * t] = m[n][0];
        s.m[warp][n * 8 + 2 * t + 1] = m[n][1];
        s.l[warp][n * 8 + 2 * t] = l[n][0];
        s.l[warp][n * 8 + 2 * t + 1] = l[n][1];
      }
    }
    const int slot = d.flags & kBegins ? 1 : 0;
    const size_t out0 = static_cast<size_t>(d.seq) * a.H * a.G + static_cast<size_t>(h) * a.G + grp * a.group_heads;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n * 8 >= heads) break;
      // (z0 + z2) + (z1 + z3): warps 0 and 1 leave their sums as they are, 2 and 3 scale both
      float* mine = s.z[warp & 1] + 2 * t * kRowPad + g;
      if (warp < 2) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[(e & 1) * kRowPad + 16 * mt + (e >> 1) * 8] = z[n][mt][e];
      }
      if (!consumer_sync()) return;
      if (warp >= 2) {
        float f[2], f0[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int hd = n * 8 + 2 * t + j;
          const float top = fmaxf(fmaxf(s.m[0][hd], s.m[1][hd]), fmaxf(s.m[2][hd], s.m[3][hd])), m0 = s.m[warp - 2][hd];
          f[j] = ex2((m[n][j] - top) * a.c);
          f0[j] = ex2((m0 - top) * a.c);
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* p = mine + (e & 1) * kRowPad + 16 * mt + (e >> 1) * 8;
            *p = *p * f0[e & 1] + z[n][mt][e] * f[e & 1];
          }
      }
      if (!consumer_sync()) return;
      const int hd = tid >> 4, dim = (tid & 15) * 8, row = n * 8 + hd;
      if (row < heads) {
        float top = kLowest, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, s.m[w][row]);
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) sum += s.l[w][row] * ex2((s.m[w][row] - top) * a.c);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s.z[0][hd * kRowPad + dim + e] + s.z[1][hd * kRowPad + dim + e];
        if (whole) {
          if (bad) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
          }
          store_out<F16>(a.out + (out0 + row) * kD + dim, v, bad || !some ? 0.0f : 1.0f / sum);
        } else {
          float* p = part_of<NT>(a, blockIdx.x, slot);
          reinterpret_cast<float4*>(p + row * kD + dim)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(p + row * kD + dim)[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (dim == 0) {
            p[NT * 8 * kD + 2 * row] = top;
            p[NT * 8 * kD + 2 * row + 1] = bad ? -1.0f : sum;  // a sum below 0 marks a bad page
          }
        }
      }
      if (!consumer_sync()) return;
    }
    if (whole) {
      if (d.flags & kRunEnds) return;
      continue;
    }
    // ---- the unit is shared with other CTAs: the last one to arrive joins the partials; of
    // many, groups of CTAs first (joined while other CTAs still compute; at once, 74 parts
    // took 59.8 us instead of 54.3, 296 of 8 heads 49 instead of 25)
    const int shares = d.c1 - d.c0 + 1;
    bool ok;
    if (shares <= 48)
      ok = join_parts<NT, F16, true>(a, s, a.tickets + 2 * d.c0 + 1, d.c0, d.c0, 1, shares, heads, out0);
    else
      ok = join_groups<NT, F16>(a, s, d.c0, shares, heads, out0);
    if (!ok || (d.flags & kRunEnds)) return;
  }
}

template <int NT, bool F16>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT))
    raw_decode_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem<NT>& s = *reinterpret_cast<Smem<NT>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 32 * kConsumers) prefetch_map(&map);
  if (tid == 0) {
    for (int i = 0; i < stages(NT); ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kConsumers);
    }
    s.dead = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  if (warp == kConsumers)
    produce<NT>(a, s, &map);
  else
    consume<NT, F16>(a, s);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

CUtensorMapDataType map_type(kvtc_dtype t) {
  return t == KVTC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

template <int NT, bool F16>
kvtc_status launch_decode(const CUtensorMap& map, const DecodeArgs& a, int grid, void* stream) {
  const size_t smem = sizeof(Smem<NT>) + 1024;
  const kvtc_status st = allow_smem<raw_decode_kernel<NT, F16>>(smem);
  if (st != KVTC_OK) return st;
  const cudaError_t e = launch(raw_decode_kernel<NT, F16>, dim3(static_cast<unsigned>(grid)), kThreads, smem, stream, map, a);
  if (e != cudaSuccess) return cuda_fail(e, "raw decode launch");
  return KVTC_OK;
}

// Query heads of a unit: one MMA column tile of 8, or two from 9 query heads per KV head on
// (K and V are then read once for up to 16 heads).
int n_col_tiles(int group) { return group <= 8 ? 1 : 2; }

}  // namespace

kvtc_status pool_map(CUtensorMap* m, const kvtc_raw_cache* c, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return fail(KVTC_ECUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD),
                              static_cast<cuuint64_t>(c->n_layers) * c->n_pages * static_cast<cuuint64_t>(c->n_kv_heads) * 2 * kPage};
  const cuuint64_t strides[1] = {kD * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, map_type(c->dtype), 2, c->pool, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(KVTC_ECUDA, "cuTensorMapEncodeTiled failed (pages)");
  return KVTC_OK;
}

kvtc_status query_map(CUtensorMap* m, const void* q, kvtc_dtype dtype, int n_tok, int n_kv_heads, int group,
                      int box_heads, int box_tok) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return fail(KVTC_ECUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(group),
                              static_cast<cuuint64_t>(n_kv_heads), static_cast<cuuint64_t>(n_tok)};
  const cuuint64_t strides[3] = {kD * 2, static_cast<cuuint64_t>(group) * kD * 2,
                                 static_cast<cuuint64_t>(group) * static_cast<cuuint64_t>(n_kv_heads) * kD * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), 1, static_cast<cuuint32_t>(box_tok)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, map_type(dtype), 4, const_cast<void*>(q), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(KVTC_ECUDA, "cuTensorMapEncodeTiled failed (queries)");
  return KVTC_OK;
}

}  // namespace raw
}  // namespace kvtc

using namespace kvtc;

// Counters (4096 bytes: two per CTA for the groups of a unit's parts, one for the groups
// themselves), then two partial slots for each CTA.
extern "C" uint64_t kvtc_raw_decode_workspace_bytes(int n_seq, int n_q_heads, int n_kv_heads, int max_seq_len) {
  if (n_seq < 1 || n_kv_heads < 1 || n_q_heads < n_kv_heads || max_seq_len < 0) return 0;
  const uint64_t rows = 8ull * raw::n_col_tiles(n_q_heads / n_kv_heads);
  return 4096 + static_cast<uint64_t>(raw::kMaxCtas) * 2 * rows * (kD + 2) * sizeof(float);
}

extern "C" kvtc_status kvtc_raw_decode_attention(const kvtc_raw_cache* cache, int layer, const void* q, int n_q_heads,
                                                 const int32_t* seq_lens, int max_seq_len, float softmax_scale,
                                                 void* out, void* workspace, uint64_t workspace_bytes, void* stream) {
  kvtc_status st = raw::check_attention(cache, layer, n_q_heads, 1024, max_seq_len, softmax_scale);
  if (st != KVTC_OK) return st;
  if (!q || !seq_lens || !out || !workspace) return fail(KVTC_EINVAL, "null device pointer");
  if (!raw::aligned16(q) || !raw::aligned16(out) || !raw::aligned16(workspace))
    return fail(KVTC_EINVAL, "q, out and workspace must be 16-byte aligned");
  if (workspace_bytes < kvtc_raw_decode_workspace_bytes(cache->n_seq, n_q_heads, cache->n_kv_heads, max_seq_len))
    return fail(KVTC_ECAPACITY, "decode workspace too small");
  st = raw::check_overlap(cache, q, out, static_cast<uint64_t>(cache->n_seq) * n_q_heads * kD * 2, workspace,
                          kvtc_raw_decode_workspace_bytes(cache->n_seq, n_q_heads, cache->n_kv_heads, max_seq_len),
                          seq_lens, nullptr);
  if (st != KVTC_OK) return st;
  int sms = 0;
  st = raw::sm_count(&sms);
  if (st != KVTC_OK) return st;
  CUtensorMap map;
  st = raw::pool_map(&map, cache, raw::kTile);
  if (st != KVTC_OK) return st;
  const int group = n_q_heads / cache->n_kv_heads, nt = raw::n_col_tiles(group);
  raw::DecodeArgs a;
  a.table = cache->block_table;
  a.seq_lens = seq_lens;
  a.n_seq = cache->n_seq;
  a.max_pages = cache->max_pages;
  a.max_len = max_seq_len;
  a.n_pages = static_cast<long long>(cache->n_pages);
  a.H = cache->n_kv_heads;
  a.G = group;
  a.groups = (group + 8 * nt - 1) / (8 * nt);
  a.group_heads = (group + a.groups - 1) / a.groups;
  a.row0 = static_cast<int>(static_cast<uint64_t>(layer) * cache->n_pages * static_cast<uint64_t>(a.H) * 2 * kPage);
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.c = raw::exp2_scale(softmax_scale);
  a.tickets = static_cast<int*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + 4096);
  a.status = cache->status;
  const long long tiles = static_cast<long long>(cache->n_seq) * a.H * a.groups * std::max(1, (max_seq_len + raw::kTile - 1) / raw::kTile);
  const int per_sm = nt == 1 ? raw::ctas_per_sm(1) : raw::ctas_per_sm(2);
  const int grid = static_cast<int>(std::min<long long>(std::min(per_sm * sms, raw::kMaxCtas), tiles));
  const bool f16 = cache->dtype == KVTC_F16;
  if (nt == 1) return f16 ? raw::launch_decode<1, true>(map, a, grid, stream) : raw::launch_decode<1, false>(map, a, grid, stream);
  return f16 ? raw::launch_decode<2, true>(map, a, grid, stream) : raw::launch_decode<2, false>(map, a, grid, stream);
}
