// kvtc_raw_cross_attention: ragged query rows over an encoder's states in uncompressed pages.
//
// o = sum_t p_t v_t / sum_t p_t with p_t = 2^(c (q . k_t - m)), c = scale * log2(e), in one
// pass with a running reference m and the running sum of every row.  m follows the maximum
// only when a row's score exceeds it by more than 2^8 in p: the sum and the accumulators are
// scaled then, otherwise not at all.
//
// Bound: the tensor cores (512 flops per query row, head and token); for few rows the bytes
// of the states.  S = Q K^T and O += P V run on tcgen05 (M = 128 rows, N = 128), both
// accumulators and P (16 bits, over S's columns) in TMEM.  Measured: 16384 queries of 32
// heads over 16384 states 3.4 ms on a cool chip (1.29 PFLOP/s), 3.9 ms in a row of calls
// under the power cap (1.13 PFLOP/s; a plain matrix product holds 1.40 there).  A step of two
// tiles takes about 3000 cycles, 2048 of them of the tensor pipe: the row warps issue about
// 1850 instructions for it on each scheduler, many of them double-width, beside 1280 cycles
// of exponentials.  Smaller calls (two tiles a unit, one unit per CTA, pages in L2): 11 us and
// 1.65 us a step; every further unit of a CTA 7 us for its start and output beside its steps.
// Times here and below are of calls replayed from a graph on the same inputs; with inputs that
// change, calls of tens of us take 3 to 6 us more.
//
// Rows of a tile: the tokens' query heads of one KV head (token-major, as many whole tokens
// as fit in 128 rows), so K and V are read once for all of them.  A unit is (sequence, KV
// head, two such tiles); a step is its 128-token K and V page against both.  All steps of
// all units in a row are cut into one equal run per CTA (one CTA per SM), found on the
// device from cu_q and seq_lens; a unit that several CTAs share leaves (m, l, O) of each
// part in the workspace, and the last CTA to arrive joins them in order, so results do not
// depend on timing.
//
// CTA: warps 0-3 and 4-7 hold one row per thread of the first and second tile (softmax,
// rescaling, output), warp 8 finds the run and loads with TMA, warp 9 issues the MMAs in the
// order PV_a(j), S_a(j+1), PV_b(j), S_b(j+1): one tile's softmax runs beside the other's
// MMAs.  P comes in two halves, so a value product starts before its softmax has ended.  A
// unit of one tile (few rows) has both row groups: the second takes every other step, and
// the first takes its sums in at the end.  Two threads per row (64 tokens each, 16 row warps)
// were slower (ragged batch of 8: 62 us, 53 with one): the schedulers, not the length of a
// row's work, are what the softmax runs against.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ptx.cuh"
#include "raw_cache.cuh"
#include "raw_device.cuh"

namespace kvtc {
namespace raw {
namespace {

constexpr int kRows = 128;                       // rows of a tile (TMEM lanes)
constexpr int kWarps = 12;                       // the last two idle: register shares go by four warps
constexpr int kThreads = 32 * kWarps;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr uint32_t kHalfBytes = 128 * 128;       // 64 elements of 128 rows
constexpr uint32_t kTileBytes = 2 * kHalfBytes;
constexpr int kStages = 4;                       // K or V tiles in flight (a power of 2)
constexpr int kMaxCtas = 160;                    // partial slots in the workspace
constexpr int kPartFloats = kRows * (kD + 2);    // (m, l) of each row, then its sums
constexpr uint32_t kTmemCols = 512;              // S_a, S_b, O_a, O_b
// Registers of a thread: 384 threads start with 168 each (64512); the row warps take what
// the others leave (2 * 208 + 88 = 3 * 168).
constexpr int kRowRegs = 208, kOtherRegs = 88;
// What a unit costs beside its steps (filling the pipeline, output or parts), in steps: the
// runs are cut by steps + kUnitCost slots a unit, the first kUnitCost of them without a step
// (a ragged batch of 8 with units of 1 and of 12 steps: 73 us with 0, 52 with 1 to 3; 16
// sequences of 40 tokens over 500 states 27.6, 26.4 with 1, 25.5 with 2, 22.6 with 3).
constexpr int kUnitCost = 3;
// Steps of a unit of one tile from which the second tile takes every other one (16 answers of
// one token and 20 heads over 500 states, 4 steps: 27.5 us, 29.3 without; 200 of 20 tokens over
// 400 states 95 and 102; over 1500 states 52 and 54.  From 2 steps on instead: no difference
// beyond 1.5 us either way).
constexpr int kTwinSteps = 4;
// Pairs of eight whose weights are formed on the FMA pipe: three balance it against the
// exponential unit (4 x 1500 states of 20 heads: none 43.0 us, 1 41.5, 2 40.4, 3 39.9, 4 41.5).
constexpr uint32_t kFmaExp = 0x92;
constexpr float kSlack = 8.0f;                   // log2 of what p may reach before m moves

// The part of a unit that this CTA computes.
struct Part {
  int steps;        // 128-token steps (0: no tokens or a bad page)
  int tail;         // tokens of the unit's last step
  int tok0, tok1;   // query tokens of the unit
  int head;         // KV head
  int two;          // whether the second tile has rows of its own
  int twin;         // whether it takes every other step of the first one's
  int first, last;  // whether the part holds the unit's first and last step
  int bad;
  int c0, c1;       // CTAs that share the unit
  int end;          // last part of the run
};

// A sequence as the kernel uses it: its query rows, tokens, units per KV head and steps.
struct Seq {
  int tok0, tok1, len, blocks, steps;
  bool bad;
};

struct __align__(1024) Smem {
  unsigned char q[2][kTileBytes];
  unsigned char kv[kStages][kTileBytes];
  unsigned char out[2][4][2048];  // [tile][warp]: rows on their way out
  Part part[2];
  uint64_t kv_full[kStages], kv_empty[kStages], q_full, q_empty, part_full[2], part_empty[2];
  uint64_t s_full[2], p_full[2][2], o_full[2], twin_full, twin_empty, drain;
  int dead;
  int arrived[2][2];       // [tile][a unit from an earlier CTA, one that goes on in the next]
  float2 twin_ml[kRows];   // the second tile's m and l of a twin part
  uint32_t tmem;
};
static_assert((kStages & (kStages - 1)) == 0, "places in the ring are taken modulo kStages");
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory of a CTA");

struct CrossArgs {
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int n_seq, max_pages, max_len, n_tok;
  long long n_pages;
  int H, G;
  int tile_tok;      // query tokens of a tile
  int row0;          // first pool row of the layer
  uint16_t* out;
  float c;           // scale * log2(e)
  int* tickets;
  float* parts;
  int32_t* status;
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
// The MMA warp runs its role as a whole (uniform control and addresses); `one` is set in the
// lane that issues.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}
// 32 columns of this warp's lanes, not waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// -inf into N columns (1 or 8) of this warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_fill(uint32_t taddr) {
  if (N == 1)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr), "r"(0xFF800000u) : "memory");
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};\n" ::"r"(taddr),
                 "r"(0xFF800000u)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Shared-memory matrix descriptors, 128-byte swizzle (layout type 2, version 1), 8-row
// groups 1024 bytes apart, as a low word that address steps are added to and a constant
// high word: an MMA of 64 cycles must not wait for its descriptor arithmetic (formed anew
// for each, a 128 x 128 x 128 product took 730 to 830 cycles instead of 516).
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
// K-major (Q, K): rows of 128 bytes.
__device__ __forceinline__ uint32_t desc_k(const void* p) { return smem_u32(p) >> 4 | 1u << 16; }
// N-major (V, whose tokens are the product's K): 64-element column blocks kHalfBytes apart.
__device__ __forceinline__ uint32_t desc_n(const void* p) { return smem_u32(p) >> 4 | (kHalfBytes >> 4) << 16; }
// Step of a K-major descriptor to elements 16 kk .., of an N-major one to tokens 16 kk ..
__device__ __forceinline__ constexpr uint32_t step_k(int kk) {
  return ((kk >> 2) * kHalfBytes + static_cast<uint32_t>(kk & 3) * 32) >> 4;
}
__device__ __forceinline__ constexpr uint32_t step_n(int kk) { return static_cast<uint32_t>(kk) * 2048 >> 4; }
// fp32 accumulate, bf16 or f16 operands, M = N = 128; B N-major for the value product.
template <bool F16>
__device__ __forceinline__ constexpr uint32_t idesc(bool b_n_major) {
  return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (b_n_major ? 1u << 16 : 0u) | ((128u >> 3) << 17) |
         ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(static_cast<uint32_t>(acc)), "n"(kDescHi), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %6, 0;\n"
      " mov.b64 b, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(static_cast<uint32_t>(acc)), "n"(kDescHi), "r"(one)
      : "memory");
}

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ Seq seq_of(const CrossArgs& a, int s) {
  Seq q;
  q.tok0 = a.cu_q[s];
  q.tok1 = a.cu_q[s + 1];
  q.len = a.seq_lens[s];
  q.bad = false;
  q.blocks = 0;
  if (q.tok0 < 0 || q.tok1 < q.tok0 || q.tok1 > a.n_tok) {
    q.bad = true;
  } else {
    q.blocks = (q.tok1 - q.tok0 + 2 * a.tile_tok - 1) / (2 * a.tile_tok);
    if (q.len < 0 || q.len > a.max_len) q.bad = true, q.len = 0;
  }
  q.steps = max(1, (q.len + kPage - 1) / kPage);
  return q;
}

// 2^x of a pair on the FMA pipe: x = n + f with n the nearest integer, 2^f by a polynomial
// (minimax in relative error on [-1/2, 1/2], fitted for this kernel: 2^-13.7 for bf16
// weights, 2^-18.5 for fp16), times 2^n.  x is held above -127, whose 2^n comes out as 0 (a
// score of -inf, and one past the end, weighs nothing); NaN stays NaN.
template <bool F16>
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
  float a, b;
  unpair(x, a, b);
  asm("max.NaN.f32 %0, %0, %1;\n" : "+f"(a) : "f"(-127.0f));
  asm("max.NaN.f32 %0, %0, %1;\n" : "+f"(b) : "f"(-127.0f));
  x = pair(a, b);
  const uint64_t t = add2(x, pair(12582912.0f, 12582912.0f));  // 1.5 * 2^23 + n
  const uint64_t n = add2(t, pair(-12582912.0f, -12582912.0f));
  const uint64_t f = fma2(n, pair(-1.0f, -1.0f), x);
  uint64_t p;
  if (F16) {
    p = fma2(f, pair(0.00957010221f, 0.00957010221f), pair(0.0559178591f, 0.0559178591f));
    p = fma2(f, p, pair(0.240247443f, 0.240247443f));
    p = fma2(f, p, pair(0.693121791f, 0.693121791f));
    p = fma2(f, p, pair(0.999999285f, 0.999999285f));
  } else {
    p = fma2(f, pair(0.0551716685f, 0.0551716685f), pair(0.242611125f, 0.242611125f));
    p = fma2(f, p, pair(0.693260968f, 0.693260968f));
    p = fma2(f, p, pair(0.999928057f, 0.999928057f));
  }
  unpair(t, a, b);
  a = __uint_as_float((__float_as_uint(a) << 23) + 0x3F800000u);
  b = __uint_as_float((__float_as_uint(b) << 23) + 0x3F800000u);
  return mul2(p, pair(a, b));
}

// ------------------------------------------------------------------ loads (one warp)
__device__ void load_role(const CrossArgs& a, Smem& s, const CUtensorMap* kv_map, const CUtensorMap* q_map) {
  const int lane = threadIdx.x & 31;
  volatile int* dead = &s.dead;
  // slots of all sequences and the longest one's steps
  int longest = 0;
  bool bad_seq = false;
  auto slots = [&](int i) {
    const Seq q = seq_of(a, i);
    bad_seq |= q.bad;
    if (q.blocks) longest = max(longest, q.steps);
    return static_cast<long long>(q.steps + kUnitCost) * q.blocks * a.H;
  };
  SlotScan<decltype(slots)> scan(a.n_seq, slots);
  const long long total = scan.total;
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (bad_seq && blockIdx.x == 0 && a.status) atomicOr(a.status, static_cast<int>(KVTC_STATUS_BAD_POS));
  // Runs of r steps take r steps and join up to longest / r parts at the end of a unit, a
  // part costing about a step of a small call: no run shorter than sqrt(longest) (3 queries
  // over 20000 states: 34.9 us, 38.6 with sqrt(longest / 2), 39.4 with sqrt(4 longest); 4
  // over 8000: 19.8, 21.7 with sqrt(2 longest)).
  const int shortest = max(1, static_cast<int>(sqrtf(static_cast<float>(longest))));
  const int n_cta = static_cast<int>(min(static_cast<long long>(gridDim.x), divide(total + shortest - 1, shortest)));
  long long f = 0, f1 = 0;
  if (static_cast<int>(blockIdx.x) < n_cta) {
    f = run_start(blockIdx.x, n_cta, total);
    f1 = run_start(blockIdx.x + 1, n_cta, total);
  }
  int n_part = 0, n_q = 0, it = 0;
  long long base = 0;  // first slot of the sequence's units
  int seq = f < f1 ? scan.find(f, base) : 0;
  Seq sq = seq_of(a, seq);
  uint32_t flags = 0;
  bool ok = true;
  auto load = [&](int row) {  // the 128 rows from `row` into the next stage (lane 0)
    const int st = it & (kStages - 1);
    if (it >= kStages && !wait_phase(&s.kv_empty[st], (it / kStages - 1) & 1, dead)) return false;
    mbar_arrive_expect_tx(&s.kv_full[st], kTileBytes);
    tma_load_2d(s.kv[st], kv_map, 0, row, &s.kv_full[st]);
    tma_load_2d(s.kv[st] + kHalfBytes, kv_map, 64, row, &s.kv_full[st]);
    ++it;
    return true;
  };
  while (f < f1 && ok) {
    while (f >= base + static_cast<long long>(sq.steps + kUnitCost) * a.H * sq.blocks) {
      base += static_cast<long long>(sq.steps + kUnitCost) * a.H * sq.blocks;
      sq = seq_of(a, ++seq);
    }
    const int u = static_cast<int>(divide(f - base, sq.steps + kUnitCost)), h = u / sq.blocks, blk = u - h * sq.blocks;
    const long long begin = base + static_cast<long long>(u) * (sq.steps + kUnitCost) + kUnitCost;  // its first step
    const int i0 = static_cast<int>(max(0ll, f - begin));
    const int i1 = static_cast<int>(min(static_cast<long long>(sq.steps), f1 - begin));
    f = begin + sq.steps;
    if (i1 <= i0) break;  // the run ends before the unit's first step
    const int32_t* pages = a.table + static_cast<size_t>(seq) * a.max_pages;
    bool good = true;
    int ids = 0;  // the next 32 page ids, one per lane
    if (sq.len > 0) {
      for (int p = i0 + 32 + lane; p < i1; p += 32) {
        const int id = pages[p];
        good &= id >= 0 && id < a.n_pages;
      }
      if (i0 + lane < i1) {
        ids = pages[i0 + lane];
        good &= ids >= 0 && ids < a.n_pages;
      }
    }
    good = __all_sync(0xffffffffu, good);
    if (!good) flags |= KVTC_STATUS_BAD_PAGE;
    const int steps = good && sq.len > 0 ? i1 - i0 : 0;
    const int tok0 = sq.tok0 + blk * 2 * a.tile_tok, tok1 = min(sq.tok1, tok0 + 2 * a.tile_tok);
    const int two = tok1 - tok0 > a.tile_tok;
    if (f1 - f <= kUnitCost) f = f1;  // no step of the next unit
    auto post = [&] {  // tells the other roles of the part (lane 0)
      Part d;
      d.steps = steps;
      d.tail = sq.len - (sq.steps - 1) * kPage;
      d.tok0 = tok0;
      d.tok1 = tok1;
      d.head = h;
      d.two = two;
      d.twin = !two && sq.steps >= kTwinSteps;
      d.first = i0 == 0;
      d.last = i1 == sq.steps;
      d.bad = !good;
      d.c0 = run_owner(begin, n_cta, total);
      d.c1 = run_owner(begin + sq.steps - 1, n_cta, total);
      d.end = f == f1;
      if (n_part >= 2) ok = wait_phase(&s.part_empty[n_part & 1], ((n_part >> 1) - 1) & 1, dead);
      if (ok) {
        s.part[n_part & 1] = d;
        mbar_arrive(&s.part_full[n_part & 1]);
      }
    };
    if (steps == 0 && lane == 0) post();
    for (int i = i0; i < i0 + steps; ++i) {
      if (i > i0 && ((i - i0) & 31) == 0) ids = i + lane < i1 ? pages[i + lane] : 0;
      const int id = __shfl_sync(0xffffffffu, ids, (i - i0) & 31);
      if (lane == 0 && ok) {
        const int row = a.row0 + (id * a.H + h) * 2 * kPage;
        ok = load(row);
        if (ok && i == i0) {
          if (n_q > 0) ok = wait_phase(&s.q_empty, (n_q - 1) & 1, dead);
          if (ok) {
            const uint32_t bytes = static_cast<uint32_t>(a.tile_tok * a.G) * 128u;  // of one half of one tile
            mbar_arrive_expect_tx(&s.q_full, bytes * (two ? 4u : 2u));
            for (int x = 0; x <= two; ++x) {
              tma_load_4d(s.q[x], q_map, 0, 0, h, tok0 + x * a.tile_tok, &s.q_full);
              tma_load_4d(s.q[x] + kHalfBytes, q_map, 64, 0, h, tok0 + x * a.tile_tok, &s.q_full);
            }
            ++n_q;
            post();  // behind the loads that the first scores wait for
          }
        }
        ok = ok && load(row + kPage);
      }
    }
    ++n_part;
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  }
  if (n_part == 0 && lane == 0) {  // nothing for this CTA
    Part d = {};
    d.first = d.last = d.end = 1;
    s.part[0] = d;
    mbar_arrive(&s.part_full[0]);
  }
  if (lane == 0) {
    if (!ok) {
      *dead = 1;
      flags |= KVTC_STATUS_TIMEOUT;
    }
    if (flags && a.status) atomicOr(a.status, static_cast<int>(flags));
    // every copy in flight lands before the CTA may exit (bounded)
    volatile int never = 0;
    for (int k = max(0, it - kStages); k < it; ++k) (void)wait_phase(&s.kv_full[k & (kStages - 1)], (k / kStages) & 1, &never);
    if (n_q > 0) (void)wait_phase(&s.q_full, (n_q - 1) & 1, &never);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ MMAs (one warp)
template <bool F16>
__device__ void mma_role(const CrossArgs& a, Smem& s, uint32_t tmem) {
  volatile int* dead = &s.dead;
  const uint32_t one = elect_one();
  uint32_t q_phase = 0, p_phase[2] = {0, 0};
  const uint32_t q0 = desc_k(s.q[0]), k0 = desc_k(s.kv[0]), v0 = desc_n(s.kv[0]);
  auto wait = [&](uint64_t* bar, uint32_t phase) { return wait_warp(bar, phase, dead); };
  // waits for tile i of the ring, and releases it
  auto loaded = [&](int i) { return wait(&s.kv_full[i & (kStages - 1)], (i / kStages) & 1); };
  auto release = [&](int i) { tc_commit(&s.kv_empty[i & (kStages - 1)], one); };
  auto scores = [&](int x, int rows, int i) {  // S_x of the rows of Q tile `rows`
    const uint32_t d = tmem + x * 128, q = q0 + rows * (kTileBytes >> 4);
    const uint32_t k = k0 + (i & (kStages - 1)) * (kTileBytes >> 4);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) mma_ss(d, q + step_k(kk), k + step_k(kk), idesc<F16>(false), kk > 0, one);
    tc_commit(&s.s_full[x], one);
  };
  // O_x += P_x V for the first `groups` groups of 16 tokens, each half of P as it arrives; in
  // between, while the row warps work on the second, tile `next` of the ring is waited for
  // (-1: none), which the scores that follow need.
  auto values = [&](int x, int i, bool acc, int groups, int next) -> bool {
    const uint32_t d = tmem + 256 + x * 128, p = tmem + x * 128, v = v0 + (i & (kStages - 1)) * (kTileBytes >> 4);
    if (!wait(&s.p_full[x][0], p_phase[x])) return false;
    tc_fence_after();
    if (groups == 8) {
#pragma unroll
      for (int g = 0; g < 4; ++g) mma_ts(d, p + 8 * g, v + step_n(g), idesc<F16>(true), acc || g > 0, one);
      if (next >= 0 && !loaded(next)) return false;
      if (!wait(&s.p_full[x][1], p_phase[x])) return false;
      tc_fence_after();
#pragma unroll
      for (int g = 4; g < 8; ++g) mma_ts(d, p + 8 * g, v + step_n(g), idesc<F16>(true), true, one);
    } else {
      if (!wait(&s.p_full[x][1], p_phase[x])) return false;
      tc_fence_after();
      for (int g = 0; g < groups; ++g) mma_ts(d, p + 8 * g, v + step_n(g), idesc<F16>(true), acc || g > 0, one);
    }
    p_phase[x] ^= 1;
    return true;
  };
  int it = 0;  // the part's first K tile in the ring; V of step j is it + 2 j + 1
  bool ok = true;
  for (int n = 0;; ++n) {
    if (!(ok = wait(&s.part_full[n & 1], (n >> 1) & 1))) break;
    const Part& d = s.part[n & 1];
    const int steps = d.steps, two = d.two, twin = d.twin, end = d.end;
    // tokens past the end add nothing: only the last step's groups of 16 that hold a token
    const int last_groups = d.last ? (d.tail + 15) >> 4 : 8;
    __syncwarp();
    if (one) mbar_arrive(&s.part_empty[n & 1]);
    if (steps > 0) {
      if (!(ok = wait(&s.q_full, q_phase))) break;
      q_phase ^= 1;
      if (!(ok = loaded(it))) break;
      tc_fence_after();
      scores(0, 0, it);
      if (two) scores(1, 1, it);
      release(it);
      if (twin && steps > 1) {
        if (!(ok = loaded(it + 2))) break;
        tc_fence_after();
        scores(1, 0, it + 2);
        release(it + 2);
      }
      if (steps <= 1 + twin) tc_commit(&s.q_empty, one);
    }
    if (!twin) {
      for (int j = 0; j < steps; ++j) {
        const int v = it + 2 * j + 1, k = v + 1;
        const bool more = j + 1 < steps;
        const int groups = more ? 8 : last_groups;
        if (!(ok = loaded(v) && values(0, v, j > 0, groups, more ? k : -1))) break;
        if (more)
          scores(0, 0, k);
        else
          tc_commit(&s.o_full[0], one);
        if (two) {
          if (!(ok = values(1, v, j > 0, groups, -1))) break;
          if (more)
            scores(1, 1, k);
          else
            tc_commit(&s.o_full[1], one);
        }
        release(v);
        if (more) release(k);
        if (j + 2 == steps) tc_commit(&s.q_empty, one);
      }
    } else {
      for (int j = 0; j < steps; ++j) {
        const int x = j & 1, v = it + 2 * j + 1, k = v + 3;
        // (the next K tile of a twin part is often still on its way: not waited for early)
        if (!(ok = loaded(v) && values(x, v, j > 1, j + 1 < steps ? 8 : last_groups, -1))) break;
        release(v);
        if (j + 2 < steps) {
          if (!(ok = loaded(k))) break;
          tc_fence_after();
          scores(x, 0, k);
          release(k);
          if (j + 3 == steps) tc_commit(&s.q_empty, one);
        } else {
          tc_commit(&s.o_full[x], one);
        }
      }
    }
    it += 2 * steps;
    if (!ok || end) break;
  }
  if (!ok && one) {
    *dead = 1;
    if (a.status) atomicOr(a.status, static_cast<int>(KVTC_STATUS_TIMEOUT));
  }
  // the MMAs issued complete before TMEM is freed (bounded)
  volatile int never = 0;
  tc_commit(&s.drain, one);
  (void)wait_phase(&s.drain, 0, &never);
  __syncwarp();
}

// ------------------------------------------------------------------ rows (four warps a tile)
// Partial slot of CTA c and tile x.  Slot 1 holds the unit that begins in the CTA, slot 0
// the one that came from an earlier CTA.
__device__ __forceinline__ float* part_of(const CrossArgs& a, int c, int slot, int x) {
  return a.parts + static_cast<size_t>((c * 2 + slot) * 2 + x) * kPartFloats;
}

// Offset of the output row of a token and a query head of a KV head.
__device__ __forceinline__ long long out_row(const CrossArgs& a, int tok, int head, int in_group) {
  return (static_cast<long long>(tok) * a.H * a.G + static_cast<long long>(head) * a.G + in_group) * kD;
}

// Writes columns 32 q .. of 32 rows, each lane giving its own (at: its offset, -1 for none),
// by way of shared memory: a row's 16 bytes per lane would take 32 lines for every store.
template <bool F16>
__device__ __forceinline__ void put_rows(unsigned char* buf, uint16_t* out, int q, const float* o, float r, long long at) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint4 w;
    w.x = pack2<F16>(o[8 * e] * r, o[8 * e + 1] * r);
    w.y = pack2<F16>(o[8 * e + 2] * r, o[8 * e + 3] * r);
    w.z = pack2<F16>(o[8 * e + 4] * r, o[8 * e + 5] * r);
    w.w = pack2<F16>(o[8 * e + 6] * r, o[8 * e + 7] * r);
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) = w;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int from = 8 * i + (lane >> 2), e = lane & 3;
    const long long dst = __shfl_sync(0xffffffffu, at, from);
    const uint4 w = *reinterpret_cast<const uint4*>(buf + from * 64 + ((e ^ ((from >> 1) & 3)) << 4));
    if (dst >= 0) *reinterpret_cast<uint4*>(out + dst + 32 * q + 8 * e) = w;
  }
}

// Takes a part (m, l, sums) in with what has been joined of its row; the reference moves on
// from part to part, so that a part's reads are all under way at once.
template <int N>
__device__ __forceinline__ void join_part(float m, float l, const float4 (&v)[N], float c, float& top, float& sum,
                                          bool& bad, float (&o)[4 * N]) {
  const float to = fmaxf(top, m);
  const float f0 = top == -INFINITY ? 0.0f : ex2((top - to) * c), f1 = m == -INFINITY ? 0.0f : ex2((m - to) * c);
  bad |= l < 0.0f;
  sum = sum * f0 + l * f1;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    o[4 * e] = o[4 * e] * f0 + v[e].x * f1;
    o[4 * e + 1] = o[4 * e + 1] * f0 + v[e].y * f1;
    o[4 * e + 2] = o[4 * e + 2] * f0 + v[e].z * f1;
    o[4 * e + 3] = o[4 * e + 3] * f0 + v[e].w * f1;
  }
  top = to;
}

// Joins the parts of a tile of up to 32 rows: its four warps take 32 columns each of the same
// rows (a row per thread left three of them idle: the first tokens of three answers over
// 1500 states 21.4 us, 19.6 so), the CTA's own part with the others.
template <bool F16>
__device__ __forceinline__ void join_few(const CrossArgs& a, Smem& s, int tok0, int head, int rows, int c0, int shares) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = warp >> 2, q = warp & 3, tk = lane / a.G;
  const bool live = lane < rows;
  const float* first = part_of(a, c0, 1, x);
  const float* second = part_of(a, c0 + 1, 0, x);
  constexpr size_t kNext = 4 * kPartFloats;  // from a CTA's slot to the next CTA's
  float top = -INFINITY, sum = 0.0f, o[32];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = 0.0f;
#pragma unroll 2
  for (int j = 0; j < shares; ++j) {
    const float* p = j == 0 ? first : second + (j - 1) * kNext;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p) + lane);
    float4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __ldcg(reinterpret_cast<const float4*>(p + 2 * kRows) + (8 * q + e) * kRows + lane);
    if (live) join_part(ml.x, ml.y, v, a.c, top, sum, bad, o);
  }
  if (bad) {
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0.0f;
  }
  put_rows<F16>(s.out[x][q], a.out, q, o, bad ? 0.0f : 1.0f / sum,
                live ? out_row(a, tok0 + tk, head, lane - tk * a.G) : -1);
}

template <bool F16>
__device__ void row_role(const CrossArgs& a, Smem& s, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = warp >> 2, row = threadIdx.x & 127;
  // fp16 weights: 2^7 at the reference, so those far below it keep clear of the subnormals
  // and 2^(7 + kSlack) stays in range
  constexpr float kBias = F16 ? 7.0f : 0.0f;
  volatile int* dead = &s.dead;
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const uint32_t ts = tmem + lanes + x * 128, to = tmem + lanes + 256 + x * 128;
  const int tok_in = row / a.G, head_in = row - tok_in * a.G;
  const uint64_t c2 = pair(a.c, a.c);
  uint32_t twin_phase = 0;
  int it = 0, n_s = 0, n_o = 0;
  auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {
    const bool ok = wait_warp(bar, phase, dead);
    if (!ok) {
      if (lane == 0) {
        *dead = 1;
        if (a.status) atomicOr(a.status, static_cast<int>(KVTC_STATUS_TIMEOUT));
      }
      __syncwarp();
      leave_barrier(1 + x, kRows);
    }
    return ok;
  };
  auto tile_sync = [&]() -> bool { return consumers_sync(1 + x, kRows, dead); };  // the tile's four warps
  for (int n = 0;; ++n) {
    if (!wait(&s.part_full[n & 1], (n >> 1) & 1)) return;
    const Part d = s.part[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.part_empty[n & 1]);
    if (x == 0 || d.two || d.twin) {
      float m = -INFINITY, l = 0.0f;
      const int stride = 1 + d.twin, t0 = d.twin ? x : 0;
      const bool some = t0 < d.steps;  // the tile has steps
      for (int t = t0; t < d.steps; t += stride) {
        const int valid = d.last && t == d.steps - 1 ? d.tail : kPage;
        if (!wait(&s.s_full[x], n_s++ & 1)) return;
        tc_fence_after();
        if (valid < kPage) {
          // scores past the end, in TMEM: the code of a full step then serves the last one
          int i = valid;
          for (; i & 7; ++i) tmem_fill<1>(ts + i);
          for (; i < kPage; i += 8) tmem_fill<8>(ts + i);
          tmem_wait_st();
        }
        float top;
        {
          float sc[128];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, sc + 32 * i);
          tmem_wait_ld();
          float m0 = sc[0], m1 = sc[1], m2 = sc[2], m3 = sc[3];
#pragma unroll
          for (int i = 4; i < 124; i += 8) {
            m0 = max3(m0, sc[i], sc[i + 1]);
            m1 = max3(m1, sc[i + 2], sc[i + 3]);
            m2 = max3(m2, sc[i + 4], sc[i + 5]);
            m3 = max3(m3, sc[i + 6], sc[i + 7]);
          }
          m0 = max3(m0, sc[124], sc[125]);
          m1 = max3(m1, sc[126], sc[127]);
          top = fmaxf(max3(m0, m1, m2), m3);
        }
        if (valid < kPage && (x == 0 || d.twin) && (valid & 15)) {
          // V rows past the end may hold anything (0 * NaN is NaN): clear those that the
          // last group of 16 tokens takes in
          const int v = it + 2 * t + 1, st = v & (kStages - 1);
          if (!wait(&s.kv_full[st], (v / kStages) & 1)) return;
          for (int e = row; e < (16 - (valid & 15)) * 16; e += 128) {
            const int r = valid + (e >> 4);
            *reinterpret_cast<uint4*>(s.kv[st] + ((e >> 3) & 1) * kHalfBytes + r * 128 + (e & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        // Each row decides for itself (the others are scaled by 1): rows of the warp that belong
        // to another sequence, or to none (heads that do not fill 128 rows, whose queries no load
        // writes), must not change the bits of these.
        const bool moves = (top - m) * a.c > kSlack;
        if (__any_sync(0xffffffffu, moves)) {
          const float to_m = moves ? top : m;
          const float f = m == -INFINITY ? 0.0f : ex2((m - to_m) * a.c);
          l *= f;
          m = to_m;
          if (t > t0) {
            // these scores were issued after the tile's last value product, so the
            // accumulators are complete
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              float o[32];
              uint32_t w[32];
              tmem_ld32(to + 32 * i, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * f);
              tmem_st32(to + 32 * i, w);
            }
          }
        }
        // (a row without a score above -inf yet: their weights are 2^-inf, not 2^(inf - inf))
        const float neg = m == -INFINITY ? 0.0f : kBias - m * a.c;
        const uint64_t neg2 = pair(neg, neg);
        uint64_t sum0 = pair(0.0f, 0.0f), sum1 = sum0;
        // The scores are read from TMEM once more, 64 columns at a time in one piece of code:
        // with 128 in registers the unrolled loop outgrew the instruction caches (half as
        // many stalls for instructions as instructions issued), the MMA warp's with it.  P
        // takes the columns of scores that have been read.
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          float sc[64];
          uint32_t w[32];
          tmem_ld32(ts + 64 * hf, sc);
          tmem_ld32(ts + 64 * hf + 32, sc + 32);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int e = 2 * i;
            uint64_t p = fma2(pair(sc[e], sc[e + 1]), c2, neg2);
            float lo, hi;
            if (kFmaExp >> (i & 7) & 1) {
              p = exp2_pair<F16>(p);
              unpair(p, lo, hi);
            } else {
              unpair(p, lo, hi);
              lo = ex2(lo);
              hi = ex2(hi);
              p = pair(lo, hi);
            }
            if (i & 1)
              sum1 = add2(sum1, p);
            else
              sum0 = add2(sum0, p);
            // P enters the value product in the pages' type (half a step of relative error
            // on each weight, as for the output; the sum l stays fp32)
            w[i] = pack2<F16>(lo, hi);
          }
          tmem_st32(ts + 32 * hf, w);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.p_full[x][hf]);
        }
        float a0, a1;
        unpair(add2(sum0, sum1), a0, a1);
        l += a0 + a1;
      }
      // ---- the tile's steps are done
      const bool whole = d.first && d.last;
      const int shares = d.c1 - d.c0 + 1;
      int* ticket = a.tickets + 2 * d.c0 + x;
      if (!whole && row == 0) s.arrived[x][d.first] = ld_acquire_gpu(ticket);
      if (some) {
        if (!wait(&s.o_full[x], n_o++ & 1)) return;
        tc_fence_after();
      }
      // a twin part: the first tile's warps take the second's sums (the same rows, so the
      // same TMEM lanes) in with their own
      float fa = 1.0f, fb = 0.0f;
      if (d.twin && x == 1) {
        s.twin_ml[row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.twin_full);
        if (!wait(&s.twin_empty, twin_phase)) return;
        twin_phase ^= 1;
        tc_fence_after();
        it += 2 * d.steps;
        if (d.end) return;
        continue;
      }
      const bool both = d.twin && d.steps > 1;
      if (d.twin) {
        if (!wait(&s.twin_full, twin_phase)) return;
        twin_phase ^= 1;
        tc_fence_after();
        if (both) {
          const float2 ml = s.twin_ml[row];
          const float to_m = fmaxf(m, ml.x);
          fa = m == -INFINITY ? 0.0f : ex2((m - to_m) * a.c);
          fb = ml.x == -INFINITY ? 0.0f : ex2((ml.x - to_m) * a.c);
          m = to_m;
          l = l * fa + ml.y * fb;
        }
      }
      const int tok = d.tok0 + x * a.tile_tok + tok_in;
      const bool live = tok_in < a.tile_tok && tok < d.tok1;
      const long long at = live ? out_row(a, tok, d.head, head_in) : -1;
      auto put = [&](int q, const float* o, float r) { put_rows<F16>(s.out[x][warp & 3], a.out, q, o, r, at); };
      auto sums = [&](int q, float* o) {  // columns 32 q .. of O
        __syncwarp();
        if (some) {
          tmem_ld32(to + 32 * q, o);
          tmem_wait_ld();
          if (both) {
            float v[32];
            tmem_ld32(to + kRows + 32 * q, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * fa + v[e] * fb;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
        }
      };
      if (whole) {
        // (a row whose every score is -inf has no softmax: 0 / 0, here as in the joins)
        const float r = some ? 1.0f / l : 0.0f;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float o[32];
          sums(q, o);
          put(q, o, r);
        }
      } else {
        // ---- the unit is shared: the last tile to arrive joins the others' sums with its own
        if (d.bad) l = -1.0f;  // a sum below 0 marks a bad page
        if (!tile_sync()) return;
        const int rows = min(a.tile_tok, d.tok1 - d.tok0 - x * a.tile_tok) * a.G;
        const bool few = rows <= 32;
        bool join = !few && s.arrived[x][d.first] == shares - 1;
        if (!join) {
          float* mine = part_of(a, blockIdx.x, d.first, x);
          if (live) reinterpret_cast<float2*>(mine)[row] = make_float2(m, l);
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float o[32];
            sums(q, o);
            if (live)
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                reinterpret_cast<float4*>(mine + 2 * kRows)[(8 * q + e / 4) * kRows + row] =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __threadfence();
          if (!tile_sync()) return;
          if (row == 0) s.arrived[x][d.first] = atomicAdd(ticket, 1);
          if (!tile_sync()) return;
          join = s.arrived[x][d.first] == shares - 1;
        }
        if (join && few) {
          __threadfence();
          if (row == 0) *ticket = 0;
          join_few<F16>(a, s, d.tok0 + x * a.tile_tok, d.head, rows, d.c0, shares);
        } else if (join) {
          __threadfence();
          if (row == 0) *ticket = 0;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            float top = -INFINITY, sum = 0.0f, o[64];
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e] = 0.0f;
#pragma unroll 1
            for (int c = d.c0; c <= d.c1; ++c) {  // in order, whoever joins
              float4 v[16];
              float2 ml = make_float2(m, l);
              if (c == static_cast<int>(blockIdx.x)) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  float w[32];
                  sums(2 * half + q, w);
#pragma unroll
                  for (int e = 0; e < 8; ++e) v[8 * q + e] = make_float4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                }
              } else if (live) {
                const float* p = part_of(a, c, c == d.c0, x);
                ml = __ldcg(reinterpret_cast<const float2*>(p) + row);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  v[e] = __ldcg(reinterpret_cast<const float4*>(p + 2 * kRows) + (16 * half + e) * kRows + row);
              }
              if (live) join_part(ml.x, ml.y, v, a.c, top, sum, bad, o);
            }
            if (bad) {
#pragma unroll
              for (int e = 0; e < 64; ++e) o[e] = 0.0f;
            }
            put(2 * half, o, bad ? 0.0f : 1.0f / sum);
            put(2 * half + 1, o + 32, bad ? 0.0f : 1.0f / sum);
          }
        }
      }
      if (d.twin) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.twin_empty);
      }
    }
    it += 2 * d.steps;
    if (d.end) return;
  }
}

template <bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    raw_cross_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CrossArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&s.tmem)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (tid == 32 * kLoadWarp) {
    prefetch_map(&kv_map);
    prefetch_map(&q_map);
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.kv_full[i], 1);
      mbar_init(&s.kv_empty[i], 1);
    }
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.drain, 1);
    mbar_init(&s.twin_full, 4);
    mbar_init(&s.twin_empty, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.part_full[i], 1);
      mbar_init(&s.part_empty[i], 9);  // the eight row warps and the MMA thread
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i][0], 4);
      mbar_init(&s.p_full[i][1], 4);
      mbar_init(&s.o_full[i], 1);
    }
    s.dead = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  griddep_wait();
  griddep_launch_dependents();
  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) load_role(a, s, &kv_map, &q_map);
    if (warp == kMmaWarp) mma_role<F16>(a, s, tmem);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRowRegs));
    row_role<F16>(a, s, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

// CTAs that a call can use: no more than it has steps.
int grid_bound(int n_seq, int n_tok, int n_kv_heads, int group, int max_seq_len) {
  const long long tile_tok = std::max(1, kRows / group);
  const long long blocks = n_tok / (2 * tile_tok) + n_seq;
  const long long steps = std::max(1, (max_seq_len + kPage - 1) / kPage);
  if (blocks >= kMaxCtas || steps >= kMaxCtas || n_kv_heads >= kMaxCtas) return kMaxCtas;
  return static_cast<int>(std::min<long long>(kMaxCtas, blocks * steps * n_kv_heads));
}

template <bool F16>
kvtc_status launch_cross(const CUtensorMap& kv_map, const CUtensorMap& q_map, const CrossArgs& a, int grid,
                         void* stream) {
  const size_t smem = sizeof(Smem) + 1024;
  const kvtc_status st = allow_smem<raw_cross_kernel<F16>>(smem);
  if (st != KVTC_OK) return st;
  const cudaError_t e = launch(raw_cross_kernel<F16>, dim3(static_cast<unsigned>(grid)), kThreads, smem, stream, kv_map, q_map, a);
  if (e != cudaSuccess) return cuda_fail(e, "raw cross launch");
  return KVTC_OK;
}

}  // namespace
}  // namespace raw
}  // namespace kvtc

using namespace kvtc;

// Counters of the CTAs (4096 bytes), then two slots of two tiles for each.
extern "C" uint64_t kvtc_raw_cross_workspace_bytes(int n_seq, int n_tok, int n_q_heads, int n_kv_heads,
                                                   int max_seq_len) {
  if (n_seq < 1 || n_tok < 0 || n_kv_heads < 1 || n_q_heads < n_kv_heads || max_seq_len < 0) return 0;
  const int ctas = raw::grid_bound(n_seq, n_tok, n_kv_heads, std::min(raw::kRows, n_q_heads / n_kv_heads), max_seq_len);
  return 4096 + static_cast<uint64_t>(ctas) * 4 * raw::kPartFloats * sizeof(float);
}

extern "C" kvtc_status kvtc_raw_cross_attention(const kvtc_raw_cache* cache, int layer, const void* q, int n_q_heads,
                                                const int32_t* cu_q, int n_tok, const int32_t* seq_lens,
                                                int max_seq_len, float softmax_scale, void* out, void* workspace,
                                                uint64_t workspace_bytes, void* stream) {
  kvtc_status st = raw::check_attention(cache, layer, n_q_heads, raw::kRows, max_seq_len, softmax_scale);
  if (st != KVTC_OK) return st;
  if (n_tok < 0) return fail(KVTC_EINVAL, "n_tok must be >= 0");
  if (n_tok == 0) return KVTC_OK;
  if (!q || !cu_q || !seq_lens || !out || !workspace) return fail(KVTC_EINVAL, "null device pointer");
  if (!raw::aligned16(q) || !raw::aligned16(out) || !raw::aligned16(workspace))
    return fail(KVTC_EINVAL, "q, out and workspace must be 16-byte aligned");
  if (workspace_bytes < kvtc_raw_cross_workspace_bytes(cache->n_seq, n_tok, n_q_heads, cache->n_kv_heads, max_seq_len))
    return fail(KVTC_ECAPACITY, "cross attention workspace too small");
  st = raw::check_overlap(cache, q, out, static_cast<uint64_t>(n_tok) * n_q_heads * kD * 2, workspace,
                          kvtc_raw_cross_workspace_bytes(cache->n_seq, n_tok, n_q_heads, cache->n_kv_heads, max_seq_len),
                          seq_lens, cu_q);
  if (st != KVTC_OK) return st;
  int sms = 0;
  st = raw::sm_count(&sms);
  if (st != KVTC_OK) return st;
  raw::CrossArgs a;
  a.table = cache->block_table;
  a.seq_lens = seq_lens;
  a.cu_q = cu_q;
  a.n_seq = cache->n_seq;
  a.max_pages = cache->max_pages;
  a.max_len = max_seq_len;
  a.n_tok = n_tok;
  a.n_pages = static_cast<long long>(cache->n_pages);
  a.H = cache->n_kv_heads;
  a.G = n_q_heads / cache->n_kv_heads;
  a.tile_tok = raw::kRows / a.G;
  a.row0 = static_cast<int>(static_cast<uint64_t>(layer) * cache->n_pages * static_cast<uint64_t>(a.H) * 2 * kPage);
  a.out = static_cast<uint16_t*>(out);
  a.c = raw::exp2_scale(softmax_scale);
  a.tickets = static_cast<int*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + 4096);
  a.status = cache->status;
  CUtensorMap kv_map, q_map;
  st = raw::pool_map(&kv_map, cache, kPage);
  if (st == KVTC_OK) st = raw::query_map(&q_map, q, cache->dtype, n_tok, a.H, a.G, a.G, a.tile_tok);
  if (st != KVTC_OK) return st;
  const int grid = std::min(sms, raw::grid_bound(a.n_seq, n_tok, a.H, a.G, max_seq_len));
  return cache->dtype == KVTC_F16 ? raw::launch_cross<true>(kv_map, q_map, a, grid, stream)
                                  : raw::launch_cross<false>(kv_map, q_map, a, grid, stream);
}
