// kvtc_step_tables: block table growth, page release and the row layout of a serving step.
//
// With c cached and n new tokens per sequence: tokens' rows are the prefix sum of n, the
// pages a sequence lacks are ceil((c + n) / 128) - ceil(c / 128), and its share of the
// free ring is the prefix sum of those needs over the sequences that fit.  Whether a
// sequence fits in the rows depends on the first sum alone, so two block scans decide a
// chunk of sequences: (rows, released pages), then (needed pages).
//
// Bound: latency for a decode step (a launch, two dependent loads, two scans), the 12
// bytes per row for large steps.  One launch without a wait between CTAs: every CTA scans
// all sequences for itself (8 bytes each, from L2) and fills its own range of rows; the rows
// find their sequences by a running maximum over the marks of the first rows, and take
// their page ids straight from the ring or the old table entries, so nothing that another
// CTA writes is read.  Where outputs replace their inputs (lengths, ring state) the last
// CTA to finish reading writes them (one counter); otherwise the first CTA does, at once.
// Up to 128 sequences a CTA has 128 threads (a step's barriers and launch cost less), for
// more 1024 with two sequences each.  Measured: 4.3 us for a step of 16 sequences (6.2 with
// 1024 threads and 64-bit scans), 7.6 us for 2048 sequences with 600000 rows (20 with two
// barriers per scan, a bisection per row and one sequence per thread).
#include <cuda_runtime.h>

#include <algorithm>

#include "ptx.cuh"
#include "raw_cache.cuh"

namespace kvtc {
namespace {

constexpr int kSmallThreads = 128, kLargeThreads = 1024, kLargePer = 2;
constexpr int kRowsPerThread = 4;

struct TablesArgs {
  const int32_t* cached;
  const int32_t* fresh;
  int n_seq;
  int32_t* ring;
  int capacity;
  const int32_t* state;
  int32_t* table;
  int max_pages;
  int32_t* seq_lens;
  int32_t* cu;
  int64_t* slots;
  int32_t* positions;
  int n_rows;
  int32_t* state_out;
  int in_place;     // seq_lens or state_out replace their inputs
  int* ticket;
  int32_t* status;
};

template <typename T, int kThreads, int kPer>
struct Smem {
  static constexpr int kWarps = kThreads / 32, kChunk = kThreads * kPer;
  T rows_sum[kWarps], released_sum[kWarps];
  int need_sum[kWarps];
  int taken;                  // pages taken from the ring's head
  int last;
  int first_row[kChunk + 1];  // rows of the chunk's sequences, clipped to n_rows
  int cached[kChunk];
  int need[kChunk];           // new pages (-1: the sequence keeps its length; -2: finished)
  int offset[kChunk];         // of its first new page from the ring's head, or of the first
                              // released one from its tail
  alignas(8) uint16_t owner[kThreads * kRowsPerThread];  // sequence (of the chunk) of each row
  int owner_max[kWarps];
};

// Exclusive sum over the block's warps of one value per thread (incl: the warp's inclusive
// sums), and the block's total; one barrier, which the caller places between put and get.
template <typename T>
__device__ __forceinline__ T warp_scan(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T p = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += p;
  }
  return v;
}
template <int kWarps, typename T>
__device__ __forceinline__ T block_prefix(const T* sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T v = warp_scan(lane < kWarps ? sums[lane] : T(0));
  total = __shfl_sync(0xffffffffu, v, kWarps - 1);
  const T p = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
  return warp ? p : T(0);
}

// Running totals before a chunk.
struct Carry {
  long long rows = 0, need = 0, released = 0;
};

// Decides the chunk of sequences from base on (kPer consecutive ones per thread) into
// shared memory; ends with a barrier.  T: the type of a chunk's sums of rows and of released
// pages; int where they fit (a length beyond n_rows then counts as n_rows + 1, which leaves
// no row to it or to a later sequence either), as 64-bit scans take twice the shuffles.
template <typename T, int kThreads, int kPer>
__device__ uint32_t decide(const TablesArgs& a, Smem<T, kThreads, kPer>& s, int base, int count, Carry& run,
                           int (&new_len)[kPer]) {
  constexpr int kWarps = kThreads / 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const long long limit = static_cast<long long>(a.max_pages) * kPage;
  int c[kPer], n[kPer], held[kPer];
  bool bad[kPer];
  uint32_t flags = 0;
  const int most_rows = sizeof(T) == 4 ? a.n_rows + 1 : INT32_MAX;
  T row_sum = 0, rel_sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int q = base + t * kPer + k;
    c[k] = q < a.n_seq ? a.cached[q] : 0;
    n[k] = q < a.n_seq ? a.fresh[q] : 0;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    bad[k] = c[k] < 0 || c[k] > limit;
    if (bad[k]) flags |= KVTC_STATUS_BAD_POS, c[k] = 0;
    held[k] = (c[k] + kPage - 1) / kPage;
    row_sum += min(max(n[k], 0), most_rows);
    rel_sum += n[k] < 0 ? held[k] : 0;
  }
  const T row_incl = warp_scan(row_sum), rel_incl = warp_scan(rel_sum);
  if (lane == 31) s.rows_sum[warp] = row_incl, s.released_sum[warp] = rel_incl;
  __syncthreads();
  T rows_total, rel_total;
  long long row = run.rows + (block_prefix<kWarps>(s.rows_sum, rows_total) + row_incl - row_sum);
  long long rel = run.released + (block_prefix<kWarps>(s.released_sum, rel_total) + rel_incl - rel_sum);
  run.rows += rows_total;
  run.released += rel_total;
  bool fits[kPer];
  int need[kPer], first_row[kPer], release0[kPer], all = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int q = base + t * kPer + k, fresh = max(n[k], 0);
    fits[k] = q < a.n_seq && n[k] >= 0 && !bad[k] && static_cast<long long>(c[k]) + fresh <= limit && row + fresh <= a.n_rows;
    if (n[k] > 0 && !fits[k]) flags |= KVTC_STATUS_BAD_POS;
    // below 2^24 pages each, and their rows (so their sum) fit n_rows
    need[k] = fits[k] ? static_cast<int>((static_cast<long long>(c[k]) + fresh + kPage - 1) / kPage) - held[k] : 0;
    all += need[k];
    first_row[k] = static_cast<int>(min(row, static_cast<long long>(a.n_rows)));
    release0[k] = static_cast<int>(min(rel, static_cast<long long>(a.capacity)));
    row += min(fresh, most_rows);
    rel += n[k] < 0 ? held[k] : 0;
  }
  const int need_incl = warp_scan(all);
  if (lane == 31) s.need_sum[warp] = need_incl;
  __syncthreads();
  int need_total;
  long long first = run.need + block_prefix<kWarps>(s.need_sum, need_total) + need_incl - all;
  run.need += need_total;
  long long taken = 0;  // the sequences that take pages are a prefix of those that need some
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int q = base + t * kPer + k, i = t * kPer + k;
    const bool grows = fits[k] && (need[k] == 0 || first + need[k] <= count);
    if (fits[k] && !grows) flags |= KVTC_STATUS_NO_PAGE;
    if (grows && need[k] > 0) taken = first + need[k];
    const bool finished = q < a.n_seq && n[k] < 0;
    s.first_row[i] = first_row[k];
    s.cached[i] = c[k];
    s.need[i] = finished ? -2 : grows ? need[k] : -1;
    s.offset[i] = finished ? release0[k] : grows ? static_cast<int>(min(first, static_cast<long long>(count))) : 0;
    new_len[k] = finished ? 0 : grows ? c[k] + n[k] : c[k];
    first += need[k];
  }
  const int most = __reduce_max_sync(0xffffffffu, static_cast<int>(taken));  // at most count
  if (lane == 0 && most > 0) atomicMax(&s.taken, most);
  if (t == kThreads - 1) s.first_row[kThreads * kPer] = static_cast<int>(min(run.rows, static_cast<long long>(a.n_rows)));
  __syncthreads();
  return flags;
}

// The sequence of each of the CTA's rows lo .. hi - 1, into shared memory: a sequence marks
// its first row there, and a running maximum over the rows carries it on (a bisection per row
// took a third of a large step's time).  Ends with a barrier.
template <typename T, int kThreads, int kPer>
__device__ __forceinline__ void find_owners(Smem<T, kThreads, kPer>& s, int n_in, int lo, int hi) {
  static_assert(kRowsPerThread == 4, "a thread's rows are one 8-byte word");
  constexpr int kWarps = kThreads / 32;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint2* words = reinterpret_cast<uint2*>(s.owner);
  words[t] = make_uint2(0u, 0u);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = t * kPer + k;
    if (i < n_in) {
      const int first = s.first_row[i], end = s.first_row[i + 1];
      if (first < end && end > lo && first < hi) s.owner[max(first, lo) - lo] = static_cast<uint16_t>(i);
    }
  }
  __syncthreads();
  const uint2 w = words[t];
  int m[4] = {static_cast<int>(w.x & 0xFFFFu), static_cast<int>(w.x >> 16), static_cast<int>(w.y & 0xFFFFu),
              static_cast<int>(w.y >> 16)};
#pragma unroll
  for (int i = 1; i < 4; ++i) m[i] = max(m[i], m[i - 1]);
  auto max_scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, p);
    }
    return v;
  };
  const int incl = max_scan(m[3]);
  if (lane == 31) s.owner_max[warp] = incl;
  __syncthreads();
  const int all = max_scan(lane < kWarps ? s.owner_max[lane] : 0);
  const int warps = __shfl_sync(0xffffffffu, all, (warp + 31) & 31), lanes = __shfl_up_sync(0xffffffffu, incl, 1);
  const int before = max(warp ? warps : 0, lane ? lanes : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max(m[i], before);
  words[t] = make_uint2(static_cast<uint32_t>(m[0] | m[1] << 16), static_cast<uint32_t>(m[2] | m[3] << 16));
  __syncthreads();
}

template <typename T, int kThreads, int kPer>
__global__ void __launch_bounds__(kThreads) step_tables_kernel(const __grid_constant__ TablesArgs a) {
  constexpr int kWarps = kThreads / 32, kChunk = kThreads * kPer, kRowsPerCta = kThreads * kRowsPerThread;
  __shared__ Smem<T, kThreads, kPer> s;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) s.taken = 0;  // (the scans' barriers come before its first use)
  griddep_wait();
  griddep_launch_dependents();
  int head = a.state[0], count = a.state[1];
  uint32_t flags = 0;
  if (head < 0 || head >= a.capacity || count < 0 || count > a.capacity) {
    head = count = 0;
    flags |= KVTC_STATUS_BAD_PAGE;
  }
  const int room = a.capacity - count;  // places a release can fill
  const int n_chunks = (a.n_seq + kChunk - 1) / kChunk;
  const int row_lo = static_cast<int>(min(static_cast<long long>(blockIdx.x) * kRowsPerCta, static_cast<long long>(a.n_rows)));
  const int row_hi = static_cast<int>(min(static_cast<long long>(row_lo) + kRowsPerCta, static_cast<long long>(a.n_rows)));
  const bool writes = !a.in_place && blockIdx.x == 0;
  Carry run;
  int new_len[kPer];
  auto write_lens = [&](int base) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = t * kPer + k;
      if (base + i < a.n_seq) {
        a.seq_lens[base + i] = new_len[k];
        a.cu[base + i] = s.first_row[i];
      }
    }
  };
  for (int ch = 0; ch < n_chunks; ++ch) {
    const int base = ch * kChunk;
    flags |= decide(a, s, base, count, run, new_len);
    if (writes) write_lens(base);
    const int n_in = min(kChunk, a.n_seq - base);
    // this CTA's rows that fall into the chunk: all of a thread's at once
    const int lo = max(row_lo, s.first_row[0]), hi = min(row_hi, s.first_row[kChunk]);
    int l[kRowsPerThread];  // their sequences
    if (lo < hi) find_owners(s, n_in, lo, hi);
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) l[i] = lo < hi ? s.owner[t + i * kThreads] : 0;
    int32_t id[kRowsPerThread];
    int pos[kRowsPerThread];
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int off = t + i * kThreads, r = lo + off;
      id[i] = -1;
      pos[i] = 0;
      if (off < hi - lo && s.need[l[i]] >= 0) {
        const int c = s.cached[l[i]], held = (c + kPage - 1) / kPage;
        pos[i] = c + (r - s.first_row[l[i]]);
        const int p = pos[i] / kPage;
        const long long at = static_cast<long long>(head) + s.offset[l[i]] + (p - held);
        id[i] = p < held ? a.table[static_cast<size_t>(base + l[i]) * a.max_pages + p]
                         : a.ring[at < a.capacity ? at : at - a.capacity];
        if (id[i] < 0) flags |= KVTC_STATUS_BAD_PAGE;
      }
    }
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
      const int off = t + i * kThreads, r = lo + off;
      if (off < hi - lo) {
        a.slots[r] = id[i] < 0 ? -1 : static_cast<int64_t>(id[i]) * kPage + pos[i] % kPage;
        a.positions[r] = id[i] < 0 ? 0 : pos[i];
      }
    }
    // new table entries and released pages: a warp per sequence, dealt over the CTAs
    for (int i = static_cast<int>(blockIdx.x) * kWarps + warp; i < n_in; i += kWarps * static_cast<int>(gridDim.x)) {
      const int c = s.cached[i], need = s.need[i], held = (c + kPage - 1) / kPage;
      int32_t* row = a.table + static_cast<size_t>(base + i) * a.max_pages;
      if (need > 0) {
        for (int p = lane; p < need; p += 32) {
          const long long at = static_cast<long long>(head) + s.offset[i] + p;
          row[held + p] = a.ring[at < a.capacity ? at : at - a.capacity];
        }
      } else if (need == -2) {
        for (int p = lane; p < held; p += 32) {
          const int32_t id = row[p];
          const long long off = static_cast<long long>(s.offset[i]) + p;
          if (id < 0 || off >= room) flags |= KVTC_STATUS_BAD_PAGE;
          if (off < room) {
            const long long at = (static_cast<long long>(head) + count + off) % a.capacity;
            a.ring[at] = id;
          }
        }
      }
    }
    if (n_chunks > 1) __syncthreads();  // the next chunk overwrites the tables
  }
  // rows behind the last sequence's
  for (long long r = max(static_cast<long long>(row_lo), min(run.rows, static_cast<long long>(a.n_rows))) + t; r < row_hi; r += kThreads) {
    a.slots[r] = -1;
    a.positions[r] = 0;
  }
  if (flags && a.status) atomicOr(a.status, static_cast<int>(flags));
  // lengths, row prefix and ring state that replace inputs: by the last CTA that has read them
  if (!writes) {
    if (!a.in_place) return;
    if (gridDim.x > 1) {
      __syncthreads();
      if (t == 0) {
        __threadfence();
        s.last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
        __threadfence();
      }
      __syncthreads();
      if (!s.last) return;
      if (t == 0) *a.ticket = 0;
    }
    Carry again;
    for (int ch = 0; ch < n_chunks; ++ch) {
      if (n_chunks > 1) (void)decide(a, s, ch * kChunk, count, again, new_len);
      write_lens(ch * kChunk);
      if (n_chunks > 1) __syncthreads();
    }
  }
  if (t == 0) {
    a.cu[a.n_seq] = static_cast<int>(min(run.rows, static_cast<long long>(a.n_rows)));
    const int kept = static_cast<int>(min(run.released, static_cast<long long>(room)));
    a.state_out[0] = static_cast<int>((static_cast<long long>(head) + s.taken) % a.capacity);
    a.state_out[1] = static_cast<int>(static_cast<long long>(count) - s.taken + kept);
  }
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" kvtc_status kvtc_step_tables(const int32_t* cached_lens, const int32_t* new_lens, int n_seq,
                                        int32_t* page_ring, int ring_capacity, const int32_t* ring_state,
                                        int32_t* block_table, int max_pages, int32_t* seq_lens, int32_t* cu_seqlens,
                                        int64_t* slot_map, int32_t* positions, int n_rows, int32_t* ring_state_out,
                                        void* workspace, int32_t* status, void* stream) {
  if (n_seq < 1 || max_pages < 1 || max_pages >= (1 << 24) || ring_capacity < 1 || n_rows < 0)
    return fail(KVTC_EINVAL, "bad sizes");
  if (!cached_lens || !new_lens || !page_ring || !ring_state || !block_table || !seq_lens || !cu_seqlens ||
      !ring_state_out || !workspace || (n_rows > 0 && (!slot_map || !positions)))
    return fail(KVTC_EINVAL, "null device pointer");
  const size_t n = static_cast<size_t>(n_seq), rows = static_cast<size_t>(n_rows);
  struct {
    const void* p;
    size_t bytes;
  } buf[] = {{cached_lens, 4 * n},  {new_lens, 4 * n},
             {page_ring, 4 * static_cast<size_t>(ring_capacity)},
             {ring_state, 8},       {block_table, 4 * n * static_cast<size_t>(max_pages)},
             {seq_lens, 4 * n},     {cu_seqlens, 4 * (n + 1)},
             {slot_map, 8 * rows},  {positions, 4 * rows},
             {ring_state_out, 8},   {workspace, 16},
             {status, 4}};
  const int count = static_cast<int>(sizeof(buf) / sizeof(buf[0]));
  for (int i = 0; i < count; ++i) {
    if (reinterpret_cast<uintptr_t>(buf[i].p) & (i == 7 ? 7 : 3)) return fail(KVTC_EINVAL, "misaligned device pointer");
    for (int j = i + 1; j < count; ++j) {
      const bool in_place = ((i == 0 && j == 5) || (i == 3 && j == 9)) && buf[i].p == buf[j].p;
      if (!in_place && raw::overlap(buf[i].p, buf[i].bytes, buf[j].p, buf[j].bytes))
        return fail(KVTC_EINVAL, "buffers overlap");
    }
  }
  TablesArgs a;
  a.cached = cached_lens;
  a.fresh = new_lens;
  a.n_seq = n_seq;
  a.ring = page_ring;
  a.capacity = ring_capacity;
  a.state = ring_state;
  a.table = block_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.cu = cu_seqlens;
  a.slots = slot_map;
  a.positions = positions;
  a.n_rows = n_rows;
  a.state_out = ring_state_out;
  a.in_place = seq_lens == cached_lens || ring_state_out == ring_state;
  a.ticket = static_cast<int*>(workspace);
  a.status = status;
  const bool small = n_seq <= kSmallThreads;
  const long long chunk = small ? kSmallThreads : static_cast<long long>(kLargeThreads) * kLargePer;
  const bool narrow = chunk * std::max<long long>(n_rows + 1ll, max_pages) < (1ll << 31);  // sums fit an int
  const long long per_cta = kRowsPerThread * (small ? kSmallThreads : kLargeThreads);
  const dim3 grid(static_cast<unsigned>(std::max<long long>(1, (n_rows + per_cta - 1) / per_cta)));
  cudaError_t e;
  if (small)
    e = narrow ? raw::launch(step_tables_kernel<int, kSmallThreads, 1>, grid, kSmallThreads, 0, stream, a)
               : raw::launch(step_tables_kernel<long long, kSmallThreads, 1>, grid, kSmallThreads, 0, stream, a);
  else
    e = narrow ? raw::launch(step_tables_kernel<int, kLargeThreads, kLargePer>, grid, kLargeThreads, 0, stream, a)
               : raw::launch(step_tables_kernel<long long, kLargeThreads, kLargePer>, grid, kLargeThreads, 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e, "step tables launch");
  return KVTC_OK;
}
