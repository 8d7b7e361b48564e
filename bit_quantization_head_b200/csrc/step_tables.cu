// kvtc_step_tables: block table growth, page release and the row layout of a serving step.
//
// With c cached and n new tokens per sequence: tokens' rows are the prefix sum of n, the
// pages a sequence lacks are ceil((c + n) / 128) - ceil(c / 128), and its share of the
// free ring is the prefix sum of those needs over the sequences that fit.  Whether a
// sequence fits in the rows depends on the first sum alone, so two block scans decide a
// chunk of 1024 sequences: (rows, released pages), then (needed pages).
//
// Bound: latency for a decode step (a launch, two dependent loads, two scans), the 12
// bytes per row for large steps.  One launch without a wait between CTAs: every CTA scans
// all sequences for itself (8 bytes each, from L2) and fills its own range of rows; a row
// finds its sequence by bisection in the chunk's prefix sums in shared memory and takes
// its page id straight from the ring or the old table entries, so nothing that another
// CTA writes is read.  The outputs that may replace their inputs (lengths, ring state) are
// written by the last CTA to finish reading (one counter).
#include <cuda_runtime.h>

#include <algorithm>

#include "ptx.cuh"
#include "raw_cache.cuh"

namespace kvtc {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerCta = 4096;

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
  int* ticket;
  int32_t* status;
};

struct Smem {
  long long warp_sum[2][kWarps];
  long long total[2];
  int first_row[kThreads + 1];  // rows of the chunk's sequences, clipped to n_rows
  int cached[kThreads];
  int page0[kThreads];   // ring offset (from the head) of the sequence's first new page
  int need[kThreads];    // new pages (-1: the sequence keeps its length; -2: finished)
  int release0[kThreads];  // ring offset (from the tail) of its first released page
  int last;
};

// Exclusive sums of a and b over the block's threads; totals in s.total.
__device__ __forceinline__ void scan2(Smem& s, long long& a, long long& b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += p, y += q;
  }
  if (lane == 31) s.warp_sum[0][warp] = x, s.warp_sum[1][warp] = y;
  __syncthreads();
  if (warp < 2) {
    long long v = s.warp_sum[warp][lane];
    const long long own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long p = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += p;
    }
    s.warp_sum[warp][lane] = v - own;
    if (lane == 31) s.total[warp] = v;
  }
  __syncthreads();
  a = x - a + s.warp_sum[0][warp];
  b = y - b + s.warp_sum[1][warp];
}

// Running totals before a chunk.
struct Carry {
  long long rows = 0, need = 0, released = 0;
  long long taken = 0;  // pages taken from the head by the sequences that fit
};

// Decides the chunk of sequences base .. base + 1023 (one per thread) into shared memory.
__device__ uint32_t decide(const TablesArgs& a, Smem& s, int base, int count, Carry& run, int& new_len) {
  const int q = base + static_cast<int>(threadIdx.x);
  const bool in = q < a.n_seq;
  int c = in ? a.cached[q] : 0;
  const int n = in ? a.fresh[q] : 0;
  const long long limit = static_cast<long long>(a.max_pages) * kPage;
  const bool bad = c < 0 || c > limit;
  uint32_t flags = bad ? KVTC_STATUS_BAD_POS : 0u;
  if (bad) c = 0;
  const int held = (c + kPage - 1) / kPage;
  const bool finished = n < 0;
  long long row = n > 0 ? n : 0, rel = finished ? held : 0;
  scan2(s, row, rel);
  row += run.rows;
  rel += run.released;
  run.rows += s.total[0];
  run.released += s.total[1];
  __syncthreads();
  const bool fits = in && !finished && !bad && static_cast<long long>(c) + n <= limit && row + n <= a.n_rows;
  if (in && n > 0 && !fits) flags |= KVTC_STATUS_BAD_POS;
  const long long need = fits ? (static_cast<long long>(c) + n + kPage - 1) / kPage - held : 0;
  long long first = need, unused = 0;
  scan2(s, first, unused);
  first += run.need;
  run.need += s.total[0];
  const bool grows = fits && (need == 0 || first + need <= count);
  if (fits && !grows) flags |= KVTC_STATUS_NO_PAGE;
  const int t = threadIdx.x;
  s.first_row[t] = static_cast<int>(min(row, static_cast<long long>(a.n_rows)));
  s.cached[t] = c;
  s.page0[t] = grows ? static_cast<int>(min(first, static_cast<long long>(count))) : 0;
  s.need[t] = !in ? -1 : finished ? -2 : grows ? static_cast<int>(need) : -1;
  s.release0[t] = static_cast<int>(min(rel, static_cast<long long>(a.capacity)));
  if (t == kThreads - 1) s.first_row[kThreads] = static_cast<int>(min(run.rows, static_cast<long long>(a.n_rows)));
  new_len = finished ? 0 : grows ? c + n : c;
  // the sequences that take pages are a prefix of those that need some: the largest end
  long long end = grows && need > 0 ? first + need : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) end = max(end, __shfl_xor_sync(0xffffffffu, end, o));
  __syncthreads();  // the totals have been read
  if ((t & 31) == 0) s.warp_sum[0][t >> 5] = end;
  __syncthreads();
  long long most = run.taken;
  for (int w = 0; w < kWarps; ++w) most = max(most, s.warp_sum[0][w]);
  run.taken = most;
  return flags;
}

__global__ void __launch_bounds__(kThreads) step_tables_kernel(const __grid_constant__ TablesArgs a) {
  __shared__ Smem s;
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  int head = a.state[0], count = a.state[1];
  uint32_t flags = 0;
  if (head < 0 || head >= a.capacity || count < 0 || count > a.capacity) {
    head = count = 0;
    flags |= KVTC_STATUS_BAD_PAGE;
  }
  const int room = a.capacity - count;  // places a release can fill
  const int n_chunks = (a.n_seq + kThreads - 1) / kThreads;
  const int row_lo = static_cast<int>(min(static_cast<long long>(blockIdx.x) * kRowsPerCta, static_cast<long long>(a.n_rows)));
  const int row_hi = static_cast<int>(min(static_cast<long long>(row_lo) + kRowsPerCta, static_cast<long long>(a.n_rows)));
  Carry run;
  int new_len = 0;
  for (int ch = 0; ch < n_chunks; ++ch) {
    const int base = ch * kThreads;
    flags |= decide(a, s, base, count, run, new_len);
    const int n_in = min(kThreads, a.n_seq - base);
    // new table entries and released pages: a warp per sequence, dealt over the CTAs
    for (int i = static_cast<int>(blockIdx.x) * kWarps + warp; i < n_in; i += kWarps * static_cast<int>(gridDim.x)) {
      const int c = s.cached[i], need = s.need[i], held = (c + kPage - 1) / kPage;
      int32_t* row = a.table + static_cast<size_t>(base + i) * a.max_pages;
      if (need > 0) {
        for (int p = lane; p < need; p += 32) {
          const long long at = static_cast<long long>(head) + s.page0[i] + p;
          row[held + p] = a.ring[at < a.capacity ? at : at - a.capacity];
        }
      } else if (need == -2) {
        for (int p = lane; p < held; p += 32) {
          const int32_t id = row[p];
          const long long off = static_cast<long long>(s.release0[i]) + p;
          if (id < 0 || off >= room) flags |= KVTC_STATUS_BAD_PAGE;
          if (off < room) {
            const long long at = (static_cast<long long>(head) + count + off) % a.capacity;
            a.ring[at] = id;
          }
        }
      }
    }
    // this CTA's rows that fall into the chunk
    const int lo = max(row_lo, s.first_row[0]), hi = min(row_hi, s.first_row[kThreads]);
    for (int r = lo + t; r < hi; r += kThreads) {
      int l = 0, h = n_in - 1;  // the last sequence whose first row is <= r
      while (l < h) {
        const int mid = (l + h + 1) >> 1;
        if (s.first_row[mid] <= r)
          l = mid;
        else
          h = mid - 1;
      }
      const int c = s.cached[l], held = (c + kPage - 1) / kPage;
      int64_t slot = -1;
      int pos = 0;
      if (s.need[l] >= 0) {
        pos = c + (r - s.first_row[l]);
        const int p = pos / kPage;
        int32_t id;
        if (p < held) {
          id = a.table[static_cast<size_t>(base + l) * a.max_pages + p];
        } else {
          const long long at = static_cast<long long>(head) + s.page0[l] + (p - held);
          id = a.ring[at < a.capacity ? at : at - a.capacity];
        }
        if (id >= 0)
          slot = static_cast<int64_t>(id) * kPage + pos % kPage;
        else
          flags |= KVTC_STATUS_BAD_PAGE, pos = 0;
      }
      a.slots[r] = slot;
      a.positions[r] = pos;
    }
    if (n_chunks > 1) __syncthreads();  // the next chunk overwrites the tables
  }
  // rows behind the last sequence's
  for (int r = max(row_lo, static_cast<int>(min(run.rows, static_cast<long long>(a.n_rows)))) + t; r < row_hi; r += kThreads) {
    a.slots[r] = -1;
    a.positions[r] = 0;
  }
  if (flags && a.status) atomicOr(a.status, static_cast<int>(flags));
  // lengths, row prefix and ring state: by the last CTA that has read its inputs
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
    const int base = ch * kThreads;
    if (n_chunks > 1) (void)decide(a, s, base, count, again, new_len);
    if (base + t < a.n_seq) {
      a.seq_lens[base + t] = new_len;
      a.cu[base + t] = s.first_row[t];
      if (base + t == a.n_seq - 1)
        a.cu[a.n_seq] = static_cast<int>(min(run.rows, static_cast<long long>(a.n_rows)));
    }
    if (n_chunks > 1) __syncthreads();
  }
  if (t == 0) {
    const int kept = static_cast<int>(min(run.released, static_cast<long long>(room)));
    a.state_out[0] = static_cast<int>((head + run.taken) % a.capacity);
    a.state_out[1] = static_cast<int>(count - run.taken + kept);
  }
}

// Whether two buffers share memory (null or empty ones do not).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
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
      if (!in_place && overlap(buf[i].p, buf[i].bytes, buf[j].p, buf[j].bytes))
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
  a.ticket = static_cast<int*>(workspace);
  a.status = status;
  const unsigned grid = static_cast<unsigned>(std::max<long long>(1, (static_cast<long long>(n_rows) + kRowsPerCta - 1) / kRowsPerCta));
  const cudaError_t e = raw::launch(step_tables_kernel, dim3(grid), kThreads, 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e, "step tables launch");
  return KVTC_OK;
}
