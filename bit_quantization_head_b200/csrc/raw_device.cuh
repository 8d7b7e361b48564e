// Device helpers of the two attention kernels on the uncompressed pages.
#pragma once
#include <cuda.h>

#include "ptx.cuh"
#include "raw_cache.cuh"

namespace kvtc {
namespace raw {

// a / b for a >= 0, b > 0, in 32 bits where they do (a 64-bit division takes a few hundred
// cycles at the head of every launch).
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// All tiles of all units in a row, cut into one run per CTA: the tile at which CTA i of n
// starts, and the CTA that holds tile t.
__device__ __forceinline__ long long run_start(long long i, long long n, long long total) { return divide(i * total, n); }
__device__ __forceinline__ int run_owner(long long t, long long n, long long total) {
  return static_cast<int>(divide((t + 1) * n + total - 1, total)) - 1;
}

// The sequences' slots in a row, by a whole warp: their total, and the sequence that holds a
// slot.  Up to 32 sequences are read once.
template <typename Slots>
struct SlotScan {
  int n_seq;
  const Slots& slots;
  long long total, mine, incl;  // incl: the sum up to the lane's sequence (of the first 32)

  __device__ __forceinline__ SlotScan(int n, const Slots& f) : n_seq(n), slots(f) {
    const int lane = threadIdx.x & 31;
    mine = lane < n ? f(lane) : 0;
    scan();
    total = __shfl_sync(0xffffffffu, incl, 31);
    if (n > 32) {
      long long more = 0;
      for (int i = lane + 32; i < n; i += 32) more += f(i);
#pragma unroll
      for (int o = 16; o; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
      total += more;
    }
  }
  __device__ __forceinline__ void scan() {
    const int lane = threadIdx.x & 31;
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
  }
  // The sequence that holds slot f (0 <= f < total); base: its first slot.
  __device__ __forceinline__ int find(long long f, long long& base) {
    const int lane = threadIdx.x & 31;
    base = 0;
    for (int i0 = 0; i0 < n_seq; i0 += 32) {
      if (i0) {
        mine = i0 + lane < n_seq ? slots(i0 + lane) : 0;
        scan();
      }
      const unsigned past = __ballot_sync(0xffffffffu, f < base + incl);
      if (past) {
        const int at = __ffs(past) - 1;
        base += __shfl_sync(0xffffffffu, incl - mine, at);
        return i0 + at;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return 0;
  }
};

// Named barrier of the `threads` threads that consume together, without an endless wait: a
// warp that leaves because the CTA gave up (the dead flag: a bounded wait ran out) arrives
// once in its place.  That completes the barrier the others may be in or come to next; the
// flag was set before it, so each of them sees it there and leaves the same way.
__device__ __forceinline__ void leave_barrier(int id, int threads) {
  __threadfence_block();
  asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool consumers_sync(int id, int threads, volatile int* dead) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
  if (!__any_sync(0xffffffffu, *dead)) return true;
  leave_barrier(id, threads);
  return false;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Bounded wait (2^16 sleeps of up to 20 us), given up at once when the CTA is dead.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t phase, volatile int* dead) {
  for (uint32_t i = 0; i < (1u << 16); ++i) {
    if (mbar_try_wait_sleep(bar, phase, 20000u)) return true;
    if (*dead) return false;
  }
  return false;
}

// The same by a whole warp, which stays together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t phase, volatile int* dead) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase))) return true;
  for (uint32_t i = 0; i < (1u << 16); ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, phase, 20000u))) return true;
    if (__any_sync(0xffffffffu, *dead)) return false;
  }
  return false;
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// Two floats rounded to the pages' type.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (F16) return pack_half2(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace raw
}  // namespace kvtc
