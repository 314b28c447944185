// target.h -- helpers shared by the kernels of the target's side of a cycle (cache.hip,
// attention.hip, logits.hip).
#pragma once

#include "../../include/dspark_target.h"
#include "dev.h"
#include "host.h"

namespace dspark {

// 64-bit inclusive scan over the whole workgroup (NT threads, a multiple of 64, every thread
// calls); `sums` is LDS of NT / 64 entries, free again after the call's last barrier.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t u = __shfl_up(v, o, kWave);
    if (lane >= o) v += u;
  }
  if (lane == kWave - 1) sums[wave] = v;
  __syncthreads();
  int64_t base = 0;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) base += w < wave ? sums[w] : 0;
  __syncthreads();
  return base + v;
}

// the same of two values at once, and their totals; `sums` has 2 * NT / 64 entries
template <int NT>
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t& all_a, int64_t& all_b,
                                            int64_t* sums) {
  constexpr int NW = NT / kWave;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t u = __shfl_up(a, o, kWave), v = __shfl_up(b, o, kWave);
    if (lane >= o) {
      a += u;
      b += v;
    }
  }
  if (lane == kWave - 1) {
    sums[wave] = a;
    sums[NW + wave] = b;
  }
  __syncthreads();
  all_a = all_b = 0;
  int64_t base_a = 0, base_b = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    base_a += w < wave ? sums[w] : 0;
    base_b += w < wave ? sums[NW + w] : 0;
    all_a += sums[w];
    all_b += sums[NW + w];
  }
  a += base_a;
  b += base_b;
  __syncthreads();
}

constexpr int kMaxRequests = 1 << 20;

inline bool page_size_ok(int ps) { return ps >= 8 && ps <= 1024 && (ps & (ps - 1)) == 0; }
inline int log2_of(int p) { return __builtin_ctz((unsigned)p); }

// a block table whose tokens leave room to count beyond them in 32 bits
inline bool table_ok(int page_size, int64_t pages) {
  return page_size_ok(page_size) && pages >= 1 && pages * page_size <= ((int64_t)1 << 30);
}

// a cache of n_pages pages whose slots fit 31 bits
inline bool pages_ok(int page_size, int64_t pages) {
  return page_size_ok(page_size) && pages >= 1 && pages * page_size < ((int64_t)1 << 31);
}

// element strides whose byte distances keep 16-byte loads aligned
inline bool stride_ok(int64_t s, size_t esz) { return s >= 0 && (s * (int64_t)esz) % 16 == 0; }

// whether two arrays of so many bytes share any
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

}  // namespace dspark
