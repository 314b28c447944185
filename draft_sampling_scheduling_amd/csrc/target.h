// target.h -- helpers shared by the kernels of the target's side of a cycle (cache.hip,
// attention.hip, logits.hip).
#pragma once

#include "../../include/dspark_target.h"
#include "dev.h"
#include "host.h"

namespace dspark {

// 64-bit inclusive scan over a wave, in registers: within rows of 16 lanes, then each row's last
// lane onto the rows behind it (with shuffles, which go through LDS, a plan of 512 trees takes 10.6
// us for 9.8).
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t moved(int64_t v) {  // lanes that nothing moves to: 0
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xf, false);
  return (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  v += moved<0x111, 0xf>(v);  // from 1, 2, 4, 8 lanes before, in the row
  v += moved<0x112, 0xf>(v);
  v += moved<0x114, 0xf>(v);
  v += moved<0x118, 0xf>(v);
  v += moved<0x142, 0xa>(v);  // lane 15 onto row 1, 47 onto row 3
  v += moved<0x143, 0xc>(v);  // lane 31 onto rows 2 and 3
  return v;
}

// 64-bit inclusive scan over the whole workgroup (NT threads, a multiple of 64, every thread
// calls); `sums` is LDS of NT / 64 entries, free again after the call's last barrier.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  v = wave_scan(v);
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
  a = wave_scan(a);
  b = wave_scan(b);
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

// Head size and strides (in bytes) of a 4-bit cache: codes in pieces of 16 bytes, and a token's
// scale bytes of one head, D / 32 for its keys and as many for its values, in one piece.
inline bool cache4_ok(int D, int64_t page, int64_t head, int64_t tok, int64_t s_page, int64_t s_head,
                      int64_t s_tok) {
  if (D != 64 && D != 128) return false;
  for (int64_t s : {page, head, tok})
    if (!stride_ok(s, 1)) return false;
  for (int64_t s : {s_page, s_head, s_tok})
    if (s < 0 || s % (D / 16) != 0) return false;
  return true;
}

// whether two arrays of so many bytes share any
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

}  // namespace dspark
