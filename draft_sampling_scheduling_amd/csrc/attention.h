// attention.h -- what the attention over a paged cache does whatever the cache holds: the rows of a
// step and what they see, the softmax of a tile, the cutting of all requests' lists over the grid,
// and the join of what was cut.  attention.hip (bf16 and float caches) and attention4.hip (4 bits)
// say how a wave takes its tiles.
#pragma once

#include <type_traits>

#include "sweep.h"
#include "target.h"

namespace dspark {

constexpr int kTok = 32;  // tokens of a tile
constexpr int kRows = 32;  // query rows of a wave
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

// A row tile whose list is cut (see attention_kernel): its pieces lie with workgroups b - 1 ..
// b - 2 + count.  A piece that begins its list is in its workgroup's slot 1, one that begins
// inside in slot 0; a workgroup has one of each at most.
struct AttJoint {
  int a, M, head, tile;  // first row and query rows of the request, cache head, row tile
  int count;             // 0: nothing to join
  int pad[3];
};

struct AttParams {
  int R, rows, Hq, Hkv, G;  // G = Hq / Hkv
  uint64_t inv_g;           // ceil(2^64 / G)
  int lg, max_pages, n_pages;
  const void* q;
  int64_t q_row;
  const void *k, *v;
  int64_t page_b, head_b, tok_b;  // strides in bytes
  const int32_t *table, *ctx, *row_off;
  const uint64_t* anc;
  float scale;
  int whole;  // rounds of a list up to which it is not cut
  void* o;
  float* lse;
  int32_t* status;
  float* part;   // [grid][2][MR][D + 2]: O, then m, then l of each row
  AttJoint* joint;  // [grid] what the second kernel joins
};

// x / G and x % G of a query row of a request, a division by multiplication: exact for 32 bits
__device__ __forceinline__ int node_of(const AttParams& p, int x) {
  return p.G == 1 ? x : (int)__umul64hi((uint64_t)(uint32_t)x, p.inv_g);
}
__device__ __forceinline__ int group_of(const AttParams& p, int x) { return x - node_of(p, x) * p.G; }

// a request's rows and tokens, as the host of the data should have them, clamped
struct AttReq {
  int a, n, ctx;
};

__device__ __forceinline__ AttReq att_req(const AttParams& p, int q, bool tell) {
  const int cap = p.max_pages << p.lg;
  int a = p.row_off[q], e = p.row_off[q + 1], c = p.ctx[q];
  bool bad = a < 0 || e < a || e > p.rows;
  a = a < 0 ? 0 : (a > p.rows ? p.rows : a);
  e = e < a ? a : (e > p.rows ? p.rows : e);
  int n = e - a;
  if (n > cap) {
    n = cap;
    bad = true;
  }
  if (n > 0 && (c < 0 || c > cap - n)) {
    c = c < 0 ? 0 : cap - n;
    bad = true;
  }
  if (tell) {
    if (bad) raise_fault(p.status, DSPARK_FAULT_LEN);
    if (p.anc && n > DSPARK_MAX_TREE_NODES) raise_fault(p.status, DSPARK_FAULT_TREE);
  }
  return {a, n, c};
}

// tokens that the query rows before row m1 of a request see: a chain's see no node after their
// last one's
__device__ __forceinline__ int att_end(const AttParams& p, const AttReq& r, int m1) {
  if (p.anc || m1 >= r.n * p.G) return r.ctx + r.n;
  return r.ctx + node_of(p, m1 - 1) + 1;
}

// uniform loads through the scalar cache (the arrays are inputs, constant during the call)
__device__ __forceinline__ int sload(const int32_t* p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t*)p)[i];
}

// a value that every lane holds alike, as a scalar
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uni(int64_t x) {
  return (int64_t)(((uint64_t)(uint32_t)uni((int)(x >> 32)) << 32) | (uint32_t)uni((int)x));
}

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
#define DSPARK_LDS __attribute__((address_space(3)))

template <class V>
__device__ __forceinline__ V lds_get(uint32_t a) {
  return *(const DSPARK_LDS V*)(uintptr_t)a;
}
template <class V>
__device__ __forceinline__ void lds_put(uint32_t a, V x) {
  *(DSPARK_LDS V*)(uintptr_t)a = x;
}
// the value, its origin hidden: what is computed from it stays where it stands (a loop's
// addresses are one instruction each, and would cost a register each if hoisted)
__device__ __forceinline__ uint32_t here(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// token of accumulator register r of half-wave h, within a tile; also d within 32 for O^T
__device__ __forceinline__ int reg_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// What one wave holds of 32 query rows: what each sees, and its running m, l and O.
template <int D>
struct AttRows {
  static constexpr int ND = D / 32;

  const AttParams& p;
  int lane, n, h;           // n: lane's column (query row of the wave's 32), h: half-wave
  // segment
  int ctx, len;             // committed tokens, tokens in all
  int seen;                 // tokens that every row of the row tile sees
  uint64_t see;             // tree: nodes (bit j - 1) the lane's row sees
  int node;                 // chain: the lane's node
  // state
  f32x16 o[ND];
  float m, l;               // m: what o and l are relative to, about the largest score so
                            // far, times scale * log2(e)

  __device__ __forceinline__ explicit AttRows(const AttParams& p_)
      : p(p_), lane(threadIdx.x & 63), n(lane & 31), h(lane >> 5) {}

  // the row tile that begins at query row m0 of a request
  __device__ __forceinline__ void begin_rows(const AttReq& rq, int m0) {
    ctx = rq.ctx;
    len = rq.ctx + rq.n;
    seen = uni(rq.ctx + 1 + (p.anc ? 0 : node_of(p, m0)));
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) o[dt] = f32x16{};
  }

  // tokens of the tile at t0 that the lane's row sees, the lane's own at bits reg_row(r, 0)
  __device__ __forceinline__ uint32_t visible(int t0) const {
    const int j0 = t0 - ctx, left = len - t0;  // node of the tile's first token, tokens from it on
    uint32_t vis;
    if (p.anc) {  // nodes from j0 on; below node 1 all are seen
      if (j0 > 0)
        vis = j0 <= 64 ? (uint32_t)(see >> (j0 - 1)) : 0;
      else
        vis = (uint32_t)see << 1 << -j0 | ((2u << -j0) - 1);
    } else {
      const int top = node - j0;
      vis = top < 0 ? 0 : ~0u >> (top < 31 ? 31 - top : 0);
    }
    if (left < 32) vis &= (1u << left) - 1;
    return vis >> 4 * h;
  }
  // scores of tokens that the lane's row does not see: -inf (t0 + 32 > ctx, as of edge tiles)
  __device__ __forceinline__ void mask(int t0, f32x16& sc) const {
    const uint32_t vis = visible(t0);
#pragma unroll
    for (int r = 0; r < 16; ++r) sc[r] = vis & (1u << reg_row(r, 0)) ? sc[r] : -INFINITY;
  }

  // the scores' weights, m, l and O's scale
  __device__ __forceinline__ void weigh(f32x16& sc) {
    const float c2 = p.scale * kLog2e;
    float mx = sc[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) mx = fmaxf(mx, sc[r]);
    mx = half_max(mx) * c2;
    // O and l are relative to m, which follows the maximum only once that is 2^kSlack past it:
    // weights of up to 2^kSlack lose nothing in float or bf16, and the rescaling of O, half a
    // tile's arithmetic, falls away on nearly all tiles
    if (__ballot(mx > m + kSlack)) {
      const float mn = fmaxf(m, mx);
      const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
      l *= f;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[dt][r] *= f;
      m = mn;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c2, -ref));
      sum += sc[r];
    }
    l += sum;  // this half-wave's tokens; the halves are added at the end
  }
};

// Where the rounds of a head go.  Each row tile of each request has a list of SETUP + rounds
// units, SETUP of them for what a list costs beside its tokens (the queries, the first
// tile's wait, the merge of the waves, the output), which no tokens stand for; all lists, head
// after head, are one row of units, cut evenly: workgroup b begins at unit begin(b).  A cut
// costs the later piece's set-up and the join; moving cuts to a near end lost more in balance
// than it saved in joins (120 requests of 180 to 254 tokens in tables of more, lists of 6 to 8
// rounds: 32 us with these kept whole, 27 cut), unless no list need be cut at all: block tables of
// no more than WHOLE tokens leave every list whole and launch no join.  Kernels alone, whole
// against cut, bf16, tables of 256 tokens, 32 heads on 8: 32 requests 15.4 and 17.1 us, 120 23.8
// and 27.5, 512 79 and 84; 17 rows, tables of 128: 32 requests 16.8 and 24.2.  In float a list's
// products take longer, and it is the call, a launch shorter, that gains: 4 requests of up to 204
// tokens 17 against 18 to 20 us a call, 19 against 13 captured in a graph.  A list that is cut has
// its pieces in the workspace; the first workgroup that begins inside one says so in joint[b].

// a / b, both at least 0; a 64-bit division is some hundred instructions
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int SETUP>
struct AttShares {
  int64_t share, more;  // units of a workgroup; the first `more` have one more
  int whole;            // lists of so many rounds stay whole
  __device__ __forceinline__ int64_t begin(int64_t b) const {
    return b * share + (b < more ? b : more);
  }
  __device__ __forceinline__ int64_t owner(int64_t u) const {  // last b with begin(b) <= u
    const int64_t big = more * (share + 1);
    return u < big ? quotient(u, share + 1) : more + quotient(u - big, share);
  }
  // where a cut at unit `at` of a list of len units falls
  __device__ __forceinline__ int64_t snapped(int64_t at, int64_t len) const {
    if (len <= SETUP + whole) return 2 * at <= len ? 0 : len;
    return at <= SETUP ? 0 : at;
  }
};

// W: what a wave does with a segment of a list (AttWave, Att4Wave), and how it sits on a CU.
template <class W>
__global__ void __launch_bounds__(W::F::THREADS, W::F::PER_SIMD)
    attention_kernel(typename W::Params p) {
  using F = typename W::F;
  using T = typename W::Out;
  constexpr int D = W::kD, NR = W::kNR;
  constexpr int MR = kRows * NR, ND = D / 32, kRound = F::ROUND, kAttThreads = F::THREADS,
                kSetup = F::SETUP;
  extern __shared__ uint4 lds[];
  __shared__ int64_t sums[F::WAVES];
  __shared__ int64_t total_s, start_off;
  __shared__ int start_s[5];
  const int tid = threadIdx.x, wave = uni(tid >> 6);
  const int b = blockIdx.x;

  auto tiles = [&](const AttReq& r) { return (r.n * p.G + MR - 1) / MR; };
  // A chain's row tile sees no tokens behind its last row's, and its list ends there.  Lists of
  // trees are all as long as the last row tile's, and so are those of pieces short beside their
  // context: alike, they divide evenly more often (16 pieces of 128 rows behind 1024 tokens: 67
  // against 87 us; past an eighth the tokens nobody sees cost more).
  auto even = [&](const AttReq& r) { return p.anc != nullptr || r.n <= (r.ctx + r.n) / 8; };
  auto list = [&](const AttReq& r, int mt) -> int64_t {
    const int end = even(r) ? r.ctx + r.n : att_end(p, r, (mt + 1) * MR);
    const int round = W::round(r.n * p.G);
    return (end + round - 1) / round + kSetup;
  };
  // Units of the first mt lists.  kPeriod * G row tiles on, a chain's lists are kMore rounds
  // longer, so a sum takes one period's lists at most.
  constexpr int kPeriod = kRound > MR ? kRound / MR : 1, kMore = MR > kRound ? MR / kRound : 1;
  auto before = [&](const AttReq& r, int mt) -> int64_t {
    if (even(r)) return mt * list(r, 0);
    const int n = tiles(r), inner = mt < n ? mt : n - 1;  // the last list ends with the rows
    const int period = kPeriod * p.G, c = inner / period, rest = inner - c * period;
    int64_t sum = 0, part = 0;
    for (int k = 0; k < (c > 0 ? period : rest); ++k) {
      const int64_t x = list(r, k);
      sum += x;
      part += k < rest ? x : 0;
    }
    if (c == 0)
      sum = part;
    else
      sum = c * sum + part + kMore * (period * ((int64_t)c * (c - 1) / 2) + (int64_t)rest * c);
    return mt < n ? sum : sum + list(r, n - 1);
  };
  auto units = [&](const AttReq& r) -> int64_t { return r.n > 0 ? before(r, tiles(r)) : 0; };
  const int per = (p.R + kAttThreads - 1) / kAttThreads;
  const int lo = min(p.R, tid * per), hi = min(p.R, lo + per);
  int64_t mine = 0;
  AttReq mine0 = {0, 0, 0};  // request lo
  for (int q = lo; q < hi; ++q) {
    const AttReq r = att_req(p, q, b == 0);
    if (q == lo) mine0 = r;
    mine += units(r);
  }
  const int64_t upto = block_scan<kAttThreads>(mine, sums);
  if (tid == kAttThreads - 1) total_s = upto;
  if (tid == 0) p.joint[b].count = 0;
  __syncthreads();
  const int64_t per_head = uni(total_s), U = per_head * p.Hkv;
  const int64_t P = U < gridDim.x ? U : gridDim.x;
  if (b >= P) return;
  AttShares<kSetup> cut;
  cut.share = quotient(U, P);
  cut.more = U - cut.share * P;
  cut.whole = p.whole;
  const int64_t u0 = cut.begin(b), u1 = cut.begin(b + 1);
  int head = (int)quotient(u0, per_head);
  {
    const int64_t w = u0 - head * per_head;
    int64_t at = upto - mine;
    if (w >= at && w < upto) {
      for (int q = lo; q < hi; ++q) {
        const AttReq r = q == lo ? mine0 : att_req(p, q, false);
        const int64_t x = units(r);
        if (w < at + x) {
          int mt = 0, end = tiles(r);  // the last list that begins at or before w
          while (end - mt > 1) {
            const int mid = mt + (end - mt) / 2;
            if (at + before(r, mid) <= w)
              mt = mid;
            else
              end = mid;
          }
          at += before(r, mt);
          start_s[0] = q;
          start_s[1] = r.a;
          start_s[2] = r.n;
          start_s[3] = r.ctx;
          start_s[4] = mt;
          start_off = w - at;
          break;
        }
        at += x;
      }
    }
  }
  __syncthreads();
  int q = uni(start_s[0]);
  AttReq rq = {uni(start_s[1]), uni(start_s[2]), uni(start_s[3])};
  int mt = uni(start_s[4]);
  int64_t at = uni(start_off);  // units of the row tile's list before this workgroup's

  const uint32_t base = (uint32_t)uni((int)lds_addr(lds));
  W wv(p, wave, base);
  int64_t u = u0;
  bool first = true;
  while (true) {
    if (mt >= tiles(rq)) {  // on to the next request, or the next head
      mt = 0;
      if (++q == p.R) {
        q = 0;
        ++head;
      }
      if (u >= u1) break;
      rq = att_req(p, q, false);
      rq = {uni(rq.a), uni(rq.n), uni(rq.ctx)};
      continue;
    }
    const int64_t len = uni(list(rq, mt)), s = u - at;  // the list's units are s .. s + len
    int64_t from = first ? cut.snapped(at, len) : at;
    const int64_t to = u1 - s >= len ? len : (u1 - s <= 0 ? 0 : cut.snapped(u1 - s, len));
    first = false;
    if (to <= 0) break;
    u += len - at;
    at = 0;
    const int mt0 = mt++;
    from = from > kSetup ? from - kSetup : 0;
    const int r0 = (int)from, nr = (int)(to - kSetup - from), rounds = (int)len - kSetup;
    if (nr <= 0) continue;
    wv.segment(rq, q, head, mt0 * MR, r0, nr);

    const bool whole = r0 == 0 && nr == rounds;
    const int M = rq.n * p.G, lane = tid & 63;
    float* part = p.part + ((int64_t)b * 2 + (r0 == 0)) * MR * (D + 2);
    // a row's O (d .. d + 3), and its m and l, to the output or the workspace
    auto put = [&](int row, int d, f32x4 z) {
      if (!whole) {
        *reinterpret_cast<f32x4*>(part + row * D + d) = z;
        return;
      }
      const int mi = mt0 * MR + row;
      T* out = static_cast<T*>(p.o) +
               ((int64_t)(rq.a + node_of(p, mi)) * p.Hq + head * p.G + group_of(p, mi)) * D + d;
      if constexpr (F::kBf) {
        bf16x4 zb;
#pragma unroll
        for (int e = 0; e < 4; ++e) zb[e] = (__bf16)z[e];
        *reinterpret_cast<bf16x4*>(out) = zb;
      } else {
        *reinterpret_cast<f32x4*>(out) = z;
      }
    };
    auto put_sums = [&](int row, float m, float l) {
      const int mi = mt0 * MR + row;
      if (!whole) {
        part[MR * D + row] = m;
        part[MR * (D + 1) + row] = l;
      } else if (p.lse) {
        p.lse[(int64_t)(rq.a + node_of(p, mi)) * p.Hq + head * p.G + group_of(p, mi)] =
            (m + __builtin_amdgcn_logf(l)) * kLn2;
      }
    };
    const auto rows_apart = [&]() {
      const int row = kRows * wave + wv.n;
      if (mt0 * MR + row < M) {
        const float f = !whole ? 1.0f : (wv.l == 0.0f ? 0.0f : 1.0f / wv.l);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
          for (int r4 = 0; r4 < 4; ++r4) {
            f32x4 z;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = wv.o[dt][4 * r4 + e] * f;
            put(row, 32 * dt + 8 * r4 + 4 * wv.h, z);
          }
        if (wv.h == 0) put_sums(row, wv.m, wv.l);
      }
    };
    const auto rows_shared = [&]() {
      // the waves' sums, through LDS: each gives the other half of its O, and finishes its own half
      constexpr int HD = ND / 2, kGive = (HD * 16 + 2) * 64;
      float* x = reinterpret_cast<float*>(lds);
      auto give = [&](auto self) {
        constexpr int S = decltype(self)::value;
        float* y = x + S * kGive + lane;
#pragma unroll
        for (int i = 0; i < HD; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) y[(i * 16 + r) * 64] = wv.o[(1 - S) * HD + i][r];
        y[HD * 16 * 64] = wv.m;
        y[(HD * 16 + 1) * 64] = wv.l;
      };
      auto finish = [&](auto self) {
        constexpr int S = decltype(self)::value;
        const float* y = x + (1 - S) * kGive + lane;
        const float m2 = y[HD * 16 * 64], l2 = y[(HD * 16 + 1) * 64];
        const float mm = fmaxf(wv.m, m2), ref = mm == -INFINITY ? 0.0f : mm;
        float f1 = __builtin_amdgcn_exp2f(wv.m - ref), f2 = __builtin_amdgcn_exp2f(m2 - ref);
        const float ll = wv.l * f1 + l2 * f2;
        if (mt0 * MR + wv.n >= M) return;
        if (whole) {
          const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
          f1 *= inv;
          f2 *= inv;
        }
#pragma unroll
        for (int i = 0; i < HD; ++i)
#pragma unroll
          for (int r4 = 0; r4 < 4; ++r4) {
            f32x4 z;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 4 * r4 + e;
              z[e] = wv.o[S * HD + i][r] * f1 + y[(i * 16 + r) * 64] * f2;
            }
            put(wv.n, 32 * (S * HD + i) + 8 * r4 + 4 * wv.h, z);
          }
        if (S == 0 && wv.h == 0) put_sums(wv.n, mm, ll);
      };
      using First = std::integral_constant<int, 0>;
      using Second = std::integral_constant<int, 1>;
      __syncthreads();
      if (wave == 0) give(First{});
      else give(Second{});
      __syncthreads();
      if (wave == 0) finish(First{});
      else finish(Second{});
    };
    if constexpr (W::kMix) {
      if (M > kRows) rows_apart();
      else rows_shared();
    } else if constexpr (NR > 1) {
      rows_apart();
    } else {
      rows_shared();
    }
    // this workgroup begins inside a list: the first to do so if the one before it did not
    if (tid == 0 && r0 > 0 && cut.begin(b - 1) <= s + kSetup)
      p.joint[b] = {rq.a, rq.n * p.G, head, mt0, (int)(cut.owner(s + len - 1) - b) + 2,
                    {0, 0, 0}};
    if (u >= u1) break;
    __syncthreads();  // LDS is the next segment's
  }
}

// Joins the pieces of the row tiles that are cut: a wave per row, 16 bytes a lane, so that
// D / 4 lanes hold a piece's row and the wave takes 256 / D pieces at a time; sums and maxima
// run over each lane's pieces and meet at the end, always in the same order.
// DEEP: lists of many pieces, twelve loads in flight where few lists leave the chip to few
// waves; otherwise four at most, in registers for twice the waves.
template <class W, bool DEEP>
__global__ void __launch_bounds__(256) attention_join_kernel(AttParams p, bool across) {
  using T = typename W::Out;
  constexpr int D = W::kD, NR = W::kNR;
  constexpr int MR = kRows * NR, LP = D / 4, NP = kWave / LP;
  const int b = across ? blockIdx.y : blockIdx.x;
  const int slice = across ? blockIdx.x : blockIdx.y, slices = across ? gridDim.x : gridDim.y;
  const AttJoint jt = p.joint[b];
  if (jt.count == 0) return;
  const int lane = threadIdx.x & 63;
  const int mine = lane / LP, d = 4 * (lane % LP);
  auto piece = [&](int k) {
    return p.part + ((int64_t)(b - 1 + k) * 2 + (k == 0)) * MR * (D + 2);
  };
  const int rows = min(MR, jt.M - jt.tile * MR);
  for (int row = slice * 4 + (threadIdx.x >> 6); row < rows; row += 4 * slices) {
    const int mi = jt.tile * MR + row;
    float m = -INFINITY, l = 0.0f;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto take = [&](auto batch, int k0) {
      constexpr int kBatch = decltype(batch)::value;
      f32x4 x[kBatch];
      float pm[kBatch], pl[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {  // pieces past the last: the last, with no weight
        const int k = k0 + u * NP + mine;
        const float* y = piece(k < jt.count ? k : jt.count - 1);
        x[u] = *reinterpret_cast<const f32x4*>(y + row * D + d);
        pm[u] = k < jt.count ? y[MR * D + row] : -INFINITY;
        pl[u] = y[MR * (D + 1) + row];
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, pm[u]);
      const float ref = mn == -INFINITY ? 0.0f : mn;
      float f = __builtin_amdgcn_exp2f(m - ref);
      l *= f;
      acc *= f;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        // where a piece has no weight its row stays out (0 * inf is none); its sum is finite, or
        // NaN where the row's scores are.  Of a cache of 4 bits NaN comes along: a group of a token
        // that the row sees, and within a piece 0 * NaN keeps it.  (A lane's elements share a group.)
        f = __builtin_amdgcn_exp2f(pm[u] - ref);
        l = fmaf(pl[u], f, l);
        const bool in = f != 0.0f || (W::kNan && x[u][0] != x[u][0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = in ? fmaf(x[u][e], f, acc[e]) : acc[e];
      }
      m = mn;
    };
    // few loads where there are few pieces: those of missing ones take their time too
    constexpr int kMost = DEEP ? 12 : 4;
    if (jt.count <= NP) {
      take(std::integral_constant<int, 1>{}, 0);
    } else if (jt.count <= 2 * NP) {
      take(std::integral_constant<int, 2>{}, 0);
    } else if (DEEP && jt.count <= 4 * NP) {
      take(std::integral_constant<int, 4>{}, 0);
    } else {
      for (int k0 = 0; k0 < jt.count; k0 += kMost * NP)
        take(std::integral_constant<int, kMost>{}, k0);
    }
#pragma unroll
    for (int w = LP; w < kWave; w *= 2) {  // the lanes that hold the same d
      const float m2 = __shfl_xor(m, w, kWave), mm = fmaxf(m, m2);
      const float ref = mm == -INFINITY ? 0.0f : mm;
      const float f1 = __builtin_amdgcn_exp2f(m - ref), f2 = __builtin_amdgcn_exp2f(m2 - ref);
      l = l * f1 + __shfl_xor(l, w, kWave) * f2;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = acc[e] * f1 + __shfl_xor(acc[e], w, kWave) * f2;
      m = mm;
    }
    if (mine != 0) continue;
    acc *= l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = (int64_t)(jt.a + node_of(p, mi)) * p.Hq + jt.head * p.G + group_of(p, mi);
    T* out = static_cast<T*>(p.o) + at * D + d;
    if constexpr (std::is_same<T, uint16_t>::value) {
      bf16x4 z;
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = (__bf16)acc[e];
      *reinterpret_cast<bf16x4*>(out) = z;
    } else {
      *reinterpret_cast<f32x4*>(out) = acc;
    }
    if (p.lse && d == 0) p.lse[at] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
// workgroups: as many as stay resident
template <class F>
static int att_grid() {
  return device_cus() * F::PER_CU;
}

// The workspace of a grid whose row tiles have MR rows.  Pieces take as much in variants of more rows
// or more; joints are counted for the most workgroups of any, so that the size does not fall where a
// step's rows take it to a variant of fewer, and a workspace for many rows serves few.
constexpr int kMostPerCu = 6;
static inline size_t att_carve(AttParams& p, void* ws, int grid, int MR, int D) {
  Carve cv(ws);
  p.joint = cv.take<AttJoint>((size_t)device_cus() * kMostPerCu);
  p.part = cv.take<float>((size_t)grid * 2 * MR * (D + 2));
  return cv.bytes();
}

static inline bool att_dims_ok(int R, int rows, int Hq, int Hkv, int D, dspark_dtype dt) {
  return R >= 0 && R <= kMaxRequests && rows >= 0 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
         (D == 64 || D == 128) && (dt == DSPARK_F32 || dt == DSPARK_BF16) &&
         (int64_t)rows * Hq <= ((int64_t)1 << 31) - 1024;  // ends of row tiles in 31 bits
}

// The arguments that the entry points share (not the cache's strides), checked and taken over.
static inline int att_args(AttParams& p, int R, int rows, int Hq, int Hkv, int D, dspark_dtype dt, int page_size,
                           int max_pages, int n_pages, const void* q, int64_t q_row, const void* k_cache,
                           const void* v_cache, const int32_t* table, const int32_t* ctx, const int32_t* row_off,
                           const uint64_t* anc, float scale, void* o, float* lse, int32_t* dev_status, void* ws) {
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  if (max_pages < 1 || !pages_ok(page_size, n_pages) || !table_ok(page_size, max_pages) || !(scale > 0.0f) ||
      !(scale * kLog2e <= FLT_MAX) || !stride_ok(q_row, e))
    return DSPARK_EINVAL;
  if (R == 0 || rows == 0) return DSPARK_OK;
  if (!q || !k_cache || !v_cache || !table || !ctx || !row_off || !o || !ws || !aligned16(q) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(ws))
    return DSPARK_EINVAL;
  // a row's heads may be read after another's output is written
  const size_t row_bytes = (size_t)Hq * D * e;
  if (overlap(q, (size_t)(rows - 1) * q_row * e + row_bytes, o, rows * row_bytes)) return DSPARK_EINVAL;
  p.R = R;
  p.rows = rows;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.inv_g = p.G > 1 ? ~(uint64_t)0 / p.G + 1 : 0;
  p.lg = log2_of(page_size);
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.q = q;
  p.q_row = q_row;
  p.k = k_cache;
  p.v = v_cache;
  p.table = table;
  p.ctx = ctx;
  p.row_off = row_off;
  p.anc = anc;
  p.scale = scale;
  p.o = o;
  p.lse = lse;
  p.status = dev_status;
  return DSPARK_OK;
}

template <class W>
static int att_launch(typename W::Params p, hipStream_t stream) {
  using F = typename W::F;
  constexpr int NR = W::kNR;
  static_assert(F::PER_CU <= kMostPerCu, "a workgroup has a joint each");
  static std::atomic<uint64_t> raised;
  auto kern = attention_kernel<W>;
  const int grid = att_grid<F>();
  ensure_dynamic_lds(reinterpret_cast<const void*>(kern), F::LDS, raised);
  p.whole = ((int64_t)p.max_pages << p.lg) <= F::WHOLE ? F::WHOLE / F::ROUND : 0;
  kern<<<grid, F::THREADS, F::LDS, stream>>>(p);
  if (p.whole > 0) return launch_status();
  // a wave per row of a row tile, as far as the host knows how many rows there are
  const int64_t m = (int64_t)((p.rows + p.R - 1) / p.R) * p.G;
  int slices = m < kRows * NR ? (int)(m + 3) / 4 : 8 * NR;
  const int64_t tiles = (m + kRows * NR - 1) / (kRows * NR);
  if (W::kMix || tiles > 1) {
    // Many workgroups have joints, each one at most: so many slices that all of them about fit the
    // chip twice (256 requests of 512 to 4096 tokens, of 4 bits: 4 slices 168, 9 172 us; 64 of 100 to
    // 2048, a quarter of whose workgroups have joints: 31 and 28.5; 2048 rows behind 4048 tokens, in 512
    // pieces of 128 rows: 4 slices 231, 16 233, 32 237; over bf16 that piece 234, as 32 slices 240, a
    // prompt of 4096 rows 198 and 204, of heads of 64 138 and 145, four of 500 rows 60 and 63.5, 16 of 128
    // behind 1000 67 and 70, 64 requests of 72 query rows 140.5 both).
    const int64_t lists = (int64_t)p.R * p.Hkv * (W::kMix ? 1 : tiles), joints = lists < grid ? lists : grid;
    const int most = (int)(4 * grid / joints);
    slices = slices < most ? slices : most;
  }
  // Workgroups go to the eight dies in turn.  The joints lie some workgroups apart, often all
  // with the same remainder by 8 or two of them, so where there is much to read (112 row tiles
  // of 128: 12 to 29 us) neighbours are the slices of one joint (13 us); where there is little,
  // one die is as good (two requests of 5 rows: 8 against 11 us).
  const bool across = slices >= 8;
  const dim3 blocks = across ? dim3(slices, grid) : dim3(grid, slices);
  if (grid / p.R / p.Hkv >= 16)  // pieces of a list, were there one row tile a request
    attention_join_kernel<W, true><<<blocks, 256, 0, stream>>>(p, across);
  else
    attention_join_kernel<W, false><<<blocks, 256, 0, stream>>>(p, across);
  return launch_status();
}

}  // namespace dspark
