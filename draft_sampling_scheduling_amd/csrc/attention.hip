// attention.hip -- attention of a step's rows (a chain or a tree of drafted tokens, one
// token, or a piece of a prompt) over the paged cache.
//
// For a request with n rows over ctx + n tokens, the n * (Hq / Hkv) query rows that share a
// cache head are the columns of two matrix products per 32 tokens, both taken transposed:
//   S^T = K Q^T   (tokens x rows)      and      O^T += V^T P^T   (D x rows),
// with one pass over K and V and the running maximum m and sum l of the softmax,
//   P = exp(S - m),  O = O exp(m_old - m) + P V,  l = l exp(m_old - m) + sum P.
// Transposed, a lane holds one query row's scores (its accumulator column), so maxima and
// sums are in-lane but for one half-wave exchange, and the 16 scores a lane ends S^T with are,
// unmoved, the operand that O^T takes: the order of the tokens in the second contraction is
// free as long as V follows it.
//
// Bound: the cache is read once, M = n Hq / Hkv multiply-adds per element of it, so HBM
// bounds it up to M of a few hundred; what the design needs is bytes in flight.
//   - Tiles of 32 tokens are copied straight to LDS, 16 bytes a lane, ahead of their use.  Up
//     to 32 query rows, a wave has tiles of its own, waits on its own copies only, and two
//     waves merge at the end; with more rows, each wave keeps 32 of them and all share each
//     tile.  m, l and O stay in registers.
//   - The tokens of all requests and heads form one list of rounds (64 or 32 tokens x one row
//     tile of one head), cut evenly over a fixed grid, so ragged lengths balance and a single long
//     request fills the chip.  A piece of a row tile's list that is not all of it goes to
//     the workspace, and a second kernel joins the pieces in order.
// Measured, bf16, D = 128, both kernels: 256 requests of 512 to 4096 tokens, 32 heads on 8, up to
// nine rows (2.44 GB) 446 us, 5.5 TB/s where a kernel that only reads gets 5.7; two single
// tokens over 100001 to 131071, 40 heads on 8 (0.95 GB) 161 to 180 us; 64 trees over 100 to
// 2048, 20 heads on 4 (145 MB) 42 to 45 us, of which 29 us are the bytes at a copy's rate.  Prompts are
// bound by the softmax's vector work, which takes as long as the products and overlaps them in
// part: 8192 rows, 32 heads on 8, 677 to 700 us, 800 TFLOP/s of the pairs seen.
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

// ---------------------------------------------------------------------------------------
// Per element type: the tile's geometry in LDS, the fragments, and the two products.
// A tile's rows lie RB bytes apart in 16-byte chunks; chunk c of row r is at chunk
// c ^ kswz(r) (K) or c ^ vswz(r) (V), which spreads what one LDS instruction reads over the
// banks: 16 rows at one chunk (K), 4 rows at 4 neighbouring chunks (V, bf16), rows 4 apart (V,
// float).  Both maps act on disjoint bits of r, so map(i | j) = map(i) ^ map(j).
// ---------------------------------------------------------------------------------------
template <class T, int D>
struct Tile {
  static constexpr bool kBf = std::is_same<T, uint16_t>::value;
  static constexpr int kE = kBf ? 2 : 4;
  static constexpr int RB = D * kE;            // bytes of a row
  static constexpr int CPR = RB / 16;          // chunks of a row
  static constexpr int RPC = kWave / CPR;      // rows one copy instruction moves
  static constexpr int NC = kTok / RPC;        // copies of one operand's tile
  static constexpr int BYTES = kTok * RB;      // one operand's tile
  static constexpr int KSTEPS = D / (kBf ? 16 : 8);  // 16-byte fragments of a row per half-wave
  static __host__ __device__ constexpr int kswz(int r) { return CPR >= 16 ? (r & 15) : ((r >> 1) & 7); }
  static __host__ __device__ constexpr int vswz(int r) {
    if (!kBf) return ((r >> 2) & 1) << 3;
    return CPR >= 16 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
  }
};

// How a variant (element type, D, NR: waves over query rows) sits on a CU.
//   NR 1, up to 32 query rows: the two waves of a workgroup take 32 tokens each, have their
//   tiles to themselves (no barrier), and merge at the end.  STAGES 2: K and V are copied two
//   tiles deep.  STAGES 1: one buffer each; K's next tile is under way as soon as the scores
//   are taken, V's as soon as O is: half the LDS, twice the workgroups.
//   NR 2 or 4, up to 64 or 128 rows: every wave has 32 rows of its own, and all share each
//   tile of 32 tokens, copied one ahead by all of them, with a barrier per tile; the cache is
//   read once for all rows.  A third stage made them slower (453 against 440 us for
//   256 requests of 512 to 4096 tokens).
//   PER_CU workgroups are resident; where registers allow two waves a SIMD, one's set-up,
//   exponentials and merge hide behind the other's tiles.
template <class T, int D, int NR>
struct Fit {
  static constexpr bool kBf = std::is_same<T, uint16_t>::value;
  static constexpr int WAVES = NR == 1 ? 2 : NR;
  static constexpr int THREADS = WAVES * kWave;
  static constexpr int ROUND = NR == 1 ? 2 * kTok : kTok;  // tokens of a round
  // what a list costs beside its tokens, in rounds: 6 to 8 us, where a round of 64 tokens takes 3,
  // of float ones more (at 3 there 16 requests of 128 rows took 136 us, at 2 133), and one of 32
  // about 1 (at 3 a prompt of 8192 rows took 750 us, at 6 704)
  static constexpr int SETUP = NR > 1 ? 6 : (kBf ? 3 : 2);
  static constexpr int TILE = 2 * kTok * D * (kBf ? 2 : 4);  // bytes of a K and a V tile
  static constexpr int STAGES = NR == 1 ? (kBf && D == 64 ? 2 : 1) : 2;
  static constexpr int LDS = (NR == 1 ? 2 : 1) * STAGES * TILE;
  // two waves a SIMD, but for float rows of 128, whose one wave takes its registers.  (bf16 of 64
  // has registers, and from 33 rows on LDS, for three: full row tiles gain, 64 requests of 72 rows
  // 98 -> 92 us, 2048 rows behind 4096 tokens 221 -> 209, others lose, 64 of 45 rows over 100 to
  // 800 tokens 27.5 -> 28.2, over 500 to 4000 78.1 -> 78.8.)
  static constexpr int PER_SIMD = !kBf && D == 128 ? 1 : 2;
  static constexpr int PER_CU = 4 * PER_SIMD / WAVES;
};

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

// K's fragment of step s times every row tile's Q fragment
template <class T>
__device__ __forceinline__ void mfma_qk(u32x4 a, u32x4 b, f32x16& acc) {
  if constexpr (std::is_same<T, uint16_t>::value) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], acc, 0, 0, 0);
  }
}

// token of accumulator register r of half-wave h, within a tile; also d within 32 for O^T
__device__ __forceinline__ int reg_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// What one wave holds: 32 query rows, and its running m, l and O of them.
template <class T, int D, int NR>
struct AttWave {
  using L = Tile<T, D>;
  using F = Fit<T, D, NR>;
  static constexpr int ND = D / 32;
  // rows of a tile that this wave copies, from row `mine` on, and groups of 8 of them
  static constexpr int CROWS = kTok / NR, CG = CROWS / 8, NC = L::NC / NR;

  const AttParams& p;
  int lane, n, h, wave;     // n: lane's column (query row of the wave's 32), h: half-wave
  int mine;                 // first row of a tile that this wave copies
  uint32_t base;            // LDS of its stages
  // segment
  const char *kh, *vh;      // cache bases of the head
  const int32_t* pages;     // the request's block table
  int ctx, len, last_page;  // committed tokens, tokens in all, page of the last token
  int seen;                 // tokens that every row of the row tile sees
  u32x4 qf[L::KSTEPS];
  uint64_t see;             // tree: nodes (bit j - 1) the lane's row sees
  int node;                 // chain: the lane's node
  // state
  f32x16 o[ND];
  float m, l;               // m: what o and l are relative to, about the largest score so
                            // far, times scale * log2(e)

  __device__ __forceinline__ AttWave(const AttParams& p_, int wave_, uint32_t lds)
      : p(p_), lane(threadIdx.x & 63), n(lane & 31), h(lane >> 5), wave(wave_),
        mine(NR == 1 ? 0 : wave_ * CROWS),
        base(NR == 1 ? lds + wave_ * F::STAGES * F::TILE : lds) {}

  // Pages of the wave's rows of tile t0, a page per 8 of them (aligned, so they share one);
  // past the last token, its page.
  __device__ __forceinline__ void page_ids(int t0, int (&pg)[CG]) const {
#pragma unroll
    for (int g = 0; g < CG; ++g) {
      int i = (t0 + mine + 8 * g) >> p.lg;
      i = i < last_page ? i : last_page;
      pg[g] = sload(pages, i);
    }
  }
  __device__ __forceinline__ void known(int (&pg)[CG]) const {
    bool bad = false;
#pragma unroll
    for (int g = 0; g < CG; ++g) {
      const bool out = pg[g] < 0 || pg[g] >= p.n_pages;
      bad = bad || out;
      pg[g] = out ? 0 : pg[g];
    }
    if (bad && lane == 0) raise_fault(p.status, DSPARK_FAULT_PAGE);
  }
  // The copies of the wave's rows of tile t0's K or V into stage s.  Rows past the last token
  // read inside its page, and are never used.  Scalar work is serial in a wave, so the 8 rows
  // of a group, which lie in one page, share an offset.
  template <bool V>
  __device__ __forceinline__ void copy(int t0, const int (&pg)[CG], int s) const {
    const int lr = lane / L::CPR, pos = lane % L::CPR;
    const uint32_t tok_b = (uint32_t)p.tok_b, row = (uint32_t)lr * tok_b;
    const uint32_t to = base + s * F::TILE + V * L::BYTES + mine * L::RB;
    const int in_page = (1 << p.lg) - 1;
    const int xl = V ? L::vswz(lr) ^ L::vswz(mine) : L::kswz(lr) ^ L::kswz(mine);
#pragma unroll
    for (int g = 0; g < CG; ++g) {
      const char* rows = (V ? vh : kh) + (uint64_t)(uint32_t)pg[g] * (uint64_t)p.page_b +
                         (uint64_t)(uint32_t)((t0 + mine + 8 * g) & in_page) * tok_b;
#pragma unroll
      for (int i = 0; i < 8; i += L::RPC) {
        const int c = (8 * g + i) / L::RPC;
        const int x = xl ^ (V ? L::vswz(8 * g + i) : L::kswz(8 * g + i));
        dma16s(rows + (uint32_t)i * tok_b, row + (uint32_t)((pos ^ x) << 4), to + c * 1024);
      }
    }
  }

  // S^T of a tile
  __device__ __forceinline__ void scores(uint32_t ks, f32x16& sc) const {
    const uint32_t krow = here(ks + n * L::RB), kx = here((uint32_t)(h ^ L::kswz(n)) << 4);
    sc = f32x16{};
    // Eight reads under way before the first is used (the fence keeps them so): one takes longer
    // than a product, and read one at a time 8192 rows take 789 us for 776.
    constexpr int kBatch = 8;
#pragma unroll
    for (int s0 = 0; s0 < L::KSTEPS; s0 += kBatch) {
      constexpr int kN = L::KSTEPS < kBatch ? L::KSTEPS : kBatch;
      u32x4 f[kN];
#pragma unroll
      for (int st = 0; st < kN; ++st) f[st] = lds_get<u32x4>(krow + (kx ^ (uint32_t)((s0 + st) << 5)));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int st = 0; st < kN; ++st) mfma_qk<T>(f[st], qf[s0 + st], sc);
    }
  }

  // scores of tokens that the lane's row does not see: -inf (t0 + 32 > ctx, as of edge tiles)
  __device__ __forceinline__ void mask(int t0, f32x16& sc) const {
    const int j0 = t0 - ctx, left = len - t0;  // node of the tile's first token, tokens from it on
    uint32_t vis;                              // tokens of the tile that the row sees
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
    vis >>= 4 * h;
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

  // O^T += V^T P^T
  __device__ __forceinline__ void values(uint32_t vs, const f32x16& sc) {
    if constexpr (L::kBf) {
      // 16 tokens a step: registers 8 st .. 8 st + 7 are the lane's 8 tokens of it, rounded to
      // bf16 (each weight off by 2^-8 of itself at most, as o is when stored: o's error against 64
      // bits is 0.0023 of its norm, one rounding's 0.0017).  The weights' remainders in products of
      // their own would leave that one rounding, and take 861 for 700 us for a prompt of 8192
      // rows, 447 for 440 for 256 requests of 512 to 4096 tokens, 46 for 44.5 for 64 trees.  V's
      // fragment is two transposing reads of 4 tokens x 16 d.  Rows 8 apart share a swizzle, so a
      // lane has one address per 32 d and the rest are immediates.
      const int j = lane & 15, g = (lane >> 4) & 1, r0 = 4 * h + (j >> 2);
      const uint32_t vrow = here(vs + r0 * L::RB + (j & 1) * 8);
      const uint32_t vx = here((uint32_t)((2 * g + ((j >> 1) & 1)) ^ L::vswz(r0)) << 4);
      union {
        s16x4 half[2];
        bf16x8 all;
      } a[2][ND];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            a[st][dt].half[b] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (DSPARK_LDS s16x4*)(uintptr_t)(vrow + (vx ^ (uint32_t)(dt << 6)) + 8 * (2 * st + b) * L::RB));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        bf16x8 pb;
#pragma unroll
        for (int e = 0; e < 8; ++e) pb[e] = (__bf16)sc[8 * st + e];
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
          o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[st][dt].all, pb, o[dt], 0, 0, 0);
      }
    } else {
      // register r is token reg_row(r, h): the two halves' tokens are one step's pair
      const uint32_t vrow = here(vs + 4 * h * L::RB + (n & 3) * 4);
      const uint32_t vx = here((uint32_t)((n >> 2) ^ L::vswz(4 * h)) << 4);
#pragma unroll
      for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) {
          const float a = lds_get<float>(vrow + (vx ^ (uint32_t)(dt << 7)) + reg_row(r, 0) * L::RB);
          o[dt] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, sc[r], o[dt], 0, 0, 0);
        }
    }
  }

  // V rows behind the last token become 0 (they may hold anything, and 0 * NaN is none);
  // whether the rows left hold infinities or NaN.  Waves that share a tile all do it alike.
  __device__ __forceinline__ bool clean_values(int t0, uint32_t vs) const {
    bool bad = false;
#pragma unroll 1
    for (int i = lane; i < L::NC * kWave; i += kWave) {
      const uint32_t at = vs + i * 16;
      if (t0 + i / L::CPR >= len) lds_put<u32x4>(at, u32x4{0, 0, 0, 0});
      const u32x4 x = lds_get<u32x4>(at);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        bad = bad || (x[w] & 0x7F800000u) == 0x7F800000u;
        if (L::kBf) bad = bad || (x[w] & 0x7F80u) == 0x7F80u;
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    return __ballot(bad) != 0;
  }

  // The product with a V tile that holds infinities or NaN: a weight of 0 leaves a token out
  // (a matrix product would make 0 * inf of it).  The weights go through the K tile's LDS,
  // which the scores no longer need, a wave at a time; the V tile is 0 afterwards, so that
  // values() adds nothing.
  __device__ __forceinline__ void odd_values(uint32_t ks, uint32_t vs, const f32x16& sc) {
#pragma unroll 1
    for (int w = 0; w < NR; ++w) {
      if (NR > 1) {
        stage_barrier();  // every wave has its scores, and is done with the weights before
        if (w != wave) continue;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) lds_put<float>(ks + (reg_row(r, h) * 32 + n) * 4, sc[r]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
      for (int t = 0; t < kTok; ++t) {
        const float wt = lds_get<float>(ks + (t * 32 + n) * 4);
        if (wt == 0.0f) continue;
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int d = 32 * dt + reg_row(r, h);
            const uint32_t at =
                vs + t * L::RB + (((d * L::kE / 16) ^ L::vswz(t)) << 4) + (d * L::kE) % 16;
            float x;
            if constexpr (L::kBf)
              x = bf16_to_f32(lds_get<uint16_t>(at));
            else
              x = lds_get<float>(at);
            o[dt][r] = fmaf(wt, x, o[dt][r]);
          }
          asm volatile("" ::: "memory");
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    if (NR > 1) stage_barrier();
#pragma unroll 1
    for (int i = lane; i < L::NC * kWave; i += kWave) lds_put<u32x4>(vs + i * 16, u32x4{0, 0, 0, 0});
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // the queries and what they see; rows m0 .. m0 + 31 of the request's M
  __device__ __forceinline__ void begin(const AttReq& rq, int q, int head, int m0, int M) {
    ctx = rq.ctx;
    pages = p.table + (int64_t)q * p.max_pages;
    kh = static_cast<const char*>(p.k) + head * p.head_b;
    vh = static_cast<const char*>(p.v) + head * p.head_b;
    len = rq.ctx + rq.n;
    last_page = (len - 1) >> p.lg;
    seen = uni(rq.ctx + 1 + (p.anc ? 0 : node_of(p, m0)));
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) o[dt] = f32x16{};
  }
  __device__ __forceinline__ void queries(const AttReq& rq, int head, int m0, int M) {
    const int mi = m0 + n;
    const bool live = mi < M;
    const int i = live ? node_of(p, mi) : 0, g = live ? group_of(p, mi) : 0;
    const char* src = static_cast<const char*>(p.q) +
                      ((int64_t)(rq.a + i) * p.q_row + (int64_t)(head * p.G + g) * D) * L::kE;
#pragma unroll
    for (int st = 0; st < L::KSTEPS; ++st) {
      qf[st] = u32x4{0, 0, 0, 0};
      if (live) qf[st] = *reinterpret_cast<const u32x4*>(src + (2 * st + h) * 16);
    }
    node = i;
    see = p.anc ? p.anc[rq.a + i] : 0;
  }

  // tokens of rounds r0 .. r0 + nr of the row tile that starts at query row m0
  __device__ __forceinline__ void segment(const AttReq& rq, int q, int head, int m0, int r0, int nr) {
    const int M = rq.n * p.G;
    begin(rq, q, head, m0, M);
    int end = uni(att_end(p, rq, m0 + NR * kRows));
    end = end < (r0 + nr) * F::ROUND ? end : (r0 + nr) * F::ROUND;
    const int first = r0 * F::ROUND + (NR == 1 ? wave * kTok : 0);
    const int nt = first < end ? (end - first + F::ROUND - 1) / F::ROUND : 0;
    if constexpr (NR == 1)
      tokens_apart(rq, head, m0, M, first, nt);
    else
      rows_apart(rq, head, m0 + wave * kRows, M, first, nt);
    l = half_sum(l);
  }

  // NR 1: this wave's tiles, kRound tokens apart, in its own LDS
  __device__ __forceinline__ void tokens_apart(const AttReq& rq, int head, int m0, int M, int first,
                                               int nt) {
    int pg[CG];
    if (nt > 0) {
      page_ids(first, pg);
      known(pg);
      copy<false>(first, pg, 0);
      copy<true>(first, pg, 0);
      page_ids(first + F::ROUND, pg);  // past the end: the last page's
    }
    queries(rq, head, m0, M);
    for (int k = 0; k < nt; ++k) {
      const int t0 = first + k * F::ROUND, t1 = t0 + F::ROUND;
      const bool more = k + 1 < nt, edge = t0 + kTok > seen;
      const int s = F::STAGES == 2 ? k & 1 : 0;
      const uint32_t ks = base + s * F::TILE, vs = ks + L::BYTES;
      if (F::STAGES == 1) {
        vm_wait<NC>();  // K's tile; V's is waited for before O
      } else if (more) {
        known(pg);
        copy<false>(t1, pg, s ^ 1);
        copy<true>(t1, pg, s ^ 1);
        page_ids(t1 + F::ROUND, pg);
        vm_wait<2 * NC>();
      } else {
        vm_wait<0>();
      }
      f32x16 sc;
      scores(ks, sc);
      if (edge) mask(t0, sc);
      if (F::STAGES == 1) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (more && !edge) {  // (an edge tile may still need K's buffer)
          known(pg);
          copy<false>(t1, pg, 0);
        }
      }
      weigh(sc);
      if (F::STAGES == 1) {
        if (more && !edge)
          vm_wait<NC>();
        else
          vm_wait<0>();
      }
      if (edge && clean_values(t0, vs)) odd_values(ks, vs, sc);
      values(vs, sc);
      // the stage is free once its reads have returned
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (F::STAGES == 1 && more) {
        if (edge) {
          known(pg);
          copy<false>(t1, pg, 0);
        }
        copy<true>(t1, pg, 0);
        page_ids(t1 + F::ROUND, pg);
      }
    }
  }

  // NR > 1: tiles that all waves share
  __device__ __forceinline__ void rows_apart(const AttReq& rq, int head, int m0, int M, int first,
                                             int nt) {
    constexpr int AHEAD = F::STAGES - 1;
    int pg[CG];
    page_ids(first, pg);
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (a < nt) {
        known(pg);
        copy<false>(first + a * kTok, pg, a);
        copy<true>(first + a * kTok, pg, a);
      }
      page_ids(first + (a + 1) * kTok, pg);
    }
    queries(rq, head, m0, M);
    const bool live = m0 < M;
    int s = 0, s_next = AHEAD;
    for (int k = 0; k < nt; ++k) {
      const int t0 = first + k * kTok;
      if (k + AHEAD - 1 < nt)  // this wave's copies of the tile; later ones stay under way
        vm_wait<(AHEAD - 1) * 2 * NC>();
      else
        vm_wait<0>();
      stage_barrier();  // the whole tile is there, and every wave is done with the one before
      if (k + AHEAD < nt) {
        known(pg);
        copy<false>(t0 + AHEAD * kTok, pg, s_next);
        copy<true>(t0 + AHEAD * kTok, pg, s_next);
        page_ids(t0 + (AHEAD + 1) * kTok, pg);
      }
      const uint32_t ks = base + s * F::TILE, vs = ks + L::BYTES;
      f32x16 sc = f32x16{};
      if (live) {
        scores(ks, sc);
        if (t0 + kTok > seen) mask(t0, sc);
        // the exponentials first: the SIMD's other wave has products to issue meanwhile (4096 rows
        // at D = 64: 164 without, 158 us; 8192 at D = 128: 697, 688)
        __builtin_amdgcn_s_setprio(1);
        weigh(sc);
        __builtin_amdgcn_s_setprio(0);
      }
      if (t0 + kTok > seen && clean_values(t0, vs)) odd_values(ks, vs, sc);
      if (live) values(vs, sc);
      s = s + 1 == F::STAGES ? 0 : s + 1;
      s_next = s_next + 1 == F::STAGES ? 0 : s_next + 1;
    }
    stage_barrier();  // the next segment's copies overwrite the stages
  }
};

// Where the rounds of a head go.  Each row tile of each request has a list of SETUP + rounds
// units, SETUP of them for what a list costs beside its tokens (the queries, the first
// tile's wait, the merge of the waves, the output), which no tokens stand for; all lists, head
// after head, are one row of units, cut evenly: workgroup b begins at unit begin(b).  A cut
// costs the later piece's set-up and the join; moving cuts to a near end lost more in balance
// than it saved in joins (120 requests of 180 to 254 tokens in tables of more, lists of 6 to 8
// rounds: 32 us with these kept whole, 27 cut), unless no list need be cut at all: block tables of
// no more than kWhole rounds leave every list whole and launch no join.  Kernels alone, whole
// against cut, bf16, tables of 256 tokens, 32 heads on 8: 32 requests 15.4 and 17.1 us, 120 23.8
// and 27.5, 512 79 and 84; 17 rows, tables of 128: 32 requests 16.8 and 24.2.  In float a list's
// products take longer, and it is the call, a launch shorter, that gains: 4 requests of up to 204
// tokens 17 against 18 to 20 us a call, 19 against 13 captured in a graph.  A list that is cut has
// its pieces in the workspace; the first workgroup that begins inside one says so in joint[b].
constexpr int kWhole = 4;

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

template <class T, int D, int NR>
__global__ void __launch_bounds__((Fit<T, D, NR>::THREADS), (Fit<T, D, NR>::PER_SIMD))
    attention_kernel(AttParams p) {
  using F = Fit<T, D, NR>;
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
    return (end + kRound - 1) / kRound + kSetup;
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
  const int64_t W = uni(total_s), U = W * p.Hkv;
  const int64_t P = U < gridDim.x ? U : gridDim.x;
  if (b >= P) return;
  AttShares<kSetup> cut;
  cut.share = quotient(U, P);
  cut.more = U - cut.share * P;
  cut.whole = p.whole;
  const int64_t u0 = cut.begin(b), u1 = cut.begin(b + 1);
  int head = (int)quotient(u0, W);
  {
    const int64_t w = u0 - head * W;
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
  AttWave<T, D, NR> wv(p, wave, base);
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
    if constexpr (NR > 1) {
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
    } else {
      // The waves' sums, through LDS: each gives the other half of its O, and finishes its own
      // half.
      constexpr int HD = ND / 2, kGive = (HD * 16 + 2) * 64;
      float* x = reinterpret_cast<float*>(lds);
      auto give = [&](auto self) {
        constexpr int W = decltype(self)::value;
        float* y = x + W * kGive + lane;
#pragma unroll
        for (int i = 0; i < HD; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) y[(i * 16 + r) * 64] = wv.o[(1 - W) * HD + i][r];
        y[HD * 16 * 64] = wv.m;
        y[(HD * 16 + 1) * 64] = wv.l;
      };
      auto finish = [&](auto self) {
        constexpr int W = decltype(self)::value;
        const float* y = x + (1 - W) * kGive + lane;
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
              z[e] = wv.o[W * HD + i][r] * f1 + y[(i * 16 + r) * 64] * f2;
            }
            put(wv.n, 32 * (W * HD + i) + 8 * r4 + 4 * wv.h, z);
          }
        if (W == 0 && wv.h == 0) put_sums(wv.n, mm, ll);
      };
      using First = std::integral_constant<int, 0>;
      using Second = std::integral_constant<int, 1>;
      __syncthreads();
      if (wave == 0) give(First{});
      else give(Second{});
      __syncthreads();
      if (wave == 0) finish(First{});
      else finish(Second{});
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
template <class T, int D, int NR, bool DEEP>
__global__ void __launch_bounds__(256) attention_join_kernel(AttParams p, bool across) {
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
        // NaN where the row's scores are
        f = __builtin_amdgcn_exp2f(pm[u] - ref);
        l = fmaf(pl[u], f, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = f != 0.0f ? fmaf(x[u][e], f, acc[e]) : acc[e];
      }
      m = mn;
    };
    // few loads where there are few pieces: those of missing ones take their time too
    constexpr int kMost = DEEP ? 12 : 4;
    if (jt.count <= 2 * NP) {
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
template <class T_, int D_, int NR_>
struct Variant {
  using T = T_;
  static constexpr int D = D_, NR = NR_;
  // workgroups: as many as stay resident
  static int grid() { return device_cus() * Fit<T, D, NR>::PER_CU; }
};

// f(variant) of the variant that runs these shapes: as many waves over query rows as a
// request's rows (rows / R, the bound the host knows, times heads to a cache head) fill, so
// that the cache is read once for all of them.  33 to 64 rows at D = 128 run four waves too,
// two of them only copying: half the workgroups cut half the lists (440 against 453 us for 256
// requests of 512 to 4096 tokens, 26 against 33 us for one of 16000, 149 against 158 us for
// 64 of 500 to 4000, 46 us both for 64 of 100 to 2048); at D = 64, with half the bytes
// under way, that costs more than it saves (89 against 77 us).  Float has only the first
// variant: its products, sixteen times as slow, bound it, and rows that are not there cost it
// as much as others (22 requests of up to 56 rows: 169 us so, 214 us with two waves over
// rows; 16 of 128 rows: 137 against 131 us).
template <class F>
static auto att_variant(int R, int rows, int G, int D, dspark_dtype dt, F f) {
  if (dt == DSPARK_F32) return D == 64 ? f(Variant<float, 64, 1>{}) : f(Variant<float, 128, 1>{});
  const int64_t m = (int64_t)((rows + R - 1) / R) * G;
  if (D == 64) {
    if (m <= 32) return f(Variant<uint16_t, 64, 1>{});
    return m <= 64 ? f(Variant<uint16_t, 64, 2>{}) : f(Variant<uint16_t, 64, 4>{});
  }
  return m <= 32 ? f(Variant<uint16_t, 128, 1>{}) : f(Variant<uint16_t, 128, 4>{});
}

static size_t att_carve(AttParams& p, void* ws, int R, int rows, int G, int D, dspark_dtype dt) {
  Carve cv(ws);
  att_variant(R, rows, G, D, dt, [&](auto v) {
    const size_t grid = (size_t)v.grid();
    p.joint = cv.take<AttJoint>(grid);
    p.part = cv.take<float>(grid * 2 * kRows * v.NR * (v.D + 2));
    return 0;
  });
  return cv.bytes();
}

static bool att_dims_ok(int R, int rows, int Hq, int Hkv, int D, dspark_dtype dt) {
  return R >= 0 && R <= kMaxRequests && rows >= 0 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
         (D == 64 || D == 128) && (dt == DSPARK_F32 || dt == DSPARK_BF16) &&
         (int64_t)rows * Hq <= ((int64_t)1 << 31) - 1024;  // ends of row tiles in 31 bits
}

template <class T, int D, int NR>
static int att_launch(AttParams p, hipStream_t stream) {
  using F = Fit<T, D, NR>;
  static std::atomic<uint64_t> raised;
  auto kern = attention_kernel<T, D, NR>;
  const int grid = Variant<T, D, NR>::grid();
  ensure_dynamic_lds(reinterpret_cast<const void*>(kern), F::LDS, raised);
  p.whole = ((int64_t)p.max_pages << p.lg) <= kWhole * F::ROUND ? kWhole : 0;
  kern<<<grid, F::THREADS, F::LDS, stream>>>(p);
  if (p.whole > 0) return launch_status();
  // a wave per row of a row tile, as far as the host knows how many rows there are
  const int64_t m = (int64_t)((p.rows + p.R - 1) / p.R) * p.G;
  const int slices = m < kRows * NR ? (int)(m + 3) / 4 : 8 * NR;
  // Workgroups go to the eight dies in turn.  The joints lie some workgroups apart, often all
  // with the same remainder by 8 or two of them, so where there is much to read (112 row tiles
  // of 128: 12 to 29 us) neighbours are the slices of one joint (13 us); where there is little,
  // one die is as good (two requests of 5 rows: 8 against 11 us).
  const bool across = slices >= 8;
  const dim3 blocks = across ? dim3(slices, grid) : dim3(grid, slices);
  if (grid / p.R / p.Hkv >= 16)  // pieces of a list, were there one row tile a request
    attention_join_kernel<T, D, NR, true><<<blocks, 256, 0, stream>>>(p, across);
  else
    attention_join_kernel<T, D, NR, false><<<blocks, 256, 0, stream>>>(p, across);
  return launch_status();
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_tree_attention_workspace_bytes(int R, int rows, int Hq, int Hkv, int D,
                                                        dspark_dtype dt) {
  if (!att_dims_ok(R, rows, Hq, Hkv, D, dt) || R == 0) return 0;
  AttParams p{};
  return att_carve(p, nullptr, R, rows, Hq / Hkv, D, dt);
}

extern "C" int dspark_tree_attention(int R, int rows, int Hq, int Hkv, int D, dspark_dtype dt,
                                     int page_size, int max_pages, int n_pages, const void* q,
                                     int64_t q_row, const void* k_cache, const void* v_cache,
                                     int64_t page_stride, int64_t head_stride, int64_t tok_stride,
                                     const int32_t* table, const int32_t* ctx,
                                     const int32_t* row_off, const uint64_t* anc, float scale,
                                     void* o, float* lse, int32_t* dev_status, void* ws,
                                     size_t ws_bytes, hipStream_t stream) {
  if (!att_dims_ok(R, rows, Hq, Hkv, D, dt) || max_pages < 1 || !pages_ok(page_size, n_pages) ||
      !table_ok(page_size, max_pages) || !(scale > 0.0f) ||
      !(scale * kLog2e <= FLT_MAX))
    return DSPARK_EINVAL;
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  if (!stride_ok(q_row, e) || !stride_ok(page_stride, e) || !stride_ok(head_stride, e) ||
      !stride_ok(tok_stride, e) || tok_stride > (1 << 24))
    return DSPARK_EINVAL;
  if (R == 0 || rows == 0) return DSPARK_OK;
  if (!q || !k_cache || !v_cache || !table || !ctx || !row_off || !o || !ws || !aligned16(q) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(ws))
    return DSPARK_EINVAL;
  // a row's heads may be read after another's output is written
  const size_t row_bytes = (size_t)Hq * D * e;
  if (overlap(q, (size_t)(rows - 1) * q_row * e + row_bytes, o, rows * row_bytes))
    return DSPARK_EINVAL;
  AttParams p{};
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
  p.page_b = page_stride * (int64_t)e;
  p.head_b = head_stride * (int64_t)e;
  p.tok_b = tok_stride * (int64_t)e;
  p.table = table;
  p.ctx = ctx;
  p.row_off = row_off;
  p.anc = anc;
  p.scale = scale;
  p.o = o;
  p.lse = lse;
  p.status = dev_status;
  if (ws_bytes < att_carve(p, ws, R, rows, p.G, D, dt)) return DSPARK_EWORKSPACE;
  return att_variant(R, rows, p.G, D, dt, [&](auto v) {
    return att_launch<typename decltype(v)::T, decltype(v)::D, decltype(v)::NR>(p, stream);
  });
}
