// attention_wave.h -- how a wave takes its tiles of 32 tokens from LDS: the tiles' geometry there, the two
// products, and, of a cache of bf16 or float, the copies that fill them.
#pragma once

#include "attention.h"

namespace dspark {

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
  static constexpr int WHOLE = 4 * ROUND;  // tokens of block tables that leave every list whole
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

// What one wave holds: 32 query rows, and its running m, l and O of them.
// L_: the tile's geometry in LDS.
template <class T, int D, int NR_, class L_ = Tile<T, D>>
struct AttWave : AttRows<D> {
  using Params = AttParams;
  using Out = T;
  using F = Fit<T, D, NR_>;
  static constexpr int kD = D, kNR = NR_;
  static constexpr bool kMix = false;
  static constexpr bool kNan = false;  // NaN of a value reaches all rows that see it, whatever its weight
  // tokens of a round of a request with M query rows to a cache head
  static __device__ constexpr int round(int) { return F::ROUND; }

  using L = L_;
  static constexpr int NR = NR_, ND = D / 32;
  // rows of a tile that this wave copies, from row `mine` on, and groups of 8 of them
  static constexpr int CROWS = kTok / NR, CG = CROWS / 8, NC = L::NC / NR;

  using B = AttRows<D>;
  using B::h;
  using B::l;
  using B::lane;
  using B::len;
  using B::n;
  using B::node;
  using B::o;
  using B::p;
  using B::see;
  using B::seen;
  int wave;
  int mine;                 // first row of a tile that this wave copies
  uint32_t base;            // LDS of its stages
  // segment
  const char *kh, *vh;      // cache bases of the head
  const int32_t* pages;     // the request's block table
  int last_page;            // page of the last token
  u32x4 qf[L::KSTEPS];

  __device__ __forceinline__ AttWave(const AttParams& p_, int wave_, uint32_t lds)
      : B(p_), wave(wave_), mine(NR == 1 ? 0 : wave_ * CROWS),
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

  // The product with a V tile that holds infinities or NaN: a weight of 0 (MARKED: below 0) leaves a
  // token out (a matrix product would make 0 * inf of it).  The weights go through the K tile's LDS,
  // which the scores no longer need, a wave at a time; the V tile is 0 afterwards, so that
  // values() adds nothing.
  template <bool MARKED = false>
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
        if (MARKED ? wt < 0.0f : wt == 0.0f) continue;
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
  __device__ __forceinline__ void begin(const AttReq& rq, int q, int head, int m0) {
    B::begin_rows(rq, m0);
    pages = p.table + (int64_t)q * p.max_pages;
    kh = static_cast<const char*>(p.k) + head * p.head_b;
    vh = static_cast<const char*>(p.v) + head * p.head_b;
    last_page = (len - 1) >> p.lg;
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
    begin(rq, q, head, m0);
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
      if (edge) B::mask(t0, sc);
      if (F::STAGES == 1) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (more && !edge) {  // (an edge tile may still need K's buffer)
          known(pg);
          copy<false>(t1, pg, 0);
        }
      }
      B::weigh(sc);
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
        if (t0 + kTok > seen) B::mask(t0, sc);
        // the exponentials first: the SIMD's other wave has products to issue meanwhile (4096 rows
        // at D = 64: 164 without, 158 us; 8192 at D = 128: 697, 688)
        __builtin_amdgcn_s_setprio(1);
        B::weigh(sc);
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

}  // namespace dspark
