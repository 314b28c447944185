// attention4.hip -- attention of a step's rows over a paged cache held in 4 bits.
//
// The products, the softmax and the cutting of the work are attention.h's.  What a cache of 4 bits
// changes is how K and V reach the matrix cores: their values, E2M1 times a power of two, are bf16
// numbers as they are (two bits of mantissa), so gfx950's conversions, two elements an instruction,
// the power included, make exact operands of them, and
//   S^T = K Q^T      O^T += V^T P^T
// are bf16 products whatever the queries' type: bf16 queries are one term, float ones the sum of three
// bf16 terms of 8 bits each, exactly, and so are the weights P beside float queries.
//
// An element is 17/32 bytes (scales included), a quarter of bf16's, so at few rows HBM wants a
// tile of 32 tokens in a quarter of the time, and the vector work of a tile (64 conversions a
// lane at D = 128, and the softmax) is what has to fit into it.
//   - K goes from memory to registers to the product: a lane holds half of a token's head, and as a sum
//     over d may be taken in any order, the queries are loaded to match.
//   - V needs tokens where memory has d, so it passes through LDS as bf16, by transposing reads.
// Measured, bf16, D = 128, both kernels: 256 requests of 512 to 4096 tokens, 32 heads on 8, up to nine rows
// (664 MB) 166 us, 4.0 TB/s where a copy gets 5.0 (vector instructions issue for 46 % of the time, LDS is
// busy for 19 %, the matrix cores for 24 %); with three rows at most 147, with nine each, 36 to a cache
// head, 235.  Two single tokens over 100001 to 131071, 40 heads on 8 (251 MB) 62 us; 64 trees over 100 to
// 2048, 20 heads on 4 (41 MB) 26 to 29.  Prompts are bound by the softmax's vector work as over bf16: 2048
// rows behind 4048 tokens 230 us, 740 TFLOP/s of the pairs seen, 8192 rows 655, 840.
#include "attention_wave.h"
#include "fp4.h"

namespace dspark {

// Strides in bytes.  Within a page, and from page to page, they fit 32 bits, so that a lane's address
// takes one multiplication of 32 bits each.
struct Att4Params : AttParams {
  uint32_t page_b4, tok_b4;
  const uint8_t* scales;
  uint32_t s_page, s_tok;
  int64_t s_head;
};

// How a variant sits on a CU.  A workgroup's two waves have their tiles to themselves.  Up to 32
// query rows they take 32 tokens each and merge at the end; more, they take 32 rows each, and the
// same tokens, which HBM sees once.  (One wave converting the keys for both and the other the values
// saves half of the conversions and costs a barrier a tile: 256 requests of 63 query rows 271 against 264
// us, 64 of 45 over 100 to 2048 tokens 36.5 and 35.)  TERMS: bf16 terms of a query and a weight.
template <int D, int TERMS>
struct Fit4 {
  static constexpr bool kBf = TERMS == 1;  // the output's type
  static constexpr int WAVES = 2;
  static constexpr int THREADS = WAVES * kWave;
  static constexpr int ROUND = kTok;  // of a list of 64 rows
  static constexpr int WHOLE = 256;   // tokens of block tables that leave every list whole
  static constexpr int SETUP = 3;
  static constexpr int TILE = kTok * D * 2;  // V as bf16
  static constexpr int MERGE = (D / 4 + 2) * kWave * 4;  // half of a wave's O, m and l
  static constexpr int LDS = WAVES * (TILE > MERGE ? TILE : MERGE) + 256;
  // Waves a SIMD: at D = 64 registers allow three (256 requests of 512 to 4096 tokens 105 us, two 121; one
  // token over 115000 41 and 47).  At D = 128 three can be had by taking addresses anew for each tile,
  // and lose: 178 against 168 us there.
  static constexpr int PER_SIMD = D == 64 ? (TERMS == 1 ? 3 : 2) : (TERMS == 1 ? 2 : 1);
  static constexpr int PER_CU = 4 * PER_SIMD / WAVES;
};

// How far V's 16-byte chunks of row t of a tile are moved, by exclusive or.  LDS takes writes of 16 bytes
// a lane from 8 lanes at a time, over 32 banks, and here those hold one chunk of 8 rows; transposing reads
// from 32 lanes, over 64 banks, 4 neighbouring chunks of 4 rows.  Neither meets itself.
template <int D>
__host__ __device__ constexpr int vswz4(int t) {
  return D == 128 ? (t & 1) << 2 ^ ((t >> 1) & 1) * 10 ^ ((t >> 2) & 1) : (t & 3) << 1 ^ ((t >> 2) & 1);
}

// What a lane holds of a tile: half h of token n's keys and values, and their powers.
template <int D>
struct Raw4 {
  static constexpr int N = D / 64;  // 16-byte pieces of half a row
  uint4 k[N], v[N];
  uint2 s;  // the token's scale bytes: keys', then values'
};

template <int D, int TERMS>
struct Att4Wave : AttRows<D> {
  using Params = Att4Params;
  using Out = typename std::conditional<TERMS == 1, uint16_t, float>::type;
  using F = Fit4<D, TERMS>;
  static constexpr int kD = D, kNR = 2;
  static constexpr bool kMix = true, kNan = true;
  static __device__ constexpr int round(int M) { return M <= kRows ? 2 * kTok : F::ROUND; }
  static constexpr int ND = D / 32, KSTEPS = D / 16, RB = D * 2, WORDS = D / 16;

  using B = AttRows<D>;
  using B::h;
  using B::l;
  using B::lane;
  using B::len;
  using B::n;
  using B::node;
  using B::o;
  using B::see;
  using B::seen;
  const Att4Params& p;
  int wave_;
  uint32_t base;            // LDS of its V tile, 256-byte aligned: chunks are found by exclusive or
  // segment
  const char *kh, *vh;      // cache bases of the head
  const uint8_t* sh;
  const int32_t* pages;     // the request's block table
  int last_page;            // page of the last token
  u32x4 qf[TERMS][KSTEPS];

  __device__ __forceinline__ Att4Wave(const Att4Params& p_, int wave, uint32_t lds)
      : B(p_), p(p_), wave_(wave), base(((lds + 255) & ~255u) + wave * F::TILE) {}

  // V's tile: row t is token t, 16-byte chunk c of it at chunk c ^ swz(t)
  static __device__ __forceinline__ int swz(int t) { return vswz4<D>(t); }

  // Pages of tile t0, a page per 8 tokens (aligned, so they share one); past the last token, its page.
  // Scalar loads: they are waited for apart from the vector loads under way.
  struct Pages {
    int a, b, c, d;
  };
  __device__ __forceinline__ int page_id(int t) const {
    const int i = t >> p.lg;
    return sload(pages, i < last_page ? i : last_page);
  }
  __device__ __forceinline__ Pages page_ids(int t0) const {
    return {page_id(t0), page_id(t0 + 8), page_id(t0 + 16), page_id(t0 + 24)};
  }

  // The loads of tile t0.  Rows past the last token are read inside its page, and are never used.
  __device__ __forceinline__ void load(int t0, Pages id, Raw4<D>& x) const {
    const int lo = n & 8 ? id.b : id.a, hi = n & 8 ? id.d : id.c;
    uint32_t pg = (uint32_t)(n & 16 ? hi : lo);
    if (pg >= (uint32_t)p.n_pages) {
      raise_fault(p.status, DSPARK_FAULT_PAGE);
      pg = 0;
    }
    const uint32_t tok = (uint32_t)(t0 + n) & ((1u << p.lg) - 1);
    const uint64_t at = (uint64_t)pg * p.page_b4 + (tok * p.tok_b4 + h * (D / 4));
    const uint4* k = reinterpret_cast<const uint4*>(kh + at);
    const uint4* v = reinterpret_cast<const uint4*>(vh + at);
#pragma unroll
    for (int i = 0; i < Raw4<D>::N; ++i) {
      x.k[i] = k[i];
      x.v[i] = v[i];
    }
    const uint8_t* s = sh + ((uint64_t)pg * p.s_page + tok * p.s_tok);
    if constexpr (D == 128)
      x.s = *reinterpret_cast<const uint2*>(s);
    else
      x.s.x = *reinterpret_cast<const uint32_t*>(s);
  }
  // byte of the group that 8-element piece w of the lane's half lies in
  static __device__ __forceinline__ uint32_t byte_of(const Raw4<D>& x, int h, bool values, int w) {
    if (D == 128) return ((values ? x.s.y : x.s.x) >> (16 * h + 8 * (w / 4))) & 255u;
    return (x.s.x >> (16 * values + 8 * h)) & 255u;
  }

  // S^T of a tile, and its V, as bf16, to LDS.  Step s of the product takes d = 8 s .. 8 s + 7 of either
  // half; V's conversions go between the steps, which have products to wait for.
  // EDGE: in V a token behind the last, and a group that reads NaN, are 0 (0 * NaN is none); sick[dt]
  // has a bit for each of the 32 tokens whose group dt was NaN.
  template <bool EDGE>
  __device__ __forceinline__ void scores(int t0, const Raw4<D>& x, f32x16& sc, uint32_t (&sick)[ND]) const {
    const uint32_t row = base + n * RB + ((h * (D / 16) ^ swz(n)) << 4);
    const uint32_t *k = reinterpret_cast<const uint32_t*>(x.k), *v = reinterpret_cast<const uint32_t*>(x.v);
    if (EDGE) {
#pragma unroll
      for (int g = 0; g < ND; ++g) sick[g] = 0;
    }
    sc = f32x16{};
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      const uint4 f = fp4_bf16x8(k[s], fp4_scale(byte_of(x, h, false, s)));
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
        sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, f),
                                                     __builtin_bit_cast(bf16x8, qf[t][s]), sc, 0, 0, 0);
      uint32_t code = v[s], byte = byte_of(x, h, true, s);
      if (EDGE) {
        const bool behind = t0 + n >= len, odd = byte >= 253;
        if (s % 4 == 0) {
          const uint64_t who = __ballot(odd && !behind);  // halves have different groups
          sick[s / 4] |= (uint32_t)who;
          sick[ND / 2 + s / 4] |= (uint32_t)(who >> 32);
        }
        code = behind || odd ? 0 : code;
        byte = behind || odd ? 127 : byte;
      }
      lds_put<u32x4>(row ^ (uint32_t)(s << 4), __builtin_bit_cast(u32x4, fp4_bf16x8(code, fp4_scale(byte))));
    }
  }

  // O^T += V^T P^T, 16 tokens a step: registers 8 st .. 8 st + 7 are the lane's 8 tokens of it.  With
  // bf16 queries the weights are rounded to bf16, each off by 2^-8 of itself at most, as o is when
  // stored; with float ones they are three terms.
  __device__ __forceinline__ void values(f32x16& sc) {
    const int j = lane & 15, g = (lane >> 4) & 1, r0 = 4 * h + (j >> 2);
    const uint32_t at = here(base + r0 * RB + (j & 1) * 8 + (((2 * g + ((j >> 1) & 1)) ^ swz(r0)) << 4));
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      union {
        s16x4 half[2];
        bf16x8 all;
      } a[ND];
#pragma unroll
      for (int dt = 0; dt < ND; ++dt)
#pragma unroll
        for (int b = 0; b < 2; ++b)  // (rows 8 apart share a swizzle)
          a[dt].half[b] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (DSPARK_LDS s16x4*)(uintptr_t)((at ^ (uint32_t)(dt << 6)) + 8 * (2 * st + b) * RB));
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        bf16x8 pb;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = sc[8 * st + e];
          if (TERMS == 1) {
            pb[e] = (__bf16)w;
          } else {
            const float top = t + 1 < TERMS ? __uint_as_float(__float_as_uint(w) & 0xFFFF0000u) : w;
            pb[e] = (__bf16)top;
            sc[8 * st + e] = w - top;
          }
        }
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
          o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[dt].all, pb, o[dt], 0, 0, 0);
      }
    }
  }

  // the rows that see a token whose group was NaN have NaN there
  __device__ __forceinline__ void spread(uint32_t vis, const uint32_t (&sick)[ND]) {
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) {
      // the half-waves hold 16 tokens of a row each
      const uint32_t mine = vis & (sick[dt] >> 4 * h) & 0x0F0F0F0Fu;
      const auto both = __builtin_amdgcn_permlane32_swap(mine, mine, false, false);
      if (both[0] | both[1]) {
#pragma unroll
        for (int r = 0; r < 16; ++r) o[dt][r] = __uint_as_float(0x7FC00000u);
      }
    }
  }

  // rows m0 .. m0 + 31 of the request's M: d of half h in a row, 8 a step
  __device__ __forceinline__ void queries(const AttReq& rq, int head, int m0, int M) {
    const int mi = m0 + n;
    const bool live = mi < M;
    const int i = live ? node_of(p, mi) : 0, g = live ? group_of(p, mi) : 0;
    const Out* src = static_cast<const Out*>(p.q) + (int64_t)(rq.a + i) * p.q_row +
                     (int64_t)(head * p.G + g) * D + h * (D / 2);
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      if constexpr (TERMS == 1) {
        qf[0][s] = u32x4{0, 0, 0, 0};
        if (live) qf[0][s] = *reinterpret_cast<const u32x4*>(src + 8 * s);
      } else {
        float x[8];
        if (live)
          ld8(src + 8 * s, x);
        else
          for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        // 8 bits at a time, the last rounded to what is left: the sum is the float.  An infinity or NaN
        // is its first term's.
        uint16_t t[TERMS][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool odd = (__float_as_uint(x[e]) & 0x7F800000u) == 0x7F800000u;
          float w = x[e];
#pragma unroll
          for (int k = 0; k < TERMS; ++k) {
            const uint32_t u = __float_as_uint(w);
            // (a NaN keeps a bit that stays)
            t[k][e] = (uint16_t)(u >> 16) | (w != w ? 0x40 : 0);
            w = odd ? 0.0f : w - __uint_as_float(u & 0xFFFF0000u);
          }
        }
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) qf[k][s][e] = (uint32_t)t[k][2 * e] | (uint32_t)t[k][2 * e + 1] << 16;
      }
    }
    node = i;
    see = p.anc ? p.anc[rq.a + i] : 0;
  }

  // one tile; next(): the loads that may go out once its own registers are free
  template <class Next>
  __device__ __forceinline__ void tile(int t0, const Raw4<D>& x, Next next) {
    const bool edge = t0 + kTok > seen;
    f32x16 sc;
    uint32_t vis = 0, sick[ND];
    // Products and conversions go before another wave's exponentials: 256 requests of 36 query rows 242 ->
    // 233 us, of 63 264 -> 256, of up to nine rows 168 -> 166.
    __builtin_amdgcn_s_setprio(1);
    // (a wave's LDS instructions take effect in their order: its reads follow its writes without a
    // wait, and the next tile's writes the reads; the fences keep the compiler to that order)
    if (edge) {
      scores<true>(t0, x, sc, sick);
      vis = B::visible(t0);
#pragma unroll
      for (int r = 0; r < 16; ++r) sc[r] = vis & (1u << reg_row(r, 0)) ? sc[r] : -INFINITY;
    } else {
      scores<false>(t0, x, sc, sick);
    }
    next();
    __builtin_amdgcn_s_setprio(0);
    B::weigh(sc);
    __builtin_amdgcn_s_setprio(1);
    asm volatile("" ::: "memory");
    values(sc);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_setprio(0);
    if (edge) spread(vis, sick);
  }

  // tokens of rounds r0 .. r0 + nr of the row tile that starts at query row m0
  __device__ __forceinline__ void segment(const AttReq& rq, int q, int head, int m0, int r0, int nr) {
    const int M = rq.n * p.G;
    const bool all = M <= kRows;  // the waves share the rows
    if (!all) m0 += wave_ * kRows;
    B::begin_rows(rq, m0);
    pages = p.table + (int64_t)q * p.max_pages;
    kh = static_cast<const char*>(p.k) + head * p.head_b;
    vh = static_cast<const char*>(p.v) + head * p.head_b;
    sh = p.scales + head * p.s_head;
    last_page = (len - 1) >> p.lg;
    const int step = all ? 2 * kTok : kTok;
    int end = uni(att_end(p, rq, m0 + kRows));
    end = end < (r0 + nr) * step ? end : (r0 + nr) * step;
    const int first = r0 * step + (all ? wave_ : 0) * kTok;
    const int nt = m0 < M && first < end ? (end - first + step - 1) / step : 0;
    if (nt > 0) {
      // A tile is under way while the one before it is computed, its page ids one further (two or
      // three tiles under way were no faster: 171, 173 and 175 us for 256 requests of 512 to 4096
      // tokens).  What would be asked for past the end is the last tile again: a load that is always
      // made leaves the compiler's wait for the one before exact.
      const int last = first + (nt - 1) * step;
      const auto next = [&](int t0) { return t0 < last ? t0 : last; };
      Raw4<D> x;
      load(first, page_ids(first), x);
      Pages id = page_ids(next(first + step));
      queries(rq, head, m0, M);
      for (int t0 = first; t0 <= last; t0 += step) {
        const Pages then = page_ids(next(t0 + 2 * step));
        tile(t0, x, [&] { load(next(t0 + step), id, x); });
        id = then;
      }
    }
    l = half_sum(l);
  }
};

// ---------------------------------------------------------------------------------------
// Many rows: four waves of 32 rows each share every tile, as bf16 in LDS, two tiles deep, with a
// barrier per tile.  Each of them converts the keys and values of 8 of the tile's tokens, a group of
// 32 elements a lane, and the products are those over a bf16 cache.
// ---------------------------------------------------------------------------------------
// (K's chunks: read from 16 rows at a time, over 64 banks, and written as V's)
template <int D>
struct Tile4 : Tile<uint16_t, D> {
  static __host__ __device__ constexpr int vswz(int r) { return vswz4<D>(r); }
  static __host__ __device__ constexpr int kswz(int r) {
    return D == 128 ? r & 15 : ((r >> 1) & 7) ^ (r & 1) << 2;
  }
};

// Three waves a SIMD at D = 64, two at D = 128.  64: 8192 rows 433 us, two waves 482; 2048 behind 4048 tokens
// 164 and 176; 64 requests of 72 over 500 to 4000 85 and 95; 16 of 128 behind 1000 32.8 and 31.4.  128, where
// three leave registers for half of the reads under way at a time: 641 and 650, 236 and 230, 119 and 122,
// 42 and 39.
template <int D>
struct Fit4Shared : Fit<uint16_t, D, 4> {
  static constexpr int PER_SIMD = D == 64 ? 3 : 2;
  static constexpr int PER_CU = PER_SIMD;  // (four waves each)
};

template <int D>
struct Att4Shared : AttWave<uint16_t, D, 4, Tile4<D>> {
  using A = AttWave<uint16_t, D, 4, Tile4<D>>;
  using Params = Att4Params;
  using F = Fit4Shared<D>;
  using L = Tile4<D>;
  static constexpr bool kNan = true;
  static constexpr int GROUPS = D / 32, LANES = 8 * GROUPS;  // lanes that a wave's 8 tokens' keys take

  using A::B::h;
  using A::B::l;
  using A::B::lane;
  using A::B::len;
  using A::B::n;
  using A::B::seen;
  using A::base;
  using A::last_page;
  using A::mine;
  using A::pages;
  using A::wave;
  const Att4Params& p;
  bool keys, any;           // the lane converts keys, or anything at all (D = 64: half of them)
  int tok, group;           // its token of the wave's 8, and group of 32
  uint32_t at;              // LDS of its first chunk, in a stage
  const char* codes;        // segment: its group's codes and scale byte at the head's first token
  const uint8_t* bytes;

  __device__ __forceinline__ Att4Shared(const Att4Params& p_, int wave_, uint32_t lds) : A(p_, wave_, lds), p(p_) {
    keys = lane < LANES;
    any = lane < 2 * LANES;
    const int i = lane % LANES;
    tok = i % 8;
    group = i / 8;
    const int x = keys ? L::kswz(mine + tok) : L::vswz(mine + tok);
    at = (uint32_t)(keys ? 0 : L::BYTES) + (uint32_t)(mine + tok) * L::RB + ((4 * group ^ x) << 4);
  }

  __device__ __forceinline__ int page_id(int t0) const {
    const int i = (t0 + mine) >> p.lg;
    return sload(pages, i < last_page ? i : last_page);
  }
  // the lane's codes and byte of tile t0; rows past the last token are read inside its page
  __device__ __forceinline__ void load(int t0, int id, uint4& x, uint32_t& byte) const {
    if ((uint32_t)id >= (uint32_t)p.n_pages) {
      if (lane == 0) raise_fault(p.status, DSPARK_FAULT_PAGE);
      id = 0;
    }
    const uint32_t t = (uint32_t)(t0 + mine) & ((1u << p.lg) - 1);  // the 8 tokens lie in one page
    x = *reinterpret_cast<const uint4*>(codes + ((uint64_t)(uint32_t)id * p.page_b4 + t * p.tok_b4));
    byte = bytes[(uint64_t)(uint32_t)id * p.s_page + t * p.s_tok];
  }
  // as bf16 to stage s
  __device__ __forceinline__ void convert(uint4 x, uint32_t byte, int s) const {
    const uint32_t to = here(at), stage = base + s * F::TILE;
    const float scale = fp4_scale(byte);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
    if (any) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        lds_put<u32x4>(stage + (to ^ (uint32_t)(j << 4)), __builtin_bit_cast(u32x4, fp4_bf16x8(w[j], scale)));
    }
  }

  // tokens of rounds r0 .. r0 + nr of the row tile that starts at query row m0
  __device__ __forceinline__ void segment(const AttReq& rq, int q, int head, int m0, int r0, int nr) {
    const int M = rq.n * p.G;
    A::begin(rq, q, head, m0);
    const uint32_t row = (uint32_t)tok * p.tok_b4, s_row = (uint32_t)tok * p.s_tok;
    codes = (keys ? A::kh : A::vh) + row + (any ? group * 16 : 0);
    bytes = p.scales + head * p.s_head + s_row + (keys ? 0 : GROUPS) + group;
    int end = uni(att_end(p, rq, m0 + 4 * kRows));
    end = end < (r0 + nr) * F::ROUND ? end : (r0 + nr) * F::ROUND;
    const int first = r0 * F::ROUND, nt = first < end ? (end - first + F::ROUND - 1) / F::ROUND : 0;
    if (nt > 0) {
      const int last = first + (nt - 1) * F::ROUND, mw = m0 + wave * kRows;
      const auto next = [&](int t) { return t < last ? t : last; };
      uint4 x;
      uint32_t byte;
      load(first, page_id(first), x, byte);
      A::queries(rq, head, mw, M);
      convert(x, byte, 0);
      load(next(first + F::ROUND), page_id(next(first + F::ROUND)), x, byte);
      int id = page_id(next(first + 2 * F::ROUND));
      const bool live = mw < M;
      int s = 0;
      for (int t0 = first; t0 <= last; t0 += F::ROUND) {
        stage_barrier();  // the whole tile is there, and every wave is done with the one before
        convert(x, byte, s ^ 1);  // (of the last tile: itself again, for nobody)
        load(next(t0 + 2 * F::ROUND), id, x, byte);
        id = page_id(next(t0 + 3 * F::ROUND));
        const uint32_t ks = base + s * F::TILE, vs = ks + L::BYTES;
        f32x16 sc = f32x16{};
        if (live) {
          A::scores(ks, sc);
          if (t0 + kTok > seen) A::B::mask(t0, sc);
          // the exponentials behind all else (before it 8192 rows take 663 for 657 us, of heads of 64
          // 434 for 420; over bf16, whose tiles are not converted, they go first)
          __builtin_amdgcn_s_setprio(0);
          A::B::weigh(sc);
          __builtin_amdgcn_s_setprio(1);
        }
        if (t0 + kTok > seen && A::clean_values(t0, vs)) {
          // a group that reads NaN reaches the rows that see its token, whatever its weight, as 0 * NaN
          // makes it in tiles without edges: what a row does not see has a weight below 0 instead
          const uint32_t vis = A::B::visible(t0);
#pragma unroll
          for (int r = 0; r < 16; ++r) sc[r] = vis & (1u << reg_row(r, 0)) ? sc[r] : -1.0f;
          A::template odd_values<true>(ks, vs, sc);
        }
        if (live) A::values(vs, sc);
        s ^= 1;
      }
      __builtin_amdgcn_s_setprio(0);
      stage_barrier();  // the next segment's tiles overwrite the stages
    }
    l = half_sum(l);
  }
};

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
// f(the variant that runs these shapes).  Past 64 query rows to a cache head (rows / R, the bound that the
// host knows, times heads to a cache head) waves that share tiles save the others' conversions: 8192 rows
// from an empty cache 655 against 791 us, 2048 behind 4048 230 and 253, 64 requests of 72 over 500 to
// 4000 114 and 123; over short contexts the barriers cost as much (16 requests of 128 rows behind 1000
// tokens 39 and 37).  Up to 64 they lose: 36 rows 343 and 242 us, 45 37 and 29, 64 rows 374 and 254, of
// heads of 64 224 and 160 (256 requests of 512 to 4096 tokens), but not in one list cut to small pieces:
// one request of 64 behind 16000 31 and 39.
template <class F>
static auto att4_variant(int R, int rows, int G, int D, dspark_dtype dt, F f) {
  if (dt == DSPARK_F32) return D == 64 ? f((Att4Wave<64, 3>*)nullptr) : f((Att4Wave<128, 3>*)nullptr);
  const int64_t m = (int64_t)((rows + R - 1) / R) * G;
  if (m > 64) return D == 64 ? f((Att4Shared<64>*)nullptr) : f((Att4Shared<128>*)nullptr);
  return D == 64 ? f((Att4Wave<64, 1>*)nullptr) : f((Att4Wave<128, 1>*)nullptr);
}

static size_t att4_carve(Att4Params& p, void* ws, int R, int rows, int G, int D, dspark_dtype dt) {
  return att4_variant(R, rows, G, D, dt, [&](auto* w) {
    using W = std::remove_pointer_t<decltype(w)>;
    return att_carve(p, ws, att_grid<typename W::F>(), kRows * W::kNR, W::kD);
  });
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_tree_attention4_workspace_bytes(int R, int rows, int Hq, int Hkv, int D,
                                                         dspark_dtype dt) {
  if (!att_dims_ok(R, rows, Hq, Hkv, D, dt) || R == 0) return 0;
  Att4Params p{};
  return att4_carve(p, nullptr, R, rows, Hq / Hkv, D, dt);
}

extern "C" int dspark_tree_attention4(int R, int rows, int Hq, int Hkv, int D, dspark_dtype dt,
                                      int page_size, int max_pages, int n_pages, const void* q,
                                      int64_t q_row, const void* k_cache, const void* v_cache,
                                      int64_t page_stride, int64_t head_stride, int64_t tok_stride,
                                      const void* scales, int64_t s_page, int64_t s_head, int64_t s_tok,
                                      const int32_t* table, const int32_t* ctx, const int32_t* row_off,
                                      const uint64_t* anc, float scale, void* o, float* lse,
                                      int32_t* dev_status, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!att_dims_ok(R, rows, Hq, Hkv, D, dt) ||
      !cache4_ok(D, page_stride, head_stride, tok_stride, s_page, s_head, s_tok) || tok_stride > (1 << 21) ||
      s_tok > (1 << 21) || page_stride >= ((int64_t)1 << 32) || s_page >= ((int64_t)1 << 32))
    return DSPARK_EINVAL;
  Att4Params p{};
  const int rc = att_args(p, R, rows, Hq, Hkv, D, dt, page_size, max_pages, n_pages, q, q_row, k_cache, v_cache,
                          table, ctx, row_off, anc, scale, o, lse, dev_status, ws);
  if (rc != DSPARK_OK || R == 0 || rows == 0) return rc;
  if (!scales || !aligned16(scales)) return DSPARK_EINVAL;
  p.page_b4 = (uint32_t)page_stride;
  p.tok_b4 = (uint32_t)tok_stride;
  p.head_b = head_stride;
  p.scales = static_cast<const uint8_t*>(scales);
  p.s_page = (uint32_t)s_page;
  p.s_tok = (uint32_t)s_tok;
  p.s_head = s_head;
  if (ws_bytes < att4_carve(p, ws, R, rows, p.G, D, dt)) return DSPARK_EWORKSPACE;
  return att4_variant(R, rows, p.G, D, dt, [&](auto* w) {
    return att_launch<std::remove_pointer_t<decltype(w)>>(p, stream);
  });
}
