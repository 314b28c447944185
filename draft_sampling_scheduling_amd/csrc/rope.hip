// rope.hip -- between a layer's projections and its cache: norms of queries and keys for each head
// and the position rotation, to rows or on the way into the paged cache (bf16, float or 4 bits),
// and the way back out of a cache of 4 bits.
//
// A head x of D elements becomes, with x^ = x / sqrt(mean x^2 + eps) * w where it is normed,
//   a' = a cos - b sin,   b' = b cos + a sin
// for the pairs (a, b) of its first `rot` elements: (i, i + rot/2), or (2i, 2i + 1); cosines and
// sines come from the row of a table that the row's position names.  About six operations an
// element, so HBM bounds it: each element is read and written once.  Measured, kernels alone, bf16, heads
// of 128: 8192 rows of 32 and 8 heads with norms to rows (172 MB) 36 us, 4.7 TB/s; 1280 rows of those and
// 8 heads of values into the cache (32 MB) 11, into 4 bits (28 MB) 13; 8192 rows with norms into 4 bits
// (181 MB) 50, 3.6 TB/s; 8192 rows of 40, 8 and 8 heads without (212 MB) 51, 4.2 TB/s; 8224 tokens of 8
// heads back out (43 MB) 11.
//
// A lane has two pieces of 8 elements of a head that hold both halves of its pairs, so a cosine and a
// sine are loaded for each pair once; D / 16 lanes work on a head, and go through heads of their row with
// the row's cosines and sines in registers.  (A piece a lane, the other halves loaded beside it, took
// twice the loads: 32 against 23 us for 1280 rows of 32 and 8 heads of 128 into 4 bits and back out.)  All of a
// head's loads return before any of it is stored, so rows may be turned in place.
// float throughout, rounded once; but keys on their way to 4 bits are taken in double: a code's
// step is up to half of its value, so at a border the last bit of a float decides about that
// much, and in double the code is that of the formula's value.
#include "fp4.h"
#include "target.h"

namespace dspark {

enum RopeTo { kToRows, kToCache, kToCache4 };

struct RopeArgs {
  int rows, Hq, Hkv, D, rot, n_pos, slices;
  bool interleaved;
  const void *q, *k, *v;
  int64_t q_row, k_row, v_row;  // elements
  const int32_t *position, *slot, *n_rows;
  const float* rope;
  const void *q_norm, *k_norm;
  double eps;
  void* q_out;
  int64_t qo_row;
  void* k_out;  // rows
  int64_t ko_row;
  int lg, n_pages;
  char *k_cache, *v_cache;
  uint8_t* scales;
  int64_t page_b, head_b, tok_b;  // strides in bytes
  int64_t s_page, s_head, s_tok;
  int32_t* status;
};

template <class T>
struct Eight {  // 8 elements as they lie in memory
  static constexpr int kE = sizeof(T), N = kE / 2;
  uint4 w[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  __device__ __forceinline__ float at(int e) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (kE == 4) return __uint_as_float(u[e]);
    return e % 2 ? bf16hi(u[e / 2]) : bf16lo(u[e / 2]);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
    if constexpr (kE == 4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(x[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bf16x2 pair;
        pair.x = (__bf16)x[2 * e];
        pair.y = (__bf16)x[2 * e + 1];
        u[e] = __builtin_bit_cast(uint32_t, pair);
      }
    }
  }
};

template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  return xlane_partner<STEP>(v);
}
template <int STEP>
__device__ __forceinline__ float partner(float v) {
  return __uint_as_float(xlane_partner<STEP>(__float_as_uint(v)));
}
template <int STEP>
__device__ __forceinline__ double partner(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = xlane_partner<STEP>((uint32_t)u), hi = xlane_partner<STEP>((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(hi << 32 | lo));
}
// over the LPR lanes (4, 8 or 16, aligned) that hold a head, the same in each
template <int LPR, class V, class Op>
__device__ __forceinline__ V head_reduce(V v, Op op) {
  v = op(v, partner<0>(v));
  v = op(v, partner<1>(v));
  if (LPR > 4) v = op(v, partner<2>(v));
  if (LPR > 8) v = op(v, partner<3>(v));
  return v;
}

// What a lane knows of its row and its place in a head.
template <class T, int LPR>
struct RopeLane {
  int ca, cb;         // its pieces of 8 elements
  int pair;           // of its pairs the first, by eights
  bool live, turns;   // it has any; its pairs turn
  bool apart;         // pairs are one element of either piece, not neighbours in one
  float c[8], s[8];   // of its pairs

  __device__ __forceinline__ void place(const RopeArgs& p, int l) {
    live = 16 * l < p.D;
    l = live ? l : 0;  // (lanes past the head do as the first, and store nothing)
    pair = l;
    apart = !p.interleaved;
    const int half = p.rot / 16;  // pieces that hold the first halves
    turns = p.rope && l < half;
    ca = 2 * l;
    cb = ca + 1;
    if (apart) {  // those behind the turned ones are taken in order
      ca = turns ? l : 2 * half + 2 * (l - half);
      cb = turns ? l + half : ca + 1;
    }
  }
  __device__ __forceinline__ void angles(const RopeArgs& p, int pos) {
    if (!turns) return;
    const float* line = p.rope + (int64_t)pos * p.rot + 8 * pair;
    ld8(line, c);
    ld8(line + p.rot / 2, s);
  }

  // a lane's pieces of a head, normed and turned, in F (float or double)
  template <class F, bool NORM>
  __device__ __forceinline__ void turn(const RopeArgs& p, const Eight<T>& a, const Eight<T>& b, const Eight<T>& wa,
                                       const Eight<T>& wb, F (&ya)[8], F (&yb)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ya[e] = (F)a.at(e);
      yb[e] = (F)b.at(e);
    }
    if (NORM) {
      F sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += ya[e] * ya[e];
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += yb[e] * yb[e];
      sum = head_reduce<LPR>(live ? sum : (F)0, [](F x, F y) { return x + y; });
      const F f = (F)1 / sqrt(sum / (F)p.D + (F)p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ya[e] = ya[e] * f * (F)wa.at(e);
        yb[e] = yb[e] * f * (F)wb.at(e);
      }
    }
    if (!turns) return;
    if (apart) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const F x = ya[e], y = yb[e];
        ya[e] = x * (F)c[e] - y * (F)s[e];
        yb[e] = y * (F)c[e] + x * (F)s[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        F* z = e < 4 ? ya + 2 * e : yb + 2 * (e - 4);
        const F x = z[0], y = z[1];
        z[0] = x * (F)c[e] - y * (F)s[e];
        z[1] = y * (F)c[e] + x * (F)s[e];
      }
    }
  }

  // a lane's pieces into a 4-bit cache: their groups' largest values meet, then their codes
  template <class F>
  __device__ __forceinline__ void put4(const RopeArgs& p, int c0, int c1, const F (&ya)[8], const F (&yb)[8],
                                       char* codes, uint8_t* scale) const {
    uint32_t a[8], b[8], ta = 0, tb = 0, ba = 0, bb = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = fp4_bits(ya[e]);
      b[e] = fp4_bits(yb[e]);
      ta = max(ta, a[e] & 0x7FFFFFFFu);
      tb = max(tb, b[e] & 0x7FFFFFFFu);
    }
    const int ga = c0 / 4, gb = c1 / 4;
#pragma unroll
    for (int g = 0; g < LPR / 2; ++g) {  // (heads of 64 have four lanes, of 128 eight)
      const uint32_t mine = max(ga == g ? ta : 0u, gb == g ? tb : 0u);
      const uint32_t byte = fp4_byte(head_reduce<LPR>(mine, [](uint32_t x, uint32_t y) { return max(x, y); }));
      ba = ga == g ? byte : ba;
      bb = gb == g ? byte : bb;
    }
    reinterpret_cast<uint32_t*>(codes)[c0] = fp4_codes(a, ba);
    reinterpret_cast<uint32_t*>(codes)[c1] = fp4_codes(b, bb);
    if (c0 % 4 == 0) scale[ga] = (uint8_t)ba;
    if (c1 % 4 == 0) scale[gb] = (uint8_t)bb;
  }
};

// A row's heads from one source (q, k or v), every slices-th of them: those of a batch are loaded
// together.
template <class T>
struct Heads {
  static constexpr int kBatch = 2;  // (four: 40 to 44 us where two take 37, 8192 rows of 32 and 8 heads)
  Eight<T> a[kBatch], b[kBatch];
  __device__ __forceinline__ void load(const T* x, int D, int ca, int cb, int h, int step, int heads) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (h + u * step < heads) {
        a[u].load(x + (int64_t)(h + u * step) * D + 8 * ca);
        b[u].load(x + (int64_t)(h + u * step) * D + 8 * cb);
      }
  }
};

template <class T, int LPR, RopeTo TO, bool NORM>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs p) {
  using H = Heads<T>;
  const int64_t group = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int i = (int)(group / p.slices), slice = (int)(group - (int64_t)i * p.slices);
  if (i >= p.rows) return;
  const int l = threadIdx.x % LPR;
  RopeLane<T, LPR> r;
  r.place(p, l);
  // what a row is needs a trip to memory each, and so do its heads: all are asked for before any is
  // looked at (a row past *n_rows, or of no position, is read and not used)
  const int live = p.n_rows ? *p.n_rows : p.rows;
  const int pos = p.rope ? p.position[i] : 0;
  const int s = TO != kToRows ? p.slot[i] : 0;
  H x;
  int h = slice;
  if (p.q) x.load(static_cast<const T*>(p.q) + i * p.q_row, p.D, r.ca, r.cb, h, p.slices, p.Hq);
  const bool tell = slice == 0 && l == 0;
  if (i >= live) return;
  if (p.rope && (pos < 0 || pos >= p.n_pos)) {
    if (tell) raise_fault(p.status, DSPARK_FAULT_PARAM);
    return;
  }
  r.angles(p, pos);
  // the heads from h on, their first batch loaded already if `loaded`: f(head, a, b, wa, wb)
  const auto each = [&](const void* src, int64_t row, const void* norm, int heads, bool loaded, auto f) {
    const T* y = static_cast<const T*>(src) + i * row;
    Eight<T> wa{}, wb{};
    if (NORM && norm) {
      wa.load(static_cast<const T*>(norm) + 8 * r.ca);
      wb.load(static_cast<const T*>(norm) + 8 * r.cb);
    }
    for (; h < heads; h += H::kBatch * p.slices) {
      if (!loaded) x.load(y, p.D, r.ca, r.cb, h, p.slices, heads);
      loaded = false;
#pragma unroll
      for (int u = 0; u < H::kBatch; ++u)
        if (h + u * p.slices < heads) f(h + u * p.slices, x.a[u], x.b[u], wa, wb);
    }
  };
  const auto put = [&](T* to, const float (&ya)[8], const float (&yb)[8]) {
    Eight<T> out;
    if (!r.live) return;
    out.set(ya);
    out.store(to + 8 * r.ca);
    out.set(yb);
    out.store(to + 8 * r.cb);
  };
  if (p.q) {
    each(p.q, p.q_row, p.q_norm, p.Hq, true, [&](int head, const Eight<T>& a, const Eight<T>& b,
                                                 const Eight<T>& wa, const Eight<T>& wb) {
      float ya[8], yb[8];
      if (NORM && p.q_norm)
        r.template turn<float, true>(p, a, b, wa, wb, ya, yb);
      else
        r.template turn<float, false>(p, a, b, wa, wb, ya, yb);
      put(static_cast<T*>(p.q_out) + i * p.qo_row + (int64_t)head * p.D, ya, yb);
    });
    // the heads after these go on with the slices where they stopped
    h = (slice + p.slices - p.Hq % p.slices) % p.slices;
  }
  if (!p.k) return;
  char *kc = nullptr, *vc = nullptr;
  uint8_t* sc = nullptr;
  if (TO != kToRows) {
    if (s < 0 || (s >> p.lg) >= p.n_pages) {
      if (s != -1 && tell) raise_fault(p.status, DSPARK_FAULT_PAGE);
      return;
    }
    const int64_t page = s >> p.lg, tok = s & ((1 << p.lg) - 1);
    kc = p.k_cache + page * p.page_b + tok * p.tok_b;
    vc = p.v_cache + page * p.page_b + tok * p.tok_b;
    if (TO == kToCache4) sc = p.scales + page * p.s_page + tok * p.s_tok;
  }
  const int k0 = h;
  each(p.k, p.k_row, p.k_norm, p.Hkv, false, [&](int head, const Eight<T>& a, const Eight<T>& b,
                                                 const Eight<T>& wa, const Eight<T>& wb) {
    typedef typename std::conditional<TO == kToCache4, double, float>::type F;
    F ya[8], yb[8];
    if (NORM && p.k_norm)
      r.template turn<F, true>(p, a, b, wa, wb, ya, yb);
    else
      r.template turn<F, false>(p, a, b, wa, wb, ya, yb);
    if constexpr (TO == kToCache4)
      r.put4(p, r.ca, r.cb, ya, yb, kc + head * p.head_b, sc + head * p.s_head);
    else if (TO == kToRows)
      put(static_cast<T*>(p.k_out) + i * p.ko_row + (int64_t)head * p.D, ya, yb);
    else
      put(reinterpret_cast<T*>(kc + head * p.head_b), ya, yb);
  });
  if (TO == kToRows) return;
  h = (k0 + p.slices - p.Hkv % p.slices) % p.slices;
  each(p.v, p.v_row, nullptr, p.Hkv, false, [&](int head, const Eight<T>& a, const Eight<T>& b,
                                                const Eight<T>&, const Eight<T>&) {
    if constexpr (TO == kToCache4) {
      float ya[8], yb[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ya[e] = a.at(e);
        yb[e] = b.at(e);
      }
      r.put4(p, r.ca, r.cb, ya, yb, vc + head * p.head_b, sc + head * p.s_head + p.D / kGroup4);
    } else if (r.live) {
      T* to = reinterpret_cast<T*>(vc + head * p.head_b);
      a.store(to + 8 * r.ca);
      b.store(to + 8 * r.cb);
    }
  });
}

// Tokens of a 4-bit cache as values: a thread per eight elements of a token's keys and values.
struct ReadArgs {
  int layers, rows, Hkv, D, lg, n_pages;
  const int32_t *slot, *n_rows;
  const char *k_cache, *v_cache;
  const uint8_t* scales;
  int64_t layer_b, page_b, head_b, tok_b;
  int64_t s_layer, s_page, s_head, s_tok;
  void *k, *v;  // [layers][rows][Hkv][D]
  int32_t* status;
};

template <class T>
__global__ void __launch_bounds__(256) cache4_read_kernel(ReadArgs p) {
  const int per = p.Hkv * p.D / 8;  // pieces of a row
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id / per;
  const int piece = (int)(id - row * per), layer = (int)(row / p.rows), i = (int)(row - (int64_t)layer * p.rows);
  const int live = p.n_rows ? min(p.rows, *p.n_rows) : p.rows;
  if (layer >= p.layers || i >= live) return;
  const int s = p.slot[i];
  if (s < 0 || (s >> p.lg) >= p.n_pages) {
    if (s != -1 && piece == 0 && layer == 0) raise_fault(p.status, DSPARK_FAULT_PAGE);
    return;
  }
  const int64_t page = s >> p.lg, tok = s & ((1 << p.lg) - 1);
  const int head = piece / (p.D / 8), c = piece - head * (p.D / 8);
  const int64_t at = layer * p.layer_b + page * p.page_b + head * p.head_b + tok * p.tok_b;
  const uint8_t* sc = p.scales + layer * p.s_layer + page * p.s_page + head * p.s_head + tok * p.s_tok + c / 4;
  const uint32_t kc = reinterpret_cast<const uint32_t*>(p.k_cache + at)[c];
  const uint32_t vc = reinterpret_cast<const uint32_t*>(p.v_cache + at)[c];
  const float ks = fp4_scale(sc[0]), vs = fp4_scale(sc[p.D / kGroup4]);
  const int64_t to = id * 8;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(static_cast<T*>(p.k) + to) = fp4_bf16x8(kc, ks);
    *reinterpret_cast<uint4*>(static_cast<T*>(p.v) + to) = fp4_bf16x8(vc, vs);
  } else {
    float x[8];
    Eight<T> out;
    fp4_f32x8(kc, ks, x);
    out.set(x);
    out.store(static_cast<T*>(p.k) + to);
    fp4_f32x8(vc, vs, x);
    out.set(x);
    out.store(static_cast<T*>(p.v) + to);
  }
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
// Whether rows of two arrays (a row's bytes apart by a_row, na bytes each) may share memory.  Slices
// of one fused projection lie between each other's rows: with equal strides it is the places
// within a row that count.
static bool rows_meet(const void* a, int64_t a_row, int64_t na, const void* b, int64_t b_row, int64_t nb,
                      int rows) {
  if (!overlap(a, (size_t)((rows - 1) * a_row + na), b, (size_t)((rows - 1) * b_row + nb))) return false;
  if (a_row != b_row || na > a_row || nb > a_row || a_row == 0) return true;
  const int64_t d = (int64_t)((uintptr_t)b - (uintptr_t)a);
  const int64_t r = ((d % a_row) + a_row) % a_row;  // where b's rows begin in a's
  return r < na || r + nb > a_row;
}

// Groups of lanes (a head each at a time) that a row's heads are spread over: few rows want all lanes
// they can get; of many, a group goes through several heads with the row's cosines and sines, loaded
// once.  us for 1, 2, 4, 8, 16 groups a row: 8192 rows to rows, 40 heads of 128, 45, 44, 41, 37, 40; to the
// cache, 48 heads, 59, 51, 48, 44, 47; into 4 bits with norms, in whose double precision a group's weights
// cost more, and back out (11), 68, 61, 60, 66, 74; 1280 rows of that (10), for 6, 12 and 25 groups, 24,
// 23, 25.
static int rope_slices(int rows, int heads, bool slow) {
  int least = 1;  // groups a row has at the least: a group takes 8 (16) heads at the most
  while (least * (slow ? 16 : 8) < heads) least *= 2;
  int64_t want = (slow ? 16384 : 32768) / (int64_t)rows;
  want = want < least ? least : want;
  return want > heads ? heads : (int)want;
}

template <class T, RopeTo TO, bool NORM>
static int rope_launch(const RopeArgs& p, hipStream_t stream) {
  const int lpr = p.D <= 64 ? 4 : (p.D <= 128 ? 8 : 16);
  const int64_t blocks = ((int64_t)p.rows * p.slices * lpr + 255) / 256;
  if (blocks >= (1 << 24)) return DSPARK_EINVAL;  // a grid holds 2^32 threads
  if (lpr == 4)
    rope_kernel<T, 4, TO, NORM><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else if (lpr == 8)
    rope_kernel<T, 8, TO, NORM><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else if constexpr (TO != kToCache4)
    rope_kernel<T, 16, TO, NORM><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return launch_status();
}

template <RopeTo TO>
static int rope_run(RopeArgs p, dspark_dtype dt, hipStream_t stream) {
  const int heads = (p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (p.v ? p.Hkv : 0);
  const bool norm = p.q_norm || p.k_norm;
  p.slices = rope_slices(p.rows, heads, TO == kToCache4 && norm);
  if (dt == DSPARK_BF16)
    return norm ? rope_launch<uint16_t, TO, true>(p, stream) : rope_launch<uint16_t, TO, false>(p, stream);
  return norm ? rope_launch<float, TO, true>(p, stream) : rope_launch<float, TO, false>(p, stream);
}

// The arguments that the calls share; outputs and caches are the callers' to check.
static int rope_args(RopeArgs& p, int rows, int Hq, int Hkv, int D, int rot, int interleaved, dspark_dtype dt,
                     const void* q, int64_t q_row, const void* k, int64_t k_row, const int32_t* position,
                     const float* rope, int n_pos, const void* q_norm, const void* k_norm, double eps,
                     const int32_t* n_rows, int32_t* status) {
  if (rows < 0 || Hkv < 0 || Hq < 0 || D < 16 || D % 16 != 0 || D > 256 || Hq > (1 << 20) || Hkv > (1 << 20) ||
      (dt != DSPARK_F32 && dt != DSPARK_BF16) || !(eps <= 1e30) || !(eps == 0.0 || eps >= 1e-30))
    return DSPARK_EINVAL;
  if (rope && (rot < 16 || rot % 16 != 0 || rot > D || n_pos < 1)) return DSPARK_EINVAL;
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  if ((q && (!stride_ok(q_row, e) || Hq < 1)) || (k && (!stride_ok(k_row, e) || Hkv < 1))) return DSPARK_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(rope) || !aligned16(q_norm) || !aligned16(k_norm))
    return DSPARK_EINVAL;
  p.rows = rows;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.rot = rope ? rot : 0;
  p.interleaved = interleaved != 0;
  p.n_pos = n_pos;
  p.q = q;
  p.k = k;
  p.q_row = q_row;
  p.k_row = k_row;
  p.position = position;
  p.n_rows = n_rows;
  p.rope = rope;
  p.q_norm = q ? q_norm : nullptr;
  p.k_norm = k ? k_norm : nullptr;
  p.eps = eps;
  p.status = status;
  return DSPARK_OK;
}

// an output of rows: its own rows apart, and either the input's very place or none of it
static bool out_ok(const void* out, int64_t o_row, const void* in, int64_t i_row, int64_t heads, int D, size_t e,
                   int rows) {
  const int64_t n = heads * D * (int64_t)e, ob = o_row * (int64_t)e;
  if (!out || !aligned16(out) || !stride_ok(o_row, e) || (rows > 1 && ob < n)) return false;
  if (out == in && (o_row == i_row || rows == 1)) return true;
  return !rows_meet(out, ob, n, in, i_row * (int64_t)e, n, rows);
}

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_qk_rope(int rows, int Hq, int Hkv, int D, int rot, int interleaved, dspark_dtype dt,
                              const void* q, int64_t q_row, const void* k, int64_t k_row,
                              const int32_t* position, const float* rope, int n_pos, const void* q_norm,
                              const void* k_norm, double eps, const int32_t* n_rows, void* q_out,
                              int64_t qo_row, void* k_out, int64_t ko_row, int32_t* dev_status,
                              hipStream_t stream) {
  RopeArgs p{};
  const int rc = rope_args(p, rows, Hq, Hkv, D, rot, interleaved, dt, q, q_row, k, k_row, position, rope,
                           n_pos, q_norm, k_norm, eps, n_rows, dev_status);
  if (rc != DSPARK_OK) return rc;
  if (rows == 0) return DSPARK_OK;
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  const int64_t nq = (int64_t)Hq * D * e, nk = (int64_t)Hkv * D * e;
  if ((!q && !k) || (rope && !position)) return DSPARK_EINVAL;
  if (q && !out_ok(q_out, qo_row, q, q_row, Hq, D, e, rows)) return DSPARK_EINVAL;
  if (k && !out_ok(k_out, ko_row, k, k_row, Hkv, D, e, rows)) return DSPARK_EINVAL;
  if (q && k &&
      (rows_meet(q_out, qo_row * e, nq, k, k_row * e, nk, rows) ||
       rows_meet(k_out, ko_row * e, nk, q, q_row * e, nq, rows) ||
       rows_meet(q_out, qo_row * e, nq, k_out, ko_row * e, nk, rows)))
    return DSPARK_EINVAL;
  p.q_out = q_out;
  p.qo_row = qo_row;
  p.k_out = k_out;
  p.ko_row = ko_row;
  return rope_run<kToRows>(p, dt, stream);
}

// What both appends check of q, k, v and the memory from a cache's first to its last element.
static int append_args(RopeArgs& p, size_t e, const void* v, int64_t v_row, const int32_t* slot, int page_size,
                       int n_pages, void* q_out, int64_t qo_row) {
  if (!pages_ok(page_size, n_pages) || p.Hkv < 1 || !stride_ok(v_row, e)) return DSPARK_EINVAL;
  if (p.rows == 0) return DSPARK_OK;
  if (!p.k || !v || !slot || !aligned16(v) || (p.rope && !p.position)) return DSPARK_EINVAL;
  const int64_t nq = (int64_t)p.Hq * p.D * e, nk = (int64_t)p.Hkv * p.D * e;
  if (p.q) {
    if (!out_ok(q_out, qo_row, p.q, p.q_row, p.Hq, p.D, e, p.rows)) return DSPARK_EINVAL;
    if (rows_meet(q_out, qo_row * e, nq, p.k, p.k_row * e, nk, p.rows) ||
        rows_meet(q_out, qo_row * e, nq, v, v_row * e, nk, p.rows))
      return DSPARK_EINVAL;
  }
  p.v = v;
  p.v_row = v_row;
  p.slot = slot;
  p.lg = log2_of(page_size);
  p.n_pages = n_pages;
  p.q_out = q_out;
  p.qo_row = qo_row;
  return DSPARK_OK;
}

// whether any of the rows lies in [m, m + bytes)
static bool rows_in(const RopeArgs& p, size_t e, const void* m, size_t bytes) {
  const auto in = [&](const void* x, int64_t row, int64_t heads) {
    return x && overlap(x, (size_t)((p.rows - 1) * row + heads * p.D) * e, m, bytes);
  };
  return in(p.q, p.q_row, p.Hq) || in(p.k, p.k_row, p.Hkv) || in(p.v, p.v_row, p.Hkv) ||
         (p.q && in(p.q_out, p.qo_row, p.Hq));
}

extern "C" int dspark_rope_append(int rows, int Hq, int Hkv, int D, int rot, int interleaved, dspark_dtype dt,
                                  int page_size, int n_pages, const void* q, int64_t q_row, const void* k,
                                  int64_t k_row, const void* v, int64_t v_row, const int32_t* slot,
                                  const int32_t* position, const float* rope, int n_pos, const void* q_norm,
                                  const void* k_norm, double eps, const int32_t* n_rows, void* q_out,
                                  int64_t qo_row, void* k_cache, void* v_cache, int64_t page_stride,
                                  int64_t head_stride, int64_t tok_stride, int32_t* dev_status,
                                  hipStream_t stream) {
  RopeArgs p{};
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  int rc = rope_args(p, rows, Hq, Hkv, D, rot, interleaved, dt, q, q_row, k, k_row, position, rope, n_pos,
                     q_norm, k_norm, eps, n_rows, dev_status);
  if (rc == DSPARK_OK) rc = append_args(p, e, v, v_row, slot, page_size, n_pages, q_out, qo_row);
  if (rc != DSPARK_OK) return rc;
  if (!stride_ok(page_stride, e) || !stride_ok(head_stride, e) || !stride_ok(tok_stride, e)) return DSPARK_EINVAL;
  if (rows == 0) return DSPARK_OK;
  if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return DSPARK_EINVAL;
  const size_t bytes = ((size_t)(n_pages - 1) * page_stride + (size_t)(Hkv - 1) * head_stride +
                        (size_t)(page_size - 1) * tok_stride + D) * e;
  if (rows_in(p, e, k_cache, bytes) || rows_in(p, e, v_cache, bytes)) return DSPARK_EINVAL;
  p.k_cache = static_cast<char*>(k_cache);
  p.v_cache = static_cast<char*>(v_cache);
  p.page_b = page_stride * (int64_t)e;
  p.head_b = head_stride * (int64_t)e;
  p.tok_b = tok_stride * (int64_t)e;
  return rope_run<kToCache>(p, dt, stream);
}

extern "C" int dspark_cache4_append(int rows, int Hq, int Hkv, int D, int rot, int interleaved, dspark_dtype dt,
                                    int page_size, int n_pages, const void* q, int64_t q_row, const void* k,
                                    int64_t k_row, const void* v, int64_t v_row, const int32_t* slot,
                                    const int32_t* position, const float* rope, int n_pos, const void* q_norm,
                                    const void* k_norm, double eps, const int32_t* n_rows, void* q_out,
                                    int64_t qo_row, void* k_cache, void* v_cache, int64_t page_stride,
                                    int64_t head_stride, int64_t tok_stride, void* scales, int64_t s_page,
                                    int64_t s_head, int64_t s_tok, int32_t* dev_status, hipStream_t stream) {
  RopeArgs p{};
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  int rc = rope_args(p, rows, Hq, Hkv, D, rot, interleaved, dt, q, q_row, k, k_row, position, rope, n_pos,
                     q_norm, k_norm, eps, n_rows, dev_status);
  if (rc == DSPARK_OK) rc = append_args(p, e, v, v_row, slot, page_size, n_pages, q_out, qo_row);
  if (rc != DSPARK_OK) return rc;
  if (!cache4_ok(D, page_stride, head_stride, tok_stride, s_page, s_head, s_tok)) return DSPARK_EINVAL;
  if (rows == 0) return DSPARK_OK;
  if (!k_cache || !v_cache || !scales || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(scales))
    return DSPARK_EINVAL;
  const size_t bytes = (size_t)(n_pages - 1) * page_stride + (size_t)(Hkv - 1) * head_stride +
                       (size_t)(page_size - 1) * tok_stride + D / 2;
  const size_t s_bytes = (size_t)(n_pages - 1) * s_page + (size_t)(Hkv - 1) * s_head +
                         (size_t)(page_size - 1) * s_tok + D / 16;
  if (rows_in(p, e, k_cache, bytes) || rows_in(p, e, v_cache, bytes) || rows_in(p, e, scales, s_bytes))
    return DSPARK_EINVAL;
  p.k_cache = static_cast<char*>(k_cache);
  p.v_cache = static_cast<char*>(v_cache);
  p.scales = static_cast<uint8_t*>(scales);
  p.page_b = page_stride;
  p.head_b = head_stride;
  p.tok_b = tok_stride;
  p.s_page = s_page;
  p.s_head = s_head;
  p.s_tok = s_tok;
  return rope_run<kToCache4>(p, dt, stream);
}

extern "C" int dspark_cache4_read(int layers, int rows, int Hkv, int D, dspark_dtype dt, int page_size,
                                  int n_pages, const int32_t* slot, const int32_t* n_rows, const void* k_cache,
                                  const void* v_cache, int64_t layer_stride, int64_t page_stride,
                                  int64_t head_stride, int64_t tok_stride, const void* scales, int64_t s_layer,
                                  int64_t s_page, int64_t s_head, int64_t s_tok, void* k, void* v,
                                  int32_t* dev_status, hipStream_t stream) {
  if (layers < 0 || rows < 0 || Hkv < 1 || Hkv > (1 << 20) || (dt != DSPARK_F32 && dt != DSPARK_BF16) ||
      !pages_ok(page_size, n_pages) ||
      !cache4_ok(D, page_stride, head_stride, tok_stride, s_page, s_head, s_tok) ||
      !stride_ok(layer_stride, 1) || s_layer < 0 || s_layer % (D / 16) != 0)
    return DSPARK_EINVAL;
  if (layers == 0 || rows == 0) return DSPARK_OK;
  if (!slot || !k_cache || !v_cache || !scales || !k || !v || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(scales) || !aligned16(k) || !aligned16(v))
    return DSPARK_EINVAL;
  const int64_t pieces = (int64_t)layers * rows;
  if (pieces >= ((int64_t)1 << 32) || pieces * Hkv >= ((int64_t)1 << 32)) return DSPARK_EINVAL;
  const int64_t blocks = (pieces * Hkv * (D / 8) + 255) / 256;
  if (blocks >= (1 << 24)) return DSPARK_EINVAL;  // a grid holds 2^32 threads
  ReadArgs p{layers, rows, Hkv, D, log2_of(page_size), n_pages, slot, n_rows, static_cast<const char*>(k_cache),
             static_cast<const char*>(v_cache), static_cast<const uint8_t*>(scales), layer_stride, page_stride,
             head_stride, tok_stride, s_layer, s_page, s_head, s_tok, k, v, dev_status};
  // outputs apart from the cache and from each other
  const size_t out = (size_t)pieces * Hkv * D * (dt == DSPARK_BF16 ? 2 : 4);
  const size_t bytes = (size_t)(layers - 1) * layer_stride + (size_t)(n_pages - 1) * page_stride +
                       (size_t)(Hkv - 1) * head_stride + (size_t)(page_size - 1) * tok_stride + D / 2;
  const size_t s_bytes = (size_t)(layers - 1) * s_layer + (size_t)(n_pages - 1) * s_page +
                         (size_t)(Hkv - 1) * s_head + (size_t)(page_size - 1) * s_tok + D / 16;
  for (const void* o : {k, v})
    if (overlap(o, out, k_cache, bytes) || overlap(o, out, v_cache, bytes) || overlap(o, out, scales, s_bytes))
      return DSPARK_EINVAL;
  if (overlap(k, out, v, out)) return DSPARK_EINVAL;
  if (dt == DSPARK_BF16)
    cache4_read_kernel<uint16_t><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else
    cache4_read_kernel<float><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return launch_status();
}
