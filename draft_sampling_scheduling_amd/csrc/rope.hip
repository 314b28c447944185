// rope.hip -- between a layer's projections and its cache: norms of queries and keys for each head
// and the position rotation, to rows or on the way into the paged cache (bf16, float or 4 bits),
// and the way back out of a cache of 4 bits.
//
// A head x of D elements becomes, with x^ = x / sqrt(mean x^2 + eps) * w where it is normed,
//   a' = a cos - b sin,   b' = b cos + a sin
// for the pairs (a, b) of its first `rot` elements: (i, i + rot/2), or (2i, 2i + 1); cosines and
// sines come from the row of a table that the row's position names.  About six operations an
// element, so HBM bounds it: each element is read and written once.
//
// A lane has 8 elements of a head, as many lanes as hold a head (8, 16 or 32) work on it, and go
// through the heads of their row with the row's cosines and sines in registers.  The other
// halves of the pairs are loaded beside a lane's own (the same lines, so HBM sees them once); all
// of a head's loads return before any of it is stored, so rows may be turned in place.
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

// sum over the LPR lanes (8, 16 or 32, aligned) that hold a head, the same in each
template <int LPR>
__device__ __forceinline__ float head_sum(float v) {
  v += __uint_as_float(xlane_partner<0>(__float_as_uint(v)));
  v += __uint_as_float(xlane_partner<1>(__float_as_uint(v)));
  v += __uint_as_float(xlane_partner<2>(__float_as_uint(v)));
  if (LPR > 8) v += __uint_as_float(xlane_partner<3>(__float_as_uint(v)));
  if (LPR > 16) v += __uint_as_float(xlane_partner<4>(__float_as_uint(v)));
  return v;
}
template <int STEP>
__device__ __forceinline__ double partner(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = xlane_partner<STEP>((uint32_t)u), hi = xlane_partner<STEP>((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(hi << 32 | lo));
}
template <int LPR>
__device__ __forceinline__ double head_sum(double v) {
  v += partner<0>(v);
  v += partner<1>(v);
  v += partner<2>(v);
  if (LPR > 8) v += partner<3>(v);
  if (LPR > 16) v += partner<4>(v);
  return v;
}

// What a lane knows of its row and its place in a head.
template <class T, int LPR>
struct RopeLane {
  static constexpr int kE = sizeof(T);
  int at, other;     // its first element, and that of the other halves of its pairs
  bool live, apart;  // it has elements at all; pairs are not neighbours
  float c[8], s[8];  // y = x c + (other of the pair) s

  __device__ __forceinline__ void begin(const RopeArgs& p, int chunk, int pos) {
    live = 8 * chunk < p.D;
    at = live ? 8 * chunk : 0;
    other = at;
    apart = !p.interleaved;
    const int half = p.rot / 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = 1.0f;
      s[e] = 0.0f;
    }
    if (!p.rope || at >= p.rot) return;
    const float* line = p.rope + (int64_t)pos * p.rot;
    if (apart) {
      const bool first = at < half;
      other = first ? at + half : at - half;
      const int i = first ? at : other;
      ld8(line + i, c);
      ld8(line + half + i, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = first ? -s[e] : s[e];
    } else {
      const float4 x = *reinterpret_cast<const float4*>(line + at / 2);
      const float4 y = *reinterpret_cast<const float4*>(line + half + at / 2);
      const float cs[4] = {x.x, x.y, x.z, x.w}, sn[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = cs[e / 2];
        s[e] = e % 2 ? sn[e / 2] : -sn[e / 2];
      }
    }
  }

  // a lane's elements of a head, in F (float or double), of its own and its pairs' other halves
  template <class F, bool NORM>
  __device__ __forceinline__ void turn(const RopeArgs& p, const Eight<T>& own, const Eight<T>& far,
                                       const Eight<T>& w, const Eight<T>& wf, F (&y)[8]) const {
    F x[8], z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = (F)own.at(e);
      z[e] = (F)(apart ? far.at(e) : own.at(e ^ 1));
    }
    if (NORM) {
      F sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += x[e] * x[e];
      sum = head_sum<LPR>(live ? sum : (F)0);
      const F f = (F)1 / sqrt(sum / (F)p.D + (F)p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = x[e] * f * (F)w.at(e);
        z[e] = z[e] * f * (F)(apart ? wf.at(e) : w.at(e ^ 1));
      }
    }
    // (a lane without pairs has c = 1, s = 0: whatever z is, it must not reach y)
    const bool turns = p.rope && at < p.rot;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = turns ? x[e] * (F)c[e] + z[e] * (F)s[e] : x[e];
  }
};

// the largest of four neighbouring lanes, which hold a group
__device__ __forceinline__ uint32_t group_top(uint32_t u) {
  u = max(u, xlane_partner<0>(u));
  return max(u, xlane_partner<1>(u));
}

template <class F>
__device__ __forceinline__ void put4(const F (&y)[8], int chunk, char* codes, uint8_t* scale) {
  uint32_t bits[8], top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bits[e] = fp4_bits(y[e]);
    top = max(top, bits[e] & 0x7FFFFFFFu);
  }
  const uint32_t byte = fp4_byte(group_top(top));
  reinterpret_cast<uint32_t*>(codes)[chunk] = fp4_codes(bits, byte);
  if (chunk % 4 == 0) scale[chunk / 4] = (uint8_t)byte;
}

template <class T, int LPR, RopeTo TO, bool NORM>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs p) {
  const int64_t group = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int i = (int)(group / p.slices), slice = (int)(group - (int64_t)i * p.slices);
  const int live = p.n_rows ? min(p.rows, *p.n_rows) : p.rows;
  if (i >= live) return;
  const int chunk = threadIdx.x % LPR;
  const bool tell = slice == 0 && chunk == 0;
  int pos = 0;
  if (p.rope) {
    pos = p.position[i];
    if (pos < 0 || pos >= p.n_pos) {
      if (tell) raise_fault(p.status, DSPARK_FAULT_PARAM);
      return;
    }
  }
  RopeLane<T, LPR> r;
  r.begin(p, chunk, pos);
  // `heads` heads of a row, from head `h0` on: f(head, own, far, w, wf)
  const auto each = [&](const void* src, int64_t row, const void* norm, int h0, int heads, auto f) {
    const T* x = static_cast<const T*>(src) + i * row;
    Eight<T> w{}, wf{};
    if (NORM && norm) {
      w.load(static_cast<const T*>(norm) + r.at);
      wf.load(static_cast<const T*>(norm) + r.other);
    }
    constexpr int kBatch = 4;  // heads whose loads are under way together
    for (int h = h0; h < heads; h += kBatch * p.slices) {
      Eight<T> own[kBatch], far[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int hu = min(h + u * p.slices, heads - 1);
        own[u].load(x + (int64_t)hu * p.D + r.at);
        far[u].load(x + (int64_t)hu * p.D + r.other);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int hu = h + u * p.slices;
        if (hu < heads) f(hu, own[u], far[u], w, wf);
      }
    }
  };
  int h = slice;
  if (p.q) {
    each(p.q, p.q_row, p.q_norm, h, p.Hq, [&](int head, const Eight<T>& own, const Eight<T>& far,
                                              const Eight<T>& w, const Eight<T>& wf) {
      float y[8];
      if (NORM && p.q_norm)
        r.template turn<float, true>(p, own, far, w, wf, y);
      else
        r.template turn<float, false>(p, own, far, w, wf, y);
      Eight<T> out;
      out.set(y);
      if (r.live) out.store(static_cast<T*>(p.q_out) + i * p.qo_row + (int64_t)head * p.D + r.at);
    });
    // the heads after these go on with the slices where they stopped
    h = (slice + p.slices - p.Hq % p.slices) % p.slices;
  }
  if (!p.k) return;
  char *kc = nullptr, *vc = nullptr;
  uint8_t* sc = nullptr;
  if (TO != kToRows) {
    const int s = p.slot[i];
    if (s < 0 || (s >> p.lg) >= p.n_pages) {
      if (s != -1 && tell) raise_fault(p.status, DSPARK_FAULT_PAGE);
      return;
    }
    const int64_t page = s >> p.lg, tok = s & ((1 << p.lg) - 1);
    kc = p.k_cache + page * p.page_b + tok * p.tok_b;
    vc = p.v_cache + page * p.page_b + tok * p.tok_b;
    if (TO == kToCache4) sc = p.scales + page * p.s_page + tok * p.s_tok;
  }
  each(p.k, p.k_row, p.k_norm, h, p.Hkv, [&](int head, const Eight<T>& own, const Eight<T>& far,
                                             const Eight<T>& w, const Eight<T>& wf) {
    typedef typename std::conditional<TO == kToCache4, double, float>::type F;
    F y[8];
    if (NORM && p.k_norm)
      r.template turn<F, true>(p, own, far, w, wf, y);
    else
      r.template turn<F, false>(p, own, far, w, wf, y);
    if constexpr (TO == kToCache4) {
      put4(y, chunk, kc + head * p.head_b, sc + head * p.s_head);
    } else {
      Eight<T> out;
      out.set(y);
      T* to = TO == kToRows ? static_cast<T*>(p.k_out) + i * p.ko_row + (int64_t)head * p.D
                            : reinterpret_cast<T*>(kc + head * p.head_b);
      if (r.live) out.store(to + r.at);
    }
  });
  if (TO == kToRows) return;
  h = (h + p.slices - p.Hkv % p.slices) % p.slices;
  const T* x = static_cast<const T*>(p.v) + i * p.v_row;
  for (; h < p.Hkv; h += p.slices) {
    Eight<T> own;
    own.load(x + (int64_t)h * p.D + r.at);
    if constexpr (TO == kToCache4) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = own.at(e);
      put4(y, chunk, vc + h * p.head_b, sc + h * p.s_head + p.D / kGroup4);
    } else {
      if (r.live) own.store(reinterpret_cast<T*>(vc + h * p.head_b) + r.at);
    }
  }
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

// Groups of lanes (a head each at a time) that a row's heads are spread over: few rows want all
// lanes they can get; many go through their heads in turn, the cosines and sines loaded once.
static int rope_slices(int rows, int heads) {
  const int64_t want = 32768 / (int64_t)rows;
  return want < 1 ? 1 : (want > heads ? heads : (int)want);
}

template <class T, RopeTo TO, bool NORM>
static int rope_launch(const RopeArgs& p, hipStream_t stream) {
  const int lpr = p.D <= 64 ? 8 : (p.D <= 128 ? 16 : 32);
  const int64_t blocks = ((int64_t)p.rows * p.slices * lpr + 255) / 256;
  if (blocks >= (1 << 24)) return DSPARK_EINVAL;  // a grid holds 2^32 threads
  if (lpr == 8)
    rope_kernel<T, 8, TO, NORM><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else if (lpr == 16)
    rope_kernel<T, 16, TO, NORM><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else if constexpr (TO != kToCache4)
    rope_kernel<T, 32, TO, NORM><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return launch_status();
}

template <RopeTo TO>
static int rope_run(RopeArgs p, dspark_dtype dt, hipStream_t stream) {
  const int heads = (p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (p.v ? p.Hkv : 0);
  p.slices = rope_slices(p.rows, heads);
  const bool norm = p.q_norm || p.k_norm;
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
      (dt != DSPARK_F32 && dt != DSPARK_BF16) || !(eps >= 0.0) || !(eps <= 1e30))
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
