// logits.hip -- the target's logits with a request's penalties, biases and grammar masks,
// moved from the step's packed rows into the layout verification reads.
//
// Bound: every logit is read and written once, so HBM bounds it.  A workgroup takes one request
// and a slice of the vocabulary and walks the request's rows (all of them, or some where there are
// few requests): it scans the history once, into a word per id in LDS (times generated, seen in
// the prompt), and from there a thread keeps the words of its ids in registers; from one row to
// the next they change only by the drafted token between them (in a tree: by the tokens above one
// of the two nodes and not the other).  A row's operands load while the row before it is worked
// on.  Ids that nothing touches are copied as they are.  Measured: 256 requests, 151936 ids, bf16,
// up to nine rows each (786 MB): 154 to 170 us, 4.6 to 5.1 TB/s, a copy's rate; loads that were not
// all issued a row ahead (the mask's bits behind the next row's logits) had made it 257 us.  4
// requests of 1024 ids, up to five rows: 5.8 us, the trips to memory.  Trees: 256 requests of nine
// nodes as long as chains; 16 of 65 nodes, 32000 ids, 52 us where chains take 32, for the tokens
// turned over between rows.
#include <type_traits>

#include "target.h"

namespace dspark {

constexpr int kLogThreads = 256;
constexpr int kLogGroups = 2;                              // groups of 8 ids per thread (4: 177 us)
constexpr int kLogSpan = kLogThreads * 8;                  // ids between a thread's groups
constexpr int kLogSlice = kLogGroups * kLogSpan;           // ids of a workgroup
constexpr uint32_t kInPrompt = 0x80000000u;                // id seen in the prompt; below: count

struct LogitsParams {
  int R, gamma, V, rows, hist_stride, nbias, n_mask, mask_stride;
  int per;  // rows of a request that a workgroup takes
  int64_t row_stride;
  const void* logits;
  const int32_t *row_off, *ell, *x, *hist, *hist_len, *prompt_len;
  const uint64_t* anc;
  const float *rep, *pres, *freq;
  const int32_t* bias_id;
  const float* bias;
  const uint32_t* mask;
  const int32_t* mask_idx;
  void* out;
  int32_t* status;
};

// 8 logits as loaded
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = bf16lo(a.x); x[1] = bf16hi(a.x); x[2] = bf16lo(a.y); x[3] = bf16hi(a.y);
    x[4] = bf16lo(a.z); x[5] = bf16hi(a.z); x[6] = bf16lo(a.w); x[7] = bf16hi(a.w);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// inputs that every lane reads alike, through the scalar cache
template <class V>
__device__ __forceinline__ V uniform_load(const V* p, int64_t i) {
  return ((const __attribute__((address_space(4))) V*)p)[i];
}

// PARTS: a request's rows go to several workgroups, p.per to each.  TREE: the drafted tokens
// that a row counts are those of its mask in p.anc, not all before it.
template <class T, bool PARTS, bool TREE>
__global__ void __launch_bounds__(kLogThreads) target_logits_kernel(LogitsParams p) {
  // one word per id of the slice: first what the history holds of it, then (its words in
  // registers) which bias entry is its last
  __shared__ __attribute__((aligned(16))) uint32_t word[kLogSlice];
  const int q = blockIdx.y, v0 = blockIdx.x * kLogSlice, tid = threadIdx.x;
  const int j0 = PARTS ? blockIdx.z * p.per : 0;
  const bool tell = blockIdx.x == 0 && tid == 0;

  // Everything that can be asked for at once is: the request's scalars, and the first ids of
  // its history and biases (clamped to the arrays, not to their lengths, which come with
  // them).  In a small step the round trips are all there is.
  int L = uniform_load(p.ell, q);
  const int64_t row0 = p.row_off ? uniform_load(p.row_off, q) : (int64_t)q * (p.gamma + 1);
  const int64_t row1 = p.row_off ? uniform_load(p.row_off, (int64_t)q + 1) : p.rows;
  const int64_t rows = row1 < p.rows ? row1 : p.rows;  // the request's end before them
  const bool has_hist = p.hist && p.hist_stride > 0;
  int hl = p.hist ? uniform_load(p.hist_len, q) : 0;
  const int pl = p.hist && p.prompt_len ? uniform_load(p.prompt_len, q) : 0;
  const float rep_in = p.rep ? uniform_load(p.rep, q) : 1.0f;
  const float pres_in = p.pres ? uniform_load(p.pres, q) : 0.0f;
  const float freq_in = p.freq ? uniform_load(p.freq, q) : 0.0f;
  constexpr int kBatch = 4;  // ids in flight per thread
  const int32_t* hist = p.hist + (int64_t)q * p.hist_stride;
  int id[kBatch];
  auto load_ids = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kLogThreads;
      id[u] = hist[i < p.hist_stride ? i : p.hist_stride - 1];
    }
  };
  if (has_hist) load_ids(tid);
  const int32_t* bias_id = p.bias_id + (int64_t)q * p.nbias;
  // tokens drafted before the workgroup's first row count as the history's
  const int drafted = PARTS && !TREE && tid < j0 ? p.x[(int64_t)q * p.gamma + tid] : -1;
  // a tree's tokens, one a lane (gamma <= 64)
  const int lane = tid & (kWave - 1);
  const int tokens = TREE ? p.x[(int64_t)q * p.gamma + (lane < p.gamma ? lane : p.gamma - 1)] : 0;
  int first_bias = -1;
  if (p.nbias > 0) first_bias = bias_id[tid < p.nbias ? tid : p.nbias - 1];

  if (L < 0 || L > p.gamma) {
    if (tell) raise_fault(p.status, DSPARK_FAULT_LEN);
    L = L < 0 ? 0 : p.gamma;
  }
  if (PARTS && j0 > L) return;
  const int last = PARTS && j0 + p.per - 1 < L ? j0 + p.per - 1 : L;
  auto param = [&](float x, float none, bool positive) {
    const bool bad = !(fabsf(x) <= FLT_MAX) || (positive && !(x >= FLT_MIN));
    if (bad && tell) raise_fault(p.status, DSPARK_FAULT_PARAM);
    return bad ? none : x;
  };
  const float rep = param(rep_in, 1.0f, true), pres = param(pres_in, 0.0f, false);
  const float freq = param(freq_in, 0.0f, false);
  // l / rep as l * (hi + lo), hi + lo = 1 / rep to 48 bits: fma(l, hi, l * lo) rounds once what is
  // off by 2^-47 of itself (of 3e9 pairs of mantissas 63 gave another float than l / rep).  hi is
  // rounded down and lo above 0, so that an infinite l stays one.  Where lo would lose its bits
  // (rep past 2^60), l is divided proper, and this leaves it so.  A product and the quotient of
  // its exact remainder leave none of the 63, but bound the kernel by its arithmetic: 169 us for
  // 159 at the headline, 26 for 21 with 16 requests.
  const bool far = !(rep >= 0x1p-60f && rep <= 0x1p60f);
  float hi = far ? 1.0f : 1.0f / rep;
  if (!far && fmaf(-rep, hi, 1.0f) < 0.0f) hi = __uint_as_float(__float_as_uint(hi) - 1);
  const float lo = far ? FLT_MIN : fmaxf(fmaf(-rep, hi, 1.0f) * hi, FLT_MIN);

  // A row's operands: its mask's bits of the thread's ids, then its logits.  Loads return in
  // order, so a row waits for its own only if all of them are issued a row ahead.
  struct Row {
    Raw8<T> x[kLogGroups];
    uint32_t bits[kLogGroups];
    uint64_t anc;  // TREE: the nodes j >= 1 (bit j - 1) on the way to the row's
  };
  auto row_ok = [&](int j) { return row0 + j >= 0 && row0 + j < rows; };
  auto load_row = [&](int j, Row& r) {
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g) r.bits[g] = 0xFFu;
    if (!row_ok(j)) return;
    if (TREE) r.anc = uniform_load(p.anc, row0 + j) & (~(uint64_t)0 >> (kMaxGamma - p.gamma));
    if (p.mask) {
      const int64_t at = (int64_t)q * (p.gamma + 1) + j;
      const int64_t i = p.mask_idx ? uniform_load(p.mask_idx, at) : at;
      if (i < -1 || i >= p.n_mask) {
        if (tell) raise_fault(p.status, DSPARK_FAULT_PARAM);
      } else if (i >= 0) {
        const uint8_t* allow = reinterpret_cast<const uint8_t*>(p.mask + i * p.mask_stride);
#pragma unroll
        for (int g = 0; g < kLogGroups; ++g) {
          const int v = v0 + g * kLogSpan + tid * 8;
          if (v < p.V) r.bits[g] = allow[v >> 3];
        }
      }
    }
    const T* src = static_cast<const T*>(p.logits) + (row0 + j) * p.row_stride;
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g) {
      const int v = v0 + g * kLogSpan + tid * 8;
      if (v < p.V) r.x[g].load(src + v);
    }
  };
  Row next;
  load_row(j0, next);  // under way while the history is scanned

  auto clear = [&]() {
    for (int i = tid; i < kLogSlice / 4; i += kLogThreads)
      reinterpret_cast<uint4*>(word)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  };
  uint32_t w[kLogGroups][8];
  float add[kLogGroups][8];
  bool touched[kLogGroups];
  clear();
  if (p.hist) {
    const bool bad = hl < 0 || hl > p.hist_stride || pl < 0 || pl > hl;
    if (bad && tell) raise_fault(p.status, DSPARK_FAULT_LEN);
    hl = hl < 0 ? 0 : (hl > p.hist_stride ? p.hist_stride : hl);
    for (int i0 = tid; i0 < hl; i0 += kBatch * kLogThreads) {
      int cur[kBatch];  // the next batch loads meanwhile (16 histories of up to 60000: 43 us, 31 so)
#pragma unroll
      for (int u = 0; u < kBatch; ++u) cur[u] = id[u];
      if (i0 + kBatch * kLogThreads < hl) load_ids(i0 + kBatch * kLogThreads);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kLogThreads;
        const uint32_t at = (uint32_t)(cur[u] - v0);
        if (i >= hl) continue;
        if (cur[u] < 0 || cur[u] >= p.V) {
          if (blockIdx.x == 0) raise_fault(p.status, DSPARK_FAULT_TOKEN);
        } else if (at < kLogSlice) {
          if (i < pl)
            atomicOr(&word[at], kInPrompt);
          else
            atomicAdd(&word[at], 1u);
        }
      }
    }
  }
  if (PARTS && !TREE && tid < j0) {
    if (drafted < 0 || drafted >= p.V) {
      if (blockIdx.x == 0) raise_fault(p.status, DSPARK_FAULT_TOKEN);
    } else if ((uint32_t)(drafted - v0) < kLogSlice) {
      atomicAdd(&word[drafted - v0], 1u);
    }
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kLogGroups; ++g) {
    touched[g] = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[g][e] = word[g * kLogSpan + tid * 8 + e];
      add[g][e] = 0.0f;
      touched[g] = touched[g] || w[g][e] != 0;
    }
  }
  if (p.nbias > 0) {
    __syncthreads();
    clear();
    for (int i = tid; i < p.nbias; i += kLogThreads) {
      const int id = i == tid ? first_bias : bias_id[i];
      const uint32_t at = (uint32_t)(id - v0);
      if (id < -1 || id >= p.V) {
        if (blockIdx.x == 0) raise_fault(p.status, DSPARK_FAULT_TOKEN);
      } else if (id >= 0 && at < kLogSlice) {
        atomicMax(&word[at], (uint32_t)i + 1);
      }
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t i = word[g * kLogSpan + tid * 8 + e];
        if (i > 0) {
          add[g][e] = p.bias[(int64_t)q * p.nbias + i - 1];
          touched[g] = true;
        }
      }
  }

  // one more drafted token (or, by = -1, one less) among what the rows count
  auto count = [&](int id, uint32_t by) {
    if ((id < 0 || id >= p.V) && tell) raise_fault(p.status, DSPARK_FAULT_TOKEN);
    const uint32_t in = (uint32_t)(id - v0);
    if (id < 0 || id >= p.V || in >= kLogSlice) return;
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g) {
      const uint32_t at = in - (uint32_t)(g * kLogSpan + tid * 8);
      touched[g] = touched[g] || at < 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[g][e] += at == (uint32_t)e ? by : 0u;
    }
  };
  uint64_t above = 0;  // TREE: the nodes counted
  for (int j = j0; j <= last; ++j) {
    Row cur = next;
    if (j < last) load_row(j + 1, next);
    if (TREE) {
      if (row_ok(j)) {
        for (uint64_t turn = above ^ cur.anc; turn != 0; turn &= turn - 1) {
          const int b = __builtin_ctzll(turn);
          count(__builtin_amdgcn_readlane(tokens, b), (cur.anc >> b) & 1 ? 1u : ~0u);
        }
        above = cur.anc;
      }
    } else if (j > j0) {  // the token drafted between the last row and this one
      count(uniform_load(p.x, (int64_t)q * p.gamma + j - 1), 1u);
    }
    if (!row_ok(j)) {
      if (tell) raise_fault(p.status, DSPARK_FAULT_LEN);
      continue;
    }
    T* dst = static_cast<T*>(p.out) + ((int64_t)q * (p.gamma + 1) + j) * p.V;
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g) {
      const int v = v0 + g * kLogSpan + tid * 8;
      if (v >= p.V) continue;
      const uint32_t bits = cur.bits[g];
      if (touched[g] || bits != 0xFFu) {
        float l[8];
        cur.x[g].get(l);
        if (far) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (w[g][e] != 0 && l[e] > 0.0f) l[e] /= rep;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // branch-free: ids that nothing touches are multiplied by 1 and lose 0
          const float c = (float)(w[g][e] & ~kInPrompt);
          const bool seen = w[g][e] != 0;
          const float x = l[e] * (seen ? rep : 1.0f), y = fmaf(l[e], hi, l[e] * lo);
          l[e] = seen && l[e] > 0.0f ? y : x;
          l[e] = fmaf(-freq, c, l[e]) - (c > 0.0f ? pres : 0.0f) + add[g][e];
          l[e] = (bits >> e) & 1 ? l[e] : -INFINITY;
        }
        cur.x[g].set(l);
      }
      cur.x[g].store(dst + v);
    }
  }
}

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_target_logits_tree(
    int R, int gamma, int V, dspark_dtype dt, const void* logits, int64_t row_stride, int rows,
    const int32_t* row_off, const int32_t* ell, const int32_t* x, const uint64_t* anc,
    const int32_t* hist, int hist_stride, const int32_t* hist_len, const int32_t* prompt_len,
    const float* rep, const float* pres, const float* freq, const int32_t* bias_id,
    const float* bias, int nbias, const uint32_t* mask, int n_mask, int mask_stride,
    const int32_t* mask_idx, void* out, int32_t* dev_status, hipStream_t stream) {
  if (R < 0 || R > 65535 || gamma < 1 || gamma > kMaxGamma || V < 8 || V > 1 << 30 || V % 8 != 0 ||
      (dt != DSPARK_F32 && dt != DSPARK_BF16) || rows < 0 || row_stride < V || nbias < 0)
    return DSPARK_EINVAL;
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  if (!stride_ok(row_stride, e)) return DSPARK_EINVAL;
  if (R == 0) return DSPARK_OK;
  if ((!logits && rows > 0) || !ell || !x || !out || !aligned16(logits) || !aligned16(out) ||
      (hist && (!hist_len || hist_stride < 0)) || (nbias > 0 && (!bias_id || !bias)) ||
      (mask && (n_mask < 1 || mask_stride < (V + 31) / 32)))
    return DSPARK_EINVAL;
  // in place only where a row stays where it is
  const size_t out_bytes = (size_t)R * (gamma + 1) * V * e;
  const bool in_place = out == logits && !row_off && row_stride == V;
  if (!in_place && rows > 0 &&
      overlap(logits, ((size_t)(rows - 1) * row_stride + V) * e, out, out_bytes))
    return DSPARK_EINVAL;
  LogitsParams p{};
  p.R = R;
  p.gamma = gamma;
  p.V = V;
  p.rows = rows;
  p.hist_stride = hist_stride;
  p.nbias = nbias;
  p.n_mask = n_mask;
  p.mask_stride = mask_stride;
  p.row_stride = row_stride;
  p.logits = logits;
  p.row_off = row_off;
  p.ell = ell;
  p.x = x;
  p.anc = anc;
  p.hist = hist;
  p.hist_len = hist_len;
  p.prompt_len = prompt_len;
  p.rep = rep;
  p.pres = pres;
  p.freq = freq;
  p.bias_id = bias_id;
  p.bias = bias;
  p.mask = mask;
  p.mask_idx = mask_idx;
  p.out = out;
  p.status = dev_status;
  // Where the requests' slices are fewer than one for two workgroups a CU, a request's rows go to
  // several workgroups, each with a scan of its own, instead of one after the other: 8 requests
  // of 32000 ids, up to 17 rows, 10.7 us against 33; 32 of 9 rows 14.5 against 18.9.
  const int slices = (V + kLogSlice - 1) / kLogSlice;
  const int64_t parts = 2 * device_cus() / ((int64_t)slices * R);
  p.per = parts > 1 ? (gamma + (int)parts) / (int)parts : gamma + 1;
  const dim3 grid(slices, R, gamma / p.per + 1);
  auto run = [&](auto kern) { kern<<<grid, kLogThreads, 0, stream>>>(p); };
  auto pick = [&](auto tree) {
    constexpr bool TREE = decltype(tree)::value;
    if (dt == DSPARK_BF16)
      run(parts > 1 ? target_logits_kernel<uint16_t, true, TREE>
                    : target_logits_kernel<uint16_t, false, TREE>);
    else
      run(parts > 1 ? target_logits_kernel<float, true, TREE>
                    : target_logits_kernel<float, false, TREE>);
  };
  if (anc)
    pick(std::true_type{});
  else
    pick(std::false_type{});
  return launch_status();
}

extern "C" int dspark_target_logits(int R, int gamma, int V, dspark_dtype dt, const void* logits,
                                    int64_t row_stride, int rows, const int32_t* row_off,
                                    const int32_t* ell, const int32_t* x, const int32_t* hist,
                                    int hist_stride, const int32_t* hist_len,
                                    const int32_t* prompt_len, const float* rep,
                                    const float* pres, const float* freq, const int32_t* bias_id,
                                    const float* bias, int nbias, const uint32_t* mask,
                                    int n_mask, int mask_stride, const int32_t* mask_idx,
                                    void* out, int32_t* dev_status, hipStream_t stream) {
  return dspark_target_logits_tree(R, gamma, V, dt, logits, row_stride, rows, row_off, ell, x,
                                   nullptr, hist, hist_stride, hist_len, prompt_len, rep, pres,
                                   freq, bias_id, bias, nbias, mask, n_mask, mask_stride, mask_idx,
                                   out, dev_status, stream);
}
