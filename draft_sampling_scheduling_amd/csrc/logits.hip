// logits.hip -- the target's logits with a request's penalties, biases and grammar masks,
// moved from the step's packed rows into the layout verification reads.
//
// Bound: every logit is read and written once, so HBM bounds it.  A workgroup takes one
// request and a slice of the vocabulary and walks the request's rows: the history is scanned
// once per slice, into a word per id in LDS (times generated, seen in the prompt), and from
// there a thread keeps the words of its ids in registers; from one row to the next they change
// only by the drafted token between them.  The next row's logits load while the current
// row's are worked on.  Ids that nothing touches are copied as they are.
#include "target.h"

namespace dspark {

constexpr int kLogThreads = 256;
constexpr int kLogGroups = 2;                              // groups of 8 ids per thread
constexpr int kLogSpan = kLogThreads * 8;                  // ids between a thread's groups
constexpr int kLogSlice = kLogGroups * kLogSpan;           // ids of a workgroup
constexpr uint32_t kInPrompt = 0x80000000u;                // id seen in the prompt; below: count

struct LogitsParams {
  int R, gamma, V, rows, hist_stride, nbias, n_mask, mask_stride;
  int64_t row_stride;
  const void* logits;
  const int32_t *row_off, *ell, *x, *hist, *hist_len, *prompt_len;
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

template <class T>
__global__ void __launch_bounds__(kLogThreads) target_logits_kernel(LogitsParams p) {
  __shared__ __attribute__((aligned(16))) uint32_t seen[kLogSlice];
  __shared__ __attribute__((aligned(16))) int last_bias[kLogSlice];  // entry + 1, 0 none
  const int q = blockIdx.y, v0 = blockIdx.x * kLogSlice, tid = threadIdx.x;
  const bool tell = blockIdx.x == 0 && tid == 0;

  int L = p.ell[q];
  if (L < 0 || L > p.gamma) {
    if (tell) raise_fault(p.status, DSPARK_FAULT_LEN);
    L = L < 0 ? 0 : p.gamma;
  }
  const int64_t row0 = p.row_off ? p.row_off[q] : (int64_t)q * (p.gamma + 1);
  auto param = [&](const float* a, float none, bool positive) {
    const float x = a ? a[q] : none;
    const bool bad = !(fabsf(x) <= FLT_MAX) || (positive && !(x > 0.0f));
    if (bad && tell) raise_fault(p.status, DSPARK_FAULT_PARAM);
    return bad ? none : x;
  };
  const float rep = param(p.rep, 1.0f, true), pres = param(p.pres, 0.0f, false);
  const float freq = param(p.freq, 0.0f, false);

  // the row pointers, and the first row's logits under way before the history is scanned
  auto row_ok = [&](int j) { return row0 + j >= 0 && row0 + j < p.rows; };
  auto load_row = [&](int j, Raw8<T> (&r)[kLogGroups]) {
    const T* src = static_cast<const T*>(p.logits) + (row0 + j) * p.row_stride;
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g) {
      const int v = v0 + g * kLogSpan + tid * 8;
      if (v < p.V) r[g].load(src + v);
    }
  };
  Raw8<T> next[kLogGroups];
  if (row_ok(0)) load_row(0, next);

  for (int i = tid; i < kLogSlice; i += kLogThreads) seen[i] = 0;
  if (p.nbias > 0)
    for (int i = tid; i < kLogSlice; i += kLogThreads) last_bias[i] = 0;
  __syncthreads();
  if (p.hist) {
    int hl = p.hist_len[q], pl = p.prompt_len ? p.prompt_len[q] : 0;
    const bool bad = hl < 0 || hl > p.hist_stride || pl < 0 || pl > hl;
    if (bad && tell) raise_fault(p.status, DSPARK_FAULT_LEN);
    hl = hl < 0 ? 0 : (hl > p.hist_stride ? p.hist_stride : hl);
    const int32_t* hist = p.hist + (int64_t)q * p.hist_stride;
    for (int i = tid; i < hl; i += kLogThreads) {
      const int id = hist[i];
      const uint32_t at = (uint32_t)(id - v0);
      if (id < 0 || id >= p.V) {
        if (blockIdx.x == 0) raise_fault(p.status, DSPARK_FAULT_TOKEN);
      } else if (at < kLogSlice) {
        if (i < pl)
          atomicOr(&seen[at], kInPrompt);
        else
          atomicAdd(&seen[at], 1u);
      }
    }
  }
  for (int i = tid; i < p.nbias; i += kLogThreads) {
    const int id = p.bias_id[(int64_t)q * p.nbias + i];
    const uint32_t at = (uint32_t)(id - v0);
    if (id < -1 || id >= p.V) {
      if (blockIdx.x == 0) raise_fault(p.status, DSPARK_FAULT_TOKEN);
    } else if (id >= 0 && at < kLogSlice) {
      atomicMax(&last_bias[at], i + 1);
    }
  }
  __syncthreads();

  uint32_t w[kLogGroups][8];
  float add[kLogGroups][8];
  bool touched[kLogGroups];
#pragma unroll
  for (int g = 0; g < kLogGroups; ++g) {
    touched[g] = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = g * kLogSpan + tid * 8 + e;
      w[g][e] = seen[at];
      const int b = p.nbias > 0 ? last_bias[at] : 0;
      add[g][e] = b > 0 ? p.bias[(int64_t)q * p.nbias + b - 1] : 0.0f;
      touched[g] = touched[g] || w[g][e] != 0 || b > 0;
    }
  }

  for (int j = 0; j <= L; ++j) {
    Raw8<T> cur[kLogGroups];
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g) cur[g] = next[g];
    if (j < L && row_ok(j + 1)) load_row(j + 1, next);
    if (j > 0) {  // the token drafted between the last row and this one
      const int id = p.x[(int64_t)q * p.gamma + j - 1];
      if ((id < 0 || id >= p.V) && tell) raise_fault(p.status, DSPARK_FAULT_TOKEN);
#pragma unroll
      for (int g = 0; g < kLogGroups; ++g) {
        const uint32_t at = (uint32_t)(id - (v0 + g * kLogSpan + tid * 8));
        if (id >= 0 && id < p.V && at < 8) {
          touched[g] = true;
#pragma unroll
          for (int e = 0; e < 8; ++e) w[g][e] += at == (uint32_t)e ? 1u : 0u;
        }
      }
    }
    if (!row_ok(j)) {
      if (tell) raise_fault(p.status, DSPARK_FAULT_LEN);
      continue;
    }
    const uint8_t* allow = nullptr;  // a bit per id
    if (p.mask) {
      const int64_t at = (int64_t)q * (p.gamma + 1) + j;
      const int64_t i = p.mask_idx ? p.mask_idx[at] : at;
      if (i < -1 || i >= p.n_mask) {
        if (tell) raise_fault(p.status, DSPARK_FAULT_PARAM);
      } else if (i >= 0) {
        allow = reinterpret_cast<const uint8_t*>(p.mask + i * p.mask_stride);
      }
    }
    T* dst = static_cast<T*>(p.out) + ((int64_t)q * (p.gamma + 1) + j) * p.V;
#pragma unroll
    for (int g = 0; g < kLogGroups; ++g) {
      const int v = v0 + g * kLogSpan + tid * 8;
      if (v >= p.V) continue;
      const uint32_t bits = allow ? allow[v >> 3] : 0xFFu;
      if (touched[g] || bits != 0xFFu) {
        float l[8];
        cur[g].get(l);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (w[g][e] != 0) {
            const float c = (float)(w[g][e] & ~kInPrompt);
            l[e] = l[e] > 0.0f ? l[e] / rep : l[e] * rep;
            l[e] -= freq * c + (c > 0.0f ? pres : 0.0f);
          }
          l[e] += add[g][e];
          l[e] = (bits >> e) & 1 ? l[e] : -INFINITY;
        }
        cur[g].set(l);
      }
      cur[g].store(dst + v);
    }
  }
}

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_target_logits(int R, int gamma, int V, dspark_dtype dt, const void* logits,
                                    int64_t row_stride, int rows, const int32_t* row_off,
                                    const int32_t* ell, const int32_t* x, const int32_t* hist,
                                    int hist_stride, const int32_t* hist_len,
                                    const int32_t* prompt_len, const float* rep,
                                    const float* pres, const float* freq, const int32_t* bias_id,
                                    const float* bias, int nbias, const uint32_t* mask,
                                    int n_mask, int mask_stride, const int32_t* mask_idx,
                                    void* out, int32_t* dev_status, hipStream_t stream) {
  if (R < 0 || R > 65535 || gamma < 1 || gamma > kMaxGamma || V < 8 || V % 8 != 0 ||
      (dt != DSPARK_F32 && dt != DSPARK_BF16) || rows < 0 || row_stride < V || nbias < 0)
    return DSPARK_EINVAL;
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  if (!stride_ok(row_stride, e)) return DSPARK_EINVAL;
  if (R == 0) return DSPARK_OK;
  if (!logits || !ell || !x || !out || !aligned16(logits) || !aligned16(out) ||
      (hist && (!hist_len || hist_stride < 0)) || (nbias > 0 && (!bias_id || !bias)) ||
      (mask && (n_mask < 1 || mask_stride < (V + 31) / 32)))
    return DSPARK_EINVAL;
  // in place only where a row stays where it is
  if (out == logits && (row_off || row_stride != V)) return DSPARK_EINVAL;
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
  const dim3 grid((V + kLogSlice - 1) / kLogSlice, R);
  if (dt == DSPARK_BF16)
    target_logits_kernel<uint16_t><<<grid, kLogThreads, 0, stream>>>(p);
  else
    target_logits_kernel<float><<<grid, kLogThreads, 0, stream>>>(p);
  return launch_status();
}
