// cache.hip -- the paged cache around the target's pass: the step plan (rows, pages and
// slots from lengths on the device), the append of a step's keys and values, and the commit
// after verification.
//
// All three are bound by latency: a plan reads and writes a few words per request and row, an
// append copies two short rows per token.  What counts is the number of launches and of
// dependent trips to memory, so each scan over the requests is one workgroup's, and all that
// follows from it is one flat kernel.
#include "target.h"

namespace dspark {

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;

struct PlanWs {
  int32_t* held;   // [R] pages held before the call
  int32_t* take;   // [R] pages handed out to q
  int32_t* first;  // [R] index of q's first page among those handed out
  int32_t* nfree;  // [1] free pages before the call
  size_t bytes;
};

static PlanWs carve_plan(void* ws, int R) {
  Carve cv(ws);
  PlanWs w{};
  w.held = cv.take<int32_t>((size_t)R);
  w.take = cv.take<int32_t>((size_t)R);
  w.first = cv.take<int32_t>((size_t)R);
  w.nfree = cv.take<int32_t>(1);
  w.bytes = cv.bytes();
  return w;
}

// Rows and pages of every request: three scans (rows asked for, pages asked for by those
// whose rows fit, rows granted), each request in its thread's consecutive run.  A request's
// rows fit in a prefix of the requests that ask for any, and of those its pages are had in a
// prefix of the ones that need any, so the exclusive sum of the needs is also the count of
// pages handed out before it.
__global__ void __launch_bounds__(kPlanThreads) plan_scan_kernel(
    int R, int rows, int lg, int max_pages, int free_len, int extra,
    const int32_t* __restrict__ lens, const int32_t* __restrict__ ctx, int32_t* held,
    int32_t* n_free, int tree_nodes, int32_t* row_off, PlanWs ws, int32_t* status) {
  __shared__ int64_t sums[kPlanThreads / kWave];
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(R, (int)threadIdx.x * per), hi = min(R, lo + per);
  int nf = *n_free;
  if (nf < 0 || nf > free_len) {
    if (threadIdx.x == 0) raise_fault(status, DSPARK_FAULT_PAGE);
    nf = nf < 0 ? 0 : free_len;
  }
  // rows request q asks for (0 where refused) and the pages they lack
  auto ask = [&](int q, bool tell, int& n, int& need) {
    const int64_t m = (int64_t)lens[q] + extra, c = ctx[q];
    const int64_t h = held[q];
    const bool bad = m < 0 || c < 0 || h < 0 || h > max_pages ||
                     c + m > ((int64_t)max_pages << lg) || m > tree_nodes;
    if (bad && tell) raise_fault(status, DSPARK_FAULT_LEN);
    n = bad ? 0 : (int)m;
    const int64_t want = n == 0 ? 0 : ((c + n + (1 << lg) - 1) >> lg) - h;
    need = want > 0 ? (int)want : 0;
  };
  int64_t s = 0;
  for (int q = lo; q < hi; ++q) {
    int n, need;
    ask(q, true, n, need);
    s += n;
  }
  int64_t base_n = block_scan<kPlanThreads>(s, sums) - s;
  // pages asked for by the requests whose rows fit
  int64_t run = base_n;
  s = 0;
  for (int q = lo; q < hi; ++q) {
    int n, need;
    ask(q, false, n, need);
    run += n;
    if (n > 0 && run > rows) raise_fault(status, DSPARK_FAULT_LEN);
    s += run <= rows ? need : 0;
  }
  int64_t base_p = block_scan<kPlanThreads>(s, sums) - s;
  // rows granted
  run = base_n;
  int64_t pages = base_p;
  s = 0;
  for (int q = lo; q < hi; ++q) {
    int n, need;
    ask(q, false, n, need);
    run += n;
    need = run <= rows ? need : 0;
    const int64_t before = pages;
    pages += need;
    const bool lack = need > 0 && pages > nf;
    if (lack) raise_fault(status, DSPARK_FAULT_PAGE);
    s += run <= rows && !lack ? n : 0;
    ws.take[q] = lack ? 0 : need;
    ws.first[q] = (int32_t)(before < nf ? before : 0);
  }
  int64_t at = block_scan<kPlanThreads>(s, sums) - s;
  run = base_n;
  pages = base_p;
  s = 0;  // pages handed out
  for (int q = lo; q < hi; ++q) {
    int n, need;
    ask(q, false, n, need);
    run += n;
    need = run <= rows ? need : 0;
    pages += need;
    const bool served = run <= rows && !(need > 0 && pages > nf);
    row_off[q] = (int32_t)at;
    at += served ? n : 0;
    const int h = held[q];
    ws.held[q] = h;
    if (served && need > 0) {
      held[q] = h + need;
      s += need;
    }
    if (q == R - 1) row_off[R] = (int32_t)at;
  }
  const int64_t out = block_scan<kPlanThreads>(s, sums);
  if (threadIdx.x == kPlanThreads - 1) {
    ws.nfree[0] = nf;
    *n_free = nf - (int32_t)out;
  }
}

// One workgroup per request and slice of its rows: its new pages into the table, and each
// row's slot, position and ancestors.  A row's ancestors are a walk up at most 64 parents,
// read from LDS.
__global__ void __launch_bounds__(kRowThreads) plan_rows_kernel(
    int lg, int max_pages, const int32_t* __restrict__ ctx, int32_t* table,
    const int32_t* __restrict__ free_pages, const int32_t* __restrict__ parent, int width,
    const int32_t* __restrict__ row_off, PlanWs ws, int32_t* __restrict__ req,
    int32_t* __restrict__ position, int32_t* __restrict__ slot, uint64_t* __restrict__ anc,
    int32_t* status) {
  __shared__ int up[DSPARK_MAX_TREE_NODES];
  const int q = blockIdx.x;
  const int a = row_off[q], n = row_off[q + 1] - a;
  const int had = ws.held[q], take = ws.take[q], c = ctx[q];
  // the k-th of q's new pages is top[-k]
  const int32_t* top = free_pages + (ws.nfree[0] - 1 - ws.first[q]);
  int32_t* row = table + (size_t)q * max_pages;
  if (n == 0) return;
  const int t0 = blockIdx.y * kRowThreads + threadIdx.x, step = gridDim.y * kRowThreads;
  for (int k = t0; k < take; k += step) row[had + k] = top[-k];
  if (parent) {
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      int p = i == 0 ? 0 : parent[(size_t)q * width + i];
      if (i > 0 && (p < 0 || p >= i)) {
        raise_fault(status, DSPARK_FAULT_TREE);
        p = i - 1;
      }
      up[i] = p;
    }
    __syncthreads();
  }
  for (int i = t0; i < n; i += step) {
    const int t = c + i, idx = t >> lg;
    const int page = idx < had ? row[idx] : top[-(idx - had)];
    int s = -1;
    if (page < 0 || page > (0x7fffffff >> lg))
      raise_fault(status, DSPARK_FAULT_PAGE);
    else
      s = (page << lg) + (t & ((1 << lg) - 1));
    int depth = i;
    if (parent) {
      uint64_t bits = 0;
      depth = 0;
      for (int j = i; j > 0; j = up[j]) {
        bits |= (uint64_t)1 << (j - 1);
        ++depth;
      }
      anc[a + i] = bits;
    }
    slot[a + i] = s;
    if (req) req[a + i] = q;
    if (position) position[a + i] = c + depth;
  }
}

// ---------------------------------------------------------------------------------------
// append: one thread per 16-byte piece of a row's keys and of its values
// ---------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) append_kernel(
    int rows, int pieces, int chunks, int lg, int n_pages, const uint4* __restrict__ k,
    const uint4* __restrict__ v, int64_t k_row, int64_t v_row, const int32_t* __restrict__ slot,
    const int32_t* __restrict__ n_rows, uint4* __restrict__ k_cache, uint4* __restrict__ v_cache,
    int64_t page_stride, int64_t head_stride, int64_t tok_stride, int32_t* status) {
  // strides in 16-byte pieces; a row is `pieces` = Hkv * chunks of them
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int i = (int)(at / pieces), p = (int)(at % pieces);
  const int live = n_rows ? min(rows, *n_rows) : rows;
  if (i >= live) return;
  const int s = slot[i];
  if (s < 0 || (s >> lg) >= n_pages) {
    if (s != -1 && p == 0) raise_fault(status, DSPARK_FAULT_PAGE);
    return;
  }
  const int64_t to = (int64_t)(s >> lg) * page_stride + (int64_t)(s & ((1 << lg) - 1)) * tok_stride +
                     (int64_t)(p / chunks) * head_stride + p % chunks;
  const uint4 a = k[i * k_row + p], b = v[i * v_row + p];
  k_cache[to] = a;
  v_cache[to] = b;
}

// ---------------------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------------------
struct CommitWs {
  int32_t* ctx;    // [R] lengths before the call
  int32_t* held;   // [R] pages held before the call
  int32_t* first;  // [R] place of q's first page on the free list
  size_t bytes;
};

static CommitWs carve_commit(void* ws, int R) {
  Carve cv(ws);
  CommitWs w{};
  w.ctx = cv.take<int32_t>((size_t)R);
  w.held = cv.take<int32_t>((size_t)R);
  w.first = cv.take<int32_t>((size_t)R);
  w.bytes = cv.bytes();
  return w;
}

// accepted nodes that fit the pages held (-1: the request had no rows)
__device__ __forceinline__ int clamp_acc(int na, int c, int h, int lg, int most) {
  const int64_t room = ((int64_t)h << lg) - c - 1;
  if (na > most) na = most;
  if (na > room) na = (int)(room < -1 ? -1 : room);
  return na < -1 ? -1 : na;
}

__global__ void __launch_bounds__(kPlanThreads) commit_scan_kernel(
    int R, int most, int lg, int max_pages, int free_len, const int32_t* __restrict__ n_acc,
    const int32_t* __restrict__ done, const int32_t* ctx, int32_t* ctx_out, int32_t* held,
    int32_t* n_free, CommitWs ws, int32_t* status) {
  __shared__ int64_t sums[kPlanThreads / kWave];
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(R, (int)threadIdx.x * per), hi = min(R, lo + per);
  int64_t s = 0;
  for (int q = lo; q < hi; ++q) {
    int h = held[q];
    if (h < 0 || h > max_pages) {
      raise_fault(status, DSPARK_FAULT_LEN);
      h = h < 0 ? 0 : max_pages;
    }
    const bool end = done && done[q] != 0;
    const int c = ctx[q];
    ws.ctx[q] = c;
    ws.held[q] = h;
    if (end) {
      s += h;
      ctx_out[q] = 0;
    } else {
      const int na = clamp_acc(n_acc[q], c, h, lg, most);
      if (na != n_acc[q]) raise_fault(status, DSPARK_FAULT_LEN);
      ctx_out[q] = c + na + 1;
    }
  }
  if (!done) return;
  int nf = *n_free;
  if (nf < 0 || nf > free_len) {
    if (threadIdx.x == 0) raise_fault(status, DSPARK_FAULT_PAGE);
    nf = nf < 0 ? 0 : free_len;
  }
  const int64_t end = block_scan<kPlanThreads>(s, sums);
  int64_t at = nf + end - s;
  for (int q = lo; q < hi; ++q) {
    ws.first[q] = (int32_t)(at < free_len ? at : free_len);
    if (done[q] != 0) {
      at += ws.held[q];
      held[q] = 0;
    }
  }
  if (threadIdx.x == kPlanThreads - 1) {
    const int64_t total = nf + end;
    if (total > free_len) raise_fault(status, DSPARK_FAULT_PAGE);
    *n_free = (int32_t)(total < free_len ? total : free_len);
  }
}

// One workgroup per request and 256 of the 16-byte columns (layer, keys or values, head,
// piece of D) of its tokens.  A thread owns its column, so the moves of one column are one
// thread's: a batch of eight tokens is read before any of them is written, and since the path
// ascends (its i-th node is at least i), no later batch reads a token that an earlier one
// wrote.  The first slice also gives a finished request's pages back.
__global__ void __launch_bounds__(256) commit_move_kernel(
    int gamma, int lg, int max_pages, int free_len, const int32_t* __restrict__ n_acc,
    const int32_t* __restrict__ path, const int32_t* __restrict__ done,
    const int32_t* __restrict__ table, int32_t* __restrict__ free_pages, int layers, int Hkv,
    int chunks, int n_pages, uint4* k_cache, uint4* v_cache, int64_t layer_stride,
    int64_t page_stride, int64_t head_stride, int64_t tok_stride, CommitWs ws, int32_t* status) {
  const int q = blockIdx.x;
  const int c = ws.ctx[q], h = ws.held[q];
  const int32_t* pages = table + (size_t)q * max_pages;
  if (done && done[q] != 0) {
    const int at = ws.first[q];
    if (blockIdx.y == 0)
      for (int k = threadIdx.x; k < h && at + k < free_len; k += 256) free_pages[at + k] = pages[k];
    return;
  }
  if (!path || c < 0) return;
  const int na = clamp_acc(n_acc[q], c, h, lg, gamma);
  if (na < 1) return;
  const int per_layer = 2 * Hkv * chunks;
  const int64_t col = (int64_t)blockIdx.y * 256 + threadIdx.x;
  const bool mine = col < (int64_t)layers * per_layer;
  int64_t at = 0;
  uint4* cache = k_cache;
  if (mine) {
    const int layer = (int)(col / per_layer);
    int r = (int)(col % per_layer);
    if (r >= Hkv * chunks) {
      cache = v_cache;
      r -= Hkv * chunks;
    }
    at = layer * layer_stride + (int64_t)(r / chunks) * head_stride + r % chunks;
  }
  const bool tell = blockIdx.y == 0 && threadIdx.x == 0;
  const int mask = (1 << lg) - 1;
  constexpr int kBatch = 8;
  int last = 0;
  bool stop = false;
  for (int i0 = 1; i0 <= na && !stop; i0 += kBatch) {
    int64_t from[kBatch], to[kBatch];  // -1: nothing moves
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u;
      const int p = path[(size_t)q * gamma + (i <= na ? i - 1 : 0)];
      const bool fine = p > last && (int64_t)c + p < ((int64_t)h << lg);
      if (i <= na && !stop && !fine && tell) raise_fault(status, DSPARK_FAULT_TREE);
      stop = stop || i > na || !fine;
      const int src = stop ? 0 : c + p, dst = stop ? 0 : c + i;
      last = stop ? last : p;
      const int ps = pages[src >> lg], pd = pages[dst >> lg];
      const bool known = ps >= 0 && ps < n_pages && pd >= 0 && pd < n_pages;
      const bool move = !stop && p != i;
      if (move && !known && tell) raise_fault(status, DSPARK_FAULT_PAGE);
      from[u] = move && known && mine ? at + ps * page_stride + (src & mask) * tok_stride : -1;
      to[u] = at + pd * page_stride + (dst & mask) * tok_stride;
    }
    uint4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) x[u] = from[u] >= 0 ? cache[from[u]] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (from[u] >= 0) cache[to[u]] = x[u];
  }
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_cache_plan_workspace_bytes(int R) {
  return R < 1 ? 0 : carve_plan(nullptr, R).bytes;
}

extern "C" int dspark_cache_plan(int R, int rows, int page_size, int max_pages, int free_len,
                                 int extra, const int32_t* lens, const int32_t* ctx,
                                 int32_t* held, int32_t* table, const int32_t* free_pages,
                                 int32_t* n_free, const int32_t* parent, int width,
                                 int32_t* row_off, int32_t* req, int32_t* position,
                                 int32_t* slot, uint64_t* anc, int32_t* dev_status, void* ws,
                                 size_t ws_bytes, hipStream_t stream) {
  if (R < 0 || rows < 0 || max_pages < 1 || free_len < 0 || extra < 0 || extra > 1 ||
      !pages_ok(page_size, max_pages))
    return DSPARK_EINVAL;
  if (R == 0) return DSPARK_OK;
  if (!lens || !ctx || !held || !table || !n_free || !row_off || !ws ||
      (free_len > 0 && !free_pages) || (rows > 0 && (!slot || (parent && !anc))) ||
      (parent && width < 1))
    return DSPARK_EINVAL;
  const PlanWs w = carve_plan(ws, R);
  if (ws_bytes < w.bytes) return DSPARK_EWORKSPACE;
  const int lg = log2_of(page_size);
  int nodes = 0x7fffffff;
  if (parent) nodes = width < DSPARK_MAX_TREE_NODES ? width : DSPARK_MAX_TREE_NODES;
  plan_scan_kernel<<<1, kPlanThreads, 0, stream>>>(R, rows, lg, max_pages, free_len, extra, lens,
                                                   ctx, held, n_free, nodes, row_off, w,
                                                   dev_status);
  // slices of a request's rows: one for steps of drafted tokens, more where few requests
  // bring long prompts
  const int slices = parent ? 1 : 1 + rows / (R < 64 ? 64 * kRowThreads : R * kRowThreads);
  plan_rows_kernel<<<dim3(R, slices < 64 ? slices : 64), kRowThreads, 0, stream>>>(
      lg, max_pages, ctx, table, free_pages, parent, width, row_off, w, req, position, slot, anc,
      dev_status);
  return launch_status();
}

extern "C" int dspark_cache_append(int rows, int Hkv, int D, dspark_dtype dt, int page_size,
                                   int n_pages, const void* k, const void* v, int64_t k_row,
                                   int64_t v_row, const int32_t* slot, const int32_t* n_rows,
                                   void* k_cache, void* v_cache, int64_t page_stride,
                                   int64_t head_stride, int64_t tok_stride, int32_t* dev_status,
                                   hipStream_t stream) {
  if (rows < 0 || Hkv < 1 || D < 8 || D % 8 != 0 || D > 1024 ||
      (dt != DSPARK_F32 && dt != DSPARK_BF16) || !pages_ok(page_size, n_pages))
    return DSPARK_EINVAL;
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  if (!stride_ok(k_row, e) || !stride_ok(v_row, e) || !stride_ok(page_stride, e) ||
      !stride_ok(head_stride, e) || !stride_ok(tok_stride, e))
    return DSPARK_EINVAL;
  if (rows == 0) return DSPARK_OK;
  if (!k || !v || !slot || !k_cache || !v_cache || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return DSPARK_EINVAL;
  const int u = (int)(16 / e);  // elements of a 16-byte piece
  const int chunks = D / u;
  const int64_t pieces = (int64_t)Hkv * chunks, blocks = (rows * pieces + 255) / 256;
  if (blocks >= (1 << 24)) return DSPARK_EINVAL;  // a grid holds 2^32 threads
  append_kernel<<<(unsigned)blocks, 256, 0, stream>>>(
      rows, (int)pieces, chunks, log2_of(page_size), n_pages, static_cast<const uint4*>(k),
      static_cast<const uint4*>(v), k_row / u, v_row / u, slot, n_rows,
      static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), page_stride / u,
      head_stride / u, tok_stride / u, dev_status);
  return launch_status();
}

extern "C" size_t dspark_cache_commit_workspace_bytes(int R) {
  return R < 1 ? 0 : carve_commit(nullptr, R).bytes;
}

extern "C" int dspark_cache_commit(int R, int gamma, int page_size, int max_pages, int free_len,
                                   const int32_t* n_acc, const int32_t* path,
                                   const int32_t* done, const int32_t* ctx, int32_t* ctx_out,
                                   int32_t* held, const int32_t* table, int32_t* free_pages,
                                   int32_t* n_free, int layers, int Hkv, int D, dspark_dtype dt,
                                   int n_pages, void* k_cache, void* v_cache,
                                   int64_t layer_stride, int64_t page_stride,
                                   int64_t head_stride, int64_t tok_stride, int32_t* dev_status,
                                   void* ws, size_t ws_bytes, hipStream_t stream) {
  if (R < 0 || max_pages < 1 || free_len < 0 || !pages_ok(page_size, max_pages))
    return DSPARK_EINVAL;
  size_t e = 4;
  if (path) {
    e = dt == DSPARK_BF16 ? 2 : 4;
    if (gamma < 1 || gamma > kMaxGamma || layers < 0 || Hkv < 1 || D < 8 || D % 8 != 0 ||
        D > 1024 || (dt != DSPARK_F32 && dt != DSPARK_BF16) || !pages_ok(page_size, n_pages) ||
        !stride_ok(layer_stride, e) || !stride_ok(page_stride, e) || !stride_ok(head_stride, e) ||
        !stride_ok(tok_stride, e) || !k_cache || !v_cache || !aligned16(k_cache) ||
        !aligned16(v_cache))
      return DSPARK_EINVAL;
  }
  if (R == 0) return DSPARK_OK;
  if (!n_acc || !ctx || !ctx_out || !held || !table || !ws ||
      (done && (!n_free || (free_len > 0 && !free_pages))))
    return DSPARK_EINVAL;
  const CommitWs w = carve_commit(ws, R);
  if (ws_bytes < w.bytes) return DSPARK_EWORKSPACE;
  const int lg = log2_of(page_size), u = (int)(16 / e), chunks = path ? D / u : 1;
  const int64_t cols = path ? (int64_t)layers * 2 * Hkv * chunks : 1;
  if ((cols + 255) / 256 > 65535) return DSPARK_EINVAL;
  commit_scan_kernel<<<1, kPlanThreads, 0, stream>>>(R, path ? gamma : 0x7fffffff, lg, max_pages,
                                                     free_len, n_acc, done, ctx, ctx_out, held,
                                                     n_free, w, dev_status);
  if (path || done)
    commit_move_kernel<<<dim3(R, cols > 0 ? (unsigned)((cols + 255) / 256) : 1), 256, 0, stream>>>(
        gamma, lg, max_pages, free_len, n_acc, path, done, table, free_pages, layers, Hkv, chunks,
        n_pages, static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), layer_stride / u,
        page_stride / u, head_stride / u, tok_stride / u, w, dev_status);
  return launch_status();
}
