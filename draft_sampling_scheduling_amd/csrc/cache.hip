// cache.hip -- the paged cache around the target's pass: the step plan (rows, pages and
// slots from lengths on the device), the append of a step's keys and values, and the commit
// after verification.
//
// All three are bound by latency: a plan reads and writes a few words per request and row, an
// append copies two short rows per token.  What counts is the number of launches and of
// dependent trips to memory, so each scan over the requests is one workgroup's, and so is all
// that follows from it while it is little; past that it is one flat kernel.  Measured (kernel
// time): a plan of 4 requests 4.0 us, of 512 trees of up to 17 nodes 10.0 us (in two launches
// 4.4 + 4.1 us and the second launch); an append of 8192 rows of 8 heads of 128 (67 MB) 12 us,
// the rate of a copy; a commit of 64 paths in 4 layers 5.8 us.  With their launches: a plan of one
// prompt of 20000 rows 23 us, a commit that gives back the pages of 256 requests of 257 pages 8.8
// us (two launches, as all of more table entries), of 64 paths of up to 16 nodes in 4 layers 12.1
// us in memory of its own and 16.0 in place (two launches).  Of a cache of 4 bits, 64 paths of up to 8
// nodes in 4 layers of 4 heads of 128, codes and scales: 7.3 us.
#include <atomic>

#include "target.h"

namespace dspark {

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;

struct PlanWs {
  int32_t* held;   // [R] pages held before the call
  int32_t* take;   // [R] pages handed out to q
  int32_t* first;  // [R] pages handed out before q's
  int32_t* nfree;  // [1] free pages before the call
  int32_t* off;    // [R + 1] the row offsets again, or null
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

struct PlanArgs {
  int R, rows, lg, max_pages, free_len, extra, width, tree_nodes;
  const int32_t *lens, *ctx;
  int32_t *held, *table;
  const int32_t* free_pages;
  int32_t* n_free;
  const int32_t* parent;
  int32_t *row_off, *req, *position, *slot;
  uint64_t* anc;
  int32_t* status;
  PlanWs ws;
};

// Rows and pages of every request, by one workgroup of NT threads, each request in its
// thread's consecutive run.  One scan of (rows asked for, pages they lack) settles a step in
// which everybody is served.  Otherwise a request's rows fit in a prefix of the requests that
// ask for any, and of those its pages are had in a prefix of the ones that need any, so the
// exclusive sum of the needs is also the count of pages handed out before it.
// `to`: where the rows' kernel, or part, finds what it needs.  Returns the pages handed out.
template <int NT>
__device__ __forceinline__ int plan_scan(const PlanArgs& p, const PlanWs& to, int64_t* sums) {
  const int R = p.R, tid = threadIdx.x;
  const int per = (R + NT - 1) / NT;
  const int lo = min(R, tid * per), hi = min(R, lo + per);
  int nf = *p.n_free;
  if (nf < 0 || nf > p.free_len) {
    if (tid == 0) raise_fault(p.status, DSPARK_FAULT_PAGE);
    nf = nf < 0 ? 0 : p.free_len;
  }
  // rows request q asks for (0 where refused) and the pages they lack
  auto ask = [&](int q, bool tell, int& n, int& need) {
    const int64_t m = (int64_t)p.lens[q] + p.extra, c = p.ctx[q];
    const int64_t h = p.held[q];
    const bool bad = m < 0 || c < 0 || h < 0 || h > p.max_pages ||
                     c + m > ((int64_t)p.max_pages << p.lg) || m > p.tree_nodes;
    if (bad && tell) raise_fault(p.status, DSPARK_FAULT_LEN);
    n = bad ? 0 : (int)m;
    const int64_t want = n == 0 ? 0 : ((c + n + (1 << p.lg) - 1) >> p.lg) - h;
    need = want > 0 ? (int)want : 0;
  };
  int64_t sn = 0, sp = 0;
  for (int q = lo; q < hi; ++q) {
    int n, need;
    ask(q, true, n, need);
    sn += n;
    sp += need;
  }
  int64_t base_n = sn, base_p = sp, all_n, all_p;
  block_scan2<NT>(base_n, base_p, all_n, all_p, sums);
  base_n -= sn;
  base_p -= sp;
  int64_t at = base_n, given = all_p;  // first row of this run; pages handed out in all
  const bool everybody = all_n <= p.rows && all_p <= nf;
  if (!everybody) {
    // pages asked for by the requests whose rows fit
    int64_t run = base_n, s = 0;
    for (int q = lo; q < hi; ++q) {
      int n, need;
      ask(q, false, n, need);
      run += n;
      if (n > 0 && run > p.rows) raise_fault(p.status, DSPARK_FAULT_LEN);
      s += run <= p.rows ? need : 0;
    }
    base_p = block_scan<NT>(s, sums) - s;
    // rows granted, pages handed out
    int64_t pages = base_p, got = 0;
    run = base_n;
    s = 0;
    for (int q = lo; q < hi; ++q) {
      int n, need;
      ask(q, false, n, need);
      run += n;
      need = run <= p.rows ? need : 0;
      pages += need;
      const bool lack = need > 0 && pages > nf;
      if (lack) raise_fault(p.status, DSPARK_FAULT_PAGE);
      s += run <= p.rows && !lack ? n : 0;
      got += lack ? 0 : need;
    }
    at = s;
    int64_t unused, all_got = got;
    block_scan2<NT>(at, all_got, unused, given, sums);
    at -= s;
  }
  int64_t run = base_n, pages = base_p;
  for (int q = lo; q < hi; ++q) {
    int n, need;
    ask(q, false, n, need);
    run += n;
    need = run <= p.rows ? need : 0;
    const int64_t before = pages;
    pages += need;
    const bool lack = need > 0 && pages > nf;
    p.row_off[q] = (int32_t)at;
    if (to.off) to.off[q] = (int32_t)at;
    at += run <= p.rows && !lack ? n : 0;
    if (q == R - 1) {
      p.row_off[R] = (int32_t)at;
      if (to.off) to.off[R] = (int32_t)at;
    }
    const int h = p.held[q];
    to.held[q] = h;
    to.take[q] = lack ? 0 : need;
    to.first[q] = (int32_t)(before < given ? before : given);
    if (!lack && need > 0) p.held[q] = h + need;
  }
  if (tid == NT - 1) {
    to.nfree[0] = nf;
    *p.n_free = nf - (int32_t)given;
  }
  return (int)given;
}

// Row i of request q, whose rows begin at a: slot, position and ancestors (a walk up at most
// 64 parents through `up`).
__device__ __forceinline__ void plan_row(const PlanArgs& p, int q, int a, int i, int had,
                                         const int32_t* top, const int* up) {
  const int c = p.ctx[q], t = c + i, idx = t >> p.lg;
  const int page = idx < had ? p.table[(size_t)q * p.max_pages + idx] : top[-(idx - had)];
  int s = -1;
  if (page < 0 || page > (0x7fffffff >> p.lg))
    raise_fault(p.status, DSPARK_FAULT_PAGE);
  else
    s = (page << p.lg) + (t & ((1 << p.lg) - 1));
  int depth = i;
  if (up) {
    uint64_t bits = 0;
    depth = 0;
    for (int j = i; j > 0; j = up[j]) {
      bits |= (uint64_t)1 << (j - 1);
      ++depth;
    }
    p.anc[a + i] = bits;
  }
  p.slot[a + i] = s;
  if (p.req) p.req[a + i] = q;
  if (p.position) p.position[a + i] = c + depth;
}

// the node above node i of request q
__device__ __forceinline__ int plan_parent(const PlanArgs& p, int q, int i) {
  if (i == 0) return 0;
  const int u = p.parent[(size_t)q * p.width + i];
  if (u >= 0 && u < i) return u;
  raise_fault(p.status, DSPARK_FAULT_TREE);
  return i - 1;
}

__global__ void __launch_bounds__(kPlanThreads) plan_scan_kernel(PlanArgs p) {
  __shared__ int64_t sums[2 * kPlanThreads / kWave];
  plan_scan<kPlanThreads>(p, p.ws, sums);
}

// One workgroup per request and slice of its rows: its new pages into the table, and its rows.
__global__ void __launch_bounds__(kRowThreads) plan_rows_kernel(PlanArgs p) {
  __shared__ int up[DSPARK_MAX_TREE_NODES];
  const int q = blockIdx.x;
  const int a = p.row_off[q], n = p.row_off[q + 1] - a;
  const int had = p.ws.held[q], take = p.ws.take[q];
  // the k-th of q's new pages is top[-k]
  const int32_t* top = p.free_pages + (p.ws.nfree[0] - 1 - p.ws.first[q]);
  if (n == 0) return;
  const int t0 = blockIdx.y * kRowThreads + threadIdx.x, step = gridDim.y * kRowThreads;
  for (int k = t0; k < take; k += step) p.table[(size_t)q * p.max_pages + had + k] = top[-k];
  if (p.parent) {
    for (int i = threadIdx.x; i < n; i += kRowThreads) up[i] = plan_parent(p, q, i);
    __syncthreads();
  }
  for (int i = t0; i < n; i += step) plan_row(p, q, a, i, had, top, p.parent ? up : nullptr);
}

// The whole plan in one workgroup, for steps of not too many requests and rows: the scan; then
// a thread per request hands out its pages, takes its tree from the anchor down (a node's mask is
// its parent's and its own bit) and names its rows' request; then a thread per row, four rows at
// a time (of chains, which may be whole prompts, it finds the request in the row offsets).
// Where a request takes more than kOwn pages, as prompts do, all pages go to a thread each, which
// finds the request likewise.  Measured (with the launch): a prompt of 8192 rows in pages of 8
// takes 11 us, handed out by its own thread 114; 256 chains that bring a page or none take 11.0
// us, with a thread a page 13.6.
template <int NT_, int R_, int ROWS_, int NODES_>
struct PlanSize {
  static constexpr int NT = NT_, R = R_, ROWS = ROWS_, NODES = NODES_;
  static bool fits(int r, int rows, int width) {
    return r <= R && rows <= ROWS && (int64_t)r * width <= NODES;
  }
  struct Lds {
    uint64_t bits[NODES];  // masks of the nodes, [R][width]
    int64_t sums[2 * NT / kWave];
    int held[R], take[R], first[R], off[R + 1], nfree[1], ctx[R];
    int many;  // a request takes more pages than its thread hands out
    uint16_t req[ROWS];  // request of each row (trees)
    uint8_t up[NODES];
  };
};
using SmallPlan = PlanSize<256, 256, 1024, 4096>;
using MidPlan = PlanSize<1024, 1024, 16384, 10240>;

template <class S>
__global__ void __launch_bounds__(S::NT) plan_small_kernel(PlanArgs p) {
  constexpr int NT = S::NT, kBatch = 4, kOwn = 2;
  extern __shared__ uint64_t plan_lds[];
  auto& m = *reinterpret_cast<typename S::Lds*>(plan_lds);
  const int tid = threadIdx.x, R = p.R, lg = p.lg;
  if (tid == 0) m.many = 0;
  if (p.parent) {  // (checked against the rows once those are known)
    constexpr int kLoads = 12;
    const int nodes = R * p.width;
    for (int k0 = tid; k0 < nodes; k0 += kLoads * NT) {
      int x[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int k = k0 + u * NT;
        x[u] = p.parent[k < nodes ? k : nodes - 1];
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int k = k0 + u * NT;
        if (k < nodes) m.up[k] = (uint8_t)(x[u] >= 0 && x[u] < k % p.width ? x[u] : 255);
      }
    }
  }
  const int given =
      plan_scan<NT>(p, PlanWs{m.held, m.take, m.first, m.nfree, m.off, 0}, m.sums);
  __syncthreads();
  const int nf = m.nfree[0];
  int half = 1;  // the largest power of two below R, or 1
  while (2 * half < R) half *= 2;
  for (int q = tid; q < R; q += NT) {
    m.ctx[q] = p.ctx[q];
    const int take = m.take[q];
    if (take > kOwn) {
      m.many = 1;
    } else {
      const int32_t* top = p.free_pages + (nf - 1 - m.first[q]);
      for (int k = 0; k < take; ++k) p.table[(size_t)q * p.max_pages + m.held[q] + k] = top[-k];
    }
    if (p.parent) {
      const int n = m.off[q + 1] - m.off[q], at = q * p.width;
      for (int i = 0; i < n; ++i) {
        int u = m.up[at + i];
        if (i > 0 && u == 255) {
          raise_fault(p.status, DSPARK_FAULT_TREE);
          u = i - 1;
        }
        m.bits[at + i] = i == 0 ? 0 : m.bits[at + u] | (uint64_t)1 << (i - 1);
        m.req[m.off[q] + i] = (uint16_t)q;
      }
    }
  }
  __syncthreads();
  if (m.many) {
    for (int k0 = tid; k0 < given; k0 += kBatch * NT) {
      int page[kBatch], q[kBatch];
  #pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + u * NT;
        page[u] = p.free_pages[nf - 1 - (k < given ? k : given - 1)];
        q[u] = 0;
      }
      for (int s = half; s > 0; s >>= 1)  // the last whose pages begin at or before page k
  #pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int next = q[u] + s;
          q[u] = next < R && m.first[next] <= k0 + u * NT ? next : q[u];
        }
  #pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + u * NT;
        if (k < given)
          p.table[(size_t)q[u] * p.max_pages + m.held[q[u]] + k - m.first[q[u]]] = page[u];
      }
    }
  }
  const int rows = m.off[R];
  for (int row0 = tid; row0 < rows; row0 += kBatch * NT) {
    int q[kBatch], t[kBatch], page[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      q[u] = p.parent && row0 + u * NT < rows ? m.req[row0 + u * NT] : 0;
    for (int s = p.parent ? 0 : half; s > 0; s >>= 1)  // the last that begins at or before the row
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int next = q[u] + s;
        q[u] = next < R && m.off[next] <= row0 + u * NT ? next : q[u];
      }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int row = row0 + u * NT;
      t[u] = row < rows ? m.ctx[q[u]] + row - m.off[q[u]] : 0;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int idx = t[u] >> lg, more = idx - m.held[q[u]];
      const int32_t* at = more < 0 ? p.table + (size_t)q[u] * p.max_pages + idx
                                   : p.free_pages + (nf - 1 - m.first[q[u]] - more);
      page[u] = row0 + u * NT < rows ? *at : 0;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int row = row0 + u * NT, i = row - m.off[q[u]];
      if (row >= rows) break;
      const bool known = page[u] >= 0 && page[u] <= (0x7fffffff >> lg);
      if (!known) raise_fault(p.status, DSPARK_FAULT_PAGE);
      p.slot[row] = known ? (page[u] << lg) + (t[u] & ((1 << lg) - 1)) : -1;
      int depth = i;
      if (p.parent) {
        const uint64_t bits = m.bits[q[u] * p.width + i];
        p.anc[row] = bits;
        depth = __popcll(bits);
      }
      if (p.req) p.req[row] = q[u];
      if (p.position) p.position[row] = t[u] - i + depth;
    }
  }
}

template <class S>
static void plan_small_launch(const PlanArgs& p, hipStream_t stream) {
  static std::atomic<uint64_t> raised;
  ensure_dynamic_lds(reinterpret_cast<const void*>(plan_small_kernel<S>), sizeof(typename S::Lds),
                     raised);
  plan_small_kernel<S><<<1, S::NT, sizeof(typename S::Lds), stream>>>(p);
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
  int32_t* ctx;    // [R] lengths before the call (null: not kept)
  int32_t* held;   // [R] pages held before the call
  int32_t* first;  // [R] place of q's first page on the free list (-1: q goes on)
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

// Entries of the block tables up to which the scanning workgroup gives pages back itself: 7 us
// where all of 4096 are, 11 us of 8192, against 8 us and a second launch.
constexpr int kGivePages = 4096, kCommitR = 1024;

struct CommitArgs {
  int R, gamma, most, lg, max_pages, free_len;
  const int32_t *n_acc, *path, *done, *ctx;
  int32_t *ctx_out, *held;
  const int32_t* table;
  int32_t *free_pages, *n_free;
  int layers, Hkv, chunks, n_pages;
  uint4 *k_cache, *v_cache;
  int64_t layer_stride, page_stride, head_stride, tok_stride;  // in 16-byte pieces
  int words;         // 4 bytes of scales of a token and head (0: a cache without)
  uint32_t* scales;
  int64_t s_layer, s_page, s_head, s_tok;  // in words
  int32_t* status;
  CommitWs ws;
};

// Lengths of every request and the places of the pages given back, by one workgroup, kept in
// `to`; GIVE: and the pages themselves.
template <int NT, bool GIVE>
__device__ __forceinline__ void commit_scan(const CommitArgs& p, const CommitWs& to, int64_t* sums) {
  const int R = p.R, tid = threadIdx.x;
  const int per = (R + NT - 1) / NT;
  const int lo = min(R, tid * per), hi = min(R, lo + per);
  int64_t s = 0;
  for (int q = lo; q < hi; ++q) {
    int h = p.held[q];
    if (h < 0 || h > p.max_pages) {
      raise_fault(p.status, DSPARK_FAULT_LEN);
      h = h < 0 ? 0 : p.max_pages;
    }
    const bool end = p.done && p.done[q] != 0;
    const int c = p.ctx[q], n = p.n_acc[q];
    if (to.ctx) to.ctx[q] = c;
    to.held[q] = h;
    if (end) {
      s += h;
      p.ctx_out[q] = 0;
    } else {
      const int na = clamp_acc(n, c, h, p.lg, p.most);
      if (na != n) raise_fault(p.status, DSPARK_FAULT_LEN);
      p.ctx_out[q] = c + na + 1;
    }
  }
  if (!p.done) return;
  int nf = *p.n_free;
  if (nf < 0 || nf > p.free_len) {
    if (tid == 0) raise_fault(p.status, DSPARK_FAULT_PAGE);
    nf = nf < 0 ? 0 : p.free_len;
  }
  const int64_t end = block_scan<NT>(s, sums);
  int64_t at = nf + end - s;
  for (int q = lo; q < hi; ++q) {
    const bool mine = p.done[q] != 0;
    to.first[q] = mine ? (int32_t)(at < p.free_len ? at : p.free_len) : -1;
    if (mine) {
      at += to.held[q];
      p.held[q] = 0;
    }
  }
  if (tid == NT - 1) {
    const int64_t total = nf + end;
    if (total > p.free_len) raise_fault(p.status, DSPARK_FAULT_PAGE);
    *p.n_free = (int32_t)(total < p.free_len ? total : p.free_len);
  }
  if (GIVE) {  // every entry of the tables, eight a thread at a time
    __syncthreads();
    constexpr int kBatch = 8;
    const int W = p.max_pages, entries = R * W;
    for (int i0 = tid; i0 < entries; i0 += kBatch * NT) {
      int at[kBatch], page[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * NT, q = i / W, k = i - q * W;
        at[u] = -1;
        if (i < entries && to.first[q] >= 0 && k < to.held[q] && to.first[q] + k < p.free_len) {
          at[u] = to.first[q] + k;
          page[u] = p.table[i];
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (at[u] >= 0) p.free_pages[at[u]] = page[u];
    }
  }
}

// The moves of one column (a piece E of a layer's keys, values or scales, at `at`) of a request's
// tokens.  A thread owns its column, so the moves of one column are one thread's: a batch of eight
// tokens is read before any of them is written, and since the path ascends (its i-th node is at
// least i), no later batch reads a token that an earlier one wrote.
template <class E>
__device__ __forceinline__ void commit_column(const CommitArgs& p, int q, int c, int h, int na, bool mine,
                                              bool tell, E* cache, int64_t at, int64_t page_stride,
                                              int64_t tok_stride) {
  const int32_t* pages = p.table + (size_t)q * p.max_pages;
  const int mask = (1 << p.lg) - 1;
  constexpr int kBatch = 8;
  int last = 0;
  bool stop = false;
  for (int i0 = 1; i0 <= na && !stop; i0 += kBatch) {
    int64_t from[kBatch], to[kBatch];  // from -1: nothing moves
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u;
      const int n = p.path[(size_t)q * p.gamma + (i <= na ? i - 1 : 0)];
      const bool fine = n > last && (int64_t)c + n < ((int64_t)h << p.lg);
      if (i <= na && !stop && !fine && tell) raise_fault(p.status, DSPARK_FAULT_TREE);
      stop = stop || i > na || !fine;
      const int src = stop ? 0 : c + n, dst = stop ? 0 : c + i;
      last = stop ? last : n;
      const int ps = pages[src >> p.lg], pd = pages[dst >> p.lg];
      const bool known = ps >= 0 && ps < p.n_pages && pd >= 0 && pd < p.n_pages;
      const bool move = !stop && n != i;
      if (move && !known && tell) raise_fault(p.status, DSPARK_FAULT_PAGE);
      from[u] = move && known && mine ? at + ps * page_stride + (src & mask) * tok_stride : -1;
      to[u] = at + pd * page_stride + (dst & mask) * tok_stride;
    }
    E x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) x[u] = from[u] >= 0 ? cache[from[u]] : E{};
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (from[u] >= 0) cache[to[u]] = x[u];
  }
}

// The moves of request q in 256 of the columns of its tokens: 16 bytes each (layer, keys or values,
// head, piece of D), then, in a cache of 4 bits, 4 bytes each (layer, head, word of the scales).
__device__ __forceinline__ void commit_move(const CommitArgs& p, int q, int slice, int c, int h) {
  if (c < 0) return;
  const int na = clamp_acc(p.n_acc[q], c, h, p.lg, p.gamma);
  if (na < 1) return;
  const int per_layer = 2 * p.Hkv * p.chunks;
  const int64_t col = (int64_t)slice * 256 + threadIdx.x, wide = (int64_t)p.layers * per_layer;
  const bool tell = slice == 0 && threadIdx.x == 0;
  const int64_t word = col - wide;
  if (p.words > 0 && word >= 0 && !tell) {
    const int per = p.Hkv * p.words;
    const int layer = (int)(word / per), r = (int)(word % per);
    if (layer < p.layers)
      commit_column(p, q, c, h, na, true, false, p.scales,
                    layer * p.s_layer + (int64_t)(r / p.words) * p.s_head + r % p.words, p.s_page, p.s_tok);
    return;
  }
  const bool mine = col < wide;
  int64_t at = 0;
  uint4* cache = p.k_cache;
  if (mine) {
    const int layer = (int)(col / per_layer);
    int r = (int)(col % per_layer);
    if (r >= p.Hkv * p.chunks) {
      cache = p.v_cache;
      r -= p.Hkv * p.chunks;
    }
    at = layer * p.layer_stride + (int64_t)(r / p.chunks) * p.head_stride + r % p.chunks;
  }
  commit_column(p, q, c, h, na, mine, tell, cache, at, p.page_stride, p.tok_stride);
}

// One launch, where the lengths go to memory of their own and the pages given back are few:
// the last workgroup scans and gives, the others move.  A move reads only what the scan leaves
// alone: ctx, and held of requests that go on.
__global__ void __launch_bounds__(256) commit_kernel(CommitArgs p, int slices) {
  __shared__ int64_t sums[256 / kWave];
  __shared__ int held[kCommitR], first[kCommitR];
  const int b = blockIdx.x;
  if (b == (int)gridDim.x - 1) {
    commit_scan<256, true>(p, CommitWs{nullptr, held, first, 0}, sums);
    return;
  }
  const int q = b / slices;
  if (p.done && p.done[q] != 0) return;
  const int h = p.held[q];
  commit_move(p, q, b % slices, p.ctx[q], h < 0 ? 0 : (h > p.max_pages ? p.max_pages : h));
}

// Two launches otherwise: the scan, then the moves from the lengths it kept, and the pages.
__global__ void __launch_bounds__(kPlanThreads) commit_scan_kernel(CommitArgs p) {
  __shared__ int64_t sums[kPlanThreads / kWave];
  commit_scan<kPlanThreads, false>(p, p.ws, sums);
}

__global__ void __launch_bounds__(256) commit_move_kernel(CommitArgs p) {
  const int q = blockIdx.x, h = p.ws.held[q];
  if (p.done && p.done[q] != 0) {
    const int at = p.ws.first[q];
    if (blockIdx.y == 0)
      for (int k = threadIdx.x; k < h && at + k < p.free_len; k += 256)
        p.free_pages[at + k] = p.table[(size_t)q * p.max_pages + k];
    return;
  }
  if (p.path) commit_move(p, q, blockIdx.y, p.ws.ctx[q], h);
}

}  // namespace dspark

using namespace dspark;

// whether one workgroup makes the whole plan
static bool plan_small(int R, int rows, int width) {
  return SmallPlan::fits(R, rows, width) || MidPlan::fits(R, rows, width);
}

extern "C" size_t dspark_cache_plan_workspace_bytes(int R, int rows, int width) {
  if (R < 1 || R > kMaxRequests || plan_small(R, rows, width)) return 0;
  return carve_plan(nullptr, R).bytes;
}

extern "C" int dspark_cache_plan(int R, int rows, int page_size, int max_pages, int free_len,
                                 int extra, const int32_t* lens, const int32_t* ctx,
                                 int32_t* held, int32_t* table, const int32_t* free_pages,
                                 int32_t* n_free, const int32_t* parent, int width,
                                 int32_t* row_off, int32_t* req, int32_t* position,
                                 int32_t* slot, uint64_t* anc, int32_t* dev_status, void* ws,
                                 size_t ws_bytes, hipStream_t stream) {
  if (R < 0 || R > kMaxRequests || rows < 0 || max_pages < 1 || free_len < 0 || extra < 0 ||
      extra > 1 ||
      !table_ok(page_size, max_pages))
    return DSPARK_EINVAL;
  if (R == 0) return DSPARK_OK;
  const bool small = plan_small(R, rows, parent ? width : 0);
  if (!lens || !ctx || !held || !table || !n_free || !row_off || (!small && !ws) ||
      (free_len > 0 && !free_pages) || (rows > 0 && (!slot || (parent && !anc))) ||
      (parent && width < 1) || !aligned16(ws))
    return DSPARK_EINVAL;
  const PlanWs w = carve_plan(ws, R);
  if (!small && ws_bytes < w.bytes) return DSPARK_EWORKSPACE;
  PlanArgs p{};
  p.R = R;
  p.rows = rows;
  p.lg = log2_of(page_size);
  p.max_pages = max_pages;
  p.free_len = free_len;
  p.extra = extra;
  p.width = width;
  p.tree_nodes = 0x7fffffff;
  if (parent) p.tree_nodes = width < DSPARK_MAX_TREE_NODES ? width : DSPARK_MAX_TREE_NODES;
  p.lens = lens;
  p.ctx = ctx;
  p.held = held;
  p.table = table;
  p.free_pages = free_pages;
  p.n_free = n_free;
  p.parent = parent;
  p.row_off = row_off;
  p.req = req;
  p.position = position;
  p.slot = slot;
  p.anc = anc;
  p.status = dev_status;
  p.ws = w;
  if (small) {
    if (SmallPlan::fits(R, rows, parent ? width : 0))
      plan_small_launch<SmallPlan>(p, stream);
    else
      plan_small_launch<MidPlan>(p, stream);
    return launch_status();
  }
  plan_scan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  // slices of a request's rows: one for steps of drafted tokens, more where few requests
  // bring long prompts
  const int slices = parent ? 1 : 1 + rows / (R < 64 ? 64 * kRowThreads : R * kRowThreads);
  plan_rows_kernel<<<dim3(R, slices < 64 ? slices : 64), kRowThreads, 0, stream>>>(p);
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
  // a row may be read after another is written
  const size_t row_bytes = (size_t)pieces * 16;
  const size_t kb = (size_t)(rows - 1) * k_row * e + row_bytes;
  const size_t vb = (size_t)(rows - 1) * v_row * e + row_bytes;
  const size_t cb = ((size_t)(n_pages - 1) * page_stride + (size_t)(Hkv - 1) * head_stride +
                     (size_t)(page_size - 1) * tok_stride + D) * e;
  for (const void* cache : {k_cache, v_cache})
    if (overlap(k, kb, cache, cb) || overlap(v, vb, cache, cb)) return DSPARK_EINVAL;
  append_kernel<<<(unsigned)blocks, 256, 0, stream>>>(
      rows, (int)pieces, chunks, log2_of(page_size), n_pages, static_cast<const uint4*>(k),
      static_cast<const uint4*>(v), k_row / u, v_row / u, slot, n_rows,
      static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), page_stride / u,
      head_stride / u, tok_stride / u, dev_status);
  return launch_status();
}

// whether one launch commits: few pages to give back, and lengths apart from those that the
// moves read
static bool commit_small(int R, int64_t pages, bool moves_in_place) {
  return R <= kCommitR && pages <= kGivePages && !moves_in_place;
}

extern "C" size_t dspark_cache_commit_workspace_bytes(int R, int max_pages, int moves_in_place) {
  if (R < 1 || R > kMaxRequests || commit_small(R, (int64_t)R * max_pages, moves_in_place)) return 0;
  return carve_commit(nullptr, R).bytes;
}

// The caches of a commit with a path: strides in bytes, a head's row `chunks` pieces of 16 bytes, its
// scales `words` of 4.
struct CommitCache {
  int layers, Hkv, chunks;
  void *k, *v;
  int64_t layer, page, head, tok;
  int words;
  void* scales;
  int64_t s_layer, s_page, s_head, s_tok;
};

static int commit_run(int R, int gamma, int page_size, int max_pages, int free_len, const int32_t* n_acc,
                      const int32_t* path, const int32_t* done, const int32_t* ctx, int32_t* ctx_out,
                      int32_t* held, const int32_t* table, int32_t* free_pages, int32_t* n_free,
                      int n_pages, const CommitCache& cache, int32_t* dev_status, void* ws,
                      size_t ws_bytes, hipStream_t stream) {
  if (R < 0 || R > kMaxRequests || max_pages < 1 || free_len < 0 ||
      !table_ok(page_size, max_pages))
    return DSPARK_EINVAL;
  if (path && (gamma < 1 || gamma > kMaxGamma || cache.layers < 0 || cache.Hkv < 1 ||
               !pages_ok(page_size, n_pages) || !cache.k || !cache.v || !aligned16(cache.k) ||
               !aligned16(cache.v)))
    return DSPARK_EINVAL;
  if (R == 0) return DSPARK_OK;
  if (!n_acc || !ctx || !ctx_out || !held || !table || !aligned16(ws) ||
      (done && (!n_free || (free_len > 0 && !free_pages))))
    return DSPARK_EINVAL;
  const size_t len_bytes = (size_t)R * sizeof(int32_t);
  const bool apart = !overlap(ctx_out, len_bytes, ctx, len_bytes);
  // what is read after the first lengths are written, or written beside them
  auto over = [&](const void* a, size_t ints) {
    return a && overlap(ctx_out, len_bytes, a, ints * sizeof(int32_t));
  };
  if ((!apart && ctx_out != ctx) || over(n_acc, R) || over(held, R) ||
      over(path, (size_t)R * gamma) || over(table, (size_t)R * max_pages) || over(done, R) ||
      (done && (over(free_pages, free_len) || over(n_free, 1))))
    return DSPARK_EINVAL;
  const bool small = commit_small(R, done ? (int64_t)R * max_pages : 0, path && !apart);
  const CommitWs w = carve_commit(ws, R);
  if (!small && !ws) return DSPARK_EINVAL;
  if (!small && ws_bytes < w.bytes) return DSPARK_EWORKSPACE;
  const int lg = log2_of(page_size);
  const int64_t cols =
      path ? (int64_t)cache.layers * cache.Hkv * (2 * cache.chunks + cache.words) : 1;
  if ((cols + 255) / 256 > 65535) return DSPARK_EINVAL;
  const int slices = cols > 256 ? (int)((cols + 255) / 256) : 1;
  CommitArgs p{};
  p.R = R;
  p.gamma = gamma;
  p.most = path ? gamma : 0x7fffffff;
  p.lg = lg;
  p.max_pages = max_pages;
  p.free_len = free_len;
  p.n_acc = n_acc;
  p.path = path;
  p.done = done;
  p.ctx = ctx;
  p.ctx_out = ctx_out;
  p.held = held;
  p.table = table;
  p.free_pages = free_pages;
  p.n_free = n_free;
  p.layers = cache.layers;
  p.Hkv = cache.Hkv;
  p.chunks = cache.chunks;
  p.n_pages = n_pages;
  p.k_cache = static_cast<uint4*>(cache.k);
  p.v_cache = static_cast<uint4*>(cache.v);
  p.layer_stride = cache.layer / 16;
  p.page_stride = cache.page / 16;
  p.head_stride = cache.head / 16;
  p.tok_stride = cache.tok / 16;
  p.words = cache.words;
  p.scales = static_cast<uint32_t*>(cache.scales);
  p.s_layer = cache.s_layer / 4;
  p.s_page = cache.s_page / 4;
  p.s_head = cache.s_head / 4;
  p.s_tok = cache.s_tok / 4;
  p.status = dev_status;
  p.ws = w;
  const int64_t blocks = path ? (int64_t)R * slices : 0;
  if (blocks >= (1 << 24) - 1) return DSPARK_EINVAL;  // a grid holds 2^32 threads
  if (small) {
    commit_kernel<<<(unsigned)blocks + 1, 256, 0, stream>>>(p, slices);
    return launch_status();
  }
  commit_scan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  if (path || done) commit_move_kernel<<<dim3(R, slices), 256, 0, stream>>>(p);
  return launch_status();
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
  CommitCache cache{};
  if (path) {
    const size_t e = dt == DSPARK_BF16 ? 2 : 4;
    if (D < 8 || D % 8 != 0 || D > 1024 || (dt != DSPARK_F32 && dt != DSPARK_BF16) ||
        !stride_ok(layer_stride, e) || !stride_ok(page_stride, e) || !stride_ok(head_stride, e) ||
        !stride_ok(tok_stride, e))
      return DSPARK_EINVAL;
    const int64_t b = (int64_t)e;
    cache = {layers, Hkv, (int)(D * e / 16), k_cache, v_cache, layer_stride * b, page_stride * b,
             head_stride * b, tok_stride * b, 0, nullptr, 0, 0, 0, 0};
  }
  return commit_run(R, gamma, page_size, max_pages, free_len, n_acc, path, done, ctx, ctx_out, held,
                    table, free_pages, n_free, n_pages, cache, dev_status, ws, ws_bytes, stream);
}

extern "C" int dspark_cache4_commit(int R, int gamma, int page_size, int max_pages, int free_len,
                                    const int32_t* n_acc, const int32_t* path, const int32_t* done,
                                    const int32_t* ctx, int32_t* ctx_out, int32_t* held,
                                    const int32_t* table, int32_t* free_pages, int32_t* n_free,
                                    int layers, int Hkv, int D, int n_pages, void* k_cache,
                                    void* v_cache, int64_t layer_stride, int64_t page_stride,
                                    int64_t head_stride, int64_t tok_stride, void* scales,
                                    int64_t s_layer, int64_t s_page, int64_t s_head, int64_t s_tok,
                                    int32_t* dev_status, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
  CommitCache cache{};
  if (path) {
    if (!cache4_ok(D, page_stride, head_stride, tok_stride, s_page, s_head, s_tok) ||
        !stride_ok(layer_stride, 1) || s_layer < 0 || s_layer % (D / 16) != 0 || !scales ||
        !aligned16(scales))
      return DSPARK_EINVAL;
    cache = {layers, Hkv, D / 32, k_cache, v_cache, layer_stride, page_stride, head_stride, tok_stride,
             D / 64, scales, s_layer, s_page, s_head, s_tok};
  }
  return commit_run(R, gamma, page_size, max_pages, free_len, n_acc, path, done, ctx, ctx_out, held,
                    table, free_pages, n_free, n_pages, cache, dev_status, ws, ws_bytes, stream);
}
