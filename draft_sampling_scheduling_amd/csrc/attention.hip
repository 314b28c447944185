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
// part: 8192 rows, 32 heads on 8, 677 to 730 us, 750 to 810 TFLOP/s of the pairs seen.
#include "attention_wave.h"

namespace dspark {

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
template <class T_, int D_, int NR_>
struct Variant {
  using T = T_;
  static constexpr int D = D_, NR = NR_;
  static int grid() { return att_grid<Fit<T, D, NR>>(); }
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
  return att_variant(R, rows, G, D, dt, [&](auto v) { return att_carve(p, ws, v.grid(), kRows * v.NR, v.D); });
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
  const size_t e = dt == DSPARK_BF16 ? 2 : 4;
  if (!att_dims_ok(R, rows, Hq, Hkv, D, dt) || !stride_ok(page_stride, e) || !stride_ok(head_stride, e) ||
      !stride_ok(tok_stride, e) || tok_stride > (1 << 24))
    return DSPARK_EINVAL;
  AttParams p{};
  const int rc = att_args(p, R, rows, Hq, Hkv, D, dt, page_size, max_pages, n_pages, q, q_row, k_cache,
                          v_cache, table, ctx, row_off, anc, scale, o, lse, dev_status, ws);
  if (rc != DSPARK_OK || R == 0 || rows == 0) return rc;
  p.page_b = page_stride * (int64_t)e;
  p.head_b = head_stride * (int64_t)e;
  p.tok_b = tok_stride * (int64_t)e;
  if (ws_bytes < att_carve(p, ws, R, rows, p.G, D, dt)) return DSPARK_EWORKSPACE;
  return att_variant(R, rows, p.G, D, dt, [&](auto v) {
    return att_launch<AttWave<typename decltype(v)::T, decltype(v)::D, decltype(v)::NR>>(p, stream);
  });
}
