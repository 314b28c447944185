"""Groups of a 4-bit cache that read NaN, at tokens whose weight underflows to 0 in float as at others:
values' reach their 32 elements of o of every row that sees the token, keys' all of such a row, and
nothing else, whichever variant takes the rows, wherever the token lies in its tile, and whether the
list is cut or not."""
import numpy as np
import pytest
import torch

from tests import cache4_ref as c4
from tests import target_ref as ref
from tests.test_gpu_cache4_attention import tol
from tests.test_gpu_target_attention import T, trees

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32

# rows and query heads to a cache head: rows shared by two waves, 32 a wave, tiles shared by four waves
SIZES = [(1, 8), (6, 8), (9, 8), (3, 40)]


def scene(n, G, ctx, D, dtype, low, tree=False):
    """One request, every score 0 but those of the tokens `low`, which are -192 sqrt(D) q's mean: their
    weights beside the others' are exp(-1000) and less, 0 in float."""
    Hkv = 2
    c = c4.Cache4(ctx + D, [ctx], [n], Hkv, D, 16, fill=255)
    c.kc[:], c.sc[..., 0, :] = 0, 127
    for t in low:
        at = c.table[0, t // 16], slice(None), t % 16
        c.kc[at], c.sc[at][:, 0] = 0xFF, 132   # all -6 * 2^5
    g = np.random.default_rng(n + G)
    q = torch.from_numpy(np.abs(g.standard_normal((n, Hkv * G, D), np.float32)) + 0.5).to(dtype)
    return c, q, trees(g, [n]) if tree else None


def check(c, q, ctx, anc, dtype, sick, keys=False):
    """Group 1 of cache head 1 reads NaN at the tokens `sick`."""
    import draft_sampling_scheduling_amd as ds
    n, Hq, D = q.shape
    G, see = Hq // 2, ref.sees(n, anc)
    c.renew()
    w = ref.attention(q.double().numpy(), c.tokens(c.k, 0, ctx + n), c.tokens(c.v, 0, ctx + n), ctx, D ** -0.5, see)
    masks = None if anc is None else T(anc, torch.int64)
    d = c.dev4()
    for t in sick:
        d[2][int(c.table[0, t // 16]), 1, t % 16, 0 if keys else 1, 1] = 255
    st = T([0])
    got = ds.tree_attention(q.to("cuda:0"), d[0], d[1], torch.from_numpy(c.table).to("cuda:0"), T([ctx]), T([0, n]),
                            scales=d[2], anc=masks, status=st)
    assert int(st) == 0
    o, lse = got["o"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    nan = np.zeros(o.shape, bool)
    for i in range(n):
        if any(t < ctx or see[i][t - ctx] for t in sick):
            nan[i, G:, slice(None) if keys else slice(32, 64)] = True
    assert np.array_equal(np.isnan(o), nan), (sick, np.argwhere(np.isnan(o) != nan)[:5])
    to, tl = tol(w, ctx + n, D, dtype is BF)
    assert (np.abs(o - w[0]) <= to)[~nan].all()
    whole = ~nan.all(-1)
    assert (np.abs(lse - w[1]) <= tl)[whole].all() and np.isnan(lse[~whole]).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", SIZES)
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
def test_one_list(n, G, tree, D, dtype):
    """A list that is not cut: in a tile that all rows see whole, in the tile where the block begins, in
    the block itself."""
    ctx = 90
    for t in (3, 70, ctx - 1, ctx, ctx + n - 1):
        for low in ([], [t], [x for x in range(ctx + n) if x != 40]):
            c, q, anc = scene(n, G, ctx, D, dtype, low, tree)
            for keys in (False, True):
                check(c, q, ctx, anc, dtype, [t], keys)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", SIZES)
def test_cut_list(n, G, D, dtype):
    """Pieces whose rows have no weight beside others', and pieces that have all of it."""
    ctx = 6000
    for low, sick in ((range(3000), [7]), (range(3000), [1500, 2990]), (range(3000), [4000]),
                      (range(3000, ctx + n), [ctx - 1]), (range(3000, ctx + n), [ctx + n - 1]), ((), [100, 5999])):
        c, q, anc = scene(n, G, ctx, D, dtype, low)
        for keys in (False, True):
            check(c, q, ctx, anc, dtype, sick, keys)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", SIZES)
@pytest.mark.parametrize("ctx", [50, 4000])
def test_odd_queries(ctx, n, G, D, dtype):
    """Infinite and NaN queries are their own row's affair."""
    import draft_sampling_scheduling_amd as ds
    c = c4.Cache4(3, [ctx], [n], 2, D, 16, fill=255)
    g = np.random.default_rng(n)
    q = torch.from_numpy(g.standard_normal((n, 2 * G, D), np.float32)).to(dtype)
    w = ref.attention(q.double().numpy(), c.tokens(c.k, 0, ctx + n), c.tokens(c.v, 0, ctx + n), ctx, D ** -0.5, ref.sees(n))
    odd = [(0, 0), (n // 2, G), (n - 1, 2 * G - 1)]
    for at, x in zip(odd, ("nan", "inf", "-inf")):
        q[(*at, 7)] = float(x)
    d = c.dev4()
    got = ds.tree_attention(q.to("cuda:0"), d[0], d[1], torch.from_numpy(c.table).to("cuda:0"), T([ctx]), T([0, n]), scales=d[2])
    o = got["o"].double().cpu().numpy()
    well = np.ones(o.shape[:2], bool)
    for at in odd:
        well[at] = False
        assert np.isnan(o[at]).any()
    assert (np.abs(o - w[0]) <= tol(w, ctx + n, D, dtype is BF)[0])[well].all()
