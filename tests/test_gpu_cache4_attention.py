"""tree_attention over a cache of 4 bits against the attention of each row taken by itself in 64
bits over the values that the cache holds, within bounds that count its roundings
(target_ref.attention_tol: the cache's values are exact operands)."""
import numpy as np
import pytest
import torch

from tests import cache4_ref as c4
from tests import target_ref as ref
from tests.test_gpu_target_attention import SHAPES, T, trees

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def tol(w, L, D, bf16):
    """Float queries and weights are three bf16 terms: a term's product with an element is exact and the
    terms' sum is the float, so a score is a sum of 3 D products and o of 3 L: thrice the steps of
    attention_tol's sums, and one weight's three terms leave nothing off."""
    o, lse, A, S = w
    return ref.attention_tol(o, lse, A, S, 3 * L if not bf16 else L, 3 * D if not bf16 else D, bf16)


def check(seed, ctx, n, Hq, Hkv, D, page, dtype, tree=False, layout="phtd", q_pad=0, slack=3, scale=None,
          spread=1.0, edit=None, anc=None, fill=255):
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(seed)
    c = c4.Cache4(seed, ctx, n, Hkv, D, page, layout, fill=fill)
    rows = sum(n) + slack
    q = torch.from_numpy(spread * g.standard_normal((rows, Hq + q_pad, D), np.float32)).to(dtype)
    if anc is None and tree:
        anc = trees(g, n)
    off = np.concatenate([[0], np.cumsum(n)])
    if edit:
        edit(c, q)
        c.renew()
    o = torch.full((rows, Hq, D), 77.0, dtype=dtype, device="cuda:0")
    lse = torch.full((rows, Hq), 77.0, device="cuda:0")
    st = T([0])
    masks = None
    if anc is not None:
        masks = T([a - 2 ** 64 if a >= 2 ** 63 else a for a in anc] + [-1] * slack, torch.int64)
    dk, dv, sc = c.dev4()
    args = (q.to("cuda:0")[:, :Hq], dk, dv, torch.from_numpy(c.table).to("cuda:0"), T(ctx), T(off.tolist()))
    ds.tree_attention(*args, scales=sc, anc=masks, scale=scale, out=dict(o=o, lse=lse), status=st)
    again = ds.tree_attention(*args, scales=sc, anc=masks, scale=scale)
    assert int(st) == 0
    live = int(off[-1])
    assert torch.equal(again["o"][:live], o[:live]) and torch.equal(again["lse"][:live], lse[:live])
    assert torch.all(o[live:] == 77.0) and torch.all(lse[live:] == 77.0)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for k, (cx, m) in enumerate(zip(ctx, n)):
        if m == 0:
            continue
        a = slice(off[k], off[k + 1])
        w = ref.attention(q[a, :Hq].double().numpy(), c.tokens(c.k, k, cx + m), c.tokens(c.v, k, cx + m), cx,
                          D ** -0.5 if scale is None else scale, ref.sees(m, None if anc is None else anc[a]))
        to, tl = tol(w, cx + m, D, dtype is BF)
        eo, el = np.abs(o[a] - w[0]) / to, np.abs(lse[a] - w[1]) / tl
        assert eo.max() <= 1 and el.max() <= 1, (k, cx, m, eo.max(), el.max())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,n", SHAPES, ids=lambda v: "-".join(map(str, v)))
def test_chain(ctx, n, D, dtype):
    check(len(ctx) + D, ctx, n, 6, 2, D, 16, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (7, 1), (10, 2), (16, 1), (48, 3)])
def test_heads(Hq, Hkv, dtype):
    check(Hq, [70, 3, 150], [4, 9, 1], Hq, Hkv, 64, 16, dtype, q_pad=2 * Hkv)
    check(Hq, [70, 3, 150], [4, 9, 1], Hq, Hkv, 128, 32, dtype, tree=True)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 1024])
@pytest.mark.parametrize("layout", ["phtd", "pthd"])
def test_pages(page, layout):
    for dtype, D in ((BF, 128), (F32, 64), (BF, 64), (F32, 128)):
        check(page, [3 * page - 2, page, 0, 95], [5, 1, 3, 33], 4, 2, D, page, dtype, layout=layout)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 5, 17, 33, 64, 65])
def test_trees(n, dtype):
    check(n, [0, 40, 31], [n, n, 1], 4, 2, 128, 16, dtype, tree=True)
    check(n + 1, [90, 7], [n, n // 2], 5, 1, 64, 8, dtype, tree=True)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ctx,n", [([0], [130]), ([100, 0], [257, 64]), ([500], [96])])
def test_prompt_pieces(ctx, n, dtype):
    check(n[0], ctx, n, 4, 2, 64, 16, dtype)
    check(n[0], ctx, n, 3, 1, 128, 64, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_long(dtype):
    check(1, [20000], [3], 2, 1, 128, 16, dtype)
    check(2, [9001, 3, 0, 4100, 64], [2, 1, 5, 1, 1], 4, 2, 64, 32, dtype)
    check(6, [7000, 40], [3, 1], 24, 1, 128, 16, dtype)   # 72 query rows to a head
    check(7, [7000, 40], [3, 5], 11, 1, 64, 16, dtype)    # 55
    check(8, [2500, 900, 3], [6, 4, 7], 40, 2, 64, 8, dtype, tree=True)  # 140


def test_many_requests():
    g = np.random.default_rng(3)
    check(3, g.integers(0, 40, 300).tolist(), g.integers(0, 4, 300).tolist(), 2, 1, 64, 8, BF)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_large_scores(dtype):
    check(4, [300, 64], [4, 9], 4, 2, 64, 16, dtype, spread=40.0)
    check(5, [300, 64], [4, 9], 4, 2, 128, 16, dtype, scale=1e-6)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_powers(D, dtype):
    """Every group of a token with a power of its own, from 2^-40 to 2^10 of the values."""
    def edit(c, q):
        g = np.random.default_rng(1)
        c.sc[..., 1, :] = g.integers(87, 138, c.sc[..., 1, :].shape)
        c.sc[..., 0, :] = g.integers(100, 128, c.sc[..., 0, :].shape)
    check(9, [150, 33], [3, 9], 4, 2, D, 16, dtype, edit=edit)
    check(9, [150, 33], [40, 39], 4, 2, D, 16, dtype, edit=edit)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [6, 14, 24])
def test_unseen_groups_hold_anything(Hq, D, dtype):
    """Groups that read NaN, of nodes that a row does not see, reach only the rows that see them: keys'
    all of the row, values' the 32 elements they stand for."""
    import draft_sampling_scheduling_amd as ds
    n, ctx = 6, 45
    anc = [0, 0b1, 0b10, 0b101, 0b1001, 0b10010]  # node 2, and 5 under it, hold it
    g = np.random.default_rng(9)
    q = torch.from_numpy(g.standard_normal((n, Hq, D), np.float32)).to(dtype)
    see = ref.sees(n, anc)
    for sick, byte in ((0, 255), (1, 255), (1, 254), (1, 253), (0, 253)):
        c = c4.Cache4(9, [ctx], [n], 2, D, 16)
        table = torch.from_numpy(c.table).to("cuda:0")

        def go():
            d = c.dev4()
            st = T([0])
            o = ds.tree_attention(q.to("cuda:0"), d[0], d[1], table, T([ctx]), T([0, n]), scales=d[2],
                                  anc=T(anc, torch.int64), status=st)["o"].double().cpu().numpy()
            assert int(st) == 0
            return o

        w = ref.attention(q.double().numpy(), c.tokens(c.k, 0, ctx + n), c.tokens(c.v, 0, ctx + n), ctx, D ** -0.5, see)
        for node in (2, 5):
            t = ctx + node
            c.sc[c.table[0, t // 16], :, t % 16, sick, 1] = byte
        after = go()
        well = [i for i in range(n) if i not in (2, 5)]
        assert (np.abs(after - w[0]) <= tol(w, ctx + n, D, dtype is BF)[0])[well].all()
        bad = ~np.isfinite(after[[2, 5]])
        if byte != 255:  # (past the largest float in part: what its own rows read is not said)
            continue
        if sick == 1:
            assert bad[..., 32:64].all() and not bad[..., :32].any() and not bad[..., 64:].any()
        else:
            assert bad.all()
    assert see[5, 2] and not see[4, 2]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_sick_token_of_the_context(dtype):
    """Seen by all: its group is NaN everywhere; away from the tiles with edges too."""
    import draft_sampling_scheduling_amd as ds
    for at in (3, 200, 299):
        c = c4.Cache4(2, [300], [2], 1, 128, 16)
        c.sc[c.table[0, at // 16], 0, at % 16, 1, 2] = 255
        d = c.dev4()
        q = torch.randn(2, 4, 128, device="cuda:0").to(dtype)
        o = ds.tree_attention(q, d[0], d[1], torch.from_numpy(c.table).to("cuda:0"), T([300]), T([0, 2]), scales=d[2])["o"]
        bad = torch.isnan(o)
        assert bad[..., 64:96].all() and not bad[..., :64].any() and not bad[..., 96:].any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_odd_queries(dtype):
    """Infinite and NaN queries are their own row's affair."""
    import draft_sampling_scheduling_amd as ds
    c = c4.Cache4(3, [90], [5], 2, 64, 16)
    d = c.dev4()
    q = torch.randn(5, 4, 64, device="cuda:0").to(dtype)
    a = (d[0], d[1], torch.from_numpy(c.table).to("cuda:0"), T([90]), T([0, 5]))
    w = ref.attention(q.double().cpu().numpy(), c.tokens(c.k, 0, 95), c.tokens(c.v, 0, 95), 90, 0.125, ref.sees(5))
    q[1, 2, 7], q[3, 0, 9], q[3, 1, 9] = float("nan"), float("inf"), float("-inf")
    o = ds.tree_attention(q, *a, scales=d[2])["o"].double().cpu().numpy()
    for i, h in ((1, 2), (3, 0), (3, 1)):
        assert np.isnan(o[i, h]).any()
        o[i, h] = w[0][i, h]
    assert (np.abs(o - w[0]) <= tol(w, 95, 64, dtype is BF)[0]).all()


def test_faults_stay_in_bounds():
    import draft_sampling_scheduling_amd as ds
    for rows_each in (3, 30):
        R = rows_each
        c = c4.Cache4(1, [40, 40, 40], [R, R, R], 2, 64, 16)
        d = c.dev4()
        q = torch.randn(3 * R, 4, 64, device="cuda:0").to(BF)

        def go(table=c.table, ctx=(40, 40, 40), off=(0, R, 2 * R, 3 * R)):
            st = T([0])
            o = torch.zeros(3 * R, 4, 64, dtype=BF, device="cuda:0")
            ds.tree_attention(q, d[0], d[1], torch.from_numpy(table).to("cuda:0"), T(list(ctx)), T(list(off)),
                              scales=d[2], out=dict(o=o), status=st)
            return int(st), o

        good = go()
        assert good[0] == 0
        bad = c.table.copy()
        bad[1, 0], bad[1, 1] = c.P, -1
        st, o = go(bad)
        assert st == ds.FAULT_PAGE
        assert torch.equal(o[:R], good[1][:R]) and torch.equal(o[2 * R:], good[1][2 * R:])
        for ctx in ((40, -1, 40), (40, 10 ** 9, 40), (40, 2 ** 31 - 1, 40)):
            st, o = go(ctx=ctx)
            assert st & ds.FAULT_LEN
            assert torch.equal(o[:R], good[1][:R]) and torch.equal(o[2 * R:], good[1][2 * R:])
        for off in ((0, R, R - 1, 3 * R), (0, R, 2 * R, 3 * R + 1), (-1, R, 2 * R, 3 * R), (0, 2 ** 31 - 1, 6, 9),
                    (5, 3, 1, -2)):
            assert go(off=off)[0] & ds.FAULT_LEN


def test_refusals():
    import draft_sampling_scheduling_amd as ds
    c = c4.Cache4(1, [40], [3], 2, 64, 16)
    k, v, s = c.dev4()
    t = torch.from_numpy(c.table).to("cuda:0")
    q = torch.randn(3, 4, 64, device="cuda:0").to(BF)

    def go(q=q, k=k, v=v, s=s):
        ds.tree_attention(q, k, v, t, T([40]), T([0, 3]), scales=s)

    go()
    for a in (dict(q=q.half()), dict(k=k.int(), v=v.int()), dict(s=s.int()), dict(s=3), dict(k=k.to(BF), v=v.to(BF)),
              dict(v=v.float())):
        with pytest.raises(TypeError):
            go(**a)
    for a in (dict(q=q[..., :32]), dict(v=v[1:]), dict(s=s[1:]), dict(s=s[..., :1]), dict(s=s.cpu()),
              dict(k=k[..., :16], v=v[..., :16]), dict(s=s.transpose(3, 4).contiguous().transpose(3, 4))):
        with pytest.raises(ValueError):
            go(**a)
    with pytest.raises(TypeError):  # codes without their scales
        ds.tree_attention(q, k, v, t, T([40]), T([0, 3]))


def test_strides_that_are_never_used():
    """A dimension of size 1 may have any stride, another one in each tensor."""
    import draft_sampling_scheduling_amd as ds
    c = c4.Cache4(3, [40], [3], 1, 64, 16)
    k, v, s = c.dev4()
    t = torch.from_numpy(c.table).to("cuda:0")
    q = torch.randn(3, 4, 64, device="cuda:0").to(BF)
    want = ds.tree_attention(q, k, v, t, T([40]), T([0, 3]), scales=s)
    odd = [x.as_strided(x.shape, (x.stride(0), w, *x.stride()[2:])) for x, w in ((k, 7), (v, 3), (s, 1))]
    got = ds.tree_attention(q, odd[0], odd[1], t, T([40]), T([0, 3]), scales=odd[2])
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])
    back = ds.cache_read(*odd, T([5, 9]))
    assert all(torch.equal(back[x], y) for x, y in ds.cache_read(k, v, s, T([5, 9])).items())
