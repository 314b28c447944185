"""tree_attention against the attention of each row taken by itself in 64 bits, within bounds
that count its roundings (target_ref.attention_tol)."""
import numpy as np
import pytest
import torch

from tests import target_ref as ref

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def T(x, dtype=I32):
    return torch.tensor(x, dtype=dtype, device="cuda:0")


def trees(g, n):
    """Masks of a random tree per request; packed."""
    out = []
    for m in n:
        up = [[]]
        for i in range(1, m):
            up.append(up[int(g.integers(0, i))] + [i])
        out += [sum(1 << (j - 1) for j in p) for p in up[:m]]
    return out


def check(seed, ctx, n, Hq, Hkv, D, page, dtype, tree=False, layout="phtd", q_pad=0, slack=3,
          scale=None, fill=float("nan"), spread=1.0, edit=None, anc=None):
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(seed)
    c = ref.Cache(seed, ctx, n, Hkv, D, page, dtype, layout, fill=fill)
    rows = sum(n) + slack
    q = torch.from_numpy(spread * g.standard_normal((rows, Hq + q_pad, D), np.float32)).to(dtype)
    if anc is None and tree:
        anc = trees(g, n)
    off = np.concatenate([[0], np.cumsum(n)])
    if edit:
        edit(c, q)
    o = torch.full((rows, Hq, D), 77.0, dtype=dtype, device="cuda:0")
    lse = torch.full((rows, Hq), 77.0, device="cuda:0")
    st = T([0])
    masks = None
    if anc is not None:
        masks = T([a - 2 ** 64 if a >= 2 ** 63 else a for a in anc] + [-1] * slack, torch.int64)
    dq = q.to("cuda:0")
    args = (dq[:, :Hq], c.dev(c.k), c.dev(c.v), torch.from_numpy(c.table).to("cuda:0"), T(ctx),
            T(off.tolist()))
    ds.tree_attention(*args, anc=masks, scale=scale, out=dict(o=o, lse=lse), status=st)
    again = ds.tree_attention(*args, anc=masks, scale=scale)
    assert int(st) == 0
    live = int(off[-1])
    assert torch.equal(again["o"][:live], o[:live]) and torch.equal(again["lse"][:live], lse[:live])
    assert torch.all(o[live:] == 77.0) and torch.all(lse[live:] == 77.0)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    worst = 0.0
    for k, (cx, m) in enumerate(zip(ctx, n)):
        if m == 0:
            continue
        a = slice(off[k], off[k + 1])
        see = ref.sees(m, None if anc is None else anc[a])
        w = ref.attention(q[a, :Hq].double().numpy(), c.tokens(c.k, k, cx + m), c.tokens(c.v, k, cx + m),
                          cx, D ** -0.5 if scale is None else scale, see)
        to, tl = ref.attention_tol(*w, cx + m, D, dtype is BF)
        eo, el = np.abs(o[a] - w[0]) / to, np.abs(lse[a] - w[1]) / tl
        worst = max(worst, eo.max(), el.max())
        assert eo.max() <= 1 and el.max() <= 1, (k, cx, m, eo.max(), el.max())
    return worst


SHAPES = [  # ctx, n
    ([0], [1]), ([31], [1]), ([32], [1]), ([63, 64, 65], [1, 1, 1]), ([1000], [1]),
    ([0, 5, 0, 200], [3, 0, 9, 5]), ([0, 0], [0, 7]), ([130, 77, 4, 260, 12], [9, 1, 4, 2, 6])]


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
    """A chain of any length: more rows than a row tile, and than a tree has nodes."""
    check(n[0], ctx, n, 4, 2, 64, 16, dtype)
    check(n[0], ctx, n, 3, 1, 128, 64, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_long(dtype):
    """One request over many workgroups, and requests of very different lengths."""
    check(1, [20000], [3], 2, 1, 128, 16, dtype)
    check(2, [9001, 3, 0, 4100, 64], [2, 1, 5, 1, 1], 4, 2, 64, 32, dtype)
    check(6, [7000, 40], [3, 1], 24, 1, 128, 16, dtype)   # 72 query rows to a head
    check(7, [7000, 40], [3, 5], 11, 1, 64, 16, dtype)    # 55
    check(8, [2500, 900, 3], [6, 4, 7], 40, 2, 64, 8, dtype, tree=True)  # 140: two row tiles


def test_many_requests():
    g = np.random.default_rng(3)
    check(3, g.integers(0, 40, 300).tolist(), g.integers(0, 4, 300).tolist(), 2, 1, 64, 8, BF)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_large_scores(dtype):
    """Scores of some hundreds: one token takes all the weight, and the maximum keeps moving."""
    check(4, [300, 64], [4, 9], 4, 2, 64, 16, dtype, spread=40.0)
    check(5, [300, 64], [4, 9], 4, 2, 128, 16, dtype, scale=1e-6)  # and next to none


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [6, 14, 24])
def test_unseen_nodes_hold_anything(Hq, bad, D, dtype):
    """Keys and values of nodes that a row does not see: infinite or NaN, they reach only the
    rows that see them (18, 42 and 72 query rows to a cache head)."""
    import draft_sampling_scheduling_amd as ds
    n, ctx = 6, 45
    anc = [0, 0b1, 0b10, 0b101, 0b1001, 0b10010]  # node 2, and 5 under it, hold it
    sick = [2, 5]
    g = np.random.default_rng(9)
    c = ref.Cache(9, [ctx], [n], 2, D, 16, dtype)
    q = torch.from_numpy(g.standard_normal((n, Hq, D), np.float32)).to(dtype)

    def go():
        return ds.tree_attention(q.to("cuda:0"), c.dev(c.k), c.dev(c.v),
                                 torch.from_numpy(c.table).to("cuda:0"), T([ctx]), T([0, n]),
                                 anc=T(anc, torch.int64))["o"].double().cpu().numpy()
    before = go()
    see = ref.sees(n, anc)
    assert [i for i in range(n) if see[i, 2] or see[i, 5]] == sick
    for x in (c.k, c.v):
        for node in (2, 5):
            t = ctx + node
            x[c.table[0, t // 16], :, t % 16] = bad
    after = go()
    well = [i for i in range(n) if i not in sick]
    assert np.isfinite(after[well]).all()
    w = ref.attention(q.double().numpy(), np.nan_to_num(c.tokens(c.k, 0, ctx + n), posinf=0, neginf=0),
                      np.nan_to_num(c.tokens(c.v, 0, ctx + n), posinf=0, neginf=0), ctx, D ** -0.5, see)
    tol, _ = ref.attention_tol(*w, ctx + n, D, dtype is BF)
    assert (np.abs(after - w[0]) <= tol)[well].all() and np.abs(after - before)[well].max() < 0.1
    assert not np.isfinite(after[[2, 5]]).any()  # who sees it has it


def test_faults_stay_in_bounds():
    import draft_sampling_scheduling_amd as ds
    c = ref.Cache(1, [40, 40, 40], [3, 3, 3], 2, 64, 16, BF)
    q = torch.randn(9, 4, 64, device="cuda:0").to(BF)

    def go(table=c.table, ctx=(40, 40, 40), off=(0, 3, 6, 9), anc=None, rows=9):
        st = T([0])
        o = torch.zeros(rows, 4, 64, dtype=BF, device="cuda:0")
        ds.tree_attention(q[:rows], c.dev(c.k), c.dev(c.v), torch.from_numpy(table).to("cuda:0"),
                          T(list(ctx)), T(list(off)), anc=anc, out=dict(o=o), status=st)
        return int(st), o

    good = go()
    assert good[0] == 0
    bad = c.table.copy()
    bad[1, 0], bad[1, 1] = c.P, -1
    st, o = go(bad)
    assert st == ds.FAULT_PAGE
    assert torch.equal(o[:3], good[1][:3]) and torch.equal(o[6:], good[1][6:])
    for ctx in ((40, -1, 40), (40, 10 ** 9, 40), (40, 2 ** 31 - 1, 40)):
        st, o = go(ctx=ctx)
        assert st & ds.FAULT_LEN
        assert torch.equal(o[:3], good[1][:3]) and torch.equal(o[6:], good[1][6:])
    for off in ((0, 3, 2, 9), (0, 3, 6, 10), (-1, 3, 6, 9), (0, 2 ** 31 - 1, 6, 9), (5, 3, 1, -2)):
        assert go(off=off)[0] & ds.FAULT_LEN
    wide = ref.Cache(2, [10], [70], 1, 64, 16, BF)
    st = T([0])
    ds.tree_attention(torch.randn(70, 1, 64, device="cuda:0").to(BF), wide.dev(wide.k),
                      wide.dev(wide.v), torch.from_numpy(wide.table).to("cuda:0"), T([10]),
                      T([0, 70]), anc=T([-1] * 70, torch.int64), status=st)
    assert int(st) == ds.FAULT_TREE


def test_refusals():
    import draft_sampling_scheduling_amd as ds
    c = ref.Cache(1, [40], [3], 2, 64, 16, BF)
    k, v, t = c.dev(c.k), c.dev(c.v), torch.from_numpy(c.table).to("cuda:0")
    q = torch.randn(3, 4, 64, device="cuda:0").to(BF)
    ok = (q, k, v, t, T([40]), T([0, 3]))

    def swap(i, x):
        return ok[:i] + (x,) + ok[i + 1:]

    for a in (swap(0, q.float()), swap(0, q.half()), swap(2, v.float()), swap(3, t.long()),
              swap(4, T([40]).float())):
        with pytest.raises(TypeError):
            ds.tree_attention(*a)
    for a in (swap(0, q[..., :32]), swap(2, v[1:]), swap(4, T([40, 1])), swap(5, T([0])),
              swap(1, k.cpu()), swap(1, k[..., :32]), swap(0, q.transpose(0, 1))):
        with pytest.raises(ValueError):
            ds.tree_attention(*a)
    for a in (swap(0, q[:, :3].contiguous()),):
        with pytest.raises(ds.DsparkError):
            ds.tree_attention(*a)
    for s in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ds.DsparkError):
            ds.tree_attention(*ok, scale=s)
    with pytest.raises(ValueError):
        ds.tree_attention(*ok, anc=T([0, 0], torch.int64))
    with pytest.raises(ValueError):
        ds.tree_attention(*ok, ws=torch.empty(256, dtype=torch.uint8, device="cuda:0"))
    none = ds.tree_attention(q[:0], k, v, t, T([40]), T([0, 0]))
    assert none["o"].shape == (0, 4, 64)


def test_cache_beyond_32_bits():
    """Caches of 5 GiB each, their last pages in use: written, read and moved where they are."""
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(5)
    P, Hkv, page, D, n, ctx = 2560, 8, 1024, 128, 5, 1500
    k, v = (torch.empty(P, Hkv, page, D, dtype=BF, device="cuda:0") for _ in range(2))
    assert k.numel() * 2 > 2 ** 32
    table = T([[P - 1, P - 3], [0, P - 2]])
    rows = torch.from_numpy(g.standard_normal((2, 2, ctx + n, Hkv, D), np.float32)).to(BF)
    t = np.arange(ctx + n)
    for q in range(2):
        slot = table[q].cpu().numpy()[t // page] * page + t % page
        ds.cache_append(rows[0, q].to("cuda:0"), rows[1, q].to("cuda:0"), k, v, T(slot.tolist()))
    qs = torch.from_numpy(g.standard_normal((2 * n, 8, D), np.float32)).to(BF)
    anc = [0, 1, 2, 0b101, 0b1010] * 2  # 1 and 2 under the anchor, 3 under 1, 4 under 2
    o = ds.tree_attention(qs.to("cuda:0"), k, v, table, T([ctx] * 2), T([0, n, 2 * n]),
                          anc=T(anc, torch.int64))["o"].double().cpu().numpy()
    for q in range(2):
        a = slice(q * n, q * n + n)
        w = ref.attention(qs[a].double().numpy(), rows[0, q].double().numpy(),
                          rows[1, q].double().numpy(), ctx, D ** -0.5, ref.sees(n, anc[a]))
        tol, _ = ref.attention_tol(*w, ctx + n, D, True)
        assert (np.abs(o[a] - w[0]) <= tol).all()
    held, free, nf = T([2, 2]), T([0] * 4), T([0])
    ds.cache_commit(T([2, 2]), T([ctx] * 2), held, table, free, nf, page, path=T([[2, 4]] * 2),
                    k_cache=k, v_cache=v)
    for q in range(2):
        for x, r in ((k, rows[0, q]), (v, rows[1, q])):
            for i, src in ((1, 2), (2, 4), (3, 3), (0, 0)):
                at = ctx + i
                assert torch.equal(x[int(table[q, at // page]), :, at % page].cpu(), r[ctx + src])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx", [0, 75])
def test_later_tokens_of_a_prompt_hold_anything(ctx, D, dtype):
    """A prompt's tokens reach no row before them, in its own row tile or in another."""
    import draft_sampling_scheduling_amd as ds
    n, Hq = 300, 4
    g = np.random.default_rng(ctx + D)
    c = ref.Cache(ctx + D, [ctx], [n], 2, D, 16, dtype)
    q = torch.from_numpy(g.standard_normal((n, Hq, D), np.float32)).to(dtype)
    clean = [c.tokens(x, 0, ctx + n) for x in (c.k, c.v)]
    w = ref.attention(q.double().numpy(), *clean, ctx, D ** -0.5, ref.sees(n, None))
    tol, _ = ref.attention_tol(*w, ctx + n, D, dtype is BF)
    for at, bad in ((299, float("nan")), (222, float("inf")), (190, float("nan")), (64, float("-inf"))):
        t = ctx + at
        for x in (c.k, c.v):
            x[c.table[0, t // 16], :, t % 16] = bad
        o = ds.tree_attention(q.to("cuda:0"), c.dev(c.k), c.dev(c.v),
                              torch.from_numpy(c.table).to("cuda:0"), T([ctx]),
                              T([0, n]))["o"].double().cpu().numpy()
        assert (np.abs(o - w[0]) <= tol)[:at].all(), at
        assert not np.isfinite(o[at]).any(), at


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 5, 7, 16])
@pytest.mark.parametrize("ctx,n", [([0], [700]), ([13, 0, 90], [333, 2, 450]),
                                   ([0] * 12, [330] + [1] * 11)], ids=["one", "three", "mixed"])
def test_prompts_of_many_row_tiles(ctx, n, G, dtype):
    """Row tiles that see more and more tokens, in every split of the waves: many rows a request on
    average, and few with one prompt among them."""
    check(G + len(n), ctx, n, 2 * G, 2, 64, 16, dtype)
    check(G + len(n), ctx, n, G, 1, 128, 32, dtype)
