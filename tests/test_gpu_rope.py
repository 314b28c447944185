"""qk_rope, rope_append and cache_read against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

from tests import cache4_ref as c4

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def T(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda:0")


def near(got, want, size, bf16):
    y = got.double().cpu().numpy()
    err = np.abs(y - want) / c4.turn_tol(want, size, bf16)
    assert err.max() <= 1, err.max()


class Rows:
    """Rows of a fused projection, positions, a table and norms; the turned heads in 64 bits."""

    def __init__(self, seed, rows, Hq, Hkv, D, rot, dtype, norm=False, interleaved=False, far=300, pad=0):
        g = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D, self.rot, self.dtype = Hq, Hkv, D, rot, dtype
        self.rows, self.interleaved, self.bf = rows, interleaved, dtype is BF
        x = torch.from_numpy(g.standard_normal((rows, Hq + 2 * Hkv + pad, D)).astype(np.float32)).to(dtype)
        self.host = x
        self.qkv = x.to("cuda:0")
        self.pos = g.integers(0, far, rows)
        self.table = c4.rope_table(far, rot) if rot else None
        self.w = [None, None]
        if norm:
            self.w = [torch.from_numpy((1 + 0.3 * g.standard_normal(D)).astype(np.float32)).to(dtype) for _ in range(2)]
        self.kw = dict(q_norm=None if not norm else self.w[0].to("cuda:0"),
                       k_norm=None if not norm else self.w[1].to("cuda:0"), interleaved=interleaved)

    def split(self, x):
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:self.Hq + 2 * self.Hkv]

    def want(self):
        q, k, v = self.split(self.host.double().numpy())
        w = [None if x is None else x.double().numpy() for x in self.w]
        a = (self.pos, self.table, self.rot, self.interleaved)
        return c4.turn(q, *a, w[0]), c4.turn(k, *a, w[1]), v

    def at(self):
        return T(self.pos), None if self.table is None else torch.from_numpy(self.table).to("cuda:0")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (128, 112), (96, 96), (96, 48), (256, 256),
                                   (256, 64), (16, 16), (48, 16), (144, 80)])
def test_rows(D, rot, interleaved, norm, dtype):
    import draft_sampling_scheduling_amd as ds
    for rows, Hq, Hkv in ((1, 1, 1), (7, 5, 2), (40, 14, 1), (3, 2, 8)):
        r = Rows(D + rows, rows, Hq, Hkv, D, rot, dtype, norm, interleaved, pad=1)
        (q, qs), (k, ks), _ = r.want()
        dq, dk, _ = r.split(r.qkv)
        st = T([0])
        got = ds.qk_rope(dq, dk, *r.at(), **r.kw, status=st)
        near(got["q"], q, qs, r.bf)
        near(got["k"], k, ks, r.bf)
        before = r.qkv.clone()
        one = ds.qk_rope(None, dk, *r.at(), **r.kw)
        assert one["q"] is None and torch.equal(one["k"], got["k"])
        one = ds.qk_rope(dq, None, *r.at(), **r.kw)
        assert one["k"] is None and torch.equal(one["q"], got["q"])
        assert torch.equal(before, r.qkv)
        ds.qk_rope(dq, dk, *r.at(), **r.kw, out=dict(q=dq, k=dk), status=st)  # in place
        assert torch.equal(dq, got["q"]) and torch.equal(dk, got["k"])
        assert torch.equal(r.qkv[:, Hq + Hkv:], before[:, Hq + Hkv:]) and int(st) == 0


@pytest.mark.parametrize("rows", [400, 8192])
def test_many_rows(rows):
    import draft_sampling_scheduling_amd as ds
    r = Rows(rows, rows, 7, 2, 128, 128, BF, True, far=70000)
    (q, qs), (k, ks), _ = r.want()
    dq, dk, _ = r.split(r.qkv)
    got = ds.qk_rope(dq, dk, *r.at(), **r.kw)
    near(got["q"], q, qs, True)
    near(got["k"], k, ks, True)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_left_alone(dtype):
    """Rows behind n_rows, and rows whose position is in no table."""
    import draft_sampling_scheduling_amd as ds
    r = Rows(5, 30, 4, 2, 64, 64, dtype, True)
    good = ds.qk_rope(*r.split(r.qkv)[:2], *r.at(), **r.kw)
    for live in (0, 1, 17, 30, 99, -4):
        pos = r.pos.copy()
        pos[[3, 11]] = [-1, 300]
        out = dict(q=torch.full((30, 4, 64), 7.0, dtype=dtype, device="cuda:0"),
                   k=torch.full((30, 2, 64), 7.0, dtype=dtype, device="cuda:0"))
        st = T([0])
        ds.qk_rope(*r.split(r.qkv)[:2], T(pos), r.at()[1], **r.kw, n_rows=T([live]), out=out, status=st)
        live = min(max(live, 0), 30)
        dead = [i for i in range(30) if i >= live or i in (3, 11)]
        alive = [i for i in range(30) if i not in dead]
        for x in ("q", "k"):
            assert torch.equal(out[x][alive], good[x][alive]) and torch.all(out[x][dead] == 7)
        assert int(st) == (ds.FAULT_PARAM if live > 3 else 0)


def test_no_pair_no_harm():
    """Elements behind `rot` are not turned: what stands there stays, and NaN elsewhere does not
    reach it; a pair's NaN reaches its other half only."""
    import draft_sampling_scheduling_amd as ds
    for interleaved in (False, True):
        r = Rows(6, 5, 2, 1, 128, 64, BF, False, interleaved)
        q = r.split(r.qkv)[0]
        q[:, :, 3] = float("nan")
        q[:, :, 100] = float("inf")
        got = ds.qk_rope(q, None, *r.at(), interleaved=interleaved)["q"]
        bad = (3, 2) if interleaved else (3, 35)
        nan = torch.isnan(got)
        assert nan[:, :, list(bad)].all() and int(nan.sum()) == 2 * 10
        assert torch.equal(got[:, :, 64:], q[:, :, 64:])


def caches(g, P, Hkv, page, D, dtype, layout):
    shape = (P, Hkv, page, D) if layout == "phtd" else (P, page, Hkv, D)
    x = [torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(dtype).to("cuda:0") for _ in range(2)]
    return x if layout == "phtd" else [y.transpose(1, 2) for y in x]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("D,rot,norm", [(64, 64, False), (128, 64, True), (96, 96, True), (256, 0, False)])
def test_append(D, rot, norm, layout, dtype):
    import draft_sampling_scheduling_amd as ds
    for rows, page in ((1, 8), (29, 16), (130, 64)):
        g = np.random.default_rng(D + rows)
        r = Rows(rows + D, rows, 6, 2, D, rot, dtype, norm)
        P = rows // page + 3
        k, v = caches(g, P, 2, page, D, dtype, layout)
        slot = g.permutation(P * page)[:rows]
        if rows > 5:
            slot[2], slot[4], slot[5] = -1, P * page, -7
        want_k, want_v = k.clone(), v.clone()
        dq, dk, dv = r.split(r.qkv)
        live = rows - 1 if rows > 1 else 1
        ok = [i for i in range(live) if 0 <= slot[i] < P * page]
        rows_only = ds.qk_rope(dq, dk, *r.at(), **r.kw)
        at = T(slot[ok], torch.int64)
        want_k[at // page, :, at % page] = rows_only["k"][ok]
        want_v[at // page, :, at % page] = dv[ok]
        st = T([0])
        out = torch.full((rows, 6, D), 7.0, dtype=dtype, device="cuda:0")
        got = ds.rope_append(dq, dk, dv, k, v, T(slot), *r.at(), **r.kw, n_rows=T([live]), out=out, status=st)
        assert got is out and torch.equal(got[:live], rows_only["q"][:live]) and torch.all(got[live:] == 7)
        assert torch.equal(k, want_k) and torch.equal(v, want_v)
        assert int(st) == (ds.FAULT_PAGE if rows > 5 else 0)
        # without queries; and with them in place
        k2, v2 = caches(np.random.default_rng(D + rows), P, 2, page, D, dtype, layout)
        assert ds.rope_append(None, dk, dv, k2, v2, T(slot), *r.at(), **r.kw, n_rows=T([live])) is None
        assert torch.equal(k2, k) and torch.equal(v2, v)
        k2, v2 = caches(np.random.default_rng(D + rows), P, 2, page, D, dtype, layout)
        ds.rope_append(dq, dk, dv, k2, v2, T(slot), *r.at(), **r.kw, n_rows=T([live]), out=dq)
        assert torch.equal(k2, k) and torch.equal(v2, v) and torch.equal(dq[:live], rows_only["q"][:live])


def test_a_bad_position_appends_nothing():
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(1)
    r = Rows(8, 4, 2, 1, 64, 64, BF)
    k, v = caches(g, 2, 1, 8, 64, BF, "phtd")
    k0, v0 = k.clone(), v.clone()
    st = T([0])
    ds.rope_append(*r.split(r.qkv), k, v, T([0, 1, 2, 3]), T([300, -1, 2 ** 31 - 1, -2 ** 31]), r.at()[1], status=st)
    assert int(st) == ds.FAULT_PARAM and torch.equal(k, k0) and torch.equal(v, v0)


@pytest.mark.parametrize("four", [False, True])
def test_rows_of_one_slot(four):
    """Of rows with the same slot either's elements (codes, scales) remain, and nobody else's change."""
    import draft_sampling_scheduling_amd as ds
    r = Rows(11, 6, 2, 3, 128, 128, BF)
    slots = [17, 4, 17, 9, 17, 4]
    alone = []
    for order in ([0, 1, 3], [2, 5, 3], [4, 1, 3]):  # each row as the only one of its slot
        g = np.random.default_rng(1)
        d = c4.Cache4(1, [40], [1], 3, 128, 16).dev4() if four else caches(g, 3, 3, 16, 128, BF, "phtd")
        kw = dict(scales=d[2]) if four else {}
        x = r.qkv[order].contiguous()
        ds.rope_append(None, *r.split(x)[1:], d[0], d[1], T([slots[i] for i in order]), T(r.pos[order]), r.at()[1], **kw)
        alone.append(d)
    g = np.random.default_rng(1)
    d = c4.Cache4(1, [40], [1], 3, 128, 16).dev4() if four else caches(g, 3, 3, 16, 128, BF, "phtd")
    kw = dict(scales=d[2]) if four else {}
    ds.rope_append(None, *r.split(r.qkv)[1:], d[0], d[1], T(slots), *r.at(), **kw)
    for got, *want in zip(d, *alone):
        assert torch.stack([got == w for w in want]).any(0).all()


def edges(g, rows, heads, D, dtype):
    """Values whose groups try the quantising: borders, zeros, one large, tiny, huge, infinite, NaN."""
    x = g.standard_normal((rows, heads, D)).astype(np.float32)
    x *= 2.0 ** g.integers(-20, 20, (rows, heads, 1))
    kinds = g.integers(0, 10, (rows, heads, D // 32))
    for i, j, k in np.ndindex(kinds.shape):
        y = x[i, j, 32 * k:32 * k + 32]
        kind = kinds[i, j, k]
        e = 2.0 ** int(g.integers(-30, 30))
        if kind == 0:
            y[:] = g.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, -7, -2.5, -0.25, 0, -0.0], 32) * e
        elif kind == 1:
            y[:] = g.choice([0.0, -0.0], 32)
        elif kind == 2:
            y[:] = 2.0 ** -126 * g.standard_normal(32)
        elif kind == 3:
            y[:] = 3e38 * g.uniform(-1, 1, 32)
        elif kind == 4:
            y[int(g.integers(32))] = g.choice([np.inf, -np.inf, np.nan])
        elif kind == 5:
            y[:] = 2.0 ** -149 * g.integers(-9, 9, 32)
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("D,rot,norm,interleaved", [(64, 64, False, False), (128, 128, True, False), (128, 64, False, True),
                                                    (128, 32, True, True), (64, 48, True, False), (64, 0, False, False),
                                                    (128, 0, True, False)])
def test_append4(D, rot, norm, interleaved, layout, dtype):
    """Codes and scale bytes are those of the definition, bit for bit, and no other byte changes."""
    import draft_sampling_scheduling_amd as ds
    for rows, page, Hkv in ((1, 8, 1), (45, 16, 3)):
        g = np.random.default_rng(rows + D + rot)
        r = Rows(rows, rows, 4, Hkv, D, rot, dtype, norm, interleaved)
        r.host[:, 4:] = edges(g, rows, 2 * Hkv, D, dtype)
        r.qkv.copy_(r.host)
        c = c4.Cache4(rows, [page * 3], [1], Hkv, D, page, layout)
        slot = g.permutation(c.P * page)[:rows]
        live = rows
        if rows > 5:
            slot[2], slot[4], live = -1, c.P * page, rows - 2
        (q, qs), (k, _), v = r.want()
        st = T([0])
        dk, dv, sc = c.dev4()
        out = ds.rope_append(*r.split(r.qkv), dk, dv, T(slot), *r.at(), scales=sc, **r.kw, n_rows=T([live]), status=st)
        assert int(st) == (ds.FAULT_PAGE if rows > 5 else 0)
        near(out[:live], q[:live], qs[:live], r.bf)
        for i in range(live):
            if 0 <= slot[i] < c.P * page:
                p, t = slot[i] // page, slot[i] % page
                c.kc[p, :, t], c.sc[p, :, t, 0] = c4.quantise(k[i])
                c.vc[p, :, t], c.sc[p, :, t, 1] = c4.quantise(v[i])
        for got, want, name in ((sc, c.sc, "scales"), (dk, c.kc, "keys"), (dv, c.vc, "values")):
            same = got.cpu().numpy() == want
            assert same.all(), (name, np.argwhere(~same)[:5])
        if rot == 0 and not norm:  # cache_append is the same without a rotation
            d2 = c4.Cache4(rows, [page * 3], [1], Hkv, D, page, layout).dev4()
            ds.cache_append(*r.split(r.qkv)[1:], d2[0], d2[1], T(slot), scales=d2[2], n_rows=T([live]))
            assert all(torch.equal(a, b) for a, b in zip(d2, (dk, dv, sc)))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layers", [0, 1, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_read(D, layers, dtype):
    """Every code and byte (253 and 254 apart) as the value it stands for."""
    import draft_sampling_scheduling_amd as ds
    for layout in ("phtd", "pthd"):
        cs = [c4.Cache4(i, [90], [1], 3, D, 16, layout) for i in range(max(layers, 1))]
        g = np.random.default_rng(D)
        for c in cs:
            c.sc[:] = g.choice([*range(253), 255], c.sc.shape)
            c.renew()
        d = [x[0] for x in zip(*(c.dev4() for c in cs))] if not layers else [torch.stack(x) for x in zip(*(c.dev4() for c in cs))]
        if layout == "pthd" and layers:  # (stack laid them out anew)
            d = [x.transpose(2, 3).contiguous().transpose(2, 3) for x in d]
        slot = g.integers(0, cs[0].P * 16, 50)
        slot[[3, 9, 12]] = [-1, cs[0].P * 16, -3]
        shape = ((layers,) if layers else ()) + (50, 3, D)
        out = dict(k=torch.full(shape, 7.0, dtype=dtype, device="cuda:0"), v=torch.full(shape, 7.0, dtype=dtype, device="cuda:0"))
        st = T([0])
        assert ds.cache_read(*d, T(slot), n_rows=T([40]), out=out, status=st) is out
        assert int(st) == ds.FAULT_PAGE
        for i, c in enumerate(cs):
            for got, x in ((out["k"], c.k), (out["v"], c.v)):
                want = x.numpy()[slot % (c.P * 16) // 16, :, slot % 16]
                want[[3, 9, 12]] = 7
                want[40:] = 7
                y = (got[i] if layers else got).double().cpu().numpy()
                assert ((y == want) | (np.isnan(y) & np.isnan(want))).all()
    fresh = ds.cache_read(*d, T([1, 2]))
    assert fresh["k"].dtype is BF and fresh["k"].shape[-3:] == (2, 3, D)


def test_written_and_read_back():
    """What comes back is off by at most half a step: a quarter of the power up to 2 of it, a half up
    to 4, one up to 7."""
    import draft_sampling_scheduling_amd as ds
    r = Rows(3, 500, 1, 4, 128, 128, F32, True)
    (_, _), (k, _), v = r.want()
    c = c4.Cache4(1, [640], [1], 4, 128, 16)
    d = c.dev4()
    slot = T(np.random.default_rng(2).permutation(c.P * 16)[:500])
    ds.rope_append(*r.split(r.qkv), d[0], d[1], slot, *r.at(), scales=d[2], **r.kw)
    back = ds.cache_read(*d, slot, dtype=F32)
    for got, x in ((back["k"], k), (back["v"], v)):
        y = x.reshape(-1, 32)
        unit = 2.0 ** np.ceil(np.log2(np.abs(y).max(1, keepdims=True) / 7))
        half = np.where(np.abs(y) <= 2 * unit, 0.25, np.where(np.abs(y) <= 4 * unit, 0.5, 1.0)) * unit
        assert (np.abs(got.double().cpu().numpy().reshape(-1, 32) - y) <= half).all()


def test_other_streams_and_replays():
    """Captured with the position, slots and rows changing between replays; eager work between."""
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(4)
    r = Rows(4, 33, 6, 2, 128, 128, BF, True)
    c = c4.Cache4(4, [300], [1], 2, 128, 16)
    d0 = c.dev4()
    d, pos, table = [x.clone() for x in d0], *r.at()
    slot, n_rows = T(np.arange(33)), T([33])
    all_slots = T(np.arange(c.P * 16))

    def run():
        for a, b in zip(d, d0):
            a.copy_(b)
        q = ds.rope_append(*r.split(r.qkv), d[0], d[1], slot, pos, table, scales=d[2], **r.kw, n_rows=n_rows,
                           out=torch.zeros(33, 6, 128, dtype=BF, device="cuda:0"))
        back = ds.cache_read(*d, all_slots)
        return [q, back["k"], back["v"], *d]

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for k in range(4):
        pos.copy_(T(g.integers(0, 300, 33)))
        slot.copy_(T(g.permutation(c.P * 16)[:33]))
        n_rows.copy_(T([int(g.integers(0, 34))]))
        r.qkv.copy_(torch.randn_like(r.qkv))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
