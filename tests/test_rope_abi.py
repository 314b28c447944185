"""Refusals of qk_rope, the appends with a rotation and the 4-bit cache's calls (no GPU needed)."""
import ctypes as C
import os

import pytest


@pytest.fixture(scope="module")
def ds():
    import draft_sampling_scheduling_amd as ds
    if not os.path.exists(ds.LIB_PATH):
        from draft_sampling_scheduling_amd import build
        build.build()
    ds.lib()
    return ds


def P(x=0x100000):
    return C.c_void_p(x)  # never dereferenced: these calls return before any launch


def test_qk_rope_refusals(ds):
    def call(rows=4, Hq=4, Hkv=2, D=64, rot=64, dt=ds.BF16, q=P(), q_row=512, k=P(0x200000), k_row=512, pos=P(),
             rope=P(), n_pos=10, qn=None, kn=None, eps=1e-6, qo=P(0x300000), qo_row=256, ko=P(0x400000), ko_row=128):
        return ds.lib().dspark_qk_rope(rows, Hq, Hkv, D, rot, 0, dt, q, q_row, k, k_row, pos, rope, n_pos, qn, kn,
                                       eps, None, qo, qo_row, ko, ko_row, None, None)

    for bad in (dict(rows=-1), dict(Hq=0), dict(Hkv=-1), dict(Hkv=0), dict(D=8), dict(D=72), dict(D=272), dict(rot=0),
                dict(rot=8), dict(rot=24), dict(rot=80), dict(dt=2), dict(n_pos=0), dict(q=None, k=None),
                dict(pos=None), dict(q=P(0x100008)), dict(k=P(0x200002)), dict(rope=P(0x100004)), dict(qn=P(0x100004)),
                dict(kn=P(0x100002)), dict(q_row=511), dict(k_row=-512), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(qo=None), dict(ko=None), dict(qo=P(0x300008)), dict(qo_row=248),
                dict(ko_row=120), dict(qo_row=0),                     # output rows over each other
                dict(qo=P(0x100010)), dict(qo=P(), qo_row=256),       # over q, not in its place
                dict(qo=P(0x200000)), dict(ko=P()), dict(ko=P(0x300000)),  # over k; over q; over q's output
                dict(k=P(0x100000 + 256), qo=P(), qo_row=512)):       # k among q's heads, q turned in place
        assert call(**bad) == ds.EINVAL, bad
    assert call(rows=0) == ds.OK
    assert call(rows=1 << 30, Hq=1 << 20) == ds.EINVAL  # no grid holds it


def append(ds, four, rows=4, Hq=4, Hkv=2, D=64, rot=64, dt=None, page=16, n=10, q=P(), k=P(0x200000), v=P(0x280000),
           row=512, slot=P(), pos=P(), rope=P(), qo=P(0x300000), kc=P(0x1000000), vc=P(0x2000000), st=1024, tok=64,
           sc=P(0x3000000), s_head=64, s_tok=4, ps=2048):
    dt = ds.BF16 if dt is None else dt
    a = [rows, Hq, Hkv, D, rot, 0, dt, page, n, q, row, k, row, v, row, slot, pos, rope, 10, None, None, 1e-6, None,
         qo, Hq * D, kc, vc, ps, st, tok]
    if four:
        return ds.lib().dspark_cache4_append(*a, sc, 128, s_head, s_tok, None, None)
    return ds.lib().dspark_rope_append(*a, None, None)


@pytest.mark.parametrize("four", [False, True])
def test_append_refusals(ds, four):
    for bad in (dict(rows=-1), dict(Hkv=0), dict(D=60), dict(rot=24), dict(dt=3), dict(page=24), dict(n=0),
                dict(n=1 << 27), dict(k=None), dict(v=None), dict(slot=None), dict(pos=None), dict(q=P(0x100008)),
                dict(k=P(0x200008)), dict(v=P(0x280008)), dict(row=250), dict(row=-256), dict(kc=None), dict(vc=None),
                dict(kc=P(0x1000004)), dict(st=1023), dict(tok=-64), dict(ps=2047), dict(qo=None), dict(qo=P(0x100010)),
                dict(qo=P(0x200000)), dict(qo=P(0x280000)), dict(kc=P(0x200000)), dict(vc=P(0x200000)),
                dict(kc=P(0x280000)), dict(vc=P(0x300000)), dict(kc=P())):
        assert append(ds, four, **bad) == ds.EINVAL, bad
    assert append(ds, four, rows=0) == ds.OK
    assert append(ds, four, rows=1 << 30, Hkv=1 << 18) == ds.EINVAL  # no grid holds it


def test_append4_refusals(ds):
    for bad in (dict(D=96), dict(D=256), dict(D=32), dict(sc=None), dict(sc=P(0x3000004)), dict(s_tok=2), dict(s_head=-64),
                dict(s_head=66), dict(sc=P(0x200000)), dict(sc=P(0x300000))):
        assert append(ds, True, **bad) == ds.EINVAL, bad


def test_read_refusals(ds):
    def call(layers=2, rows=4, Hkv=2, D=64, dt=ds.BF16, page=16, n=10, slot=P(), kc=P(0x1000000), vc=P(0x2000000), ls=65536,
             st=1024, sc=P(0x3000000), sl=8192, s_tok=4, k=P(0x100000), v=P(0x200000)):
        return ds.lib().dspark_cache4_read(layers, rows, Hkv, D, dt, page, n, slot, None, kc, vc, ls, 2048, st, 32, sc, sl,
                                           128, 64, s_tok, k, v, None, None)

    for bad in (dict(layers=-1), dict(rows=-1), dict(Hkv=0), dict(D=32), dict(D=96), dict(dt=2), dict(page=12), dict(n=0),
                dict(slot=None), dict(kc=None), dict(vc=P(0x2000008)), dict(ls=-16), dict(ls=8), dict(st=1), dict(sc=None),
                dict(sc=P(0x3000008)), dict(sl=2), dict(s_tok=3), dict(k=None), dict(v=P(0x200004)), dict(v=P(0x100000)),
                dict(k=P(0x1000000)), dict(v=P(0x2000000)), dict(k=P(0x3000000))):
        assert call(**bad) == ds.EINVAL, bad
    assert call(rows=0) == ds.OK and call(layers=0) == ds.OK
    assert call(rows=1 << 30, layers=4) == ds.EINVAL and call(rows=1 << 28, Hkv=16) == ds.EINVAL  # no grid holds it


def test_binding_wants_device_tensors(ds):
    import torch
    i, x, u = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 64), torch.zeros(2, 2, 16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ds.qk_rope(x, x, i, torch.zeros(9, 64))
    with pytest.raises(ValueError):
        ds.rope_append(x, x, x, x, x, i, i, torch.zeros(9, 64))
    with pytest.raises(ValueError):
        ds.cache_append(x, x, u, u, i, scales=u)
    with pytest.raises(ValueError):
        ds.cache_read(u, u, u, i)
    with pytest.raises(TypeError):
        ds.qk_rope([0], None, i, None)
    with pytest.raises(TypeError):
        ds.qk_rope(None, None, i, None)


def test_attention4_refusals(ds):
    ws = ds.tree_attention_workspace_bytes(4, 20, 8, 2, 64, ds.BF16, True)
    assert ws > 0 and ds.tree_attention_workspace_bytes(4, 20, 8, 2, 96, ds.BF16, True) == 0
    assert ds.tree_attention_workspace_bytes(0, 20, 8, 2, 64, ds.BF16, True) == 0

    def call(R=4, rows=20, Hq=8, Hkv=2, D=64, dt=ds.BF16, page=16, W=10, n=40, q=P(), q_row=512, k=P(), ps=2048, st=1024,
             tok=32, sc=P(), sp=128, s_tok=4, table=P(), scale=0.125, o=P(0x200000), wsp=P(), ws_bytes=ws):
        return ds.lib().dspark_tree_attention4(R, rows, Hq, Hkv, D, dt, page, W, n, q, q_row, k, P(), ps, st, tok, sc, sp, 64,
                                               s_tok, table, P(), P(), None, scale, o, None, None, wsp, ws_bytes, None)

    for bad in (dict(R=(1 << 20) + 1), dict(Hq=9), dict(Hkv=0), dict(D=80), dict(dt=2), dict(page=10), dict(W=0),
                dict(W=(1 << 26) + 1), dict(n=0), dict(q=None), dict(q=P(0x100002)), dict(q_row=511), dict(k=None),
                dict(k=P(0x100008)), dict(ps=8), dict(st=1), dict(tok=-64), dict(tok=1 << 25), dict(sc=None),
                dict(sc=P(0x100004)), dict(sp=2), dict(s_tok=-4), dict(s_tok=1 << 25), dict(table=None),
                dict(scale=0.0), dict(scale=float("nan")), dict(scale=3e38), dict(o=None), dict(o=P()), dict(wsp=None),
                dict(wsp=P(0x100008)), dict(rows=-1), dict(rows=1 << 28)):
        assert call(**bad) == ds.EINVAL, bad
    assert call(ws_bytes=ws - 1) == ds.EWORKSPACE
    assert call(R=0) == ds.OK and call(rows=0) == ds.OK


def test_commit4_refusals(ds):
    ws = ds.cache_commit_workspace_bytes(4, 10, True)

    def call(R=4, gamma=4, page=16, W=10, n_acc=P(), path=P(), layers=1, Hkv=2, D=64, n=40, k=P(), ls=0, st=1024, tok=32, sc=P(),
             sl=0, s_tok=4, ws_bytes=ws, ctx=P(0x200000), out=P(0x200000)):
        return ds.lib().dspark_cache4_commit(R, gamma, page, W, 8, n_acc, path, None, ctx, out, P(0x300000), P(), P(), P(),
                                             layers, Hkv, D, n, k, P(), ls, 2048, st, tok, sc, sl, 128, 64, s_tok, None, P(),
                                             ws_bytes, None)

    for bad in (dict(R=-1), dict(gamma=0), dict(gamma=65), dict(page=20), dict(W=0), dict(n_acc=None), dict(layers=-1),
                dict(Hkv=0), dict(D=32), dict(D=256), dict(n=0), dict(k=None), dict(k=P(0x100008)), dict(ls=8), dict(st=8),
                dict(tok=-16), dict(sc=None), dict(sc=P(0x100004)), dict(sl=-4), dict(sl=2), dict(s_tok=2), dict(out=P(0x200004)),
                dict(out=P())):
        assert call(**bad) == ds.EINVAL, bad
    assert call(ws_bytes=ws - 1) == ds.EWORKSPACE
    assert call(R=0) == ds.OK


def test_eps_that_float_loses(ds):
    """An eps that is nothing as a float would turn a head of zeros into NaN: refused."""
    for eps, rc in ((1e-46, ds.EINVAL), (9e-31, ds.EINVAL), (1.1e30, ds.EINVAL), (0.0, ds.OK), (1e-30, ds.OK),
                    (1e30, ds.OK)):
        assert ds.lib().dspark_qk_rope(0, 4, 2, 64, 64, 0, ds.BF16, P(), 512, P(0x200000), 512, P(), P(), 10, None,
                                       None, eps, None, P(0x300000), 256, P(0x400000), 128, None, None) == rc, eps
