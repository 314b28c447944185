"""Host-side checks of include/dspark_target.h: the library exports what it declares, and
each call refuses bad arguments before anything reaches a device (no GPU needed)."""
import ctypes as C
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ds():
    import draft_sampling_scheduling_amd as ds
    if not os.path.exists(ds.LIB_PATH):
        from draft_sampling_scheduling_amd import build
        build.build()
    ds.lib()
    return ds


def P(x=0x1000):
    return C.c_void_p(x)  # never dereferenced: these calls return before any launch


def test_exports_every_declared_symbol(ds):
    src = open(os.path.join(ROOT, "include", "dspark_target.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(dspark_\w+)\s*\(", src))
    assert names == set(ds.TARGET_EXPORTS)
    for n in names:
        assert hasattr(ds.lib(), n), n


def test_workspace_sizes(ds):
    assert ds.cache_plan_workspace_bytes(0, 5000) == 0
    assert ds.cache_plan_workspace_bytes(256, 1024) == 0          # small: needs none
    assert ds.cache_plan_workspace_bytes(256, 16385) >= 3 * 4 * 256
    assert ds.cache_plan_workspace_bytes(1025, 300) >= 3 * 4 * 1025
    assert ds.cache_plan_workspace_bytes(200, 1000, 65) >= 3 * 4 * 200
    assert ds.cache_commit_workspace_bytes(-1, 10) == 0
    assert ds.cache_commit_workspace_bytes(7, 100) == 0
    assert ds.cache_commit_workspace_bytes(7, 100, True) >= 3 * 4 * 7
    assert ds.cache_commit_workspace_bytes(1025, 1) >= 3 * 4 * 1025
    assert ds.cache_commit_workspace_bytes(512, 8) == 0
    assert ds.cache_commit_workspace_bytes(512, 9) >= 3 * 4 * 512
    assert ds.tree_attention_workspace_bytes(4, 20, 8, 2, 64, ds.BF16) > 0
    assert ds.tree_attention_workspace_bytes(0, 20, 8, 2, 64, ds.BF16) == 0
    for bad in (dict(Hq=7), dict(Hkv=0), dict(D=96), dict(dt=2), dict(rows=-1)):
        a = dict(R=4, rows=20, Hq=8, Hkv=2, D=64, dt=ds.BF16, **{})
        a.update(bad)
        assert ds.tree_attention_workspace_bytes(**a) == 0, bad


def test_plan_refusals(ds):
    ws = ds.cache_plan_workspace_bytes(4, 20000)

    def call(R=4, rows=20000, page=16, W=10, free_len=8, extra=1, lens=P(), free=P(), parent=None,
             width=0, slot=P(), anc=None, wsp=P(), ws_bytes=ws):
        return ds.lib().dspark_cache_plan(R, rows, page, W, free_len, extra, lens, P(), P(), P(),
                                          free, P(), parent, width, P(), None, None, slot, anc,
                                          None, wsp, ws_bytes, None)

    for bad in (dict(R=-1), dict(R=(1 << 20) + 1), dict(rows=-1), dict(page=12), dict(page=4), dict(page=2048),
                dict(W=0), dict(W=(1 << 26) + 1), dict(free_len=-1), dict(extra=2), dict(lens=None),
                dict(free=None), dict(parent=P(), width=5), dict(parent=P(), anc=P(), width=0),
                dict(slot=None), dict(wsp=None), dict(wsp=P(0x1002)),
                dict(rows=20, lens=None, wsp=None)):
        assert call(**bad) == ds.EINVAL, bad
    assert call(ws_bytes=ws - 1) == ds.EWORKSPACE
    assert call(R=0) == ds.OK


def test_append_refusals(ds):
    def call(rows=4, Hkv=2, D=64, dt=ds.BF16, page=16, n=10, k=P(), row=256, cache=P(), st=1024):
        return ds.lib().dspark_cache_append(rows, Hkv, D, dt, page, n, k, P(), row, 256, P(), None,
                                            cache, P(), 2048, st, 64, None, None)

    for bad in (dict(rows=-1), dict(Hkv=0), dict(D=60), dict(D=2048), dict(dt=3), dict(page=24),
                dict(n=0), dict(n=1 << 27), dict(k=None), dict(k=P(0x1008)), dict(row=250),
                dict(row=-256), dict(cache=P(0x1004)), dict(st=1023)):
        assert call(**bad) == ds.EINVAL, bad
    assert call(rows=0) == ds.OK
    assert call(rows=1 << 30, Hkv=1 << 20) == ds.EINVAL  # no grid holds it


def test_attention_refusals(ds):
    ws = ds.tree_attention_workspace_bytes(4, 20, 8, 2, 64, ds.BF16)

    def call(R=4, rows=20, Hq=8, Hkv=2, D=64, dt=ds.BF16, page=16, W=10, n=40, q=P(), q_row=512,
             k=P(), st=1024, tok=64, table=P(), scale=0.125, o=P(0x100000), wsp=P(), ws_bytes=ws):
        return ds.lib().dspark_tree_attention(R, rows, Hq, Hkv, D, dt, page, W, n, q, q_row, k, P(),
                                              2048, st, tok, table, P(), P(), None, scale, o, None,
                                              None, wsp, ws_bytes, None)

    for bad in (dict(R=(1 << 20) + 1), dict(Hq=9), dict(Hkv=0), dict(D=80), dict(D=256), dict(dt=2), dict(page=10),
                dict(W=0), dict(W=(1 << 26) + 1), dict(n=0), dict(q=None), dict(q=P(0x1002)), dict(q_row=511),
                dict(k=None), dict(st=1), dict(tok=-64), dict(table=None), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(o=None), dict(wsp=None), dict(wsp=P(0x1008)), dict(rows=-1),
                dict(o=P()), dict(o=P(0x1000 + 19 * 1024)),  # over q
                dict(rows=1 << 28, Hq=8)):
        assert call(**bad) == ds.EINVAL, bad
    assert call(ws_bytes=ws - 1) == ds.EWORKSPACE
    assert call(R=0) == ds.OK and call(rows=0) == ds.OK


def test_logits_refusals(ds):
    def call(R=4, gamma=4, V=1024, dt=ds.BF16, lg=P(), stride=1024, rows=20, off=P(), ell=P(),
             hist=None, hl=None, nb=0, ids=None, mask=None, n_mask=0, words=0, out=P(0x9000)):
        return ds.lib().dspark_target_logits(R, gamma, V, dt, lg, stride, rows, off, ell, P(), hist,
                                             16, hl, None, None, None, None, ids, None, nb, mask,
                                             n_mask, words, None, out, None, None)

    for bad in (dict(R=-1), dict(R=65536), dict(gamma=0), dict(gamma=65), dict(V=1020),
                dict(dt=2), dict(lg=None), dict(lg=P(0x1004)), dict(stride=1016),
                dict(stride=1025), dict(rows=-1), dict(ell=None), dict(hist=P()), dict(nb=-1),
                dict(nb=2), dict(mask=P(), n_mask=0, words=32), dict(mask=P(), n_mask=1, words=31),
                dict(out=None), dict(out=P()),  # in place with packed rows
                dict(off=None, out=P(0x1800)), dict(lg=P(0x10000))):  # over each other
        assert call(**bad) == ds.EINVAL, bad
    assert call(off=None, out=P(), stride=1032) == ds.EINVAL  # in place, rows spaced
    assert call(R=0) == ds.OK


def test_commit_refusals(ds):
    ws = ds.cache_commit_workspace_bytes(4, 10, True)

    def call(R=4, gamma=4, page=16, W=10, n_acc=P(), path=P(), done=None, n_free=P(), free=P(),
             layers=1, Hkv=2, D=64, dt=ds.BF16, n=40, k=P(), st=1024, ws_bytes=ws, free_len=8,
             ctx=P(0x2000), out=P(0x2000), held=P(0x3000)):
        return ds.lib().dspark_cache_commit(R, gamma, page, W, free_len, n_acc, path, done, ctx,
                                            out, held, P(), free, n_free, layers, Hkv, D, dt, n, k,
                                            P(), 0, 2048, st, 64, None, P(), ws_bytes, None)

    for bad in (dict(R=-1), dict(R=(1 << 20) + 1), dict(gamma=0), dict(gamma=65), dict(page=20), dict(W=0),
                dict(n_acc=None), dict(done=P(), n_free=None), dict(done=P(), free=None),
                dict(layers=-1), dict(Hkv=0), dict(D=12), dict(dt=5), dict(n=0), dict(k=None),
                dict(k=P(0x1001)), dict(st=1022), dict(free_len=-1),
                dict(out=P(0x2004)), dict(out=P(0x1000)), dict(out=P(0x3008))):
        assert call(**bad) == ds.EINVAL, bad
    assert call(ws_bytes=ws - 1) == ds.EWORKSPACE
    assert call(R=0) == ds.OK


def test_binding_wants_device_tensors(ds):
    import torch
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ds.cache_plan(i, i, i, i.view(4, 1), i, i[:1], 16, rows=20)
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        ds.tree_attention(q, q, q, i.view(4, 1), i, i)
    with pytest.raises(ValueError):
        ds.cache_append(q, q, q, q, i)
    with pytest.raises(ValueError):
        ds.target_logits(torch.zeros(4, 2, 8), i, i.view(4, 1))
    with pytest.raises(ValueError):
        ds.cache_commit(i, i, i, i.view(4, 1), i, i[:1], 16)
    with pytest.raises(TypeError):
        ds.cache_plan([0], i, i, i, i, i, 16, rows=20)
