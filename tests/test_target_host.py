"""Host-side checks of the calls around the target's pass (no GPU needed)."""
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


def P(x=0x1000):
    return C.c_void_p(x)  # never dereferenced: these calls return before any launch


def test_verify_rows_refusals(ds):
    ws = ds.verify_workspace_bytes(4, 4, 1024, 16)

    def call(row_off=P(), x0=P(), x_next=P(), ws_bytes=ws, ell=P(), R=4):
        return ds.lib().dspark_verify_rows(R, 4, 1024, 16, ds.BF16, P(), P(), P(), P(), ds.BF16, P(), P(),
                                           P(), ell, row_off, x0, 0, 0, P(), P(), P(), x_next, None, P(),
                                           ws_bytes, None)

    assert call(x0=None) == ds.EINVAL  # nothing to keep in x_next
    assert call(ell=None) == ds.EINVAL
    assert call(R=0) == ds.OK
    for k in (dict(), dict(x0=None, x_next=None), dict(row_off=None, x0=None)):
        assert call(ws_bytes=ws - 1, **k) == ds.EWORKSPACE  # past the checks of arguments


def test_logits_tree_refusals(ds):
    def call(lg=P(), out=P(0x9000), off=P(), ell=P(), R=4):
        return ds.lib().dspark_target_logits_tree(R, 4, 1024, ds.BF16, lg, 1024, 20, off, ell, P(), P(),
                                                  None, 0, None, None, None, None, None, None, None, 0, None,
                                                  0, 0, None, out, None, None)

    for bad in (dict(lg=None), dict(out=None), dict(ell=None), dict(R=65536), dict(out=P()),
                dict(lg=P(0x10000))):
        assert call(**bad) == ds.EINVAL, bad
    assert call(R=0) == ds.OK


def test_logits_vocabulary_limit(ds):
    def call(V, logits=P(), rows=20):
        return ds.lib().dspark_target_logits(0, 4, V, ds.BF16, logits, V, rows, P(), P(), P(), None, 0, None,
                                             None, None, None, None, None, None, 0, None, 0, 0, None, P(0x9000),
                                             None, None)

    assert call(1 << 30) == ds.OK  # (no requests: returns before any launch)
    assert call((1 << 30) + 8) == ds.EINVAL
    assert call((1 << 31) - 8) == ds.EINVAL  # a slice's end would pass 31 bits


def test_commit_lengths_over_other_arguments(ds):
    """ctx_out may be ctx itself; over anything else that the call reads or writes it is refused."""
    ws = ds.cache_commit_workspace_bytes(4, 10, True)

    def call(out, ctx=0x2000, done=0x4000, ws_bytes=ws):
        return ds.lib().dspark_cache_commit(4, 4, 16, 10, 8, P(0x1000), P(0x5000), P(done) if done else None,
                                            P(ctx), P(out), P(0x3000), P(0x6000), P(0x7000), P(0x8000), 1, 2,
                                            64, ds.BF16, 40, P(0x10000), P(0x20000), 0, 2048, 1024, 64, None,
                                            P(0x9000), ws_bytes, None)

    assert call(0x2000, ws_bytes=ws - 1) == ds.EWORKSPACE          # ctx: past the checks
    for base, ints in ((0x1000, 4), (0x3000, 4), (0x4000, 4), (0x5000, 16), (0x6000, 40), (0x7000, 8),
                       (0x8000, 1)):
        for at in (base - 12, base, base + 4 * ints - 4):
            assert call(at) == ds.EINVAL, (hex(base), hex(at))
    assert call(0x2004) == ds.EINVAL
    # the list is not touched without `done`
    assert call(0x7000, ctx=0x7000, done=0, ws_bytes=ws - 1) == ds.EWORKSPACE


def test_attention_rows_limit(ds):
    """The end of the last row tile is counted in 31 bits."""
    b = ds.tree_attention_workspace_bytes
    assert b(1, (1 << 28) - 128, 8, 1, 64, ds.BF16) > 0
    for rows, Hq in (((1 << 28) - 127, 8), ((1 << 28) - 1, 8), ((1 << 31) - 1, 1)):
        assert b(1, rows, Hq, 1, 64, ds.BF16) == 0, (rows, Hq)


def test_attention_scale_limit(ds):
    """Scores are taken in powers of two: scale * log2(e) has to be a float."""
    def call(scale):
        return ds.lib().dspark_tree_attention(4, 20, 8, 2, 64, ds.BF16, 16, 10, 40, P(), 512, P(), P(), 2048,
                                              1024, 64, P(), P(), P(), None, scale, P(0x100000), None, None, P(),
                                              0, None)

    for scale in (0.125, 1e-40, 2.3e38):
        assert call(scale) == ds.EWORKSPACE, scale  # past the checks of arguments
    for scale in (2.4e38, 3.4e38, float("inf"), float("nan"), 0.0, -0.125):
        assert call(scale) == ds.EINVAL, scale


def test_append_rows_inside_the_caches(ds):
    """Rows that lie in a cache are refused, whichever of the two."""
    rows, Hkv, D, page, n = 4, 2, 64, 16, 10
    size = 2 * n * Hkv * page * D       # bytes of a cache: 40960
    row = 2 * Hkv * D                   # of a row: 256

    def call(k, v=0x900000, kc=0x100000, vc=0x200000):
        return ds.lib().dspark_cache_append(rows, Hkv, D, ds.BF16, page, n, P(k), P(v), 128, 128, P(0x1000),
                                            None, P(kc), P(vc), Hkv * page * D, page * D, D, None, None)

    for base in (0x100000, 0x200000):
        for at in (base - rows * row + 16, base, base + 4096, base + size - 16):
            assert call(at) == ds.EINVAL, hex(at)
            assert call(0x900000, v=at) == ds.EINVAL, hex(at)
