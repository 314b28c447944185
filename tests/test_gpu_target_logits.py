"""target_logits against its definition in 64 bits.  Bound of the error: a handful of float
steps on the terms added up (8 * 2^-24 of their sizes), and the stored type's rounding (at
most half a step: 2^-8 of a bf16 value, 2^-24 of a float)."""
import numpy as np
import pytest
import torch

from tests import target_ref as ref

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def T(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda:0")


def check(seed, R, gamma, V, dtype, n_hist=50, nb=6, n_mask=5, packed=True, in_place=False,
          use=("hist", "prompt", "rep", "pres", "freq"), every_row=False, edit=None, pad=0):
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(seed)
    ell = g.integers(0, gamma + 1, R)
    off = np.concatenate([[0], np.cumsum(ell + 1)])
    rows = int(off[-1]) + 2 if packed else R * (gamma + 1)
    lg = torch.from_numpy((4 * g.standard_normal((rows, V + pad))).astype(np.float32)).to(dtype)
    x = (V * g.random((R, gamma)) ** 3).astype(int)
    hist = (V * g.random((R, n_hist)) ** 3).astype(int)
    hl = g.integers(0, n_hist + 1, R)
    pl = (hl * g.random(R)).astype(int)
    rep, pres, freq = 0.5 + g.random(R), g.standard_normal(R), g.standard_normal(R)
    ids = g.integers(-1, V, (R, nb))
    if nb > 2:
        ids[:, 2] = ids[:, 0]  # twice the same id: the later counts
    bias = 3 * g.standard_normal((R, nb))
    words = ref.cdiv(V, 32) + 1
    if every_row:
        n_mask = R * (gamma + 1)
    mask = g.integers(0, 2 ** 32, (n_mask, words), dtype=np.uint64).astype(np.uint32)
    if n_mask:
        mask[0] = 0           # allows nothing
        mask[-1] = 0xFFFFFFFF
    idx = g.integers(-1, max(n_mask, 1), (R, gamma + 1))
    f32 = np.float32
    a = dict(row_off=T(off) if packed else None)
    if "hist" in use:
        a.update(hist=T(hist), hist_len=T(hl))
    if "prompt" in use:
        a.update(prompt_len=T(pl))
    for k, val in (("rep", rep), ("pres", pres), ("freq", freq)):
        if k in use:
            a[k] = T(val.astype(f32), F32)
    if nb:
        a.update(bias_id=T(ids), bias=T(bias.astype(f32), F32))
    if n_mask:
        a["mask"] = torch.from_numpy(mask.view(np.int32)).to("cuda:0")
        if not every_row:
            a["mask_idx"] = T(idx)
    if edit:
        edit(lg)
    st = T([0])
    d = lg.to("cuda:0")[:, :V] if pad else lg.to("cuda:0")
    if not packed:
        d = d.view(R, gamma + 1, V)
    out = d if in_place else torch.full((R, gamma + 1, V), 55.0, dtype=dtype, device="cuda:0")
    got = ds.target_logits(d, T(ell), T(x), out=out, status=st, **a)
    assert got is out and int(st) == 0
    got = out.double().cpu().numpy()
    src = lg.double().numpy()[:, :V]
    for q in range(R):
        L = ell[q]
        r0 = off[q] if packed else q * (gamma + 1)
        ms = []
        for j in range(L + 1):
            i = (q * (gamma + 1) + j if every_row else idx[q, j]) if n_mask else -1
            ms.append(None if i < 0 else (mask[i][np.arange(V) // 32] >> (np.arange(V) % 32)) & 1 == 1)
        w, size = ref.logits(
            src[r0:r0 + L + 1], x[q], hist[q, :hl[q]] if "hist" in use else [],
            pl[q] if "prompt" in use else 0,
            float(f32(rep[q])) if "rep" in use else 1.0, float(f32(pres[q])) if "pres" in use else 0.0,
            float(f32(freq[q])) if "freq" in use else 0.0,
            [(int(i), float(f32(b))) for i, b in zip(ids[q], bias[q]) if i >= 0], ms)
        u = 2.0 ** -8 if dtype is BF else 2.0 ** -24
        with np.errstate(invalid="ignore"):
            tol = np.where(np.isfinite(w), u * np.abs(w) + (1 + u) * 8 * 2.0 ** -24 * size, 0)
            same = (w == got[q, :L + 1]) | (np.isnan(w) & np.isnan(got[q, :L + 1]))
            assert (same | (np.abs(got[q, :L + 1] - w) <= tol)).all(), q
        rest = src[(r0 + L + 1):(r0 + gamma + 1)] if in_place else 55.0
        assert (got[q, L + 1:] == rest).all()  # rows that are not checked stay as they were


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,gamma,V", [(1, 1, 8), (4, 4, 1024), (3, 8, 4096), (5, 3, 4104),
                                       (2, 64, 520), (40, 2, 12296), (2, 5, 32000)])
def test_sizes(R, gamma, V, dtype):
    check(V + R, R, gamma, V, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_forms(dtype):
    check(1, 5, 4, 1000, dtype, packed=False)
    check(2, 5, 4, 5000, dtype, packed=False, in_place=True)
    check(3, 5, 4, 1000, dtype, every_row=True)
    check(4, 5, 4, 1000, dtype, pad=24)
    check(5, 3, 4, 9000, dtype, n_hist=3000)
    check(6, 3, 4, 72, dtype, n_hist=700, nb=300)   # the same ids over and over


@pytest.mark.parametrize("drop", ["hist", "prompt", "rep", "pres", "freq", "bias", "mask", "all"])
def test_parts_left_out(drop):
    use = tuple(k for k in ("hist", "prompt", "rep", "pres", "freq") if drop not in (k, "all"))
    check(7, 4, 3, 800, F32, use=use, nb=0 if drop in ("bias", "all") else 6,
          n_mask=0 if drop in ("mask", "all") else 5)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_many_requests(dtype):
    """Enough slices that a workgroup walks all rows of its request."""
    check(12, 130, 3, 8200, dtype)
    check(13, 600, 2, 264, dtype, packed=False, in_place=True)


def test_headline_vocabulary():
    check(8, 3, 8, 151936, BF, n_hist=2000, nb=20)


def test_beyond_32_bits():
    """5 GB of logits: the last requests as they come out alone."""
    import draft_sampling_scheduling_amd as ds
    R, gamma, V = 520, 16, 151936
    gen = torch.Generator(device="cuda").manual_seed(1)
    lg = torch.randn(R, gamma + 1, V, device="cuda", generator=gen)
    assert lg.numel() * 4 > 2 ** 32
    x = torch.randint(0, V, (R, gamma), device="cuda", dtype=I32, generator=gen)
    ell = torch.full((R,), gamma, device="cuda", dtype=I32)
    one = torch.ones(R, device="cuda")
    out = ds.target_logits(lg, ell, x, pres=one, freq=one)
    for s in (slice(0, 1), slice(R - 2, R)):
        alone = ds.target_logits(lg[s].contiguous(), ell[s], x[s], pres=one[s], freq=one[s])
        assert torch.equal(out[s], alone)
    q = R - 1
    assert float(out[q, gamma, x[q, 0].long()]) < float(lg[q, gamma, x[q, 0].long()]) - 1.5
    ds.target_logits(lg, ell, x, pres=one, freq=one, out=lg)
    assert torch.equal(out, lg)


def test_infinities_and_nan():
    def edit(lg):
        f = lg.view(-1)
        f[::7], f[1::11], f[2::13] = float("inf"), float("-inf"), float("nan")

    def lowest(lg):
        lg.view(-1)[::3] = -torch.finfo(lg.dtype).max

    for dtype in (BF, F32):
        check(9, 4, 4, 1024, dtype, edit=edit)
        check(10, 4, 4, 1024, dtype, edit=lowest, use=("hist", "pres", "freq"))


def test_faults():
    import draft_sampling_scheduling_amd as ds
    R, gamma, V = 3, 2, 64
    lg = torch.randn(9, V, device="cuda:0")
    ell, x = T([2, 2, 2]), T([[1, 2], [3, 4], [5, 6]])
    off = T([0, 3, 6, 9])
    hist, hl = T([[1, 2, 3]] * 3), T([3, 3, 3])

    def go(**k):
        st = T([0])
        a = dict(row_off=off, hist=hist, hist_len=hl, pres=T([1.0] * 3, F32))
        e, xx = k.pop("ell", ell), k.pop("x", x)
        a.update(k)
        out = torch.zeros(R, gamma + 1, V, device="cuda:0")
        ds.target_logits(lg, e, xx, out=out, status=st, **a)
        return int(st), out

    st, good = go()
    assert st == 0
    st, o = go(ell=T([2, 7, -1]))
    assert st == 4 and torch.equal(o[:2], good[:2]) and torch.equal(o[2, :1], good[2, :1])
    assert torch.all(o[2, 1:] == 0)
    st, o = go(row_off=T([0, 3, -5, 9]))
    assert st == 4 and torch.equal(o[0], good[0]) and torch.all(o[1:] == 0)
    # requests that a step gave fewer rows than they have tokens, or none, take no one else's
    st, o = go(row_off=T([0, 3, 8, 9]))
    assert st == 4 and torch.equal(o[0], good[0]) and torch.all(o[2, 1:] == 0)
    st, o = go(row_off=T([0, 0, 2, 11]))
    assert st == 4 and torch.all(o[0] == 0) and torch.all(o[1, 2:] == 0)
    st, want = go(row_off=T([0, 3, 5, 8]), ell=T([2, 1, 2]))
    assert st == 0 and torch.all(want[1, 2:] == 0)
    st, o = go(row_off=T([0, 3, 5, 8]))
    assert st == 4 and torch.equal(o, want)
    for k in (dict(hist_len=T([4, 3, 3])), dict(prompt_len=T([0, 4, 0])), dict(hist_len=T([3, -1, 3]))):
        st, o = go(**k)
        assert st == 4 and torch.equal(o[2], good[2])
    for k in (dict(x=T([[1, 64], [3, 4], [5, 6]])), dict(hist=T([[1, -2, 3]] + [[1, 2, 3]] * 2)),
              dict(bias_id=T([[-2], [-1], [-1]]), bias=T([[1.0]] * 3, F32)),
              dict(bias_id=T([[64], [-1], [-1]]), bias=T([[1.0]] * 3, F32))):
        st, o = go(**k)
        assert st == 1 and torch.equal(o[1:], good[1:])
    for k in (dict(rep=T([0.0, 1, 1], F32)), dict(rep=T([1e-39, 1, 1], F32)), dict(rep=T([-1.0, 1, 1], F32)),
              dict(rep=T([float("inf"), 1, 1], F32)), dict(freq=T([float("nan"), 0, 0], F32)),
              dict(mask=T([[-1, -1]]), mask_idx=T([[1, 0, 0]] + [[0, 0, -1]] * 2)),
              dict(mask=T([[-1, -1]]), mask_idx=T([[-2, 0, 0]] + [[0, 0, -1]] * 2))):
        st, o = go(**k)
        assert st == 32 and torch.equal(o, good), k
    st, o = go(pres=T([float("inf"), 1, 1], F32))
    assert st == 32 and torch.equal(o[1:], good[1:])


def test_refusals():
    import draft_sampling_scheduling_amd as ds
    lg, ell, x = torch.randn(2, 3, 64, device="cuda:0"), T([1, 1]), T([[1, 2], [3, 4]])
    ds.target_logits(lg, ell, x)
    h = T([[1], [2]])
    for k in (dict(hist=h), dict(bias=torch.zeros(2, 1, device="cuda:0")),
              dict(mask=T([[1, 1]])), dict(row_off=T([0, 1])), dict(hist=h, hist_len=T([1]))):
        with pytest.raises(ValueError):
            ds.target_logits(lg, ell, x, **k)
    with pytest.raises(ValueError):
        ds.target_logits(lg[:, :2].contiguous(), ell, x)
    with pytest.raises(TypeError):
        ds.target_logits(lg.half(), ell, x)
    with pytest.raises(TypeError):
        ds.target_logits(lg, ell.long(), x)
    with pytest.raises(ds.DsparkError):
        ds.target_logits(lg, ell, x, mask=T([[1]]), mask_idx=T([[0] * 3] * 2))  # too few words
    with pytest.raises(ds.DsparkError):
        ds.target_logits(lg.view(6, 64), ell, x, row_off=T([0, 2, 4]), out=lg)  # packed, in place
    off = T([0, 2, 4])
    for bad in (lg.view(6, 64)[:1].expand(4, 64), lg.view(6, 64)[:4, :32].contiguous().view(-1)[:72]
                .as_strided((4, 64), (2, 1))):  # rows over each other
        with pytest.raises(ds.DsparkError):
            ds.target_logits(bad, ell, x, row_off=off)
    one = ds.target_logits(lg.view(6, 64)[:1], T([0]), x[:1], row_off=T([0, 1]))
    assert torch.equal(one[0, 0], lg[0, 0])
    for k in (dict(hist=[[1]], hist_len=ell), dict(mask=3), dict(bias=[0.0], bias_id=h)):
        with pytest.raises(TypeError):
            ds.target_logits(lg, ell, x, **k)
