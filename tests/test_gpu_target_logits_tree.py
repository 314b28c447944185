"""target_logits of drafted trees: a node's row counts the tokens on the way to it, against the
definition in 64 bits (bounds as in test_gpu_target_logits)."""
import numpy as np
import pytest
import torch

from tests import target_ref as ref

pytestmark = pytest.mark.gpu
I32, I64, BF, F32 = torch.int32, torch.int64, torch.bfloat16, torch.float32


def T(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda:0")


def signed(a):
    return a - 2 ** 64 if a >= 2 ** 63 else a


def tree(g, n):
    """Ways (lists of nodes) of a random tree of n nodes."""
    ways = [[]]
    for i in range(1, n):
        ways.append(ways[int(g.integers(0, i))] + [i])
    return ways


def check(seed, R, gamma, V, dtype, packed=True, in_place=False, n_hist=40, junk=False):
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(seed)
    ell = g.integers(0, gamma + 1, R)
    ell[0] = gamma
    off = np.concatenate([[0], np.cumsum(ell + 1)])
    rows = int(off[-1]) + 2 if packed else R * (gamma + 1)
    ways = [tree(g, gamma + 1) for _ in range(R)]
    anc = np.full(rows, -1, np.int64)
    for q in range(R):
        r0 = off[q] if packed else q * (gamma + 1)
        for j in range(ell[q] + 1):
            bits = sum(1 << (i - 1) for i in ways[q][j])
            if junk and gamma < 64:
                bits |= 1 << gamma  # a node past gamma: ignored
            anc[r0 + j] = signed(bits)
    lg = torch.from_numpy((4 * g.standard_normal((rows, V))).astype(np.float32)).to(dtype)
    x = (V * g.random((R, gamma)) ** 3).astype(int)  # the same ids on different branches
    hist = (V * g.random((R, n_hist)) ** 3).astype(int)
    hl = g.integers(0, n_hist + 1, R)
    pl = (hl * g.random(R)).astype(int)
    f32 = np.float32
    rep, pres, freq = (f32(0.5 + g.random(R)), f32(g.standard_normal(R)), f32(g.standard_normal(R)))
    mask = g.integers(0, 2 ** 32, (3, ref.cdiv(V, 32)), dtype=np.uint64).astype(np.uint32)
    idx = g.integers(-1, 3, (R, gamma + 1))
    st = T([0])
    d = lg.to("cuda:0") if packed else lg.to("cuda:0").view(R, gamma + 1, V)
    out = d if in_place else torch.full((R, gamma + 1, V), 55.0, dtype=dtype, device="cuda:0")
    ds.target_logits(d, T(ell), T(x), row_off=T(off) if packed else None, anc=T(anc, I64), hist=T(hist),
                     hist_len=T(hl), prompt_len=T(pl), rep=T(rep, F32), pres=T(pres, F32),
                     freq=T(freq, F32), mask=torch.from_numpy(mask.view(np.int32)).to("cuda:0"),
                     mask_idx=T(idx), out=out, status=st)
    assert int(st) == 0
    got, src = out.double().cpu().numpy(), lg.double().numpy()
    u = 2.0 ** -8 if dtype is BF else 2.0 ** -24
    for q in range(R):
        r0 = off[q] if packed else q * (gamma + 1)
        for j in range(ell[q] + 1):
            k = idx[q, j]
            m = None if k < 0 else (mask[k][np.arange(V) // 32] >> (np.arange(V) % 32)) & 1 == 1
            text = hist[q, :hl[q]].tolist() + [int(x[q, i - 1]) for i in ways[q][j]]
            w, size = ref.logits(src[r0 + j:r0 + j + 1], [], text, pl[q], float(rep[q]), float(pres[q]),
                                 float(freq[q]), [], [m])
            tol = np.where(np.isfinite(w), u * np.abs(w) + (1 + u) * 8 * 2.0 ** -24 * size, 0)
            with np.errstate(invalid="ignore"):
                bad = (w[0] != got[q, j]) & ~(np.abs(got[q, j] - w[0]) <= tol[0])
            assert not bad.any(), (q, j)
        rest = src[(r0 + ell[q] + 1):(r0 + gamma + 1)] if in_place else 55.0
        assert (got[q, ell[q] + 1:] == rest).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,gamma,V", [(1, 1, 8), (4, 4, 1024), (5, 16, 4104), (2, 64, 520), (3, 64, 8200),
                                       (150, 6, 8200)])
def test_trees(R, gamma, V, dtype):
    check(R + gamma, R, gamma, V, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_tree_forms(dtype):
    check(1, 6, 9, 1000, dtype, packed=False)
    check(2, 6, 9, 5000, dtype, packed=False, in_place=True)
    check(3, 300, 5, 264, dtype, packed=False, in_place=True)
    check(4, 6, 9, 1000, dtype, junk=True)


def test_a_chain_as_a_tree():
    """A chain's masks give the chain's result, bit for bit."""
    import draft_sampling_scheduling_amd as ds
    for R, V in ((3, 4096), (200, 8200)):
        gamma = 7
        g = np.random.default_rng(R)
        lg = torch.randn(R, gamma + 1, V, device="cuda:0")
        x, ell = T(g.integers(0, V, (R, gamma))), T(g.integers(0, gamma + 1, R))
        a = dict(rep=torch.full((R,), 1.25, device="cuda:0"), pres=torch.ones(R, device="cuda:0"),
                 freq=torch.ones(R, device="cuda:0"))
        anc = T([(1 << j) - 1 for _ in range(R) for j in range(gamma + 1)], I64)
        outs = [ds.target_logits(lg, ell, x, anc=m, out=torch.zeros_like(lg), **a) for m in (None, anc)]
        assert torch.equal(*outs)


def test_tree_faults_and_plan():
    """A token out of range only where it is on a row's way; a plan's masks; refusals."""
    import draft_sampling_scheduling_amd as ds
    R, gamma, V, page = 2, 3, 64, 8
    x = T([[1, 99, 1], [5, 6, 7]])
    parent = T([[0, 0, 0, 1], [0, 0, 1, 2]])
    held, n_free, st = T([0, 0]), T([4]), T([0])
    p = ds.cache_plan(T([3, 3]), T([0, 0]), held, T([[-1] * 2] * 2), T([0, 1, 2, 3]), n_free, page, rows=8,
                      extra=1, parent=parent, status=st)
    lg = torch.zeros(8, V, device="cuda:0")
    one = torch.ones(2, device="cuda:0")
    out = ds.target_logits(lg, T([3, 3]), x, row_off=p["row_off"], anc=p["anc"], freq=one, status=st)
    assert int(st) == ds.FAULT_TOKEN
    want = torch.zeros(2, 4, V)
    want[0, 1, 1], want[0, 3, 1] = -1, -2      # node 3 is under node 1, and the same id
    want[1, 1, 5] = want[1, 2, 5] = want[1, 2, 6] = -1
    want[1, 3, 5] = want[1, 3, 6] = want[1, 3, 7] = -1
    assert torch.equal(out.cpu(), want)
    st.zero_()
    ds.target_logits(lg, T([1, 3]), x, row_off=p["row_off"], anc=p["anc"], freq=one, status=st)
    assert int(st) == 0  # no row has the unknown token on its way
    with pytest.raises(ValueError):
        ds.target_logits(lg, T([3, 3]), x, row_off=p["row_off"], anc=p["anc"][:7])
    with pytest.raises(TypeError):
        ds.target_logits(lg, T([3, 3]), x, row_off=p["row_off"], anc=p["anc"].int())
