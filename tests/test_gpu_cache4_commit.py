"""cache_commit of caches of 4 bits: codes and scales of the accepted path move together, and nothing
else does (bytes, exact)."""
import numpy as np
import pytest
import torch

from tests import target_ref as ref
from tests.test_gpu_target_cache import T, case, commit_ref

pytestmark = pytest.mark.gpu


def run(seed, R, gamma, page, ctx_hi, layers, Hkv, D, layout="phtd", change=None, in_place=False, known=None):
    import draft_sampling_scheduling_amd as ds
    g = np.random.default_rng(seed)
    c = case(seed, R, gamma, page, ctx_hi, 3)
    c["held"] = [ref.cdiv(x + gamma + 1, page) for x in c["ctx"]]
    P = sum(c["held"]) + 3
    order, at = g.permutation(P).tolist(), 0
    for q, h in enumerate(c["held"]):
        c["table"][q][:h] = order[at:at + h]
        at += h
    n_acc = g.integers(-1, gamma + 1, R).tolist()
    path = [sorted((g.permutation(gamma) + 1).tolist()[:max(k, 0)]) + [0] * (gamma - max(k, 0)) for k in n_acc]
    done = (g.random(R) < 0.3).astype(int).tolist()
    c["free"] = order[at:] + [-5] * (P - 3)
    if change:
        change(c, n_acc, path, done)
    shapes = [(layers, P, Hkv, page, D // 2)] * 2 + [(layers, P, Hkv, page, 2, D // 32)]
    host = [torch.from_numpy(g.integers(0, 256, s, dtype=np.uint8)) for s in shapes]
    dev = [x.to("cuda:0") for x in host]
    if layout == "pthd":
        dev = [x.transpose(2, 3).contiguous().transpose(2, 3) for x in dev]
    known = known or P
    view = [x[:, :known] if layers > 1 else x[0, :known] for x in dev]
    st = T([0])
    ctx, held, free, nf = T(c["ctx"]), T(c["held"]), T(c["free"]), T([c["n_free"]])
    out = ds.cache_commit(T(n_acc), ctx, held, T(c["table"]), free, nf, page, path=T(path), done=T(done),
                          k_cache=view[0], v_cache=view[1], scales=view[2], out=ctx if in_place else None, status=st)
    want = commit_ref(c, n_acc, path, done, page, host, len(c["free"]), known)
    assert out.tolist() == want[0] and held.tolist() == want[1]
    assert free.tolist() == want[2] and nf.tolist() == [want[3]] and int(st) == want[4]
    for a, b in zip(dev, host):
        assert torch.equal(a.cpu(), b)
    return want[4]


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("R,gamma,page,ctx_hi,layers,Hkv,D", [
    (1, 1, 8, 0, 1, 1, 64), (4, 4, 16, 200, 2, 2, 64), (64, 8, 16, 256, 4, 4, 128), (9, 64, 8, 100, 3, 1, 128),
    (3, 33, 64, 70, 1, 8, 64), (1500, 2, 16, 30, 1, 1, 64), (5, 6, 16, 40, 3, 40, 128)])
def test_commit(R, gamma, page, ctx_hi, layers, Hkv, D, layout):
    assert run(R, R, gamma, page, ctx_hi, layers, Hkv, D, layout, in_place=R % 2 == 0) == 0


def test_commit_faults():
    def change(c, n_acc, path, done):
        done[:6] = [0] * 6
        n_acc[:6] = [9, 6, 6, 6, 3, 2]
        path[0] = list(range(1, 9))
        path[1] = [1, 2, 2, 5, 6, 8, 0, 0]        # does not ascend
        path[2] = [0, 2, 3, 4, 5, 6, 7, 8]        # node 0 is the anchor
        path[3] = [2, 4, 5, 6, 7, 900, 0, 0]      # past the pages held
        path[4] = [3, 5, 8, 0, 0, 0, 0, 0]
        c["table"][4][c["ctx"][4] // 8] = -1      # an unknown page
        c["held"][5] = 0                          # nothing fits
        path[5] = [1, 2] + [0] * 6

    assert run(3, 12, 8, 8, 90, 2, 2, 64, change=change) & 28 == 28
    assert run(4, 10, 6, 8, 60, 1, 2, 128, known=20) & 8


def test_refusals():
    import draft_sampling_scheduling_amd as ds
    k, s = torch.zeros(2, 5, 2, 16, 32, dtype=torch.uint8, device="cuda:0"), None
    s = torch.zeros(2, 5, 2, 16, 2, 2, dtype=torch.uint8, device="cuda:0")

    def go(k=k, v=k.clone(), s=s, page=16):
        ds.cache_commit(T([1]), T([3]), T([1]), T([[0]]), T([0]), T([0]), page, path=T([[2]]), k_cache=k, v_cache=v, scales=s)

    go()
    go(k[0], k[1], s[0])
    for a in (dict(s=s.int()), dict(s=1), dict(k=k.float(), v=k.float()), dict(s=None), dict(v=k.int())):
        with pytest.raises(TypeError):
            go(**a)
    for a in (dict(s=s[0]), dict(s=s[:, 1:]), dict(k=k[0]), dict(page=32), dict(k=k[..., :8], v=k[..., :8])):
        with pytest.raises(ValueError):
            go(**a)
