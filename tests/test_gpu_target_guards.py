"""Plans repeated under every fault, and workspaces of exactly the stated size inside memory that
must not change."""
import numpy as np
import pytest
import torch

from tests import target_ref as ref
from tests.test_gpu_target_cache import T, case

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


@pytest.mark.parametrize("rows", [12 * 7, 3000, 20000])
@pytest.mark.parametrize("n_free", [-3, 0, 2, 60, 1000])
def test_a_plan_repeated_under_faults(n_free, rows):
    """Shortage, a clamped count of free pages, unknown pages and parents, refused requests: the
    second plan of the step changes nothing, and says the same."""
    import draft_sampling_scheduling_amd as ds
    c = case(9, 12, 6, 16, 300, 60, tree=True)
    c["ctx"][0], c["lens"][1], c["held"][2] = -1, -5, len(c["table"][0]) + 1
    c["lens"][5], c["parent"][5][3] = 6, 3
    c["ctx"][7], c["lens"][7], c["held"][7] = 40, 3, 3
    c["table"][7][:3] = [5, 6, -1]
    d = {k: T(c[k]) for k in ("ctx", "lens", "held", "table", "free", "parent")}
    nf, count = T([n_free]), min(max(n_free, 0), len(c["free"]))
    table = [list(r) for r in c["table"]]
    want, bits = ref.plan(c["lens"], c["ctx"], c["held"], table, c["free"], count, 16, rows, 1, c["parent"])
    n = want["row_off"][-1]
    for turn in range(3):
        st = T([0])
        out = {k: torch.full((rows,), -9, dtype=I32, device="cuda:0") for k in ("req", "position", "slot")}
        out.update(row_off=T([-9] * 13), anc=torch.full((rows,), -9, dtype=torch.int64, device="cuda:0"))
        ds.cache_plan(d["lens"], d["ctx"], d["held"], d["table"], d["free"], nf, 16, rows=rows, extra=1,
                      parent=d["parent"], out=out, status=st)
        assert out["row_off"].tolist() == want["row_off"], turn
        for k in ("req", "position", "slot", "anc"):
            assert out[k].tolist() == want[k] + [-9] * (rows - n), (turn, k)
        assert d["table"].tolist() == table and d["held"].tolist() == want["held"], turn
        assert nf.tolist() == [want["n_free"]], turn
        # (an impossible count of free pages is one no longer)
        assert int(st) == bits | (8 if count != n_free and turn == 0 else 0), turn


GUARD = 4096


def guarded(nbytes, fill):
    """A workspace of nbytes inside a patterned allocation; the check that the rest is whole."""
    big = (torch.arange(nbytes + 2 * GUARD, device="cuda:0") % 251).to(torch.uint8)
    whole = big.clone()
    ws = big[GUARD:GUARD + nbytes]
    ws.fill_(fill)

    def check():
        return torch.equal(big[:GUARD], whole[:GUARD]) and torch.equal(big[-GUARD:], whole[-GUARD:])

    return ws, check


@pytest.mark.parametrize("fill", [0, 127, 255])
def test_workspaces_of_the_stated_size(fill):
    import draft_sampling_scheduling_amd as ds
    # plan: two launches, for its rows, its requests and its trees
    for R, rows, width in ((40, 20000, 0), (1100, 3000, 0), (200, 1500, 60)):
        c = case(R, R, 6, 16, 200, 3 * R, tree=width > 0, width=width)
        outs = []
        for own in (False, True):
            d = {k: T(c[k]) for k in ("ctx", "lens", "held", "table", "free")}
            nf, check, ws = T([c["n_free"]]), lambda: True, None
            nbytes = ds.cache_plan_workspace_bytes(R, rows, width)
            assert nbytes > 0
            if own:
                ws, check = guarded(nbytes, fill)
            p = ds.cache_plan(d["lens"], d["ctx"], d["held"], d["table"], d["free"], nf, 16, rows=rows,
                              extra=1, parent=T(c["parent"]) if width else None, ws=ws)
            n = int(p["row_off"][-1])
            assert check() and 0 < n <= min(rows, sum(c["lens"]) + R)  # (1100 ask for more than 3000)
            outs.append([p["row_off"], p["slot"][:n], p["req"][:n], d["held"], d["table"], nf])
        assert all(torch.equal(a, b) for a, b in zip(*outs)), (R, rows, width)
    # commit: in place with a path; many pages back
    g = np.random.default_rng(5)
    for R, gamma, W, in_place, path in ((30, 6, 4, True, True), (1500, 3, 2, False, True),
                                        (300, 3, 40, False, False)):
        P, page = R * W, 16
        ctx = g.integers(0, page * (W - 1), R)
        n_acc = g.integers(-1, gamma + 1, R)
        ways = [sorted((g.permutation(gamma) + 1)[:max(k, 0)]) + [0] * (gamma - max(k, 0)) for k in n_acc]
        done = (g.random(R) < 0.3).astype(int)
        order = g.permutation(P).reshape(R, W)
        kv = torch.randn(2, P, 2, page, 64, device="cuda:0")
        outs = []
        for own in (False, True):
            nbytes = ds.cache_commit_workspace_bytes(R, W, in_place)
            assert nbytes > 0
            check, ws = lambda: True, None
            if own:
                ws, check = guarded(nbytes, fill)
            cx, held, free, nf = T(ctx.tolist()), T([W] * R), T([-1] * P), T([0])
            k, v = kv[0].clone(), kv[1].clone()
            a = dict(path=T([[int(i) for i in w] for w in ways]), k_cache=k, v_cache=v) if path else {}
            o = ds.cache_commit(T(n_acc.tolist()), cx, held, T(order.tolist()), free, nf, page,
                                done=T(done.tolist()), out=cx if in_place else None, ws=ws, **a)
            assert check() and int(nf) == W * done.sum()
            outs.append([o, held, free, nf, k, v])
        assert all(torch.equal(a, b) for a, b in zip(*outs)), (R, W)
    # attention: one variant of each kind of tile
    for R, rows, Hq, Hkv, D, dtype in ((5, 15, 4, 2, 64, torch.float32), (5, 15, 4, 2, 128, BF),
                                       (4, 60, 8, 2, 128, BF), (4, 48, 8, 2, 64, BF), (3, 90, 8, 1, 64, BF)):
        n = rows // R
        ctx = [700 + 31 * q for q in range(R)]
        c = ref.Cache(R, ctx, [n] * R, Hkv, D, 16, dtype)
        q = torch.randn(rows, Hq, D, device="cuda:0").to(dtype)
        a = (q, c.dev(c.k), c.dev(c.v), T(c.table.tolist()), T(ctx), T([n * i for i in range(R + 1)]))
        nbytes = ds.tree_attention_workspace_bytes(R, rows, Hq, Hkv, D, ds.BF16 if dtype is BF else ds.F32)
        ws, check = guarded(nbytes, fill)
        want, got = ds.tree_attention(*a), ds.tree_attention(*a, ws=ws)
        assert check() and torch.equal(want["o"], got["o"]) and torch.equal(want["lse"], got["lse"])
