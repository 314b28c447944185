"""Calls of the target's side at the ends of what their documentation allows."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
I32, F32, BF = torch.int32, torch.float32, torch.bfloat16


def T(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda:0")


def test_logits_of_a_step_without_rows():
    """Nobody was served: every request is reported, nothing is written."""
    import draft_sampling_scheduling_amd as ds
    for dtype in (F32, BF):
        out, st = torch.full((3, 3, 64), 5.0, dtype=dtype, device="cuda:0"), T([0])
        got = ds.target_logits(torch.empty(0, 64, dtype=dtype, device="cuda:0"), T([2, 0, 1]),
                               T([[1, 2]] * 3), row_off=T([0, 0, 0, 0]), out=out, status=st)
        assert got is out and torch.all(out == 5) and int(st) == ds.FAULT_LEN


def test_logits_of_a_history_without_places():
    import draft_sampling_scheduling_amd as ds
    lg, x, ell = torch.randn(2, 3, 64, device="cuda:0"), T([[1, 2], [3, 4]]), T([2, 2])
    hist = torch.empty(2, 0, dtype=I32, device="cuda:0")
    pres = torch.ones(2, device="cuda:0")
    want = ds.target_logits(lg, ell, x, pres=pres)
    for lens, fault in (([0, 0], 0), ([0, 5], ds.FAULT_LEN), ([-1, 0], ds.FAULT_LEN)):
        st = T([0])
        got = ds.target_logits(lg, ell, x, hist=hist, hist_len=T(lens), pres=pres, status=st)
        assert int(st) == fault and torch.equal(got, want), lens


def test_commit_of_a_path_without_places():
    """Not taken for a chain, whose n_acc has no such bound."""
    import draft_sampling_scheduling_amd as ds
    ctx, held, nf = T([0, 0]), T([1, 1]), T([0])
    kc = torch.zeros(2, 1, 8, 64, device="cuda:0")
    with pytest.raises(ValueError):
        ds.cache_commit(T([2, 0]), ctx, held, T([[0], [1]]), T([0]), nf, 8, k_cache=kc, v_cache=kc.clone(),
                        path=torch.empty(2, 0, dtype=I32, device="cuda:0"))


def test_workspaces_that_are_no_tensors():
    import draft_sampling_scheduling_amd as ds
    one, zero, nf = T([1, 1]), T([0, 0]), T([0])
    kc = torch.zeros(2, 1, 8, 64, device="cuda:0")
    for ws in (3, [0] * 4, np.zeros(64, np.uint8)):
        with pytest.raises(TypeError):
            ds.cache_plan(one, zero, one, T([[0], [1]]), T([0]), nf, 8, rows=2, ws=ws)
        with pytest.raises(TypeError):
            ds.cache_commit(zero, zero, one, T([[0], [1]]), T([0]), nf, 8, ws=ws)
        with pytest.raises(TypeError):
            ds.tree_attention(torch.zeros(2, 1, 64, device="cuda:0"), kc, kc, T([[0], [1]]), zero, T([0, 1, 2]),
                              ws=ws)
    # nor are caches
    with pytest.raises(TypeError):
        ds.cache_commit(zero, zero, one, T([[0], [1]]), T([0]), nf, 8, path=T([[1], [1]]), k_cache=[0],
                        v_cache=kc)


def test_append_from_beside_a_cache():
    """Rows right before and right behind the caches in one allocation are taken; rows in them are
    refused, and leave them as they were."""
    import draft_sampling_scheduling_amd as ds
    n, rows = 3 * 2 * 8 * 64, 4
    for dtype in (F32, BF):
        mem = torch.randn(2 * n + 2 * rows * 128, device="cuda:0").to(dtype)
        before, behind = mem[:rows * 128].view(rows, 2, 64), mem[-rows * 128:].view(rows, 2, 64)
        kc, vc = mem[rows * 128:-rows * 128].view(2, 3, 2, 8, 64)
        slot = T([3, 8, 23, 0])
        ds.cache_append(before, behind, kc, vc, slot)
        for i, s in enumerate(slot.tolist()):
            assert torch.equal(kc[s // 8, :, s % 8], before[i]) and torch.equal(vc[s // 8, :, s % 8], behind[i])
        was = mem.clone()
        for at in (8, rows * 128, rows * 128 + n - 64, mem.numel() - rows * 128 - 8):
            inside = mem[at:at + rows * 128].view(rows, 2, 64)
            for a in ((inside, behind), (behind, inside)):
                with pytest.raises(ds.DsparkError):
                    ds.cache_append(*a, kc, vc, slot)
        assert torch.equal(mem, was)
