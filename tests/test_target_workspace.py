"""Workspaces of the attention: one sized for a program's largest step serves its smaller ones (no GPU
needed for the sizes)."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def ds():
    import draft_sampling_scheduling_amd as ds
    if not os.path.exists(ds.LIB_PATH):
        from draft_sampling_scheduling_amd import build
        build.build()
    ds.lib()
    return ds


@pytest.mark.parametrize("four", [False, True], ids=["cache16_32", "cache4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (1, 1), (40, 1)])
def test_never_smaller_with_more_rows_a_request(ds, Hq, Hkv, D, four):
    for dt in (ds.BF16, ds.F32):
        for R in (1, 8, 256):
            sizes = [ds.tree_attention_workspace_bytes(R, rows, Hq, Hkv, D, dt, four)
                     for rows in (*range(0, 40 * R, max(R // 8, 1)), 100 * R, 8192 * R)]
            assert sizes[0] > 0 and sizes == sorted(sizes)
        # nor with fewer requests of as many rows
        sizes = [ds.tree_attention_workspace_bytes(R, 300, Hq, Hkv, D, dt, four) for R in range(300, 0, -1)]
        assert sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True], ids=["cache16_32", "cache4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bf", [True, False], ids=["bf16", "f32"])
def test_one_workspace_for_all_steps(ds, bf, D, four):
    from tests import cache4_ref as c4
    from tests import target_ref as ref
    Hq, Hkv, R, dtype = 8, 2, 3, torch.bfloat16 if bf else torch.float32
    T = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda:0")
    nbytes = ds.tree_attention_workspace_bytes(1, 120, Hq, Hkv, D, ds.BF16 if bf else ds.F32, four)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda:0")
    for n in (40, 12, 8, 1):  # rows a request
        ctx = [700, 31, 2000]
        if four:
            c = c4.Cache4(n, ctx, [n] * R, Hkv, D, 16)
            k, v, s = c.dev4()
        else:
            c = ref.Cache(n, ctx, [n] * R, Hkv, D, 16, dtype)
            k, v, s = c.dev(c.k), c.dev(c.v), None
        q = torch.randn(R * n, Hq, D, device="cuda:0").to(dtype)
        a = (q, k, v, T(c.table), T(ctx), T([n * i for i in range(R + 1)]))
        want, got = ds.tree_attention(*a, scales=s), ds.tree_attention(*a, scales=s, ws=ws)
        assert torch.equal(want["o"], got["o"]) and torch.equal(want["lse"], got["lse"])
