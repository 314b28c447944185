"""The repetition penalty alone is one division or one product in float, rounded once: bit for bit
what the host's float arithmetic gives, and its bf16 rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32
TINY, HUGE = float(np.finfo(np.float32).tiny), float(np.finfo(np.float32).max)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_quotients(dtype):
    import draft_sampling_scheduling_amd as ds
    V, gamma = 4096, 1
    reps = np.array([1.3, 0.7, 1.1, 1.0, 2.0, 1.9999999, 3.0, 1e30, 1e-30, TINY, HUGE, 2.0 ** 60, 1.5 * 2.0 ** 60,
                     2.0 ** -60, 1.2e-19], np.float32)
    R = len(reps)
    g = np.random.default_rng(3)
    l = (4 * g.standard_normal((R, gamma + 1, V))).astype(np.float32)
    l[:, 0, ::5] *= np.float32(1e-25)      # quotients at the ends of the range
    l[:, 0, 1::5] = l[:, 0, 1::5] * np.float32(1e37)
    l[:, 0, 2::50] = np.inf
    l[:, 0, 3::50] = -np.inf
    l[:, 0, 4::50] = np.nan
    l[:, 0, 5::50] = 0.0
    l[:, 0, 6::50] = HUGE
    l[:, 0, 7::50] = TINY / 8
    l[:, 0, 8::50] = -TINY / 8
    lg = torch.from_numpy(l).to(dtype)
    hist = torch.arange(V, dtype=I32).expand(R, V).contiguous()
    seen = np.arange(V) % 3 > 0            # the others are not in the history
    hist[:, ~seen] = 1
    full = torch.full((R,), V, dtype=I32, device="cuda:0")
    st = torch.zeros(1, dtype=I32, device="cuda:0")
    out = ds.target_logits(lg.to("cuda:0"), torch.ones(R, dtype=I32, device="cuda:0"),
                           torch.ones(R, gamma, dtype=I32, device="cuda:0"), hist=hist.to("cuda:0"),
                           hist_len=full, prompt_len=full, rep=torch.from_numpy(reps).to("cuda:0"), status=st)
    assert int(st) == 0
    src = lg.float().numpy()
    with np.errstate(all="ignore"):
        r = reps[:, None, None]
        want = np.where(src > 0, src / r, src * r)
    want = torch.from_numpy(np.where(seen, want, src)).to(dtype)
    got = out.cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    assert same.all(), [(q, float(lg[q, j, v]), float(reps[q]), float(got[q, j, v]), float(want[q, j, v]))
                        for q, j, v in (~same).nonzero()[:5].tolist()]
