"""lse_sample with top_p and min_p where the whole is summed in 32 bits and what min_p leaves ends
just behind the cut of top_p: the cut is that of exact arithmetic.

The row's heavy token passes through additions each of which rounds up by nearly half a step, so
the 32-bit whole is too large, and a share of it lies beyond what min_p leaves.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
from test_gpu_sample_heavy import DT, OPEN, _need_gpu, numbers  # noqa: E402, F401


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_cut_next_to_the_floor(dtype):
    N, E, lights = 8192, 4 if dtype == "f32" else 8, 12
    r = torch.full((N,), -float("inf"), dtype=torch.float64)
    r[0] = 0.0
    for c in (1, 2, 32 * E, 64 * E) + (() if dtype == "f32" else (4,)):  # one for each addition of the lane's
        r[c] = -16.5  # 6.8e-8: 0.57 of the step of a sum in [1, 2); below min_p
    r[N // 2:N // 2 + lights] = -15.9375  # 1.2e-7
    row = r.to(DT[dtype])
    x64 = row.double()
    order = torch.sort(x64, descending=True, stable=True).indices
    w = torch.exp(x64)
    run, total = torch.cumsum(w[order], 0), float(w.sum())
    p = numbers(float(run[lights]) / total, 24)
    need = p.double() * total
    reach = torch.searchsorted(run, need).clamp(max=lights)  # min_p leaves the heavy token and the lights
    below = torch.where(reach > 0, run[(reach - 1).clamp(min=0)], torch.zeros_like(need))
    far = torch.minimum((run[reach] - need).abs(), (need - below).abs()) > OPEN * total
    x = row.expand(p.numel(), N).contiguous().cuda()
    got = L.lse_sample(x, torch.full((p.numel(),), 1.0 - 2.0 ** -24, device="cuda"), top_p=p.cuda(), min_p=1e-7)
    want = torch.stack([order[:int(k) + 1].max() for k in reach])
    assert far.sum() > 15 and len(set(want.tolist())) > 3
    assert torch.equal(got.token.cpu()[far], want[far]), (got.token.cpu() - want)[far]
