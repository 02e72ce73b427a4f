"""Of every row that is a distribution: entropy >= 0, log-probabilities <= 0 and
lse >= max, also where a rounding is all that is left of them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
import test_gpu_stats as ts  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,N", [(4000, 1), (4000, 5), (4000, 300), (3000, 3001), (60, 20011), (3, 200003)])
def test_signs(dtype, B, N):
    g = torch.Generator().manual_seed(N)
    top = (2.0 ** (torch.rand(B, generator=g, dtype=torch.float64) * 25) * torch.where(torch.rand(B, generator=g) < 0.5, -1, 1))
    if dtype == "f16":
        top = top.clamp(-60000, 60000)
    top = top.to(ts.DT[dtype])
    at = torch.randint(0, N, (B,), generator=g)
    x = (top.double()[:, None] - 40 - torch.rand((B, N), generator=g, dtype=torch.float64) * 100).to(ts.DT[dtype])
    x = torch.minimum(x, top[:, None])
    x[::2] = -np.inf                              # the others masked
    x[::3] = torch.finfo(ts.DT[dtype]).min
    x[torch.arange(B), at] = top
    for K in (0, 4):
        s = ts.check(x.cuda(), x, at, K)
        assert (s.entropy >= 0).all() and not torch.signbit(s.entropy).any()
        assert (s.logprob <= 0).all() and (s.lse.cpu() >= x.float().amax(1)).all()
        assert K == 0 or (s.top_logprob <= 0).all()
