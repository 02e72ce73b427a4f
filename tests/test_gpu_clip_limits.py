"""Clipping where the quotient max_norm / (norm + eps) has a limit case."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, math.inf])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_zero_gradients_stay_zero(dtype, max_norm, eps):
    for n in (1, 5, 40001):
        g = torch.zeros(n, dtype=dtype, device="cuda")
        out = torch.full_like(g, 3.0)
        assert float(L.lse_grad_clip(L.GradList([g], [out]), max_norm, eps)) == 0.0
        assert (out == 0).all()
        assert float(L.lse_grad_clip([g], max_norm, eps)) == 0.0
        assert (g == 0).all()


def test_infinite_limits():
    for max_norm, finite, infinite in ((1.0, 0.0, math.nan), (math.inf, math.nan, math.nan)):
        g = torch.ones(100, device="cuda")
        g[7] = math.inf
        assert float(L.lse_grad_clip([g], max_norm)) == math.inf
        got = g.tolist()
        assert math.isnan(got[7]) and all(v == finite or (math.isnan(v) and math.isnan(finite)) for v in got[:7] + got[8:])
    g = torch.full((100,), 2.0, device="cuda")
    assert float(L.lse_grad_clip([g], math.inf)) == 20.0 and (g == 2.0).all()
