"""A matrix made by Weights4.from_values is its own: a later write to the given scales does not reach it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
from test_gpu_linear4 import _need_gpu, random_weights  # noqa: E402, F401


@pytest.mark.parametrize("strided", [False, True])
def test_scales_are_copied(strided):
    q, s, _ = random_weights(20, 256, 64, "bf16", 1)
    s = torch.cat((s, s), 1)[:, :4] if strided else s.clone()
    w = L.Weights4.from_values(q, s, 64)
    before = L.lse_dequantize4(w)
    s.fill_(7.0)
    q.zero_()
    assert torch.equal(L.lse_dequantize4(w), before) and w.scales.is_contiguous()
