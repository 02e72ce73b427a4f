"""The gradient takes any object with the attributes of a TokenStats, as it did before
there was an lse_low."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


def test_without_a_second_part():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.randn((9, 301), generator=torch.Generator().manual_seed(1)).cuda()
    g = torch.ones(9, device="cuda")
    s = L.lse_token_stats(x, top_k=2)
    other = SimpleNamespace(lse=s.lse, entropy=s.entropy, top_index=s.top_index)
    d = L.lse_token_stats_backward(x, other, grad_entropy=g)
    assert torch.equal(d, L.lse_token_stats_backward(x, L.TokenStats(*s), grad_entropy=g))
    other.lse_low = s.lse_low
    assert torch.equal(L.lse_token_stats_backward(x, other, grad_entropy=g),
                       L.lse_token_stats_backward(x, s, grad_entropy=g))
