"""A row whose own settings are out of range is marked, as settings for all rows are refused."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("N", [5, 300, 5000, 60001])
def test_out_of_range(N):
    B = 12
    x = torch.randn((B, N), generator=torch.Generator().manual_seed(N)).cuda()
    u = torch.rand(B, generator=torch.Generator().manual_seed(N)).cuda()
    bad = torch.tensor([-0.5, -1e-30, -float("inf"), float("nan")], device="cuda")
    for name, good in (("temperature", 0.8), ("top_p", 0.9), ("min_p", 0.01)):
        rows = torch.full((B,), good, device="cuda")
        rows[1:9:2] = bad
        for more in ({}, {"top_k": 3}):
            got, want = L.lse_sample(x, u, **{name: rows}, **more), L.lse_sample(x, u, **{name: good}, **more)
            marked = torch.zeros(B, dtype=torch.bool, device="cuda")
            marked[1:9:2] = True
            assert (got.token[marked] == -1).all() and torch.isnan(got.logprob[marked]).all(), name
            assert torch.equal(got.token[~marked], want.token[~marked]) and torch.equal(got.logprob[~marked], want.logprob[~marked])
    # -0 is 0, and a top_k below 0 is off
    zero = torch.full((B,), -0.0, device="cuda")
    assert torch.equal(L.lse_sample(x, u, top_p=zero).token, L.lse_sample(x, u, top_p=0.0).token)
    assert torch.equal(L.lse_sample(x, u, min_p=zero).token, L.lse_sample(x, u).token)
    off = torch.full((B,), -2, dtype=torch.int64, device="cuda")
    assert torch.equal(L.lse_sample(x, u, top_k=off).token, L.lse_sample(x, u).token)
