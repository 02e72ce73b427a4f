"""The end of a block: rows of no columns."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("T", [1, 5, 300])
def test_no_columns(T):
    """The mean of nothing is NaN, and so is what is made of it: never what memory held before."""
    x, w = torch.empty((T, 0), device="cuda"), torch.empty(0, device="cuda")
    for y, post in ((x, w), (x, None), (None, None)):
        stale = [torch.full((T,), 7.0, device="cuda") for _ in range(4)]
        del stale
        got = L.lse_residual_norm(x, y, w, post_weight=post)
        assert got.out.shape == (T, 0) and torch.isnan(got.rstd).all()
        assert post is None or torch.isnan(got.post_rstd).all()
        d = L.lse_residual_norm_backward(x, None, x, y, got, w, post_weight=post)
        assert d.x.shape == (T, 0) and d.weight.shape == (0,)


def test_no_columns_in_c():
    """The C call does no device work then, and says so: rstd is left as it was."""
    rstd = torch.full((4,), 7.0, device="cuda")
    args = (None, 0, 4, 0, 0, None, 0, None, 0, 0, None, None, 0, 1.0, 1e-6, None, 0, None, 0)
    assert L.load().lse_residual_norm(*args, rstd.data_ptr(), None, torch.cuda.current_stream().cuda_stream) == 0
    assert (rstd == 7.0).all()
