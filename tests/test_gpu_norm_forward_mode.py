"""residual_norm: forward-mode derivatives are refused, not dropped, and second ones as well."""
import pytest

torch = pytest.importorskip("torch")
from torch.autograd import forward_ad as fwd  # noqa: E402

pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("which", ["x", "y", "weight", "post_weight", "gate"])
def test_tangents(which):
    a = dict(x=torch.randn(4, 16, device="cuda"), y=torch.randn(4, 16, device="cuda"), weight=torch.rand(16, device="cuda"),
             post_weight=torch.rand(16, device="cuda"), gate=torch.rand(16, device="cuda"))
    with fwd.dual_level():
        dual = dict(a, **{which: fwd.make_dual(a[which], torch.ones_like(a[which]))})
        for grad in (True, False):
            with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError):
                L.residual_norm(**dual)
        assert L.residual_norm(**a)[1].shape == (4, 16)


def test_second_derivatives():
    x = torch.randn(4, 16, device="cuda", requires_grad=True)
    h, out = L.residual_norm(x, torch.randn(4, 16, device="cuda"), torch.rand(16, device="cuda"))
    (d,) = torch.autograd.grad(out.sum() + h.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(d.sum(), x)
