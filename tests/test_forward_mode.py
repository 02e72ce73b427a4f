"""Forward-mode derivatives are refused, not dropped."""
import pytest

torch = pytest.importorskip("torch")
from torch.autograd import forward_ad as fwd  # noqa: E402

import log_sum_exp_gb300 as L  # noqa: E402
import log_sum_exp_gb300._model_ops as M  # noqa: E402


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is a CUDA tensor."""
    is_cuda = property(lambda self: True)


def make_dual(t):
    return fwd.make_dual(t, torch.ones_like(t))


@pytest.fixture
def no_kernels(monkeypatch):
    def stats(x, target=None, top_k=0, entropy=True, stream=None):
        v = x.detach().sum(-1)
        return M._token_stats((None, v.clone(), v, None, None), v.clone())

    monkeypatch.setattr(M, "lse_token_stats", stats)
    monkeypatch.setattr(M, "lse_embedding", lambda table, ids, scale=1.0, stream=None: table.detach()[ids])
    monkeypatch.setattr(M, "_FUNCTIONS", {})


def test_a_tangent_reaches_the_function(no_kernels):
    x, table = torch.randn(4, 7), torch.randn(5, 6)
    ids = torch.tensor([1, 3])
    with fwd.dual_level():
        d = make_dual(x).as_subclass(OnDevice)
        assert fwd.unpack_dual(d).tangent is not None
        for call in (lambda: L.token_stats(d), lambda: L.embedding(ids, make_dual(table))):
            for grad in (True, False):
                with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError):
                    call()
        # Without a tangent nothing changes.
        assert L.token_stats(x.as_subclass(OnDevice)).lse.shape == (4,)
        assert L.embedding(ids, table).shape == (2, 6)


@pytest.mark.gpu
def test_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x, table = torch.randn(4, 7, device="cuda"), torch.randn(5, 6, device="cuda")
    ids = torch.tensor([1, 3], device="cuda")
    with fwd.dual_level():
        for call in (lambda: L.token_stats(make_dual(x)), lambda: L.embedding(ids, make_dual(table))):
            with pytest.raises(NotImplementedError):
                call()
        assert L.token_stats(x).lse.shape == (4,)
