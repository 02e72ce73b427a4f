"""Copies made inside a call run on the stream that the call was given: the caller has
ordered the inputs before that stream and cannot order what it does not see."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import log_sum_exp_gb300 as L  # noqa: E402
import log_sum_exp_gb300._model_ops as M  # noqa: E402

current = [None]
copied_on = []


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is a CUDA tensor and notes where it is copied."""
    is_cuda = property(lambda self: True)

    def contiguous(self, *args, **kwargs):
        if not self.is_contiguous():
            copied_on.append(current[0])
        return super().contiguous(*args, **kwargs)


@pytest.fixture
def fake(monkeypatch):
    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    def stats(x, target, top_k, stream=None):
        return M._token_stats((target, target, target, None, None), target)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(M, "lse_token_stats", stats)
    copied_on.clear()


def make(t):
    return t.as_subclass(OnDevice)


@pytest.mark.parametrize("stream", [None, "side"])
def test_target(fake, stream):
    x = make(torch.zeros((2, 3, 7)))
    t = torch.arange(6).reshape(3, 2).t()
    s = L.token_stats(x, make(t), stream=stream)
    assert copied_on == [stream]
    assert torch.equal(s.logprob.as_subclass(torch.Tensor), t)
    L.token_stats(x, make(t.contiguous()), stream=stream)  # nothing to copy
    assert copied_on == [stream]
