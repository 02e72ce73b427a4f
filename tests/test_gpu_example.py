"""The policy-step example: its gradients against a 64-bit model, and that it learns."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_gradients_of_a_step():
    """In f32: every gradient within 1e-4 of its tensor's largest entry (the f32 matrix
    products of 512-long sums err by about 512 * 2^-24 = 3e-5 of it)."""
    import policy_step as ex

    torch.backends.cuda.matmul.allow_tf32 = False
    model = ex.TokenModel(1009, 72, dtype=torch.float32)
    ids = torch.randint(0, 1009, (512,), device="cuda")
    ids[::3] = 17
    actions = torch.randint(0, 1009, (512,), device="cuda")
    adv = torch.randn(512, device="cuda")
    loss, _ = ex.policy_loss(model.logits(ids), actions, adv, 0.1)
    loss.backward()
    ref = [p.detach().double().requires_grad_() for p in model.params]
    logp = torch.log_softmax((ref[0][ids] * model.scale) @ ref[1].t(), 1)
    want = -(adv.double() * logp.gather(1, actions[:, None])[:, 0]).mean() + 0.1 * (logp.exp() * logp).sum(1).mean()
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) < 1e-4
    for p, r in zip(model.params, ref):
        assert (p.grad.double() - r.grad).abs().max() <= 1e-4 * r.grad.abs().max()
    before = [p.grad.clone() for p in model.params]
    norm = torch.cat([b.double().reshape(-1) for b in before]).norm()
    masters = [m.clone() for m in model.master]
    got = model.update(lr=1.0, max_norm=float(norm) / 2)
    assert abs(float(got) - float(norm)) <= 1e-6 * float(norm)
    for m, old, b in zip(model.master, masters, before):
        assert ((old - m) - b * 0.5).abs().max() <= 1e-4 * b.abs().max()


def test_it_learns():
    import policy_step as ex

    _, rewards = ex.train(steps=40, quiet=True)
    assert sum(rewards[-10:]) / 10 > 0.9 and rewards[0] < 0.1
