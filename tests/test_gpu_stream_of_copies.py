"""A call on another stream reads its own copies of the inputs after they are made."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("grad", [False, True])
def test_transposed_target(grad):
    st = torch.cuda.Stream()
    g = torch.Generator().manual_seed(1)
    x = torch.randn((40, 30, 1009), generator=g).cuda()
    t = torch.randint(0, 1009, (30, 40), generator=g).cuda().t()
    want = torch.log_softmax(x.double(), -1).gather(-1, t[..., None])[..., 0]
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        leaf = x.clone().requires_grad_(grad)
        st.wait_stream(torch.cuda.current_stream())  # the inputs are there
        for _ in range(8):                           # and the current stream is busy
            big = big @ big / 64
        s = L.token_stats(leaf, t, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        assert ((s.logprob - want).abs() <= 1e-5 + 1e-6 * want.abs()).all()
        if grad:
            s.logprob.sum().backward()
            ref = torch.nn.functional.one_hot(t, 1009) - torch.softmax(x.double(), -1)
            assert ((leaf.grad - ref).abs() <= 1e-6 + 2.0 ** -20 * ref.abs()).all()
