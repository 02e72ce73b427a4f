"""The same call on the same values at the same offsets gives the same bits, wherever the
memory is."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def copies(x, offset):
    """Two device copies of x, each ``offset`` elements behind an allocation's start."""
    out = []
    for _ in range(2):
        buf = torch.full((offset + x.numel() + 16,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf[offset:offset + x.numel()].view(x.shape)
        view.copy_(x)
        out.append(view)
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_every_operator(dtype, offset):
    g = torch.Generator().manual_seed(offset)
    for B, N in ((1000, 90), (300, 3001), (40, 40003)):
        a, b = copies(torch.randn((B, N), generator=g).to(dtype), offset)
        t = torch.randint(0, N, (B,), generator=g).cuda()
        w = torch.randn(B, generator=g).cuda()
        s, r = L.lse_token_stats(a, t, 5), L.lse_token_stats(b, t, 5)
        assert all(torch.equal(x, y) for x, y in zip((*s, s.lse_low), (*r, r.lse_low)))
        assert torch.equal(L.lse_token_stats_backward(a, s, t, w, w), L.lse_token_stats_backward(b, r, t, w, w))
    a, b = copies(torch.randn(1_000_003, generator=g).to(dtype), offset)
    assert torch.equal(L.lse_grad_norm([a]), L.lse_grad_norm([b]))
    for T, V, D in ((300, 50, 40), (9000, 400, 260)):
        ids = torch.randint(0, V, (T,), generator=g).cuda() ** 2 // V
        a, b = copies(torch.randn((T, D), generator=g).to(dtype), offset)
        assert torch.equal(L.lse_embedding_backward(a, ids, V), L.lse_embedding_backward(b, ids, V))
