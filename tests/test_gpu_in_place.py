"""Results written over their inputs are those written elsewhere, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
import test_gpu_stats as ts  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,N", [(5000, 60), (5000, 250), (4000, 1000), (3000, 2049), (300, 4100), (64, 20011),
                                 (3, 200001)])
def test_gradient_of_token_statistics(dtype, B, N):
    """Every mapping, with elements that are read first and written last: targets, and
    alternatives that repeat the target or one another."""
    x, t = ts.rows(B, N, dtype, seed=N)
    g = torch.Generator().manual_seed(B)
    for K, lay in ((0, {}), (8, {"offset": 1, "row_stride": N + 3}), (16, {"row_stride": N + 8}), (32, {"offset": 2})):
        xd = ts.place(x, **lay)
        s = L.lse_token_stats(xd, t.cuda(), K)
        if K:
            s.top_index[::3, 1] = t[::3].cuda()
            s.top_index[::5, 2] = s.top_index[::5, 3]
        on = [torch.randn(B, generator=g).cuda() for _ in range(3)]
        gt = torch.randn((B, K), generator=g).cuda() if K else None
        apart = ts.place(torch.zeros_like(x), **lay)
        want = L.lse_token_stats_backward(xd, s, t.cuda(), on[0], on[1], gt, on[2], dx=apart).clone()
        got = L.lse_token_stats_backward(xd, s, t.cuda(), on[0], on[1], gt, on[2], dx=xd)
        assert got.data_ptr() == xd.data_ptr() and torch.equal(got, want)


def test_clipping():
    g = torch.Generator().manual_seed(4)
    flat = torch.randn(3_000_011, generator=g)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        whole = flat.to(dtype).cuda()
        cuts = [0, 1, 4, 4100, 70001, 70002, 1_000_003, 3_000_011]  # neighbours share vectors
        grads = [whole[a:b] for a, b in zip(cuts, cuts[1:])]
        out = [torch.empty_like(v) for v in grads]
        L.lse_grad_clip(L.GradList(grads, out), 1.0)
        L.lse_grad_clip(grads, 1.0)
        for a, b in zip(grads, out):
            assert torch.equal(a, b)
