"""Sizes at which the model operators' kernels take paths that ordinary ones do not:
maxima kept of several batches at once, several rounds of a sorting block, three sorting
passes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
import test_gpu_stats as ts  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype,B,N", [("f32", 200, 262147), ("bf16", 700, 140001), ("f16", 250, 300007),
                                       ("f32", 2, 5_000_003), ("bf16", 3, 9_000_001)])
def test_rows_of_more_batches_than_maxima(dtype, B, N):
    """Masked, tied and ordered rows too; every copy of a row gives the same bits."""
    x = torch.cat([ts.special_rows(N, dtype, seed=N), ts.rows(3, N, dtype, seed=N)[0]])[-min(B, 25):]
    n = x.shape[0]
    t = torch.randint(0, N, (n,), generator=torch.Generator().manual_seed(N))
    row = torch.arange(B) % n
    rs = (N + 7) // 8 * 8 + 8
    buf = torch.full((1 + B * rs,), float("nan"), dtype=x.dtype, device="cuda")
    xd = buf[1:].reshape(B, rs)[:, :N]
    xd.copy_(x.cuda()[row.cuda()])
    td = t[row].cuda()
    for K in (20, 32):
        s = L.lse_token_stats(xd, td, K)
        ts.check(None, x, t, K, s._replace(**{f: getattr(s, f)[:n].contiguous() for f in s._fields}))
        for f in s._fields:
            v = torch.nan_to_num(getattr(s, f))
            assert torch.equal(v, v[:n][row.cuda()])


def whole_numbers(T, D, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-8, 9, (T, D), generator=g).float()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D", [(300001, 70000, 8), (300001, 700, 5), (5000, 1_100_000, 8), (70001, 2_000_003, 3),
                                   (600_000, 1_048_576, 2)])
def test_sorts_of_many_tokens_and_of_many_rows(dtype, T, V, D):
    """Whole numbers, so every sum is exact in f32 and rounded once."""
    g = torch.Generator().manual_seed(T + V)
    ids = torch.randint(0, V, (T,), generator=g)
    ids[::3] = torch.randint(0, 40, (ids[::3].numel(),), generator=g) * (V // 41)  # frequent tokens
    ids[5::7] = -1
    grad = whole_numbers(T, D, T)
    ok = (ids >= 0) & (ids != 7)
    want = torch.zeros((V, D), dtype=torch.float64).index_add_(0, ids[ok], grad.double()[ok])
    on = grad.to(ts.DT[dtype]).cuda()
    for out in {torch.float32, ts.DT[dtype]}:
        d = torch.full((V, D), 3.0, dtype=out, device="cuda")
        L.lse_embedding_backward(on, ids.cuda(), V, padding=7, dtable=d)
        assert torch.equal(d.cpu(), want.to(out))
        d.fill_(1.0)
        L.lse_embedding_backward(on, ids.cuda(), V, padding=7, dtable=d, accumulate=True)
        assert torch.equal(d.cpu(), (want + 1).to(out))
