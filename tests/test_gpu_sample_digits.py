"""Log-probabilities near 0 keep their digits.

A row whose drawn token is its largest has logprob = -log(1 + r), r the weights of the other
kept tokens.  Each weight is off by at most 3e-7 of itself (2^z in f32: 1.5e-7, two roundings
of 6e-8) and by the rounding of x - m (2^-24 of it, here at most 14: 8.4e-7), a sum's terms
pass through at most 20 roundings of 6e-8, and log(1 + r) adds two more: less than
2.6e-6 = 2^-18.5 of r, and of logprob, which is r / (1 + r) or more.  Sums held to 2^-44 add as
much of every part of a row (272 at most): 2^-35.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL, ABS = 2.6e-6, 2.0 ** -35


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def peaked(N, dtype, rest, seed, B=24):
    """Rows with one token at 0 and others whose weights come to about `rest`, none lighter than
    e^-14 of it as far as `rest` goes (more of them are then masked)."""
    g = torch.Generator().manual_seed(seed)
    z = torch.rand((B, N), generator=g, dtype=torch.float64) * 4 - 14.0
    n = min(N - 1, max(1, int(rest / float(torch.exp(z).mean()))))
    z[:, n:] = -float("inf")
    z = z.gather(1, torch.argsort(torch.rand((B, N), generator=g), 1))
    at = torch.randint(0, N, (B,), generator=g)
    z[torch.arange(B), at] = 0.0
    z += torch.tensor([0.0, 0.0, 8.0])[torch.arange(B) % 3, None]  # (a shift that 16-bit types round: weights follow the rounded row)
    return z.to(DT[dtype]).cuda(), at


def check(x, at, keep=None, **settings):
    x64 = x.double().cpu()
    m = x64.amax(1, keepdim=True)
    w = torch.exp((x64 - m) / settings.get("temperature", 1.0))
    if keep is not None:
        w = torch.where(keep(x64 - m), w, torch.zeros_like(w))
    if "top_k" in settings:
        rank = torch.argsort(torch.sort(x64, dim=1, descending=True, stable=True).indices, 1)
        w = torch.where(rank < settings["top_k"], w, torch.zeros_like(w))
    w[torch.arange(len(at)), at] = 0.0
    want = -torch.log1p(w.sum(1))
    # A number inside the largest token's share of the row.
    run = torch.cumsum(torch.where(torch.arange(x.shape[1])[None] < at[:, None], w, torch.zeros_like(w)), 1)[:, -1]
    u = ((run + 0.5) / (w.sum(1) + 1)).float().cuda()
    got = L.lse_sample(x, u, **settings)
    assert torch.equal(got.token.cpu(), at)
    err = (got.logprob.double().cpu() - want).abs()
    assert (err <= REL * want.abs() + ABS).all(), float((err / want.abs()).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [60, 261, 500, 1000, 2000, 8200, 50001, 128256])
@pytest.mark.parametrize("rest", [1e-5, 1e-3, 0.02, 0.5])
def test_uncut(dtype, N, rest):
    check(*peaked(N, dtype, rest, N))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [261, 1000, 50001])
def test_cut(dtype, N):
    x, at = peaked(N, dtype, 0.02, N)
    check(x, at, keep=lambda d: d >= torch.log(torch.tensor(3e-6, dtype=torch.float64)), min_p=3e-6)
    check(x, at, top_p=0.9999999)
    x, at = peaked(N, dtype, 0.5, N)
    check(x, at, top_k=N - 1)
    check(x, at, top_k=N // 2)
