"""lse_sample next to borders in rows with one or two heavy tokens, where the roundings of 32-bit
sums do not average out: the token is that of exact arithmetic.

The rows are built so that every addition that a heavy token's weight passes through meets a
term of just under half a step of the sum and loses it.  Weights are 64-bit exponentials of the
logits; a number closer than 4e-9 of the sum to a border may give either side.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
OPEN = 4e-9
LOST = -16.6875  # weight 5.66e-8, 0.475 of the step of a sum in [1, 2)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def heavy_row(dtype, N, first, second, light, tail=0):
    """A heavy token at column 0 whose 1024 (f32: 512) columns hold the terms that get lost, a
    second one behind `light` tokens of 1e-6, and a tail of tokens of 1e-9."""
    E = 4 if dtype == "f32" else 8
    r = torch.full((N,), -float("inf"), dtype=torch.float64)
    r[0] = first
    for j in range(1, 4):
        r[j * 32 * E] = LOST            # the same lane's next loads
    r[1:E] = LOST                       # its other columns
    for lane in (16, 8, 4, 2, 1):       # lanes that are added to it one after the other
        r[lane * E] = LOST
    start = 128 * E
    r[start:start + light] = -13.8125
    r[N // 2] = second
    if tail:
        r[N - tail:] = -20.75
    return r.to(DT[dtype])


def check(row, u, **settings):
    """The tokens of one row for many numbers."""
    w = torch.exp(row.double() - row.double().max())
    run = torch.cumsum(w, 0)
    target = u.double() * run[-1]
    want = torch.searchsorted(run, target, right=True)
    lower = torch.where(want > 0, run[(want - 1).clamp(min=0)], torch.zeros_like(target))
    far = torch.minimum(target - lower, run[want] - target) > OPEN * run[-1]
    x = row.expand(u.numel(), row.numel()).contiguous().cuda()
    got = L.lse_sample(x, u.cuda(), **settings).token.cpu()
    assert far.sum() > 0.9 * u.numel()
    assert torch.equal(got[far], want[far]), (int((got != want)[far].sum()), u[far & (got != want)][:4].tolist())


def numbers(centre, count=300, steps=1):
    """f32 numbers around `centre`, one every `steps` of their steps."""
    at = torch.tensor([centre], dtype=torch.float32).view(torch.int32)
    return (at + steps * torch.arange(-count // 2, count // 2, dtype=torch.int32)).view(torch.float32)


def centre(row, dtype):
    """The number that lies in the middle of the light tokens."""
    w = torch.exp(row.double())
    return float((w[:128 * (4 if dtype == "f32" else 8)].sum() + 6e-6) / w.sum())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [8192, 16384, 40000])
@pytest.mark.parametrize("second", [0.0, -0.25])
def test_two_heavy_tokens(dtype, N, second):
    row = heavy_row(dtype, N, 0.0, second, 12)
    check(row, numbers(centre(row, dtype)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("second", [-4.0, -9.0])
def test_one_heavy_token(dtype, second):
    row = heavy_row(dtype, 8192, 0.0, second, 12)
    check(row, numbers(centre(row, dtype)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_cut_by_min_p(dtype):
    """More tokens than the list holds are kept, so what is kept is summed in 32 bits."""
    row = heavy_row(dtype, 16384, 0.0, 0.0, 12, tail=3000)
    check(row, numbers(centre(row, dtype)), min_p=5e-10)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_cut_by_top_p(dtype):
    """The cut falls among the light tokens behind the heavy one: the shortest prefix that reaches
    top_p by 64-bit sums.  The number next to 1 draws the last kept token, which is a light one."""
    N = 8192
    row = heavy_row(dtype, N, 0.0, -float("inf"), 0)
    row[N // 2:N // 2 + 12] = -13.8125
    x64 = row.double()
    order = torch.sort(x64, descending=True, stable=True).indices
    w = torch.exp(x64)
    run, total = torch.cumsum(w[order], 0), float(w.sum())
    p = numbers((1.0 + 6e-6) / total, 180)
    need = p.double() * total
    reach = torch.searchsorted(run, need)
    below = torch.where(reach > 0, run[(reach - 1).clamp(min=0)], torch.zeros_like(need))
    far = torch.minimum(run[reach] - need, need - below) > OPEN * total
    assert far.sum() > 0.9 * p.numel() and (reach > 0).all() and (reach < 13).all()
    x = row.expand(p.numel(), N).contiguous().cuda()
    got = L.lse_sample(x, torch.full((p.numel(),), 1.0 - 2.0 ** -24, device="cuda"), top_p=p.cuda())
    want = torch.stack([order[:int(r) + 1].max() for r in reach])
    assert torch.equal(got.token.cpu()[far], want[far]), int((got.token.cpu() != want)[far].sum())
