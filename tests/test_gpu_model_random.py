"""Seeded random cases over every mapping of the model operators: shapes, types, strides,
offsets, K, and values with ties and masks.  Bars as in the operators' own tests."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
import test_gpu_embed as te  # noqa: E402
import test_gpu_grads as tg  # noqa: E402
import test_gpu_stats as ts  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def values(B, N, dtype, r, g):
    """Rows of one of several kinds each: smooth, few levels, masked, shifted far."""
    x = torch.randn((B, N), generator=g) * 3
    kind = torch.randint(0, 5, (B,), generator=g)
    few = torch.randint(-2, 3, (B, N), generator=g).float()
    x = torch.where(kind[:, None] == 1, few, x)
    masked = torch.rand((B, N), generator=g) < r.choice([0.1, 0.9, 0.999])
    low = r.choice([-float("inf"), torch.finfo(ts.DT[dtype]).min])
    x = torch.where((kind[:, None] == 2) & masked, torch.tensor(low), x)
    x = torch.where(kind[:, None] == 3, x + (1000.0 if dtype == "f16" else 30000.0), x)
    return x.to(ts.DT[dtype])


@pytest.mark.parametrize("seed", range(60))
def test_stats(seed):
    r = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    dtype = r.choice(["f32", "bf16", "f16"])
    N = int(round(2 ** r.uniform(0, 18)))
    B = max(1, min(3000, int(2 ** r.uniform(0, 12)), 3_000_000 // N))
    K = r.choice([0, 1, 2, 4, 5, 8, 9, 16, 20, 24, 25, 32])
    x = values(B, N, dtype, r, g)
    t = torch.randint(-2, N + 2, (B,), generator=g)
    lay = {"row_stride": N + r.choice([0, 0, 1, 5, 8, 64]), "offset": r.choice([0, 0, 1, 2, 3, 8])}
    xd = ts.place(x, **lay)
    s = ts.check(xd, x, t, K)
    for a, b in zip(s, L.lse_token_stats(xd, t.cuda(), K)):
        assert a is None or torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    dx = xd if r.random() < 0.5 else ts.place(torch.zeros_like(x), **lay) if r.random() < 0.5 else None
    finite = torch.isfinite(s.lse.cpu())  # (rows of only -inf are the special tests' part)
    gl, gh, gt, gs = ts.gradients(B, K, seed)
    gl, gh, gs = gl * finite, gh * finite, gs * finite
    gt = gt * finite[:, None] if K else None
    on = [None if v is None else v.cuda() for v in (gl, gh, gt, gs)]
    d = L.lse_token_stats_backward(xd, s, t.cuda(), *on, dx=dx)
    ts.check_gradient(d.cpu(), x, s, t, gl, gh, gt, gs, dtype)


@pytest.mark.parametrize("seed", range(25))
def test_gradient_lists(seed):
    r = random.Random(seed)
    sizes = [int(2 ** r.uniform(0, r.choice([6, 12, 20]))) for _ in range(r.choice([1, 3, 47, 49, 250, 1100]))]
    if sum(sizes) > 20_000_000:
        sizes = [n // 16 + 1 for n in sizes]
    ins = tg.make(sizes, r.choice([["f32"], ["bf16"], ["f16"], ["f32", "bf16", "f16"]]), seed, r.choice([1.0, 1e-6, 100.0]))
    lst = L.GradList(ins, [torch.empty_like(t) for t in ins])
    want = tg.check_norm(L.lse_grad_norm(lst), ins)
    max_norm = want * r.choice([0.1, 0.9, 2.0])
    L.lse_grad_clip(lst, max_norm)
    tg.check_clipped(lst.out, ins, want, max_norm)


@pytest.mark.parametrize("seed", range(40))
def test_embedding(seed):
    r = random.Random(seed)
    dtype = r.choice(["f32", "bf16", "f16"])
    D = int(2 ** r.uniform(0, 11)) if r.random() < 0.5 else 8 * int(2 ** r.uniform(0, 8))
    V = int(2 ** r.uniform(0, 17))
    T = int(2 ** r.uniform(0, 16))
    T = max(1, min(T, 8_000_000 // D))
    V = max(1, min(V, 16_000_000 // D))
    stride, off = D + r.choice([0, 0, 2, 3, 8]), r.choice([0, 0, 1, 2, 4, 8])
    _, grad = te.spread(T, D, dtype, seed, stride, off)
    ids = te.tokens(T, V, seed) if r.random() < 0.7 else torch.randint(-1, V + 1, (T,), generator=torch.Generator().manual_seed(seed))
    out = r.choice(["f32", dtype])
    buf, dt = te.spread(V, D, out, seed + 1, D + r.choice([0, 0, 2, 8, 5]), r.choice([0, 0, 1, 4, 8]), fill=3.0)
    accumulate = r.random() < 0.4
    base = dt.clone() if accumulate else None
    padding = r.choice([-1, 0, V // 2])
    L.lse_embedding_backward(grad, ids.cuda(), V, 1.25, padding, dtable=dt, accumulate=accumulate)
    te.check_gradient(dt, grad, ids, V, 1.25, padding, base)
    got = L.lse_embedding(dt, ids.cuda(), 0.5)
    ok = ((ids >= 0) & (ids < V)).cuda()
    assert torch.equal(got[ok], (dt[ids.cuda().clamp(0, V - 1)].float() * 0.5).to(dt.dtype)[ok])
    assert torch.isnan(got[~ok]).all()
    dt.fill_(3.0)
    assert (buf == 3.0).all()
