"""The gradient of lse_token_stats where the logits are large, against a float64 softmax
of x itself (not of the kernel's rounded row value).

Bars, with logp = log p, H the entropy, and c, gH as in the formula, G = |c| + |gH| (|logp| + |H|):
  - log sum exp(x - max) in f32: 2^-22 of the exponentials, sums of up to N / 128 terms in a
    row (2^-24 each), the logarithm: D = 2^-20 + N 2^-31, which is p's relative error and
    log p's absolute one; none of it grows with the row's offset;
  - the exponent's roundings: 2^-22 |logp| of p;
  - the kernel's entropy: 1e-5 + 2^-19 (H + M), M = sum p (1 + |logp|) |logp + H|;
  - the bracket and the unit terms: 2^-22 of their magnitudes; the element type's rounding.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
import test_gpu_stats as ts  # noqa: E402

OFFSETS = [0.0, 20.0, -1e3, 1e3, 3e4, -3e4, 1e6, -1e6, 3e7, 1e12]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def shifted_rows(N, dtype, seed):
    """Rows around each offset (their spread at least two of the type's steps there), a
    row of nothing but the type's lowest value, and one where half of those are -inf."""
    g = torch.Generator().manual_seed(seed)
    info = torch.finfo(ts.DT[dtype])
    out = []
    for o in OFFSETS:
        if abs(o) > 3e4 and dtype == "f16":
            continue
        spread = max(3.0, 2 * abs(o) * info.eps)
        out.append(o + torch.randn(N, generator=g, dtype=torch.float64) * spread)
    out.append(torch.full((N,), info.min, dtype=torch.float64))
    half = torch.full((N,), info.min, dtype=torch.float64)
    half[1::2] = -np.inf
    out.append(half)
    return torch.stack(out).to(ts.DT[dtype])


def reference(x, t, idx, gl, gh, gt, gs):
    xd = x.double()
    B, N = xd.shape
    m = xd.amax(1, keepdim=True)
    logs = torch.log(torch.exp(xd - m).sum(1, keepdim=True))
    logp = (xd - m) - logs
    p = torch.exp(logp)
    lp = torch.where(p > 0, logp, 0.0)
    h = -(p * lp).sum(1, keepdim=True)
    mom = (p * (1 + lp.abs()) * (lp + h).abs()).sum(1, keepdim=True)
    gl, gh, gs, gt = (v.double()[:, None] if v.dim() == 1 else v.double() for v in (gl, gh, gs, gt))
    unit, mag = torch.zeros_like(xd), torch.zeros_like(xd)
    unit.scatter_add_(1, t[:, None], gl)
    unit.scatter_add_(1, idx, gt)
    mag.scatter_add_(1, t[:, None], gl.abs())
    mag.scatter_add_(1, idx, gt.abs())
    c = gs - gl - gt.sum(1, keepdim=True)
    ca = gs.abs() + gl.abs() + gt.abs().sum(1, keepdim=True)
    ref = p * (c - gh * (lp + h)) + unit
    G = ca + gh.abs() * (lp.abs() + h)
    D = 2.0 ** -20 + N * 2.0 ** -31
    bar = p * (G * (D + 2.0 ** -22 * lp.abs()) + gh.abs() * (D + 1e-5 + 2.0 ** -19 * (h + mom)) + 2.0 ** -22 * G) \
        + 2.0 ** -22 * mag + 1e-37 * (G + mag)
    return ref, bar, p


def check(d, ref, bar, dtype):
    lim = bar + ts.Q[dtype] * ref.abs() + (2.0 ** -24 if dtype == "f16" else 2.0 ** -133 if dtype == "bf16" else 0)
    bad = ~((d.double() - ref).abs() <= lim)
    assert not bad.any(), [(tuple(i.tolist()), float(d[tuple(i)]), float(ref[tuple(i)])) for i in bad.nonzero()[:4]]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [5, 40, 261, 3000, 32000, 70001])
def test_gradient_does_not_depend_on_the_offset(dtype, N):
    x = shifted_rows(N, dtype, N)
    B = x.shape[0]
    g = torch.Generator().manual_seed(N)
    t = 2 * torch.randint(0, (N + 1) // 2, (B,), generator=g)
    gl, gh, gs = torch.randn(B, generator=g), torch.randn(B, generator=g), torch.randn(B, generator=g)
    gt = torch.randn((B, 2), generator=g)
    for place in (dict(), dict(offset=1, row_stride=N + 3)):
        xd = ts.place(x, **place)
        s = L.lse_token_stats(xd, t.cuda(), 2)
        zero = torch.zeros(B)
        for on in ((gl, gh, gt, gs), (zero, gh, 0 * gt, zero), (gl, zero, 0 * gt, zero)):
            ref, bar, _ = reference(x, t, s.top_index.cpu(), on[0], on[1], on[2], on[3])
            d = L.lse_token_stats_backward(xd, s, t.cuda(), *[v.cuda() for v in on])
            check(d.cpu(), ref, bar, dtype)


@pytest.mark.parametrize("N", [5, 261, 32000])
def test_probabilities_sum_to_one(N):
    x = shifted_rows(N, "f32", N)
    s = L.lse_token_stats(x.cuda(), None, entropy=False)
    p = L.lse_token_stats_backward(x.cuda(), s, grad_lse=torch.ones(x.shape[0], device="cuda"))
    # sum p (D + 2^-22 |logp|) + roundings, sum p |logp| <= log N < 16
    assert ((p.double().sum(1) - 1).abs() <= 2.0 ** -20 + N * 2.0 ** -31 + 2.0 ** -18).all()


def test_autograd_of_large_logits():
    x = shifted_rows(3001, "f32", 7)
    t = torch.full((x.shape[0],), 1500)
    leaf = x.cuda().requires_grad_()
    s = L.token_stats(leaf, t.cuda())
    w = torch.linspace(-1, 1, x.shape[0])
    ((s.logprob - 0.5 * s.entropy) * w.cuda()).sum().backward()
    none = torch.zeros((x.shape[0], 1))
    ref, bar, _ = reference(x, t, t[:, None], w, -0.5 * w, none, torch.zeros_like(w))
    check(leaf.grad.cpu(), ref, bar, "f32")


def test_the_two_parts_of_the_row_value():
    """lse + lse_low against float64, beyond f32's digits; what carries them along."""
    x = shifted_rows(3000, "f32", 1)
    s = L.lse_token_stats(x.cuda())
    xd = x.double()
    m = xd.amax(1)
    logs = torch.log(torch.exp(xd - m[:, None]).sum(1))
    low = s.lse_low.cpu().double()
    got = (s.lse.cpu().double() - m) + low
    assert ((got - logs).abs() <= 2.0 ** -20 + 3000 * 2.0 ** -31 + 2.0 ** -23 * logs).all()
    lse = s.lse.cpu().double()
    assert (low.abs()[:-2] <= 2.0 ** -24 * lse.abs()[:-2]).all()
    assert len(s) == 5 and s._replace(entropy=None).lse_low is s.lse_low
    assert s._replace(lse=s.lse).lse_low is None and L.TokenStats(*s).lse_low is None
    special = torch.tensor([[np.inf, 1.0], [-np.inf, -np.inf], [np.nan, 1.0]], device="cuda")
    assert (L.lse_token_stats(special).lse_low == 0).all()
    assert (L.lse_token_stats(torch.empty((3, 0), device="cuda")).lse_low == 0).all()
    assert L.lse_token_stats(x[0].cuda()).lse_low.shape == ()
    assert L.token_stats(x.cuda().reshape(2, -1, 3000)).lse_low.shape == (2, x.shape[0] // 2)


def test_the_row_value_alone():
    """A tuple without lse_low, and the C entry points that have none: the gradient of
    the rounded lse, within the bars of its own test."""
    x, t = ts.rows(6, 3001, "f32", 3)
    xd, td = x.cuda(), t.cuda()
    s = L.lse_token_stats(xd, td, 3)
    gl, gh, gt, gs = ts.gradients(6, 3, 0)
    on = [v.cuda() for v in (gl, gh, gt, gs)]
    d = L.lse_token_stats_backward(xd, L.TokenStats(*s), td, *on)
    ts.check_gradient(d.cpu(), x, s, t, gl, gh, gt, gs, "f32")
    lib = L.load()
    c = [torch.empty_like(v) for v in s]
    stream = torch.cuda.current_stream().cuda_stream
    ptr = [v.data_ptr() for v in c]
    assert lib.lse_token_stats(xd.data_ptr(), 0, 6, 3001, 3001, td.data_ptr(), 3, *ptr, stream) == 0
    for a, b in zip(c, s):
        assert torch.equal(a, b)
    e = torch.empty_like(d)
    assert lib.lse_token_stats_backward(xd.data_ptr(), 0, 6, 3001, 3001, ptr[2], ptr[1], td.data_ptr(), ptr[4], 3,
                                        *[v.data_ptr() for v in on], e.data_ptr(), 3001, stream) == 0
    assert torch.equal(d, e)


def test_refused_parts():
    x = torch.zeros((4, 10), device="cuda")
    s = L.lse_token_stats(x)
    g = torch.ones(4, device="cuda")
    for low in (g[:2], g.double(), g.cpu()):
        s.lse_low = low
        with pytest.raises(ValueError):
            L.lse_token_stats_backward(x, s, grad_lse=g)
