"""lse_residual_norm and its gradient against the formulas in 64 bits.

Bounds.  f32 arithmetic: a sum of D terms taken in chains of at most 40 and a tree of ten
levels is off by less than 64 * 2^-24 = 2^-18 of the sum of magnitudes; with the products
around it the tests allow E = 2^-17.  h is off by E of |x| + |s g a|, which where the two
cancel is more of h and of its norm: A = rms(|x| + |s g a|) / rms(h) carries that through.
Each output is then rounded to its type (Q, half a step).
"""
import itertools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
Q = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
E = 2.0 ** -17


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def spread(rows, D, dtype, seed, scale=1.0, stride=None, offset=0, fill=float("nan")):
    """A random [rows, D] matrix whose rows lie ``stride`` apart in a larger buffer."""
    stride = D if stride is None else stride
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((offset + max(rows, 1) * stride + 32,), fill, dtype=DT[dtype])
    v = buf[offset:offset + rows * stride].reshape(rows, stride)[:, :D]
    v.copy_(torch.randn((rows, D), generator=g) * scale)
    buf = buf.cuda()
    return buf, buf[offset:offset + rows * stride].reshape(rows, stride)[:, :D]


def vector(D, dtype, seed, mean=1.0):
    return (torch.randn(D, generator=torch.Generator().manual_seed(seed)) * 0.3 + mean).to(DT[dtype]).cuda()


def forward64(x, y, w, post, gate, scale, eps):
    d = torch.float64
    x, w = x.to(d), w.to(d)
    r1 = None
    add = torch.zeros_like(x)
    if y is not None:
        a = y.to(d)
        if post is not None:
            r1 = 1 / torch.sqrt((a * a).mean(1, keepdim=True) + eps)
            a = a * r1 * post.to(d)
        add = scale * (1.0 if gate is None else gate.to(d)) * a
    h = x + add
    r2 = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    mag = x.abs() + add.abs()
    A = torch.sqrt((mag * mag).mean(1, keepdim=True)) * r2
    return h, h * r2 * w, r1, r2, mag, A.clamp(min=1.0)


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol + want.abs() * Q[got.dtype] + TINY[got.dtype])
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].max()), float(want[bad].abs().max()))


def check_forward(s, x, y, w, post, gate, scale, eps):
    h, out, r1, r2, mag, A = forward64(x, y, w, post, gate, scale, eps)
    if y is not None:
        close(s.h, h, E * mag, "h")
    close(s.out, out, 2 * E * w.double().abs() * r2 * (mag + h.abs() * A), "out")
    close(s.rstd, r2[:, 0], 2 * E * A[:, 0] * r2[:, 0], "rstd")
    if r1 is not None:
        close(s.post_rstd, r1[:, 0], E * r1[:, 0], "post_rstd")


def check_backward(d, go, gh, x, y, w, post, gate, scale, eps, weights=True):
    h, _, r1, r2, mag, A = forward64(x, y, w, post, gate, scale, eps)
    T, D = x.shape
    n, w64 = go.double() * w.double(), w.double()
    up = torch.zeros_like(n) if gh is None else gh.double()
    G = up + r2 * n - h * r2 ** 3 / D * (n * h).sum(1, keepdim=True)
    Gm = up.abs() + r2 * n.abs() + mag * r2 ** 3 / D * (n.abs() * mag).sum(1, keepdim=True)
    F = 8 * E * A * A
    close(d.x, G, F * Gm, "dx")
    rows = (T + 64) * 2.0 ** -24
    dw = (go.double() * h * r2)
    dwm = (go.double().abs() * mag * r2)
    if weights:
        close(d.weight, dw.sum(0), ((F + rows) * dwm).sum(0), "dweight")
    if y is None:
        assert d.y is None and d.gate is None and d.post_weight is None
        return
    y64 = y.double()
    rr = torch.ones_like(r2) if r1 is None else r1
    p = torch.ones_like(w64) if post is None else post.double()
    g = torch.ones_like(x, dtype=torch.float64) if gate is None else gate.double().expand_as(x)
    e, em = scale * g * p * G, (scale * g * p).abs() * Gm
    if post is None:
        close(d.y, e, F * em, "dy")
    else:
        dy = r1 * e - y64 * r1 ** 3 / D * (e * y64).sum(1, keepdim=True)
        close(d.y, dy, 2 * F * (r1 * em + y64.abs() * r1 ** 3 / D * (em * y64.abs()).sum(1, keepdim=True)), "dy")
        if weights:
            close(d.post_weight, (scale * g * G * y64 * rr).sum(0),
                  ((2 * F + rows) * (scale * g * y64).abs() * rr * Gm).sum(0), "dpost")
    if gate is not None:
        dg, dgm = scale * p * y64 * rr * G, (scale * p * y64).abs() * rr * Gm
        if gate.dim() == 1:
            if weights:
                close(d.gate, dg.sum(0), ((2 * F + rows) * dgm).sum(0), "dgate")
        else:
            close(d.gate, dg, 2 * F * dgm, "dgate")


def both(x, y, w, post, gate, scale, go, gh, eps=1e-6):
    s = L.lse_residual_norm(x, y, w, post_weight=post, gate=gate, scale=scale, eps=eps)
    check_forward(s, x, y, w, post, gate, scale, eps)
    d = L.lse_residual_norm_backward(go, gh, x, y, s, w, post_weight=post, gate=gate, scale=scale)
    check_backward(d, go, gh, x, y, w, post, gate, scale, eps)
    return s, d


WIDTHS = [1, 2, 3, 7, 8, 16, 33, 64, 65, 100, 128, 129, 255, 256, 260, 511, 512, 1001, 1024, 1030, 2048, 2050, 4096, 4099,
          8192, 8200, 16383, 16384]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(dtype, D):
    for T, post, kind, wdt in [(1, True, "none", dtype), (5, True, "channel", "f32"), (37, True, "element", dtype),
                               (6, False, "channel", dtype), (9, False, "none", "f32"), (3, False, "element", "f32")]:
        x, y, go, gh, ge = (spread(T, D, dtype, D + i, s)[1] for i, s in enumerate((1.5, 0.4, 1.0, 0.7, 0.5)))
        w = vector(D, wdt, 5)
        p = vector(D, wdt, 6) if post else None
        gate = {"none": None, "channel": vector(D, wdt, 7, 0.5), "element": ge}[kind]
        both(x, y, w, p, gate, 0.7, go, gh)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [40, 333, 1024, 2056])
def test_strides_and_offsets(dtype, D):
    """Rows at the same offset in every array, at different ones, and what lies behind them."""
    for strides, offsets in [([D + 8] * 5, [8] * 5), ([D + 1] * 5, [1] * 5), ([D + 1, D, D + 3, D + 8, D], [1, 0, 2, 3, 5])]:
        T = 11
        (xb, x), (yb, y), (gb, go), (hb, gh), (eb, ge) = (
            spread(T, D, dtype, 10 * D + i, 1.0, st, of) for i, (st, of) in enumerate(zip(strides, offsets)))
        w, p = vector(D, dtype, 1), vector(D, dtype, 2)
        both(x, y, w, p, ge, 0.9, go, gh)
        hbuf, h = spread(T, D, dtype, 0, 1.0, strides[0], offsets[0], 7.0)
        obuf, o = spread(T, D, dtype, 0, 1.0, strides[1] + 2, offsets[1] + 1, 7.0)
        s = L.lse_residual_norm(x, y, w, post_weight=p, gate=ge, scale=0.9, h=h, out=o)
        check_forward(s, x, y, w, p, ge, 0.9, 1e-6)
        h.fill_(7.0), o.fill_(7.0)
        assert (hbuf == 7.0).all() and (obuf == 7.0).all()
    # weights off a 16-byte boundary
    w = vector(D + 3, dtype, 1)[3:]
    both(x, y, w, vector(D + 1, dtype, 2)[1:], vector(D + 2, dtype, 3)[2:], -1.3, go, gh)


@pytest.mark.parametrize("dtype,D,T", [("bf16", 64, 70000), ("bf16", 2048, 3000), ("f32", 1001, 4000), ("f16", 257, 20000),
                                       ("bf16", 4096, 1500), ("f32", 16384, 700), ("bf16", 16384, 900), ("f16", 8, 9000)])
def test_many_rows(dtype, D, T):
    x, y, go, gh = (spread(T, D, dtype, D + i, s)[1] for i, s in enumerate((1.5, 0.4, 1.0, 0.7)))
    w, p, g = vector(D, dtype, 1), vector(D, dtype, 2), vector(D, dtype, 3, 0.5)
    s, d = both(x, y, w, p, g, 0.7, go, gh)
    again = L.lse_residual_norm_backward(go, gh, x, y, s, w, post_weight=p, gate=g, scale=0.7)
    for a, b in zip(d, again):
        assert torch.equal(a, b)


def test_without_a_block_and_without_sums():
    x, go, gh, y = (spread(50, 200, "bf16", i)[1] for i in range(4))
    w = vector(200, "bf16", 1)
    both(x, None, w, None, None, 1.0, go, gh)
    both(x, None, w, None, None, 1.0, go, None)
    s = L.lse_residual_norm(x, None, w)
    assert s.h is x and s.post_rstd is None
    s = L.lse_residual_norm(x, y, w, post_weight=w, gate=w)
    d = L.lse_residual_norm_backward(go, gh, x, y, s, w, post_weight=w, gate=w, weights=False)
    assert d.weight is None and d.post_weight is None and d.gate is None
    check_backward(d, go, gh, x, y, w, w, w, 1.0, 1e-6, weights=False)


def test_in_place():
    for D, dtype in itertools.product((64, 1001, 4096, 16384), ("bf16", "f32")):
        x, y = (spread(33, D, dtype, i)[1].clone() for i in range(2))
        w, p = vector(D, dtype, 1), vector(D, dtype, 2)
        want = L.lse_residual_norm(x, y, w, post_weight=p)
        got = L.lse_residual_norm(x, y, w, post_weight=p, h=x, out=y)
        assert got.h is x and got.out is y
        assert torch.equal(x, want.h) and torch.equal(y, want.out)


def test_cancelling_and_empty_rows():
    """Rows in which x and the block cancel, zeros, infinities and NaN: each row by itself."""
    D = 512
    x, y = (spread(8, D, "f32", i)[1].clone() for i in range(2))
    w = vector(D, "f32", 1)
    x[0] = -y[0]
    x[0, 0] += 2.0 ** -10
    x[1], y[1] = 0.0, 0.0
    x[2, 5] = float("inf")
    y[3, 7] = float("nan")
    s = L.lse_residual_norm(x, y, w)
    for i in (0, 1, 4, 5, 6, 7):
        check_forward(L.ResidualNorm(s.h[i:i + 1], s.out[i:i + 1], s.rstd[i:i + 1], None), x[i:i + 1], y[i:i + 1], w, None,
                      None, 1.0, 1e-6)
    assert (s.out[1] == 0).all() and s.rstd[2] == 0 and torch.isnan(s.out[2, 5]) and (s.out[2, :5] == 0).all()
    assert torch.isnan(s.out[3]).all() and not torch.isnan(s.out[4:]).any()


def test_no_rows():
    x = torch.empty((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    s = L.lse_residual_norm(x, x, w, post_weight=w, gate=w)
    d = L.lse_residual_norm_backward(x, x, x, x, s, w, post_weight=w, gate=w)
    assert s.out.shape == (0, 64) and (d.weight == 0).all() and (d.post_weight == 0).all() and (d.gate == 0).all()


def test_against_differences():
    """The gradient against central differences of the 64-bit formulas."""
    T, D = 3, 10
    t = [spread(T, D, "f32", i)[1] for i in range(5)]
    x, y, go, gh, gate = t
    w, p = vector(D, "f32", 1), vector(D, "f32", 2)
    s = L.lse_residual_norm(x, y, w, post_weight=p, gate=gate, scale=0.8)
    d = L.lse_residual_norm_backward(go, gh, x, y, s, w, post_weight=p, gate=gate, scale=0.8)

    def value(*a):
        h, out, *_ = forward64(a[0], a[1], a[2], a[3], a[4], 0.8, 1e-6)
        return float((out * go.double()).sum() + (h * gh.double()).sum())

    base = [v.double().clone() for v in (x, y, w, p, gate)]
    for v, grad in zip(base, d):
        flat = v.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + 1e-5
            up = value(*base)
            flat[i] = keep - 1e-5
            down = value(*base)
            flat[i] = keep
            # differences: 1e-10 times the third derivative (here below 100) and 64-bit noise
            assert abs((up - down) / 2e-5 - float(grad.reshape(-1)[i])) < 2e-5 * max(1.0, float(grad.abs().max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_autograd(dtype):
    g = torch.Generator().manual_seed(3)
    x, y, ge = (torch.randn((2, 5, 96), generator=g).to(dtype).cuda().requires_grad_() for _ in range(3))
    w, p, gc = (torch.randn(96, generator=g).to(dtype).cuda().requires_grad_() for _ in range(3))
    for gate in (None, gc, ge):
        for t in (x, y, w, p, gc, ge):
            t.grad = None
        h, out = L.residual_norm(x, y, w, p, gate, scale=0.6)
        assert h.shape == out.shape == x.shape
        (h.float() * 0.5 + out.float() * 2).sum().backward()
        flat = [t.detach().reshape(10, 96) if t is not None and t.dim() == 3 else None if t is None else t.detach()
                for t in (x, y, w, p, gate)]
        s = L.lse_residual_norm(*flat, scale=0.6)
        d = L.lse_residual_norm_backward(torch.full_like(flat[0], 2), torch.full_like(flat[0], 0.5), flat[0], flat[1], s,
                                         flat[2], flat[3], flat[4], scale=0.6)
        for t, want in zip((x, y, w, p, gate), d):
            if t is not None:
                assert torch.equal(t.grad.reshape(-1), want.reshape(-1))
    # expanded and missing gradients, no gradient for some inputs
    x2 = x.detach()
    h, out = L.residual_norm(x2, y, w.detach())
    y.grad = None
    out.sum().backward()
    assert y.grad is not None and torch.isfinite(y.grad).all()
    h, out = L.residual_norm(x, None, w)
    assert h is x
    h2, _ = L.residual_norm(x, y, w)
    x.grad = None
    h2.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))
    with pytest.raises(RuntimeError):
        h, out = L.residual_norm(x, y, w)
        (dx,) = torch.autograd.grad(out.float().sum(), x, create_graph=True)
        dx.sum().backward()


def test_another_stream_and_graph():
    x, y, go = (spread(300, 512, "bf16", i)[1] for i in range(3))
    w, p = vector(512, "bf16", 1), vector(512, "bf16", 2)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s = L.lse_residual_norm(x, y, w, post_weight=p, stream=st)
    d = L.lse_residual_norm_backward(go, None, x, y, s, w, post_weight=p, stream=st)
    st.synchronize()
    check_backward(d, go, None, x, y, w, p, None, 1.0, 1e-6)
    graphs = []
    for _ in range(2):  # each has scratch of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s = L.lse_residual_norm(x, y, w, post_weight=p)
            d = L.lse_residual_norm_backward(go, None, x, y, s, w, post_weight=p)
        graphs.append((graph, s, d))
    x.copy_(spread(300, 512, "bf16", 9)[1])
    for graph, _, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, s, d in graphs:
        check_forward(s, x, y, w, p, None, 1.0, 1e-6)
        check_backward(d, go, None, x, y, w, p, None, 1.0, 1e-6)


def test_gradient_on_the_forward_stream():
    st = torch.cuda.Stream()
    x, y = (spread(4000, 512, "f32", i)[1] for i in range(2))
    w = vector(512, "f32", 1)
    want = []
    for stream in (None, st):
        leaf = y.clone().requires_grad_()
        if stream is not None:
            st.wait_stream(torch.cuda.current_stream())
        _, out = L.residual_norm(x, leaf, w, post_weight=w, stream=stream)
        torch.cuda.current_stream().wait_stream(st)
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):  # the incoming gradient is late
            big = big @ big / 64
        (out * (1 + 0 * big[0, 0].nan_to_num(0.0, 0.0, 0.0))).sum().backward()
        want.append(leaf.grad * 2)
    assert torch.equal(want[0], want[1])


def test_refusals():
    x = torch.zeros((4, 8), device="cuda")
    w = torch.ones(8, device="cuda")
    s = L.lse_residual_norm(x, x, w, post_weight=w)
    for call in [lambda: L.lse_residual_norm(x, x[:3], w), lambda: L.lse_residual_norm(x, x.half(), w),
                 lambda: L.lse_residual_norm(x, x, w[:7]), lambda: L.lse_residual_norm(x, x, w.half()),
                 lambda: L.lse_residual_norm(x, x, w, post_weight=w.half()), lambda: L.lse_residual_norm(x, x, w, gate=w[:3]),
                 lambda: L.lse_residual_norm(x, None, w, gate=w), lambda: L.lse_residual_norm(x, None, w, h=x),
                 lambda: L.lse_residual_norm(x.t(), x.t(), w), lambda: L.lse_residual_norm(x[0], x[0], w),
                 lambda: L.lse_residual_norm(x, x, w, out=x.half()), lambda: L.lse_residual_norm(x, x, w.cpu()),
                 lambda: L.lse_residual_norm_backward(x[:2], None, x, x, s, w),
                 lambda: L.lse_residual_norm_backward(x, None, x, x, L.ResidualNorm(x, x, s.rstd, None), w, post_weight=w),
                 lambda: L.lse_residual_norm_backward(x, None, x, x, L.ResidualNorm(x, x, s.rstd[:2], None), w),
                 lambda: L.residual_norm(x.t(), x.t(), w), lambda: L.residual_norm(x, x[:2], w)]:
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros((2, 16385), device="cuda")
    with pytest.raises(L.LseError):
        L.lse_residual_norm(wide, wide, torch.ones(16385, device="cuda"))
    with pytest.raises(L.LseError):
        L.lse_residual_norm(x, x, w, eps=-1.0)
    with pytest.raises(TypeError):
        L.lse_residual_norm(x.double(), x.double(), w.double())
