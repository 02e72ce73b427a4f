"""lse_token_stats and its gradient against plain 64-bit formulas.

Bars.  Row values and log-probabilities: the library's bar (1e-5 + 1e-6 of the
magnitudes).  Entropy H = -sum p log p: an exponential is off by a relative
2^-21 + 2^-22 |log p| (its argument's roundings), which moves H by at most the
p-weighted sum of that times |log p + H|; sums and logs add a few 2^-22 of H.  With
M = sum p (1 + |log p|) |log p + H| the bar is 1e-5 + 2^-19 (H + M).  Gradient,
with c and H as in the formula and G = |c| + |gH| (|log p| + |H|): the exponential's
error p G (2^-21 + 2^-23 (|lse| + |log p|)), the bracket's own rounding
p 2^-22 (G + |gH| (|lse| + |x|)), 2^-22 of the added unit terms, and the element
type's rounding.  Columns are exact.
"""
import numpy as np
import pytest

from lse_testutil import canary_array, compare, torch_view

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
Q = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def place(x, row_stride=None, offset=0):
    """A device copy of the CPU rows ``x`` inside a buffer of NaNs."""
    B, N = x.shape
    rs = N if row_stride is None else row_stride
    buf = torch.full((offset + B * rs + 64,), float("nan"), dtype=x.dtype)
    view = buf[offset:offset + B * rs].reshape(B, rs)[:, :N] if B else buf[offset:offset].reshape(0, N)
    view.copy_(x)
    dev = buf.cuda()
    return dev[offset:offset + B * rs].reshape(B, rs)[:, :N] if B else dev[offset:offset].reshape(0, N)


def reference(x, target, K):
    """The definitions in float64 on the CPU tensor x."""
    xd = x.double()
    B, N = xd.shape
    lse = torch.logsumexp(xd, 1) if N else torch.full((B,), -np.inf, dtype=torch.float64)
    has_nan = torch.isnan(xd).any(1)
    top_inf = (xd == np.inf).any(1) & ~has_nan
    lse = torch.where(has_nan, torch.nan, torch.where(top_inf, torch.inf, lse))
    # log p against the maximum: lse itself has no digits left for log N next to
    # a row of the lowest value.
    m = xd.amax(1) if N else lse
    m = torch.where(torch.isfinite(m), m, 0.0)
    logs = torch.where(torch.isfinite(lse), torch.log(torch.exp(xd - m[:, None]).sum(1)), lse)
    logp = (xd - m[:, None]) - logs[:, None]
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp.clamp(min=-1e300), 0.0)
    ent = torch.where(torch.isfinite(lse), -plogp.sum(1), torch.nan)
    mom = torch.where(p > 0, p * (1 + logp.abs()) * (logp + ent[:, None]).abs(), 0.0).sum(1)
    lp = None
    if target is not None:
        ok = (target >= 0) & (target < N)
        at = target.clamp(0, max(N - 1, 0))
        lp = torch.where(ok, logp[torch.arange(B), at] if N else torch.nan, torch.nan)
    # (value descending, NaN first, column ascending): a stable sort of the values.
    rank = torch.where(torch.isnan(xd), np.inf, xd) + 0.0
    order = torch.from_numpy(np.lexsort((np.broadcast_to(np.arange(N), (B, N)), -rank.numpy(),
                                         ~torch.isnan(xd).numpy()), axis=1)) if N else \
        torch.zeros((B, 0), dtype=torch.int64)
    idx = torch.full((B, K), -1, dtype=torch.int64)
    tlp = torch.full((B, K), -np.inf, dtype=torch.float64)
    k = min(K, N)
    idx[:, :k] = order[:, :k]
    tlp[:, :k] = logp.gather(1, order[:, :k]) if k else tlp[:, :0]
    # A difference beyond the f32 range is infinite in f32.
    lp = None if lp is None else lp.float().double()
    return lp, ent, lse, tlp.float().double(), idx, mom


def check(xd, x, target, K, stats=None):
    s = L.lse_token_stats(xd, target.cuda() if target is not None else None, K) if stats is None else stats
    torch.cuda.synchronize()
    lp, ent, lse, tlp, idx, mom = reference(x, target, K)
    compare(s.lse.cpu().numpy(), lse.numpy())
    big = np.abs(np.nan_to_num(lse.numpy(), posinf=0, neginf=0))
    if target is not None:
        compare(s.logprob.cpu().numpy(), lp.numpy(),
                scale=big + np.abs(np.nan_to_num(lp.numpy(), posinf=0, neginf=0)))
    bar = (ent + mom).numpy()
    compare(s.entropy.cpu().numpy(), ent.numpy(), atol=1e-5, rtol=2.0 ** -19,
            scale=np.nan_to_num(bar))
    if K:
        assert torch.equal(s.top_index.cpu(), idx)
        compare(s.top_logprob.cpu().numpy(), tlp.numpy(),
                scale=big[:, None] + np.abs(np.nan_to_num(tlp.numpy(), posinf=0, neginf=0)))
    else:
        assert s.top_index is None and s.top_logprob is None
    return s


def rows(B, N, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, N), generator=g) * scale + torch.rand((B, 1), generator=g) * 20 - 10
    return x.to(DT[dtype]), torch.randint(0, max(N, 1), (B,), generator=g)


LAYOUTS = [{}, {"row_stride": 8}, {"row_stride": 3}, {"offset": 1}, {"offset": 3, "row_stride": 1}]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 63, 65, 100, 127, 130, 255, 256, 257,
                               261, 511, 513, 1000, 1023, 1025, 2047, 2049, 4095, 4097, 8191, 10007])
def test_lengths_and_layouts(dtype, N):
    x, t = rows(5, N, dtype, seed=N)
    t[3] = -100
    t[4] = N
    for i, lay in enumerate(LAYOUTS):
        lay = dict(lay)
        if "row_stride" in lay:
            lay["row_stride"] += N
        check(place(x, **lay), x, t, (0, 1, 5, 20, 32)[(i + N) % 5])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,N,K", [(1, 128256, 20), (3, 50257, 32), (17, 32000, 7), (1, 1048579, 32),
                                   (2, 300001, 1), (160, 20011, 20), (700, 4099, 8), (5000, 261, 8),
                                   (40000, 33, 4), (3, 200000, 0), (400, 9000, 32)])
def test_shapes(dtype, B, N, K):
    x, t = rows(B, N, dtype, seed=B + N)
    s = check(place(x), x, t, K)
    again = L.lse_token_stats(place(x), t.cuda(), K)
    for a, b in zip(s, again):
        assert a is None or torch.equal(a, b)


def special_rows(N, dtype, seed=0):
    """Rows that a mask, a tie or an overflow makes hard."""
    g = torch.Generator().manual_seed(seed)
    low = torch.finfo(DT[dtype]).min
    out = []
    out.append(torch.full((N,), -np.inf))                        # nothing left
    out.append(torch.zeros(N))                                   # all equal
    out.append(torch.full((N,), low))                            # all the lowest value
    x = torch.full((N,), -np.inf); x[N // 2] = 1.5; out.append(x)      # one left
    x = torch.full((N,), -np.inf); x[N - 1] = -2.0; x[N // 3] = 4.0; out.append(x)
    x = torch.full((N,), low); x[N // 2] = 1.5; x[N - 1] = 1.5; out.append(x)
    x = torch.randint(0, 3, (N,), generator=g).float(); out.append(x)  # many ties
    x = torch.randn(N, generator=g); x[::2] = -np.inf; out.append(x)
    x = torch.randn(N, generator=g); x[N // 2] = np.nan; out.append(x)
    x = torch.randn(N, generator=g); x[::3] = np.nan; out.append(x)
    out.append(torch.full((N,), np.nan))
    x = torch.randn(N, generator=g); x[N // 2] = np.inf; out.append(x)
    x = torch.randn(N, generator=g); x[::2] = np.inf; x[N - 1] = np.nan; out.append(x)
    x = torch.randn(N, generator=g); x[N // 2] = np.inf; x[0] = -np.inf; x[N - 1] = low; out.append(x)
    x = torch.zeros(N); x[::2] = -0.0; out.append(x)                 # zeros of both signs
    x = torch.full((N,), -1.0); x[1::2] = -0.0; x[::4] = 0.0; out.append(x)
    out.append(torch.linspace(-8, 8, N))                            # ascending
    out.append(torch.linspace(8, -8, N))                            # descending
    x = torch.randn(N, generator=g); x[N - min(N, 40):] = 30.0; out.append(x)  # ties at the end
    x = torch.randn(N, generator=g); x[:min(N, 100)] += 50.0; out.append(x)    # a cluster
    x = torch.randn(N, generator=g) * 1e4; out.append(x)
    x = torch.randn(N, generator=g); x[0] = low; x[N - 1] = -low; out.append(x)
    return torch.stack(out).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [1, 2, 5, 31, 40, 64, 261, 1000, 2050, 4096, 9001, 40000, 131072])
def test_special_rows(dtype, N):
    x = special_rows(N, dtype)
    t = torch.full((x.shape[0],), N // 2)
    for K in (1, 20, 32):
        check(place(x), x, t, K)
    check(place(x, offset=1, row_stride=N + 1), x, t, 5)
    # A single row takes the mapping for few rows.
    for i in range(x.shape[0]):
        if N in (40000, 131072):
            check(place(x[i:i + 1]), x[i:i + 1], t[i:i + 1], 20)


def test_empty_inputs_and_missing_outputs():
    x, t = rows(4, 50, "f32", 1)
    s = L.lse_token_stats(x.cuda(), None, 0, entropy=False)
    assert s.logprob is None and s.entropy is None and s.lse.shape == (4,)
    s = L.lse_token_stats(torch.empty((0, 50), device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 3)
    assert s.top_index.shape == (0, 3) and s.lse.shape == (0,)
    s = L.lse_token_stats(torch.empty((3, 0), device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"), 2)
    assert torch.isnan(s.logprob).all() and torch.isnan(s.entropy).all()
    assert (s.lse == -np.inf).all() and (s.top_index == -1).all() and (s.top_logprob == -np.inf).all()
    one = L.lse_token_stats(x[0].cuda(), t[:1].cuda(), 4)
    assert one.lse.shape == () and one.top_index.shape == (4,)
    check(None, x[:1], t[:1], 4, L.TokenStats(*[v.reshape((1,) + v.shape) for v in one]))


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 bytes and 2^31 elements into the tensor."""
    N, rs, B = 5003, (1 << 28) + 3, 9
    buf = torch.empty(8 * rs + N, dtype=torch.bfloat16, device="cuda")
    x, t = rows(B, N, "bf16", 5)
    view = torch.as_strided(buf, (B, N), (rs, 1))
    view.copy_(x)
    s = check(view, x, t, 6)
    g = torch.linspace(-1, 1, B, device="cuda")
    d = L.lse_token_stats_backward(view, s, t.cuda(), grad_logprob=g, grad_entropy=g, dx=view)
    assert d.data_ptr() == buf.data_ptr()
    check_gradient(view.cpu(), x, s, t, g.cpu(), g.cpu(), None, None, "bf16")


def test_another_stream():
    x, t = rows(64, 30011, "bf16", 9)
    xd, td = x.cuda(), t.cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s = L.lse_token_stats(xd, td, 9, stream=st)
    g = torch.ones(64, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    d = L.lse_token_stats_backward(xd, s, td, grad_logprob=g, stream=st)
    st.synchronize()
    check(xd, x, t, 9, s)
    check_gradient(d.cpu(), x, s, t, g.cpu(), None, None, None, "bf16")


def test_graph_capture():
    x, t = rows(2, 128256, "bf16", 3)
    xd, td = x.cuda(), t.cuda()
    L.lse_token_stats(xd, td, 20)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = L.lse_token_stats(xd, td, 20)
    y, u = rows(2, 128256, "bf16", 4)
    xd.copy_(y)
    td.copy_(u)
    graph.replay()
    check(xd, y, u, 20, s)


# ---------------------------------------------------------------------------
# Gradient
# ---------------------------------------------------------------------------
def gradient_reference(x, lse, ent, target, idx, gl, gh, gt, gs):
    """The formula in float64 and the bar of the module's docstring (without the
    element type's rounding), for the f32 lse and entropy that the kernel has."""
    xd, l = x.double(), lse.double()[:, None]
    B, N = xd.shape
    z = torch.zeros(B, dtype=torch.float64)
    gl = z if gl is None else gl.double()
    if target is not None:
        ok = (target >= 0) & (target < N)
        gl = torch.where(ok, gl, 0.0)
    gh = z if gh is None else gh.double()
    gs = z if gs is None else gs.double()
    K = 0 if gt is None else gt.shape[1]
    unit = torch.zeros_like(xd)
    mag = torch.zeros_like(xd)
    c = gs - gl
    ca = gs.abs() + gl.abs()
    at = torch.arange(B)
    if target is not None:
        unit[at, target.clamp(0, N - 1)] += gl
        mag[at, target.clamp(0, N - 1)] += gl.abs()
    zero = (gl == 0) & (gh == 0) & (gs == 0)
    for k in range(K):
        i = idx[:, k]
        g = torch.where((i >= 0) & (i < N), gt[:, k].double(), 0.0)
        unit[at, i.clamp(0, N - 1)] += g
        mag[at, i.clamp(0, N - 1)] += g.abs()
        c = c - g
        ca = ca + g.abs()
        zero &= g == 0
    logp = xd - l
    p = torch.exp(logp)
    h = torch.where(gh != 0, ent.double() if ent is not None else 0.0, 0.0)[:, None]
    lp = logp.clamp(min=-16384.0)
    lp = torch.where(torch.isnan(logp), 0.0, lp)
    ref = p * (c[:, None] - gh[:, None] * (lp + h)) + unit
    G = ca[:, None] + gh.abs()[:, None] * (lp.abs() + h.abs())
    la = torch.nan_to_num(l.abs(), posinf=0)
    xa = torch.nan_to_num(xd.abs(), posinf=0).clamp(max=1e6)
    bar = p * G * (2.0 ** -21 + 2.0 ** -23 * (la + lp.abs())) \
        + p * 2.0 ** -22 * (G + gh.abs()[:, None] * (la + xa)) + 2.0 ** -22 * mag + 1e-37 * (G + mag)
    ref[zero] = 0.0
    bar[zero] = 0.0
    return ref, bar


def check_gradient(d, x, s, target, gl, gh, gt, gs, dtype):
    idx = s.top_index.cpu() if s.top_index is not None else None
    ent = s.entropy.cpu() if s.entropy is not None else None
    ref, bar = gradient_reference(x, s.lse.cpu(), ent, target if gl is not None else None, idx, gl, gh, gt, gs)
    got = d.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    fin = torch.isfinite(ref)
    lim = bar + Q[dtype] * ref.abs() + (2.0 ** -24 if dtype == "f16" else 2.0 ** -133 if dtype == "bf16" else 0)
    err = (got - ref).abs()
    bad = fin & ~(err <= lim)
    assert not bad.any(), (int(bad.sum()), [(tuple(i.tolist()), float(got[tuple(i)]), float(ref[tuple(i)]))
                                            for i in bad.nonzero()[:4]])


def gradients(B, K, seed):
    g = torch.Generator().manual_seed(seed)
    gl = torch.randn(B, generator=g)
    gh = torch.randn(B, generator=g) * 0.5
    gs = torch.randn(B, generator=g) * 0.1
    gt = torch.randn((B, K), generator=g) if K else None
    used = (torch.arange(B) % 4 != 1).float()
    return gl * used, gh * used, gt * used[:, None] if K else None, gs * used


def run_gradient(xd, x, t, K, dtype, parts="lhts", dx=None, seed=0):
    s = L.lse_token_stats(xd, t.cuda(), K)
    gl, gh, gt, gs = gradients(x.shape[0], K, seed)
    gl, gh = gl if "l" in parts else None, gh if "h" in parts else None
    gt, gs = gt if "t" in parts else None, gs if "s" in parts else None
    on = [None if v is None else v.cuda() for v in (gl, gh, gt, gs)]
    d = L.lse_token_stats_backward(xd, s, t.cuda(), *on, dx=dx)
    torch.cuda.synchronize()
    check_gradient(d.cpu(), x, s, t, gl, gh, gt, gs, dtype)
    return d


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [1, 2, 3, 7, 8, 9, 16, 17, 31, 33, 65, 130, 257, 261, 1000, 2049, 4097, 10007])
def test_gradient_lengths_and_layouts(dtype, N):
    x, t = rows(6, N, dtype, seed=N)
    t[3] = -1
    t[4] = N + 5
    for i, lay in enumerate(LAYOUTS):
        lay = dict(lay)
        if "row_stride" in lay:
            lay["row_stride"] += N
        run_gradient(place(x, **lay), x, t, (0, 4, 32)[(i + N) % 3], dtype, seed=i)
        # Into rows of another layout, and in place; nothing outside the rows changes.
        dx = place(torch.zeros_like(x), **lay)
        run_gradient(place(x), x, t, 5, dtype, dx=dx, seed=i)
        xd = place(x, **lay)
        run_gradient(xd, x, t, 5, dtype, dx=xd, seed=i)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradient_writes_its_rows_only(dtype):
    for N, rs, off in [(13, 20, 1), (261, 264, 0), (1003, 1010, 3), (40001, 40010, 2)]:
        x, t = rows(4, N, dtype, seed=N)
        buf = torch.full((off + 4 * rs + 64,), 7.0, dtype=DT[dtype], device="cuda")
        dx = buf[off:off + 4 * rs].reshape(4, rs)[:, :N]
        run_gradient(x.cuda(), x, t, 3, dtype, dx=dx)
        dx.fill_(7.0)
        assert (buf == 7.0).all()


@pytest.mark.parametrize("parts", ["l", "h", "t", "s", "lh", "lt", "hs"])
def test_gradient_parts(parts):
    for dtype, B, N, K in [("bf16", 9, 32000, 8), ("f32", 300, 261, 20), ("f16", 2, 128256, 32)]:
        x, t = rows(B, N, dtype, seed=B)
        run_gradient(x.cuda(), x, t, K, dtype, parts)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [5, 40, 261, 2050, 40000])
def test_gradient_special_rows(dtype, N):
    x = special_rows(N, dtype)
    t = torch.full((x.shape[0],), N // 2)
    run_gradient(place(x), x, t, 0, dtype, "l")
    run_gradient(place(x), x, t, min(N, 4), dtype, "lt")
    run_gradient(place(x), x, t, 0, dtype, "h")
    # Rows left out of the loss get zeros whatever they hold.
    s = L.lse_token_stats(x.cuda(), t.cuda(), 2)
    z = torch.zeros(x.shape[0], device="cuda")
    d = L.lse_token_stats_backward(x.cuda(), s, t.cuda(), z, z, torch.zeros((x.shape[0], 2), device="cuda"), z)
    assert (d == 0).all()


def test_target_among_the_alternatives_and_repeats():
    x, _ = rows(8, 500, "f32", 2)
    t = x.argmax(1)
    run_gradient(x.cuda(), x, t, 6, "f32")
    s = L.lse_token_stats(x.cuda(), t.cuda(), 3)
    s = s._replace(top_index=torch.stack([s.top_index[:, 0]] * 2 + [torch.full((8,), -1, device="cuda")], 1).contiguous())
    gl, gh, gt, gs = gradients(8, 3, 1)
    d = L.lse_token_stats_backward(x.cuda(), s, t.cuda(), gl.cuda(), gh.cuda(), gt.cuda(), gs.cuda())
    check_gradient(d.cpu(), x, s, t, gl, gh, gt, gs, "f32")


def test_gradient_against_differences():
    """Central differences of the 64-bit definition, step 1e-5: their error is about
    1e-10 / 1e-5 from rounding plus 1e-10 from the cubic term; f32 adds 1e-6 G."""
    x, t = rows(3, 23, "f32", 11, scale=1.0)
    K = 4
    gl, gh, gt, gs = (torch.randn(3), torch.randn(3), torch.randn(3, K), torch.randn(3))
    s = L.lse_token_stats(x.cuda(), t.cuda(), K)
    d = L.lse_token_stats_backward(x.cuda(), s, t.cuda(), gl.cuda(), gh.cuda(), gt.cuda(), gs.cuda())

    def f(xd):
        lse = torch.logsumexp(xd, 1)
        logp = xd - lse[:, None]
        ent = -(logp.exp() * logp).sum(1)
        top = logp.gather(1, s.top_index.cpu())
        return (gl * logp[torch.arange(3), t] + gh * ent + gs * lse).sum() + (gt * top).sum()

    x64 = x.double()
    for b in range(3):
        for n in range(23):
            e = torch.zeros_like(x64)
            e[b, n] = 1e-5
            num = (f(x64 + e) - f(x64 - e)) / 2e-5
            assert abs(float(num) - float(d[b, n])) < 2e-5


def test_autograd():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((2, 5, 301), generator=g).cuda().requires_grad_()
    t = torch.randint(0, 301, (2, 5), generator=g).cuda()
    s = L.token_stats(x, t, top_k=3)
    assert s.logprob.shape == (2, 5) and s.top_index.shape == (2, 5, 3)
    w = torch.randn((2, 5), generator=g).cuda()
    loss = (s.logprob * w).sum() - 0.1 * s.entropy.sum() + (s.top_logprob[..., 1] * w).sum() + s.lse.mean()
    loss.backward()
    y = x.detach().double().requires_grad_()
    logp = torch.log_softmax(y, -1)
    lp = logp.gather(-1, t[..., None])[..., 0]
    top = logp.gather(-1, s.top_index)
    ref = (lp * w).sum() + 0.1 * (logp.exp() * logp).sum() + (top[..., 1] * w).sum() \
        + torch.logsumexp(y, -1).mean()
    ref.backward()
    assert abs(float(loss) - float(ref)) < 1e-3
    assert (x.grad.double() - y.grad).abs().max() < 1e-5
    with torch.no_grad():
        assert not L.token_stats(x, t).logprob.requires_grad
    x2 = x.detach().requires_grad_()
    L.token_stats(x2, None).entropy.sum().backward()  # the other outputs carry no gradient
    assert torch.isfinite(x2.grad).all()


def test_second_derivatives_are_refused():
    x = torch.randn((3, 40), device="cuda", requires_grad=True)
    s = L.token_stats(x)
    (g,) = torch.autograd.grad(s.entropy.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_refusals():
    x = torch.zeros((4, 10), device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    s = L.lse_token_stats(x, t, 2)
    g = torch.zeros(4, device="cuda")
    for call in [
        lambda: L.lse_token_stats(x.cpu()),
        lambda: L.lse_token_stats(x, t, 33),
        lambda: L.lse_token_stats(x, t, -1),
        lambda: L.lse_token_stats(x, t.int()),
        lambda: L.lse_token_stats(x, t[:3]),
        lambda: L.lse_token_stats(x, t.cpu()),
        lambda: L.lse_token_stats(x.t(), None),
        lambda: L.lse_token_stats(x[None], None),
        lambda: L.lse_token_stats_backward(x, s, None, grad_logprob=g),
        lambda: L.lse_token_stats_backward(x, s._replace(entropy=None), t, grad_entropy=g),
        lambda: L.lse_token_stats_backward(x, s, t, grad_logprob=g.double()),
        lambda: L.lse_token_stats_backward(x, s, t, grad_top=g),
        lambda: L.lse_token_stats_backward(x, s._replace(lse=g[:2]), t, grad_lse=g),
        lambda: L.lse_token_stats_backward(x, s, t, grad_lse=g, dx=x.half()),
        lambda: L.lse_token_stats_backward(x, s, t, grad_lse=g, dx=x[:, :5]),
        lambda: L.lse_token_stats_backward(x.cpu(), s, t, grad_lse=g),
        lambda: L.token_stats(x.t()),
        lambda: L.token_stats(x, t[:, None]),
    ]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.lse_token_stats(x.double())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K", [(1500, 20), (2311, 8), (4000, 24), (4103, 1), (8191, 0), (5003, 32)])
def test_special_rows_by_the_thousand(dtype, N, K):
    """Many rows of middling length take a mapping of their own."""
    x = special_rows(N, dtype, seed=N)
    x = x.repeat(2600 // x.shape[0] + 1, 1)
    t = torch.randint(0, N, (x.shape[0],), generator=torch.Generator().manual_seed(N))
    xd = place(x, offset=1, row_stride=N + 3)
    check(xd, x, t, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K", [(1500, 32), (2311, 25), (4000, 31), (4100, 28), (8190, 32)])
def test_many_alternatives_by_the_thousand(dtype, N, K):
    """For K > 24 their bound comes from the kept 16-bit maxima: ties, masks, values that
    round up (to infinity too) and one column that holds nearly all of the row."""
    x = special_rows(N, dtype, seed=N)
    g = torch.Generator().manual_seed(N + K)
    more = torch.randn((8, N), generator=g)
    more[0] = torch.finfo(torch.float32).max * (1 - 2.0 ** -12 * torch.rand(N, generator=g)) if dtype == "f32" else 60000.0
    more[1] = 1.0 + 2.0 ** -9 * torch.rand(N, generator=g)     # one bf16 value, many f32 ones
    more[2] = -1.0 - 2.0 ** -9 * torch.rand(N, generator=g)
    more[3, :N - K] = -float("inf")                             # K left
    more[4, :N - K + 1] = -float("inf")                         # one too few
    more[5] = torch.arange(N) * 2.0 ** -6                       # the largest all at the end
    more[6] = -torch.arange(N) * 2.0 ** -6
    more[7] = torch.randint(0, 40, (N,), generator=g).float()
    x = torch.cat([x, more.to(DT[dtype])])
    x = x.repeat(2600 // x.shape[0] + 1, 1)
    t = torch.randint(0, N, (x.shape[0],), generator=torch.Generator().manual_seed(N))
    check(place(x, offset=2, row_stride=N + 1), x, t, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [1, 63, 64, 65, 250, 257, 511, 1020, 1030, 2047, 4100])
def test_gradient_of_many_short_rows(dtype, N):
    """A few lanes per row, each row's gradients among them alone."""
    x, t = rows(1300, N, dtype, seed=N)
    t[::7] = -100
    for i, K in enumerate((0, 7, 8, 9, 16, 17)):
        lay = dict(offset=i % 4, row_stride=N + (0, 1, 8)[i % 3])
        xd = place(x, **lay)
        dx = (None, xd, place(torch.zeros_like(x)))[i % 3]
        run_gradient(xd, x, t, min(K, N), dtype, dx=dx, seed=i)


def test_gradient_on_the_forward_stream():
    """autograd's own work runs on the current stream; the gradient kernel on the one that
    the forward was given, after the incoming gradients and before their use."""
    st = torch.cuda.Stream()
    x, t = rows(4000, 4096, "f32", 11)
    xd, td = x.cuda(), t.cuda()
    w = torch.randn(4000, device="cuda")
    want = []
    for stream in (None, st):
        leaf = xd.clone().requires_grad_()
        st.wait_stream(torch.cuda.current_stream())
        s = L.token_stats(leaf, td, 4, stream=stream)
        torch.cuda.current_stream().wait_stream(st)
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):  # the incoming gradient is late
            big = big @ big / 64
        y = (s.logprob + s.entropy) * (w + 0 * big[:4000, 0].nan_to_num(0.0, 0.0, 0.0))
        y.sum().backward()
        want.append(leaf.grad * 2)
    assert torch.equal(want[0], want[1])


@pytest.mark.parametrize("dtype,N,K", [("f32", 33001, 32), ("bf16", 66000, 20), ("f16", 65539, 0)])
def test_about_as_many_long_rows_as_processors(dtype, N, K):
    """Long rows of which each takes two blocks."""
    x = special_rows(N, dtype, seed=N)
    x = x.repeat(150 // x.shape[0] + 1, 1)[:150]
    t = torch.randint(0, N, (150,), generator=torch.Generator().manual_seed(N))
    check(place(x, offset=1, row_stride=N + 1), x, t, K)
