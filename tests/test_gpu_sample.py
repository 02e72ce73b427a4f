"""lse_sample against the definition in 64 bits: tokens are equal.

A token is left open only where the drawn number lies within 4e-9 of the sum from one of its
borders (weights are off by up to 2^-30 of themselves on either side), and the threshold of
top-p where a sum lies as near to its target; the cases are drawn from seeds, and a row that
is left open has to give one of the two tokens.  logprob: two f32 roundings of quantities
no larger than |z| + |log sum|, and an f32 logarithm: 2^-21 of their magnitudes.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
OPEN = 4e-9


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def column(v, B):
    v = v.cpu() if isinstance(v, torch.Tensor) else torch.full((B,), float(v))
    return v.to(torch.float32).double()


def reference(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(tokens, alternative tokens, logprob, magnitude of the logprob's terms) row by row."""
    x64, u64 = x.double().cpu(), u.double().cpu()
    B, N = x64.shape
    t, k, p, low = (column(v, B) for v in (temperature, top_k, top_p, min_p))
    out = []
    for b in range(B):
        r = x64[b]
        if N == 0 or torch.isnan(r).any() or not math.isfinite(float(r.max())) or not 0 <= float(t[b]) <= 1e20 \
                or math.isnan(float(p[b])) or math.isnan(float(low[b])):
            out.append((-1, -1, math.nan, 0.0))
            continue
        m = r.max()
        if float(t[b]) < 1e-20:
            a = int((r == m).nonzero()[0])
            out.append((a, a, 0.0, 0.0))
            continue
        order = torch.sort(r, descending=True, stable=True).indices
        z = (r - m) / t[b]
        w = torch.exp(z)[order]
        kk = int(k[b])
        if 0 < kk < N:
            w[kk:] = 0
        choices = []
        for nudge in (-OPEN, 0.0, OPEN):
            v = w.clone()
            if float(p[b]) < 1:
                before = torch.cumsum(v, 0) - v
                keep = before < (p[b] + nudge * (nudge != 0)) * v.sum()
                keep[0] = True
                v = torch.where(keep, v, torch.zeros_like(v))
            if float(low[b]) > 0:
                v = torch.where(r[order] - m >= t[b] * math.log(min(float(low[b]), 1.0)), v, torch.zeros_like(v))
            back = torch.zeros_like(v).scatter_(0, order, v)
            run = torch.cumsum(back, 0)
            uu = min(max(float(u64[b]), 0.0), 1.0) if not math.isnan(float(u64[b])) else 0.0
            border = uu * run[-1] + nudge * run[-1]
            if uu >= 1.0:
                at = int((back > 2.0 ** -44).nonzero()[-1])
            else:
                at = int(torch.searchsorted(run, border.clamp(min=0.0), right=True).clamp(max=N - 1))
                at = min(at, int((back > 0).nonzero()[-1]))
            choices.append((at, float(z[at] - torch.log(run[-1])), float(z[at].abs() + torch.log(run[-1]).abs())))
        out.append((choices[1][0], {c[0] for c in choices}, choices[1][1], choices[1][2]))
    return out


def check(x, u, **settings):
    got = L.lse_sample(x, u, **settings)
    left_open = 0
    for b, (token, others, logprob, mag) in enumerate(reference(x, u, **settings)):
        g = int(got.token[b])
        if token == -1:
            assert g == -1 and math.isnan(float(got.logprob[b])), b
            continue
        if g != token:
            assert g in others, (b, g, token, others, {k: (v[b] if isinstance(v, torch.Tensor) else v) for k, v in settings.items()})
            left_open += 1
            continue
        assert abs(float(got.logprob[b]) - logprob) <= 2.0 ** -21 * (1 + mag), (b, float(got.logprob[b]), logprob)
    assert left_open <= 1
    again = L.lse_sample(x, u, **settings)
    assert torch.equal(again.token, got.token) and torch.equal(again.logprob.nan_to_num(7.0), got.logprob.nan_to_num(7.0))
    return got


def logits(B, N, dtype, seed, spread=3.0, peak=9.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, N), generator=g) * spread + torch.rand((B, 1), generator=g) * 40 - 20
    if N > 1:
        x[torch.arange(B), torch.randint(0, N, (B,), generator=g)] += peak
    return x.to(DT[dtype]).cuda(), torch.rand(B, generator=g).cuda()


SETTINGS = [dict(), dict(temperature=0.7, top_k=50, top_p=0.95), dict(top_p=0.9), dict(temperature=1.3, min_p=0.02),
            dict(top_k=5), dict(temperature=0.0), dict(temperature=2.0, top_k=200, top_p=0.8, min_p=0.01), dict(top_p=0.3),
            dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0), dict(temperature=0.05), dict(temperature=30.0, top_p=0.99)]
WIDTHS = [1, 2, 3, 7, 31, 32, 33, 100, 261, 500, 1000, 1023, 2049, 4097, 8200, 20011]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_widths(dtype, N):
    x, u = logits(13, N, dtype, N)
    for s in SETTINGS:
        check(x, u, **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,N", [(3, 50257), (2, 128256), (700, 33000)])
@pytest.mark.parametrize("spread,peak", [(3.0, 9.0), (0.5, 0.0)])
def test_long_rows(dtype, B, N, spread, peak):
    x, u = logits(B, N, dtype, N, spread, peak)
    few = slice(0, 6)
    for s in [dict(), dict(top_p=0.9), dict(temperature=0.7, top_k=50, top_p=0.95), dict(top_k=3001, top_p=0.99), dict(min_p=0.05)]:
        if B <= 6:
            check(x, u, **s)
            continue
        got = L.lse_sample(x, u, **s)
        part = check(x[few], u[few], **s)
        assert torch.equal(got.token[few], part.token) and torch.equal(got.logprob[few], part.logprob)
        assert (got.token >= 0).all() and (got.token < N).all()


def test_rows_of_more_than_a_million():
    x, u = logits(2, 3_000_001, "bf16", 5)
    for s in (dict(), dict(top_p=0.9), dict(top_k=40), dict(temperature=0.0)):
        check(x, u, **s)


@pytest.mark.parametrize("N", [200, 5000, 60001])
def test_settings_of_each_row(N):
    B = 60
    x, u = logits(B, N, "bf16", N)
    g = torch.Generator().manual_seed(N)

    def pick(values, dtype=torch.float32):
        return torch.tensor(values, dtype=dtype)[torch.randint(0, len(values), (B,), generator=g)].cuda()

    t = pick([0.0, 0.3, 0.8, 1.0, 1.7, -1.0, float("nan"), 1e30, 1e-30])
    check(x, u, temperature=t, top_k=pick([0, 1, 20, 1000, -3, 1 << 40], torch.int64), top_p=pick([1.0, 0.9, 0.5, 0.0, 2.0]),
          min_p=pick([0.0, 0.05, 1.0, 3.0]))
    check(x, u, top_p=pick([0.5, float("nan")]), temperature=0.9)
    check(x, u, min_p=pick([0.05, float("nan")]), top_k=30)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [40, 3000, 40000])
def test_masks_and_special_rows(dtype, N):
    low = torch.finfo(DT[dtype]).min
    x, u = logits(16, N, dtype, 1)
    x[0] = -math.inf
    x[1] = low
    x[2, :] = -math.inf
    x[2, N // 2] = low
    x[3, 3] = math.nan
    x[4, 5] = math.inf
    x[5, 1:] = -math.inf
    x[6, : N - 1] = low
    x[7, ::2] = -math.inf
    x[8] = 0.0
    x[9, N // 3:] = x[9, 0]
    x[10, : N // 2] = low
    x[11] = 2.0
    x[11, N - 1] = -0.0
    x[12, 0] = torch.finfo(DT[dtype]).max
    x[13, 7] = -math.nan
    for s in SETTINGS:
        check(x, u, **s)


@pytest.mark.parametrize("N", [64, 5000, 70000])
def test_equal_values(N):
    """Rows of equal values: cuts go by column, and borders are exact."""
    B = 24
    x = torch.zeros((B, N), dtype=torch.bfloat16, device="cuda")
    x[B // 2:] = torch.where(torch.arange(N, device="cuda") % 3 == 1, 1.5, -0.5)
    u = torch.linspace(0, 1, B, device="cuda")
    u[-1] = 1.0 - 2.0 ** -24
    u[:4] = torch.tensor([0.0, 0.5, 0.25, 0.125])
    for s in (dict(), dict(top_k=N // 2), dict(top_k=N - 1), dict(top_p=0.5), dict(top_p=0.25), dict(top_p=0.7), dict(min_p=0.5),
              dict(top_k=N // 2, top_p=0.5)):
        check(x, u, **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [64, 230, 628, 1653, 4096, 8669, 21247, 70001])
def test_few_distinct_values(dtype, N):
    """Cuts that fall into runs of equal values, close to the run's end: more elements than any
    list, and sums that differ by less than the bins of a histogram are wide."""
    B = 10
    g = torch.Generator().manual_seed(N)
    x = torch.empty((B, N))
    for b, values in enumerate([2, 3, 5, 40]):
        x[b] = torch.randint(0, values, (N,), generator=g) * 3.0
    x[4] = torch.randint(0, 3, (N,), generator=g) * 0.01
    x[5], x[6], x[7], x[8] = -20.0, -20.0, 100.0, 0.0
    x[5, N // 3], x[6, N // 2], x[6, 7], x[7, 9] = 0.5, -2.4375, -2.375, 50.0
    x[8, N // 4: N // 4 + 40] = 3.0
    x[9] = torch.where(torch.rand(N, generator=g) < 0.6, -math.inf, x[1])
    x = x.to(DT[dtype]).cuda()
    u = torch.rand(B, generator=g).cuda()
    for s in (dict(top_p=0.95), dict(top_p=0.99, temperature=1.3), dict(top_p=0.999999), dict(top_p=0.95, min_p=1e-4),
              dict(top_k=N - 1, top_p=0.95), dict(top_k=3, top_p=0.999999), dict(top_p=0.7)):
        check(x, u, **s)


@pytest.mark.parametrize("N,k", [(125, 124), (700, 600), (5000, 3000)])
def test_nearly_equal_weights(N, k):
    """At a temperature of 1e10 half of an even count of tokens is a border to 1e-9: one more or not."""
    x, u = logits(6, N, "f16", N)
    got = L.lse_sample(x, u, temperature=1e10, top_k=k, top_p=0.5)
    assert (got.token >= 0).all()
    kept = torch.exp(-got.logprob.double())
    assert ((kept - k / 2 > -1e-2 * k / 2 / 50) & (kept - k / 2 < 1 + 1e-2 * k / 2 / 50)).all(), kept
    for b in range(6):
        order = torch.sort(x[b].double(), descending=True, stable=True).indices
        assert int(got.token[b]) in order[: k // 2 + 1].tolist()


@pytest.mark.parametrize("N", [300, 5000, 70000])
def test_numbers_of_zero_and_light_columns(N):
    """u = 0 draws the first column that weighs 2^-45 or more, behind many that weigh less."""
    x = torch.full((3, N), -31.5, device="cuda")  # 2^-45.4
    x[0, N - 1] = 0.0
    x[1, N // 2] = -10.0
    x[1, N - 1] = 0.0
    x[2, 0] = 0.0
    u = torch.tensor([0.0, 0.0, 1.0 - 2.0 ** -24], device="cuda")
    for s in (dict(), dict(temperature=0.9), dict(top_k=N - 1)):
        got = L.lse_sample(x, u, **s)
        assert got.token.tolist() == [N - 1, N // 2, 0], got.token
        assert (got.logprob <= 0).all()


def test_numbers_outside_the_unit_interval():
    x, _ = logits(6, 500, "f32", 2)
    u = torch.tensor([-1.0, math.nan, 1.0, 2.0, math.inf, 0.0], device="cuda")
    check(x, u)
    check(x, u, top_k=10)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [50, 301, 5003])
def test_strides_and_offsets(dtype, N):
    for stride, off in [(N + 8, 8), (N + 1, 1), (N + 5, 3)]:
        buf = torch.full((9 * stride + 64,), math.nan, dtype=DT[dtype], device="cuda")
        x = buf[off:off + 9 * stride].reshape(9, stride)[:, :N]
        v, u = logits(9, N, dtype, off)
        x.copy_(v)
        want = L.lse_sample(v, u, temperature=0.9, top_p=0.9)
        got = check(x, u, temperature=0.9, top_p=0.9)
        assert torch.equal(got.token, want.token)
        check(x, u)
    one = L.lse_sample(x[0], u[:1])
    assert one.token.dim() == 0 and one.logprob.dim() == 0


def test_frequencies():
    """Over evenly spaced numbers every token is drawn as often as its probability says."""
    N, B = 37, 4096
    row = torch.randn(N, generator=torch.Generator().manual_seed(1)) * 2
    u = ((torch.arange(B) + 0.5) / B).cuda()
    got = L.lse_sample(row.expand(B, N).contiguous().cuda(), u, temperature=1.1)
    count = torch.bincount(got.token.cpu(), minlength=N)
    p = torch.softmax(row.double() / torch.tensor(1.1).double(), 0)
    assert ((count - B * p).abs() <= 1.0).all()
    assert (torch.diff(got.token.cpu()) >= 0).all()


def test_close_borders():
    """Numbers next to the borders of tokens, where 32-bit sums would give a neighbour."""
    N, B = 20000, 300
    row = torch.randn(N, generator=torch.Generator().manual_seed(3))
    p = torch.softmax(row.double(), 0)
    run = torch.cumsum(p, 0)
    at = torch.randint(0, N - 1, (B,), generator=torch.Generator().manual_seed(4))
    u = run[at].float()
    x = row.expand(B, N).contiguous().cuda()
    got = L.lse_sample(x, u.cuda()).token.cpu()
    want = torch.searchsorted(run, u.double(), right=True)
    far = (u.double() - run[at]).abs() > OPEN  # (an f32 number is 3e-8 from a border on average)
    assert far.sum() > 200 and torch.equal(got[far], want[far])


def test_no_columns_and_no_rows():
    s = L.lse_sample(torch.empty((3, 0), device="cuda"), torch.rand(3, device="cuda"))
    assert (s.token == -1).all() and torch.isnan(s.logprob).all()
    assert L.lse_sample(torch.empty((0, 5), device="cuda"), torch.empty(0, device="cuda")).token.shape == (0,)


def test_beyond_32_bits():
    B, N = 20000, 128256
    x = torch.zeros((B, N), dtype=torch.bfloat16, device="cuda")
    x[B - 1, N - 5] = 60.0
    x[B - 2, 17] = 60.0
    got = L.lse_sample(x, torch.full((B,), 0.5, device="cuda"), top_p=0.5)
    assert int(got.token[B - 1]) == N - 5 and int(got.token[B - 2]) == 17
    assert (got.token[:B - 2] == N // 4).all()


def test_another_stream_and_graph():
    x, u = logits(40, 5003, "bf16", 1)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = L.lse_sample(x, u, top_p=0.9, stream=st)
    st.synchronize()
    want = L.lse_sample(x, u, top_p=0.9)
    assert torch.equal(got.token, want.token)
    graph = torch.cuda.CUDAGraph()
    k = torch.full((40,), 7, dtype=torch.int64, device="cuda")
    with torch.cuda.graph(graph):
        got = L.lse_sample(x, u, top_k=k)
    x.copy_(logits(40, 5003, "bf16", 2)[0])
    k.fill_(3)
    graph.replay()
    assert torch.equal(got.token, L.lse_sample(x, u, top_k=3).token)


def test_refusals():
    x, u = logits(4, 30, "f32", 1)
    for call in [lambda: L.lse_sample(x, u[:3]), lambda: L.lse_sample(x, u.double()), lambda: L.lse_sample(x, u.cpu()),
                 lambda: L.lse_sample(x.t(), u), lambda: L.lse_sample(x, u, temperature=-1.0),
                 lambda: L.lse_sample(x, u, temperature=math.nan), lambda: L.lse_sample(x, u, temperature=1e21),
                 lambda: L.lse_sample(x, u, top_k=-1), lambda: L.lse_sample(x, u, top_p=-0.1),
                 lambda: L.lse_sample(x, u, min_p=math.nan), lambda: L.lse_sample(x, u, top_k=u),
                 lambda: L.lse_sample(x, u, temperature=u[:2]), lambda: L.lse_sample(x, u, top_p=u.double())]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.lse_sample(x.double(), u)
