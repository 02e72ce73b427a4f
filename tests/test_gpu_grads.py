"""lse_grad_norm and lse_grad_clip against 64-bit sums.

Bars.  A thread adds at most 16 squares in a row in f32 before its sums go to 64
bits, so the sum of squares is off by a relative 16 * 2^-24 at most, the norm by half
of that, and it is rounded to f32: 1e-6.  Clipped values: the coefficient carries
the norm's error and three more roundings, then the element type's.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = 1e-6
Q = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -148, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def norm64(ts):
    """The norm from 64-bit sums, as the f32 value that holds it."""
    norm = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))
    return float(torch.tensor(norm, dtype=torch.float64).float())


def check_norm(got, ts):
    want = norm64(ts)
    assert float(got) == want or abs(float(got) - want) <= REL * want, (float(got), want)
    return want


def check_clipped(outs, ins, want_norm, max_norm, eps=1e-6):
    c = min(1.0, max_norm / (want_norm + eps))
    for o, i in zip(outs, ins):
        ref = i.double() * c
        if c == 1.0:
            assert torch.equal(o, i)
            continue
        lim = ref.abs() * (2 * REL + Q[o.dtype]) + TINY[o.dtype]
        assert ((o.double() - ref).abs() <= lim).all(), (o.shape, o.dtype)


def make(sizes, dtypes, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(DT[dtypes[i % len(dtypes)]]).cuda()
            for i, n in enumerate(sizes)]


SIZES = [[1], [0, 5, 0], [7, 1, 31, 33], [255, 256, 257, 1000], [16384, 16385, 16383, 3],
         [100003, 17, 65536, 1], [5000000, 12, 4097], [3] * 1000, list(range(2100))]


@pytest.mark.parametrize("dtypes", [["f32"], ["bf16"], ["f16"], ["f32", "bf16", "f16"]])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_sizes(dtypes, case):
    ts = make(SIZES[case], dtypes, case)
    want = check_norm(L.lse_grad_norm(ts), ts)
    for max_norm in (want * 0.3, want * 3 + 1, 0.0):
        outs = [torch.empty_like(t) for t in ts]
        got = L.lse_grad_clip(L.GradList(ts, outs), max_norm)
        check_norm(got, ts)
        check_clipped(outs, ts, want, max_norm)
        here = [t.clone() for t in ts]
        got2 = L.lse_grad_clip(here, max_norm)
        assert torch.equal(got, got2)
        for a, b in zip(here, outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_unaligned_views_and_neighbours(dtype):
    """Slices at every offset of a buffer: all of each is scaled, nothing else."""
    sizes = [1, 2, 3, 5, 8, 13, 21, 100, 257, 1021, 5003, 20011]
    buf = torch.full((sum(sizes) + 3 * len(sizes) + 64,), 2.0, device="cuda", dtype=DT[dtype])
    views, at = [], 1
    for n in sizes:
        views.append(buf[at:at + n])
        at += n + 3
    inside = torch.zeros_like(buf, dtype=torch.bool)
    for v in views:
        o = (v.data_ptr() - buf.data_ptr()) // buf.element_size()
        inside[o:o + v.numel()] = True
    before = [v.clone() for v in views]
    want = check_norm(L.lse_grad_norm(views), before)
    # Into buffers at other offsets from a 16-byte boundary.
    outs = [torch.zeros(n + 9, device="cuda", dtype=DT[dtype])[i % 8:i % 8 + n] for i, n in enumerate(sizes)]
    L.lse_grad_clip(L.GradList(views, outs), want / 7)
    check_clipped(outs, before, want, want / 7)
    L.lse_grad_clip(views, want / 7)
    check_clipped(views, before, want, want / 7)
    assert (buf[~inside] == 2.0).all()


@pytest.mark.parametrize("scale", [1e30, 3e37, 1e-20, 1e-30, 1e-42, 0.0])
def test_range(scale):
    """Squares beyond the f32 range in both directions, and mixtures."""
    ts = make([1000, 70001, 3], ["f32"], 5, scale)
    check_norm(L.lse_grad_norm(ts), ts)
    b = make([1000, 70001], ["bf16"], 6, scale)
    check_norm(L.lse_grad_norm(b), b)
    mixed = ts + make([5000, 3], ["f16", "bf16"], 7, 1e-3)
    check_norm(L.lse_grad_norm(mixed), mixed)
    spike = torch.full((100000,), 1e-25, device="cuda")
    spike[777] = 1e-12
    check_norm(L.lse_grad_norm([spike]), [spike])


def test_infinite_and_nan():
    a = torch.randn(5000, device="cuda")
    bad = a.clone()
    bad[4321] = float("inf")
    assert float(L.lse_grad_norm([a, bad])) == float("inf")
    here = [a.clone(), bad.clone()]
    L.lse_grad_clip(here, 1.0)
    assert (here[0] == 0).all() and torch.isnan(here[1][4321]) and (here[1][:4321] == 0).all()
    bad[17] = float("nan")
    assert math.isnan(float(L.lse_grad_norm([bad.bfloat16(), a])))
    here = [a.clone(), bad.clone()]
    L.lse_grad_clip(here, 1.0)
    assert torch.isnan(here[0]).all()
    # The norm itself beyond f32.
    assert float(L.lse_grad_norm([torch.full((100,), 3e38, device="cuda")])) == float("inf")


def test_shapes_and_orders():
    x = torch.randn(6, 50, 40, device="cuda")
    ts = [x.permute(2, 0, 1), torch.randn(3, 4, device="cuda"), torch.randn(64, 64, device="cuda").t()]
    want = check_norm(L.lse_grad_norm(ts), ts)
    before = [t.clone() for t in ts]
    L.lse_grad_clip(ts, want / 2)
    check_clipped(ts, before, want, want / 2)


def test_same_bits_every_time():
    ts = make([400001, 77, 900000], ["bf16", "f32"], 1)
    first = L.lse_grad_norm(ts)
    for _ in range(5):
        assert torch.equal(L.lse_grad_norm(ts), first)


def test_another_stream_and_graph():
    ts = make([300001, 5], ["f32"], 2)
    lst = L.GradList(ts, [torch.empty_like(t) for t in ts])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    n = L.lse_grad_clip(lst, 0.5, stream=st)
    st.synchronize()
    want = check_norm(n, ts)
    check_clipped(lst.out, ts, want, 0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = L.lse_grad_clip(lst, 0.25)
    ts[0].mul_(2.0)
    graph.replay()
    want = check_norm(n, ts)
    check_clipped(lst.out, ts, want, 0.25)


def test_beyond_32_bits():
    t = torch.full(((1 << 32) + 5,), 0.5, dtype=torch.bfloat16, device="cuda")
    n = L.lse_grad_clip([t], 0.25 * math.sqrt(float(t.numel())))
    want = 0.5 * math.sqrt(float(t.numel()))
    assert abs(float(n) - want) <= REL * want
    assert (t[-5:] == 0.25).all() and (t[(1 << 31) - 3:(1 << 31) + 3] == 0.25).all() and t[0] == 0.25


def test_empty_views_next_to_their_tensor():
    t = torch.randn(1000, device="cuda")
    check_norm(L.lse_grad_norm([t[:0], t, t[:0]]), [t])


def test_refusals():
    a = torch.zeros(4, device="cuda")
    for call in [lambda: L.lse_grad_norm([]), lambda: L.lse_grad_norm([a.cpu()]),
                 lambda: L.lse_grad_norm([a, a]), lambda: L.lse_grad_norm([torch.zeros(4, 4, device="cuda")[:, :2]]),
                 lambda: L.lse_grad_norm([a.expand(3, 4)]),
                 lambda: L.GradList([a], []), lambda: L.GradList([a], [a[:3]]),
                 lambda: L.GradList([a], [a.half()]),
                 lambda: L.GradList([torch.zeros(3, 4, device="cuda").t()], [torch.zeros(4, 3, device="cuda")])]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.lse_grad_norm([a.double()])
    for bad in (-1.0, float("nan")):
        with pytest.raises(L.LseError):
            L.lse_grad_clip([a], bad)
    with pytest.raises(L.LseError):
        L.lse_grad_clip([a], 1.0, eps=-1.0)


def test_lists_that_share_memory_are_refused():
    buf = torch.zeros(1000, device="cuda")
    with pytest.raises(ValueError, match="share memory"):
        L.GradList([buf[:600], buf[599:]])
    with pytest.raises(ValueError, match="share memory"):
        L.GradList([buf[:300], buf[300:600]], [buf[600:900], buf[200:500]])
    L.GradList([buf[:600], buf[600:], buf[:0]])
    L.GradList([buf[:300], buf[300:600]], [buf[:300], buf[600:900]])
