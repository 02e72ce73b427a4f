"""lse_embedding (exact) and lse_embedding_backward against 64-bit sums.

The lookup multiplies and rounds once, as torch does on the f32 value: bits are
equal.  Gradient: a row of n tokens is summed in f32, off by at most n 2^-24 of
the sum of magnitudes, times the scale, then rounded to the table's type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
Q = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def spread(rows, D, dtype, seed, stride=None, offset=0, fill=float("nan")):
    """A random [rows, D] matrix whose rows lie ``stride`` apart in a larger buffer."""
    stride = D if stride is None else stride
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((offset + rows * stride + 32,), fill, dtype=DT[dtype])
    v = buf[offset:offset + rows * stride].reshape(rows, stride)[:, :D]
    v.copy_(torch.randn((rows, D), generator=g))
    buf = buf.cuda()
    return buf, buf[offset:offset + rows * stride].reshape(rows, stride)[:, :D]


def tokens(T, V, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.exp(torch.rand(T, generator=g, dtype=torch.float64) * np.log(V + 1)).long().sub(1).clamp(0, V - 1)


WIDTHS = [1, 2, 3, 7, 8, 9, 16, 33, 64, 100, 128, 255, 256, 512, 1000, 1001, 1024, 2048, 4104, 8200]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_lookup(dtype, D):
    V = 57
    for T, stride, off, ostride, ooff in [(1, D, 0, D, 0), (9, D + 8, 0, D + 8, 8), (33, D + 1, 1, D + 3, 1),
                                          (400, D, 3, D, 0)]:
        _, table = spread(V, D, dtype, D, stride, off)
        ids = tokens(T, V, T).cuda()
        ids[0] = V - 1
        if T > 5:
            ids[3], ids[4], ids[5] = -1, V, 1 << 40
        obuf, out = spread(T, D, dtype, 1, ostride, ooff, fill=7.0)
        for scale in (1.0, 45.25):
            got = L.lse_embedding(table, ids, scale, out=out)
            ok = (ids >= 0) & (ids < V)
            want = (table[ids.clamp(0, V - 1)].float() * scale).to(DT[dtype])
            assert torch.equal(got[ok], want[ok])
            assert torch.isnan(got[~ok]).all()
        out.fill_(7.0)
        assert (obuf == 7.0).all()
    assert L.lse_embedding(table, ids.reshape(2, 200)).shape == (2, 200, D)


def check_gradient(got, grad, ids, V, scale, padding=-1, base=None):
    ids, g = ids.cpu(), grad.double().cpu()
    keep = (ids >= 0) & (ids < V) & (ids != padding)
    D = g.shape[1]
    want = torch.zeros((V, D), dtype=torch.float64).index_add_(0, ids[keep], g[keep]) * scale
    mag = torch.zeros((V, D), dtype=torch.float64).index_add_(0, ids[keep], g[keep].abs()) * abs(scale)
    n = torch.bincount(ids[keep], minlength=V).double()[:, None]
    if base is not None:
        want += base.double().cpu()
        mag += base.double().cpu().abs()
    lim = mag * (n + 4) * 2.0 ** -24 + want.abs() * Q[got.dtype] + TINY[got.dtype] * (n > 0)
    err = (got.double().cpu() - want).abs()
    assert (err <= lim).all(), (int((~(err <= lim)).sum()), float(err.max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_gradient_widths(dtype, D):
    V, T = 61, 300
    ids = tokens(T, V, D)
    ids[5], ids[6], ids[7] = -1, V, 1 << 33
    for stride, off, dstride, doff in [(D, 0, D, 0), (D + 8, 8, D + 8, 0), (D + 1, 1, D + 3, 2)]:
        _, grad = spread(T, D, dtype, D, stride, off)
        buf, dt = spread(V, D, dtype, 3, dstride, doff, fill=5.0)
        got = L.lse_embedding_backward(grad, ids.cuda(), V, 0.75, padding=2, dtable=dt)
        check_gradient(got, grad, ids, V, 0.75, padding=2)
        dt.fill_(5.0)
        assert (buf == 5.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V", [(0, 10), (1, 1), (1, 70000), (31, 5), (1000, 100000), (4097, 300), (20000, 50257),
                                 (70001, 1000), (65536, 128256), (150000, 70000)])
def test_gradient_tokens(dtype, T, V):
    D = 40
    g = torch.Generator().manual_seed(T)
    grad = torch.randn((T, D), generator=g).to(DT[dtype]).cuda()
    ids = tokens(T, V, T + 1) if T else torch.empty(0, dtype=torch.int64)
    got = L.lse_embedding_backward(grad, ids.cuda(), V, 2.0)
    check_gradient(got, grad, ids, V, 2.0)
    assert torch.equal(got, L.lse_embedding_backward(grad, ids.cuda(), V, 2.0))
    wide = torch.empty((V, D), device="cuda")
    L.lse_embedding_backward(grad, ids.cuda(), V, 2.0, dtable=wide)
    check_gradient(wide, grad, ids, V, 2.0)


@pytest.mark.parametrize("make", ["one", "two", "ascending", "descending", "none", "ends"])
@pytest.mark.parametrize("T", [5, 64, 1000, 9001])
def test_gradient_of_few_and_many(make, T):
    V, D = 20000, 264
    ids = {"one": torch.full((T,), 4321), "two": torch.arange(T) % 2 * 19999,
           "ascending": torch.arange(T) % V, "descending": (V - 1 - torch.arange(T)) % V,
           "none": torch.full((T,), -1), "ends": torch.where(torch.arange(T) < T // 2, 0, V - 1)}[make]
    grad = torch.randn((T, D), generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    got = L.lse_embedding_backward(grad, ids.cuda(), V)
    check_gradient(got, grad, ids, V, 1.0)


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("D", [72, 333])
def test_accumulate(dtype, out, D):
    V, T = 5000, 3000
    ids = tokens(T, V, 4)
    _, grad = spread(T, D, dtype, 1)
    _, dt = spread(V, D, out, 2)
    base = dt.clone()
    L.lse_embedding_backward(grad, ids.cuda(), V, 0.5, dtable=dt, accumulate=True)
    untouched = torch.ones(V, dtype=torch.bool)
    untouched[ids] = False
    assert torch.equal(dt[untouched.cuda()], base[untouched.cuda()])
    check_gradient(dt, grad, ids, V, 0.5, base=base)


def test_gradient_against_differences():
    """The lookup is linear in the table: differences of <g, out> are exact up to
    rounding (64-bit lookup, step 1)."""
    V, D, T = 7, 5, 12
    ids = tokens(T, V, 8)
    g = torch.randn((T, D))
    got = L.lse_embedding_backward(g.cuda(), ids.cuda(), V, 1.5).cpu()
    for v in range(V):
        for d in range(D):
            e = torch.zeros((V, D), dtype=torch.float64)
            e[v, d] = 1.0
            diff = float((g.double() * e[ids] * 1.5).sum())
            assert abs(diff - float(got[v, d])) < 1e-5


def test_autograd():
    table = torch.randn((50, 24), device="cuda", requires_grad=True)
    ids = torch.randint(0, 50, (3, 7), device="cuda")
    ids[1, 2] = 9
    out = L.embedding(ids, table, scale=3.0, padding=9)
    w = torch.randn_like(out)
    (out * w).sum().backward()
    y = table.detach().clone().requires_grad_()
    ref = torch.nn.functional.embedding(ids, y, padding_idx=9) * 3.0
    (ref * w).sum().backward()
    assert torch.equal(out, ref)
    assert (table.grad - y.grad).abs().max() < 1e-4


def test_another_stream_and_graph():
    grad = torch.randn((5000, 128), device="cuda").bfloat16()
    ids = tokens(5000, 9000, 1).cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = L.lse_embedding_backward(grad, ids, 9000, stream=st)
    st.synchronize()
    check_gradient(got, grad, ids, 9000, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = L.lse_embedding_backward(grad, ids, 9000)
    ids.copy_(tokens(5000, 9000, 2))
    graph.replay()
    check_gradient(got, grad, ids, 9000, 1.0)


def test_beyond_32_bits():
    V, D = 300000, 8192
    dt = torch.full((V, D), 3.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 5, V - 1, 280000], device="cuda")
    grad = torch.randn((4, D), device="cuda").bfloat16()
    L.lse_embedding_backward(grad, ids, V, dtable=dt)
    want = (grad[0].float() + grad[2].float()).bfloat16()
    assert torch.equal(dt[V - 1], want) and torch.equal(dt[5], grad[1]) and torch.equal(dt[280000], grad[3])
    assert (dt[6:280000:997] == 0).all() and (dt[280001:V - 1:97] == 0).all() and (dt[:5] == 0).all()
    out = L.lse_embedding(dt, ids)
    assert torch.equal(out[0], want) and torch.equal(out[3], grad[3])


def test_refusals():
    t = torch.zeros((5, 8), device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    g = torch.zeros((3, 8), device="cuda")
    for call in [lambda: L.lse_embedding(t.cpu(), ids), lambda: L.lse_embedding(t, ids.int()),
                 lambda: L.lse_embedding(t.t(), ids), lambda: L.lse_embedding(t[0], ids),
                 lambda: L.lse_embedding(t, ids, out=t), lambda: L.lse_embedding(t, ids, out=g.half()),
                 lambda: L.lse_embedding_backward(g, ids[:2], 5), lambda: L.lse_embedding_backward(g.cpu(), ids, 5),
                 lambda: L.lse_embedding_backward(g, ids, 5, accumulate=True),
                 lambda: L.lse_embedding_backward(g, ids, 5, dtable=t[:4]),
                 lambda: L.lse_embedding_backward(g, ids, 5, dtable=t.half())]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.lse_embedding(t.double(), ids)


def test_gradient_on_the_forward_stream():
    st = torch.cuda.Stream()
    table = torch.randn(9000, 256, device="cuda")
    ids = torch.randint(0, 9000, (20000,), device="cuda")
    w = torch.randn(20000, 256, device="cuda")
    want = []
    for stream in (None, st):
        leaf = table.clone().requires_grad_()
        if stream is not None:
            st.wait_stream(torch.cuda.current_stream())
        out = L.embedding(ids, leaf, scale=0.5, stream=stream)
        torch.cuda.current_stream().wait_stream(st)
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):  # the incoming gradient is late
            big = big @ big / 64
        (out * w * (1 + 0 * big[0, 0].nan_to_num(0.0, 0.0, 0.0))).sum().backward()
        want.append(leaf.grad * 2)
    assert torch.equal(want[0], want[1])


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 255, 257, 1000, 4095, 4096, 4097, 8193])
@pytest.mark.parametrize("V,D", [(1, 40), (7, 33), (300, 64), (20011, 96)])
def test_gradient_of_few_tokens(T, V, D):
    """Up to 4096 tokens are put in order by counting, more by sorting: the same sums."""
    g = torch.Generator().manual_seed(T * 31 + V)
    ids = torch.randint(-1, V + 1, (T,), generator=g)
    ids[::3] = ids[0].clamp(0, V - 1)  # a frequent one
    grad = torch.randint(-8, 9, (T, D), generator=g).float()  # sums without rounding
    want = torch.zeros(V, D)
    ok = (ids >= 0) & (ids < V) & (ids != 2)
    want.index_add_(0, ids[ok], grad[ok])
    got = L.lse_embedding_backward(grad.cuda(), ids.cuda(), V, padding=2)
    assert torch.equal(got.cpu(), want)
    held = torch.randint(-8, 9, (V, D), generator=g).float()
    dt = held.cuda()
    L.lse_embedding_backward(grad.cuda(), ids.cuda(), V, padding=2, dtable=dt, accumulate=True)
    assert torch.equal(dt.cpu(), held + want)
