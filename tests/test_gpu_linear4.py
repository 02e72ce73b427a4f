"""Matrices held in 4 bits: quantising and reading back (exact), products against 64 bits.

Products: a group's products are summed in f32 by matrix instructions of 16 columns, 8 of
them at most (f32 tokens: 24), each adding with an error of at most 2^-22 of the magnitudes
so far, and the groups' sums follow in f32: (24 + K / group + 8) * 2^-22 of the sum of
magnitudes covers them, then one rounding to the output's type.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
Q = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def plain_quantize(w, G):
    """(scales, whole numbers) by 64-bit quotients."""
    N, K = w.shape
    v = torch.nn.functional.pad(w.double(), (0, -K % G)).reshape(N, -1, G)
    s = (v.abs().amax(2) / 7).to(w.dtype)
    wide = s.double()[:, :, None]
    q = torch.where(wide > 0, v / wide, torch.zeros((), dtype=torch.float64, device=w.device)).round().clamp(-8, 7)
    return s, q.reshape(N, -1)[:, :K]


def values_of(w4):
    """The whole numbers behind the codes, by the documented layout."""
    N, K = w4.shape
    b = w4.codes.cpu().reshape(N, -1, 4, 4, 4).int()  # block, c, w, byte
    word = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | (b[..., 3].long() << 24)
    word = word.long()
    out = torch.zeros((N, word.shape[1], 128), dtype=torch.int64)
    for c in range(4):
        for w in range(4):
            for i in range(4):
                out[:, :, 32 * w + 8 * c + 2 * i] = (word[:, :, c, w] >> (4 * i)) & 15
                out[:, :, 32 * w + 8 * c + 2 * i + 1] = (word[:, :, c, w] >> (16 + 4 * i)) & 15
    out = out.reshape(N, -1) - 8
    assert (out[:, K:] == 0).all()
    return out[:, :K]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,K,pad", [(1, 1, 0), (3, 31, 0), (7, 32, 8), (5, 100, 3), (9, 128, 0), (4, 129, 1), (17, 257, 0),
                                     (6, 1001, 0), (33, 1024, 0), (130, 640, 8), (2, 8200, 0)])
def test_quantize(dtype, G, N, K, pad):
    g = torch.Generator().manual_seed(N * K)
    buf = (torch.randn((N, K + pad), generator=g) * 0.02).to(DT[dtype])
    w = buf[:, :K]
    w[0, :min(K, 20)] = 0
    w = buf.cuda()[:, :K]
    w4 = L.lse_quantize4(w, group=G)
    s, q = plain_quantize(w, G)
    assert torch.equal(w4.scales, s)
    assert torch.equal(values_of(w4), q.cpu().long())
    want = (q * s.double().repeat_interleave(G, 1)[:, :K]).to(DT[dtype])
    assert torch.equal(L.lse_dequantize4(w4), want)
    out = torch.full((N, K + 5), 3.0, dtype=DT[dtype], device="cuda")
    L.lse_dequantize4(w4, out=out[:, :K])
    assert torch.equal(out[:, :K], want) and (out[:, K:] == 3.0).all()
    again = L.Weights4.from_values(q.to(torch.int8), s, G)
    assert torch.equal(again.codes, w4.codes)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_halves_and_extremes(dtype):
    """Quotients on a half, small and large magnitudes, NaN and infinities."""
    dt = DT[dtype]
    G = 32
    w = torch.zeros((9, 64), dtype=dt)
    w[0, :15] = torch.arange(-7, 8).to(dt)            # whole
    w[1, :14] = (torch.arange(-7, 7) + 0.5).to(dt)    # halves, scale 1
    w[1, 20] = 7
    w[2, :3] = torch.tensor([torch.finfo(dt).max, -torch.finfo(dt).max, torch.finfo(dt).max / 2])
    w[3, :5] = torch.tensor([7., -3., 1., 2., 5.]) * torch.finfo(dt).smallest_normal * 2.0 ** -4
    w[4, 3] = float("nan")
    w[5, 40] = float("inf")
    w[6, :8] = torch.rand(8, generator=torch.Generator().manual_seed(1)).to(dt)
    w[7] = torch.finfo(dt).tiny
    w[8, :] = -1.0
    w4 = L.lse_quantize4(w.cuda(), group=G)
    ok = [0, 1, 2, 3, 6, 7, 8]
    s, q = plain_quantize(w[ok].cuda(), G)
    assert torch.equal(w4.scales[ok], s) and torch.equal(values_of(w4)[ok], q.cpu().long())
    back = L.lse_dequantize4(w4)
    assert torch.isnan(back[4, :32]).all() and (back[4, 32:] == 0).all()
    assert torch.isnan(back[5, 32:]).all() and (back[5, :32] == 0).all()


def test_values_are_cut_off():
    v = torch.tensor([[-128, -9, -8, -1, 0, 6, 7, 8, 127]], dtype=torch.int8).cuda()
    w = L.Weights4.from_values(v, torch.ones((1, 1), device="cuda"), 32)
    assert values_of(w).tolist() == [[-8, -8, -8, -1, 0, 6, 7, 7, 7]]


def random_weights(N, K, G, sdtype, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-8, 8, (N, K), generator=g).to(torch.int8).cuda()
    s = ((torch.rand((N, -(-K // G)), generator=g) + 0.5) * 0.01).to(DT[sdtype]).cuda()
    return q, s, L.Weights4.from_values(q, s, G)


def check_product(got, x, q, s, G):
    K = q.shape[1]
    w = q.double() * s.double().repeat_interleave(G, 1)[:, :K]
    want, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    tol = mag * (24 + K / G + 8) * 2.0 ** -22 + want.abs() * Q[got.dtype] + TINY[got.dtype]
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (int((err > tol).sum()), float((err / tol).max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 33, 70])
def test_tokens(dtype, G, T):
    for N, K in [(1, 1), (15, 33), (16, 128), (17, 129), (100, 1001), (1000, 640), (5003, 256)]:
        q, s, w = random_weights(N, K, G, dtype, N + K)
        x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(DT[dtype]).cuda()
        check_product(L.lse_linear4(x, w), x, q, s, G)
        check_product(L.lse_linear4(x, w, out_dtype=torch.float32), x, q, s, G)


@pytest.mark.parametrize("dtype,sdtype", [("bf16", "f32"), ("f32", "f16"), ("f16", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,N,K", [(1, 70000, 640), (5, 40001, 1000), (24, 33000, 512), (32, 300, 16000), (16, 2000, 8192)])
def test_sizes(dtype, sdtype, T, N, K):
    q, s, w = random_weights(N, K, 64, sdtype, N)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(DT[dtype]).cuda()
    got = L.lse_linear4(x, w)
    check_product(got, x, q, s, 64)
    assert torch.equal(got, L.lse_linear4(x, w))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strides(dtype):
    q, s, w = random_weights(333, 300, 32, dtype, 1)
    for stride, off in [(300, 0), (304, 8), (301, 1), (307, 3)]:
        buf = torch.full((5 * stride + 64,), float("nan"), dtype=DT[dtype], device="cuda")
        x = buf[off:off + 5 * stride].reshape(5, stride)[:, :300]
        x.copy_(torch.randn((5, 300)))
        out = torch.full((5, 340), 7.0, dtype=DT[dtype], device="cuda")
        L.lse_linear4(x, w, out=out[:, :333])
        check_product(out[:, :333], x, q, s, 32)
        assert (out[:, 333:] == 7.0).all()
        wide = torch.empty((5, 333), device="cuda")
        assert L.lse_linear4(x, w, out=wide) is wide
        check_product(wide, x, q, s, 32)
    one = torch.randn(300).to(DT[dtype]).cuda()
    y = L.lse_linear4(one, w)
    assert y.shape == (333,)
    check_product(y[None], one[None], q, s, 32)
    out = torch.empty(333, dtype=DT[dtype], device="cuda")
    assert torch.equal(L.lse_linear4(one, w, out=out), y)


def test_exact_sums_and_magnitudes():
    """Whole numbers come out exactly; f32 tokens count with all their bits and range."""
    q, s, w = random_weights(64, 256, 128, "f32", 3)
    s.fill_(1.0)
    w = L.Weights4.from_values(q, s, 128)
    x = torch.randint(-64, 65, (9, 256), generator=torch.Generator().manual_seed(1)).float().cuda()
    assert torch.equal(L.lse_linear4(x, w), (x.double() @ q.double().t()).float())
    x.zero_()
    x[0, 5], x[1, 6], x[2, 200], x[3, 0] = 1.0 + 2.0 ** -23, 3.4e38, 2.0 ** -100, float("inf")
    y = L.lse_linear4(x, w)
    # x = 1 + 2^-23 has 24 bits: times a power of two that is an f32, and no sum on the way to it
    # rounds (its parts are 1 and 2^-23 times the same power); times 3, 5, 6 or 7 it is not, and
    # each of the two additions of the parts' products may cut off less than one step of the
    # result, at most 2^-23 of it.
    for t, k in ((0, 5), (2, 200)):
        want = x[t, k].double() * q[:, k].double()
        held = want == want.float().double()
        assert torch.equal(y[t][held].double(), want[held]) and held.sum() > 20
        assert ((y[t].double() - want).abs() <= 2 * 2.0 ** -23 * want.abs()).all()
    small = q[:, 6].abs() <= 1
    assert torch.equal(y[1][small], x[1, 6] * q[small, 6].float())
    col = q[:, 0]
    assert (y[3][col > 0] == float("inf")).all() and (y[3][col < 0] == -float("inf")).all()
    assert torch.isnan(y[3][col == 0]).all()


def test_no_columns_and_no_rows():
    w = L.Weights4(torch.empty((5, 0), dtype=torch.uint8, device="cuda"), torch.empty((5, 0), device="cuda"), (5, 0), 64)
    assert (L.lse_linear4(torch.empty((3, 0), device="cuda"), w) == 0).all()
    q, s, w = random_weights(5, 40, 32, "f32", 3)
    assert L.lse_linear4(torch.empty((0, 40), device="cuda"), w).shape == (0, 5)
    assert L.lse_dequantize4(L.lse_quantize4(torch.empty((0, 40), device="cuda"))).shape == (0, 40)


def test_beyond_32_bits():
    """Codes beyond 2^32 bytes."""
    N, K = 1_100_000, 8192
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.ones((N, K // 128), dtype=torch.bfloat16, device="cuda")
    last = (torch.arange(K) % 16 - 8).to(torch.int8)[None].cuda()
    codes[N - 1] = L.Weights4.from_values(last, scales[:1], 128).codes[0]
    w = L.Weights4(codes, scales, (N, K), 128)
    x = (torch.arange(K) % 5 - 2).to(torch.bfloat16)[None].cuda()
    y = L.lse_linear4(x, w, out_dtype=torch.float32)[0]
    assert float(y[N - 1]) == float((x.double() * last.double()).sum()) and (y[:N - 1] == 0).all()


def test_another_stream_and_graph():
    q, s, w = random_weights(3000, 512, 64, "bf16", 3)
    x = torch.randn((4, 512)).bfloat16().cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = L.lse_linear4(x, w, stream=st)
    st.synchronize()
    check_product(y, x, q, s, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = L.lse_linear4(x, w)
        z = L.lse_dequantize4(L.lse_quantize4(x.float()))
    x.copy_(torch.randn((4, 512)))
    graph.replay()
    check_product(y, x, q, s, 64)
    assert (z - x.float()).abs().max() <= 0.5 * x.float().abs().max() / 7 * (1 + 2.0 ** -20)


def test_refusals():
    q, s, w = random_weights(8, 64, 32, "f32", 3)
    x = torch.zeros((2, 64), device="cuda")
    for call in [lambda: L.lse_quantize4(x, group=16), lambda: L.lse_quantize4(x.t()), lambda: L.lse_quantize4(x[0]),
                 lambda: L.lse_linear4(x[:, :32], w), lambda: L.lse_linear4(x, w, out_dtype=torch.float16),
                 lambda: L.lse_linear4(x, w, out=torch.empty((2, 7), device="cuda")),
                 lambda: L.lse_linear4(x.t(), w), lambda: L.lse_linear4(x.half(), w, out_dtype=torch.bfloat16),
                 lambda: L.Weights4.from_values(q.float(), s, 32), lambda: L.Weights4.from_values(q, s, 64),
                 lambda: L.Weights4(w.codes[:, :32], s, (8, 64), 32), lambda: L.Weights4(w.codes.float(), s, (8, 64), 32),
                 lambda: L.Weights4(w.codes, s.cpu(), (8, 64), 32), lambda: L.Weights4(w.codes, s, (8, 64), 20),
                 lambda: L.lse_dequantize4(w, out=torch.empty((8, 64), dtype=torch.float16, device="cuda"))]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.lse_quantize4(x.double())
