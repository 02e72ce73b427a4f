"""f32 tokens of lse_linear4 count with all their bits down to the smallest f32.

Bounds.  One element per token: its product with a whole number of -8 .. 7 is rounded once in
f32 if it does not fit, or is the sum of at most three parts' products (two additions, each off
by less than a step, 2^-23 of the result); times a scale that is a power of two nothing more is
lost: 3 * 2^-23.  Whole rows: as in test_gpu_linear4.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
from test_gpu_linear4 import _need_gpu, check_product, random_weights  # noqa: E402, F401


def scaled(N, K, G, exponent, seed=3):
    q, s, _ = random_weights(N, K, G, "f32", seed)
    s.fill_(2.0 ** exponent)
    return q, s, L.Weights4.from_values(q, s, G)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("K", [100, 1001, 8200, 20000])
def test_one_element(T, G, K):
    q, s, w = scaled(48, K, G, 100)
    bits = torch.Generator().manual_seed(T * K)
    for e in (-90, -105, -111, -115, -120, -126, -128, -133, -140):
        x = torch.zeros((T, K))
        at = torch.randint(0, K, (T,), generator=bits)
        # 24 bits, or as many as an f32 of this magnitude has
        x[torch.arange(T), at] = ((torch.rand(T, generator=bits, dtype=torch.float64) + 1.0) * 2.0 ** e).float()
        x = x.cuda()
        got = L.lse_linear4(x, w).double()
        want = x.double() @ q.double().t() * 2.0 ** 100
        assert ((got - want).abs() <= 3 * 2.0 ** -23 * want.abs()).all(), (e, float(((got - want).abs() / want.abs()).nan_to_num(0).max()))


@pytest.mark.parametrize("T", [1, 4, 7, 12, 40])
@pytest.mark.parametrize("N,K,G", [(40, 777, 32), (5003, 256, 128), (130, 9000, 64), (33, 128, 32)])
def test_rows(T, N, K, G):
    """Rows of small numbers, and rows in which the large ones meet whole numbers of 0."""
    q, s, w = scaled(N, K, G, 100)
    x = (torch.randn((T, K), generator=torch.Generator().manual_seed(T)).double() * 2.0 ** -118).float().cuda()
    check_product(L.lse_linear4(x, w), x, q, s, G)
    q[:, ::3] = 0
    s.fill_(1.0)
    w = L.Weights4.from_values(q, s, G)
    big = x.clone()
    big[:, ::3] = (torch.randn_like(big[:, ::3]) * 2.0 ** 100)
    s.fill_(2.0 ** 20)
    w = L.Weights4.from_values(q, s, G)
    check_product(L.lse_linear4(big, w) * 2.0 ** 80, x, q, s * 2.0 ** 80, G)


@pytest.mark.parametrize("dtype,e", [("bf16", -120), ("bf16", -128), ("f16", -16), ("f16", -23)])
@pytest.mark.parametrize("T", [1, 9, 20])
def test_small_16_bit_tokens(dtype, e, T):
    """16-bit tokens below their type's normal range."""
    N, K, G = 48, 300, 32
    q, s, w = scaled(N, K, G, 40)
    x = (torch.randn((T, K), generator=torch.Generator().manual_seed(T)).double() * 2.0 ** e)
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float16).cuda()
    assert (x != 0).any()
    check_product(L.lse_linear4(x, w, out_dtype=torch.float32), x, q, s, G)
