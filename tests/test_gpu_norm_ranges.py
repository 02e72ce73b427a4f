"""The gradient of the end of a block for rows far from 1, against the formulas in 64 bits.

The bounds are those of test_gpu_norm: they are relative to the formulas' terms, whatever the
rows' magnitude, as long as the terms and the sums of squares are ordinary f32 numbers.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_norm import _need_gpu, both, spread, vector  # noqa: E402, F401


def along(go, h, share=1.0):
    """go with a part along the rows h, so that the gradient's second term counts."""
    unit = h.double() / h.double().pow(2).mean(1, keepdim=True).sqrt()
    return (go.double() + share * unit).to(go.dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("magnitude", [1e-17, 1e-13, 1e-10, 1e10, 1e13, 1e14, 1e17])
@pytest.mark.parametrize("T,D", [(7, 100), (5, 1001), (3, 4096), (2, 16384)])
def test_magnitudes(dtype, magnitude, T, D):
    """Rows of an rms from 1e-17 (eps = 0) to 1e17: the squares' sums are from 1e-34 up to 1e38."""
    if magnitude == 1e17 and D > 1024:
        magnitude = 2e16  # (the sum of h^2 stays an f32)
    eps = 0.0 if magnitude < 1 else 1e-6
    g = torch.Generator().manual_seed(D)
    x, y = (spread(T, D, dtype, D + i, magnitude * s)[1] for i, s in enumerate((1.5, 0.4)))
    gh = spread(T, D, dtype, D + 2, 0.7 / magnitude)[1]
    ge = torch.rand((T, D), generator=g).to(x.dtype).cuda()
    w, p, gc = vector(D, dtype, 5), vector(D, dtype, 6), vector(D, dtype, 7, 0.5)
    go = along(spread(T, D, dtype, D + 3)[1], x)
    both(x, None, w, None, None, 1.0, go, None, eps)
    both(x, y, w, None, gc, 0.7, go, gh, eps)
    both(x, y, w, None, ge, 0.7, go, gh, eps)
    # The block's norm takes its magnitude off, so the scale brings it back.
    both(x, y, w, p, gc, 0.7 * magnitude, go, gh, eps)
    both(x, y, w, p, ge, 0.7 * magnitude, go, gh, eps)
    # A block far from the stream's magnitude: h is an ordinary row, y is not.
    plain = spread(T, D, dtype, D + 4, 1.5)[1]
    both(plain, y, w, p, gc, 0.7, along(go, plain), None, eps)


def test_rows_of_zeros():
    """Zeros with an eps far below the squares of ordinary rows: rstd = 1e15, and its cube is beyond f32."""
    for D in (64, 1001, 16384):
        x = torch.zeros((3, D), device="cuda")
        y = torch.zeros_like(x)
        w, p = vector(D, "f32", 1), vector(D, "f32", 2)
        go = spread(3, D, "f32", 3)[1]
        both(x, None, w, None, None, 1.0, go, None, 1e-30)
        both(x, y, w, p, None, 1.0, go, None, 1e-30)
