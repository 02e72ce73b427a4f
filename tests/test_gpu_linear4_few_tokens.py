"""Up to four f32 tokens: every number of them, groups, strides and offsets, and what lies around the output."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
from test_gpu_linear4 import _need_gpu, check_product, random_weights  # noqa: E402, F401


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("sdtype", ["f32", "bf16", "f16"])
def test_sizes_and_strides(T, G, sdtype):
    for N, K in [(1, 1), (15, 33), (17, 129), (100, 1001), (333, 300), (1000, 640), (30001, 1025), (3, 4500)]:
        q, s, w = random_weights(N, K, G, sdtype, N + K)
        g = torch.Generator().manual_seed(N)
        for stride, off in [(K, 0), (K + 8, 8), (K + 1, 1), (K + 7, 3)]:
            buf = torch.full((T * stride + 64,), float("nan"), device="cuda")
            x = buf[off:off + T * stride].reshape(T, stride)[:, :K]
            x.copy_(torch.randn((T, K), generator=g))
            out = torch.full((T, N + 7), 7.0, device="cuda")
            L.lse_linear4(x, w, out=out[:, :N])
            check_product(out[:, :N], x, q, s, G)
            assert (out[:, N:] == 7.0).all()
            assert torch.equal(L.lse_linear4(x, w), out[:, :N])
