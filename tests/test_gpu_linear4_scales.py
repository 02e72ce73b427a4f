"""lse_linear4 with scales that are no ordinary numbers: a group's products are summed and the
sum is multiplied by the scale, so an infinite scale gives an infinity of the sum's sign (NaN
for a sum of 0), whatever the shape of the matrix and the kernel it takes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402
from test_gpu_linear4 import DT, _need_gpu, random_weights  # noqa: E402, F401


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sdtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 9, 20])
def test_infinite_scales(dtype, sdtype, G, T):
    N = 40
    for K in (20, 130, 200, 256, 1001, 2100, 20000):
        q, s, _ = random_weights(N, K, G, sdtype, K)
        groups = s.shape[1]
        x = torch.randint(-3, 4, (T, K), generator=torch.Generator().manual_seed(T + K)).to(DT[dtype]).cuda()
        inf = torch.zeros((N, groups), dtype=torch.bool, device="cuda")
        rows = torch.arange(0, N, 2, device="cuda")
        inf[rows, rows % groups] = True
        inf[::4, groups - 1] = True  # the last group, behind which a block of codes has room for more
        s[inf] = float("inf")
        s[2::8] *= -1
        q[4, (groups - 1) * G:] = 0  # sums of 0
        w = L.Weights4.from_values(q, s, G)
        got = L.lse_linear4(x, w, out_dtype=torch.float32).cpu()
        pad = torch.nn.functional.pad
        qs, xs = pad(q.double(), (0, -K % G)).reshape(N, groups, G).cpu(), pad(x.double(), (0, -K % G)).reshape(T, groups, G).cpu()
        want = (torch.einsum("tgk,ngk->tng", xs, qs) * s.double().cpu()).sum(2)  # (whole numbers: the sums are exact)
        assert torch.equal(torch.isnan(got), torch.isnan(want)), K
        assert torch.equal(got == float("inf"), want == float("inf")) and torch.equal(got == -float("inf"), want == -float("inf")), K
        assert torch.isfinite(want[:, 1::4]).all() and torch.isinf(want[:, ::4]).any()


def test_nan_scales():
    for dtype, T in (("f32", 1), ("f32", 9), ("bf16", 1), ("f16", 20)):
        q, s, _ = random_weights(20, 130, 32, "f32", 1)
        s[3, 4] = float("nan")
        got = L.lse_linear4(torch.ones((T, 130), dtype=DT[dtype], device="cuda"), L.Weights4.from_values(q, s, 32), out_dtype=torch.float32)
        assert torch.isnan(got[:, 3]).all() and torch.isfinite(got[:, :3]).all() and torch.isfinite(got[:, 4:]).all()
