"""A GradList keeps the memory that it refers to, whatever its tensors are given later."""
import gc
import weakref

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import log_sum_exp_gb300 as L  # noqa: E402


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    device = property(lambda self: torch.device("cuda", 0))


def watched(n):
    a = np.ones(n, np.float32)
    return torch.Tensor._make_subclass(OnDevice, torch.from_numpy(a)), weakref.ref(a)


def test_memory_outlives_a_reallocated_gradient():
    (g, held), (o, held_out) = watched(8), watched(8)
    lst = L.GradList([g], [o])
    g.data = torch.zeros(8)
    o.data = torch.zeros(8)
    gc.collect()
    assert held() is not None and held_out() is not None
    assert held().ctypes.data == lst._table[0].data and held_out().ctypes.data == lst._table[0].out
    del lst, g, o
    gc.collect()
    assert held() is None and held_out() is None


@pytest.mark.gpu
def test_other_tensors_are_not_clipped():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = 1 << 20
    g = torch.full((n,), 2.0, device="cuda")
    lst = L.GradList([g])
    where = g.data_ptr()
    g.data = torch.full((n,), 3.0, device="cuda")
    others = [torch.full((n,), 7.0, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != where for t in others)
    assert float(L.lse_grad_clip(lst, 1.0)) == 2048.0  # of the memory as it was
    torch.cuda.synchronize()
    assert (g == 3.0).all() and all((t == 7.0).all() for t in others)
