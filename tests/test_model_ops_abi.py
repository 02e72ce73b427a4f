"""The model operators' C entry points without a GPU: bad arguments are refused
before any device work, and empty calls need none."""
import ctypes

import pytest

import log_sum_exp_gb300 as L
from log_sum_exp_gb300 import build as lse_build


@pytest.fixture(scope="module")
def lib():
    lse_build.build()
    return L.load()


STATS = dict(x=256, dtype=0, B=4, N=8, row_stride=8, target=512, top_k=3, logprob=1024, entropy=2048,
             lse=4096, top_logprob=8192, top_index=16384, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(row_stride=7), 1), (dict(x=None), 1), (dict(x=258), 1),
    (dict(dtype=3), 2), (dict(top_k=33), 1), (dict(top_k=-1), 1), (dict(target=None), 1),
    (dict(logprob=None), 1), (dict(target=516), 1), (dict(logprob=1026), 1), (dict(entropy=2049), 1),
    (dict(lse=4098), 1), (dict(top_logprob=None), 1), (dict(top_index=None), 1), (dict(top_index=16388), 1),
    (dict(N=1 << 31, row_stride=1 << 31), 1), (dict(B=1 << 40, row_stride=1 << 30), 1),
    (dict(target=None, logprob=None, entropy=None, lse=None, top_k=0), 1),
    (dict(B=0), 0),
])
def test_stats_arguments(lib, change, status):
    a = dict(STATS, **change)
    assert lib.lse_token_stats(*a.values()) == status


BACK = dict(x=256, dtype=1, B=4, N=8, row_stride=8, lse=512, entropy=1024, target=2048, top_index=4096,
            top_k=2, gl=8192, gh=16384, gt=32768, gs=65536, dx=131072, dx_stride=8, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), 1), (dict(row_stride=7), 1), (dict(dx_stride=7), 1), (dict(dtype=9), 2), (dict(x=257), 1),
    (dict(x=None), 1), (dict(dx=None), 1), (dict(dx=131073), 1), (dict(lse=None), 1), (dict(lse=514), 1),
    (dict(target=None), 1), (dict(entropy=None), 1), (dict(top_index=None), 1), (dict(top_k=40), 1),
    (dict(gl=8194), 1), (dict(gh=16386), 1), (dict(gt=32770), 1), (dict(gs=65538), 1),
    (dict(dx_stride=1 << 62), 1), (dict(B=0), 0), (dict(N=0, row_stride=0), 0),
])
def test_stats_backward_arguments(lib, change, status):
    a = dict(BACK, **change)
    assert lib.lse_token_stats_backward(*a.values()) == status


def _tensors(*entries):
    t = (L.LseTensor * max(1, len(entries)))()
    for i, e in enumerate(entries):
        t[i] = L.LseTensor(*e)
    return t


@pytest.mark.parametrize("entry,status", [
    ((256, None, -1, 0), 1), ((None, None, 5, 0), 1), ((258, None, 5, 0), 1), ((256, 514, 5, 0), 1),
    ((257, None, 5, 1), 1), ((256, None, 5, 3), 2), ((256, None, 1 << 62, 0), 1),
])
def test_gradient_list_arguments(lib, entry, status):
    t = _tensors((256, None, 4, 0), entry)
    assert lib.lse_grad_norm(t, 2, 512, None) == status
    assert lib.lse_grad_clip(t, 2, 1.0, 1e-6, 512, None) == status


def test_gradient_scalars(lib):
    t = _tensors((256, None, 4, 0))
    assert lib.lse_grad_norm(t, -1, 512, None) == 1
    assert lib.lse_grad_norm(None, 1, 512, None) == 1
    assert lib.lse_grad_norm(t, 1, None, None) == 1
    assert lib.lse_grad_norm(t, 1, 514, None) == 1
    for max_norm, eps in ((-1.0, 0.0), (float("nan"), 0.0), (1.0, -1.0), (1.0, float("nan"))):
        assert lib.lse_grad_clip(t, 1, max_norm, eps, 512, None) == 1


EMBED = dict(table=256, dtype=0, V=5, D=8, stride=8, ids=512, T=3, scale=1.0, out=1024, out_stride=8,
             stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(V=-1), 1), (dict(D=-1), 1), (dict(T=-1), 1), (dict(stride=7), 1), (dict(out_stride=7), 1),
    (dict(dtype=4), 2), (dict(table=258), 1), (dict(out=1026), 1), (dict(ids=516), 1), (dict(table=None), 1),
    (dict(ids=None), 1), (dict(out=None), 1), (dict(V=1 << 40, stride=1 << 40), 1), (dict(T=0), 0),
    (dict(D=0, stride=0, out_stride=0), 0),
])
def test_embedding_arguments(lib, change, status):
    a = dict(EMBED, **change)
    assert lib.lse_embedding(*a.values()) == status


EMBACK = dict(grad=256, dtype=1, T=3, D=8, stride=8, ids=512, V=5, scale=1.0, padding=-1, dtable=1024,
              ddtype=1, dstride=8, accumulate=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(V=-1), 1), (dict(D=-1), 1), (dict(stride=7), 1), (dict(dstride=7), 1),
    (dict(dtype=4), 2), (dict(ddtype=7), 2), (dict(ddtype=2), 2), (dict(grad=257), 1), (dict(dtable=1025), 1),
    (dict(ids=516), 1), (dict(grad=None), 1), (dict(ids=None), 1), (dict(dtable=None), 1),
    (dict(T=1 << 31), 1), (dict(V=1 << 31), 1), (dict(V=0), 0), (dict(D=0, stride=0, dstride=0), 0),
])
def test_embedding_backward_arguments(lib, change, status):
    a = dict(EMBACK, **change)
    assert lib.lse_embedding_backward(*a.values()) == status


def test_tensor_struct_layout(tmp_path):
    import os
    import subprocess

    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "lse.h"\nint main(void){printf("%zu", '
                   "sizeof(lse_tensor));" + "".join(f'printf(" %zu", offsetof(lse_tensor, {f}));'
                                                    for f, _ in L.LseTensor._fields_) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", lse_build.INCLUDE, "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(L.LseTensor)] + [getattr(L.LseTensor, f).offset for f, _ in L.LseTensor._fields_]
    assert os.path.exists(exe)
