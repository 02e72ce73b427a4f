"""The C entry points between a model's last block and its next token, without a GPU: bad
arguments are refused before any device work, and empty calls need none."""
import ctypes
import os
import subprocess

import pytest

import log_sum_exp_gb300 as L
from log_sum_exp_gb300 import build as lse_build


@pytest.fixture(scope="module")
def lib():
    lse_build.build()
    return L.load()


NORM = dict(x=256, dtype=1, T=4, D=8, xs=8, y=512, ys=8, gate=1024, kind=2, gs=8, post=2048, w=4096, wdt=1, scale=1.0,
            eps=1e-6, h=8192, hs=8, out=16384, os=8, rstd=32768, prstd=65536, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(D=-1), 1), (dict(D=16385, xs=16385, ys=16385, gs=16385, hs=16385, os=16385), 1), (dict(xs=7), 1),
    (dict(ys=7), 1), (dict(gs=7), 1), (dict(hs=7), 1), (dict(os=7), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(w=None), 1), (dict(gate=None), 1), (dict(kind=3), 1), (dict(kind=-1), 1), (dict(x=257), 1), (dict(y=513), 1),
    (dict(h=8193), 1), (dict(out=16385), 1), (dict(gate=1025), 1), (dict(w=4097), 1), (dict(post=2049), 1),
    (dict(wdt=0, w=4098), 1), (dict(wdt=0, post=2050), 1), (dict(dtype=5), 2), (dict(wdt=5), 2), (dict(wdt=2), 2),
    (dict(dtype=0, wdt=1), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(rstd=32770), 1), (dict(prstd=65538), 1), (dict(y=None), 1),
    (dict(T=1 << 31), 1), (dict(T=1 << 30, xs=1 << 40), 1), (dict(T=0), 0),
    (dict(D=0, xs=0, ys=0, gs=0, hs=0, os=0), 0),
])
def test_norm_arguments(lib, change, status):
    a = dict(NORM, **change)
    assert lib.lse_residual_norm(*a.values()) == status


BACK = dict(go=256, gos=8, gh=512, ghs=8, x=1024, dtype=1, T=4, D=8, xs=8, y=2048, ys=8, gate=4096, kind=1, gs=8,
            post=8192, w=16384, wdt=1, scale=1.0, rstd=32768, prstd=65536, dx=1 << 17, dxs=8, dy=1 << 18, dys=8,
            dgate=1 << 19, dgs=8, dpost=1 << 20, dw=1 << 21, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(D=16385), 1), (dict(gos=7), 1), (dict(ghs=7), 1), (dict(xs=7), 1), (dict(dxs=7), 1),
    (dict(dys=7), 1), (dict(kind=2, dgs=7), 1), (dict(go=None), 1), (dict(go=257), 1), (dict(gh=513), 1),
    (dict(dx=(1 << 17) + 1), 1), (dict(dw=(1 << 21) + 1), 1), (dict(dpost=(1 << 20) + 1), 1), (dict(dgate=(1 << 19) + 1), 1),
    (dict(rstd=None), 1), (dict(prstd=None), 1), (dict(rstd=32769), 1), (dict(kind=0), 1), (dict(post=None), 1),
    (dict(y=None), 1), (dict(dtype=7), 2), (dict(D=0, gos=0, ghs=0, xs=0, ys=0, gs=0, dxs=0, dys=0, dgs=0), 0),
])
def test_norm_backward_arguments(lib, change, status):
    a = dict(BACK, **change)
    assert lib.lse_residual_norm_backward(*a.values()) == status


QUANT = dict(w=256, dtype=0, N=4, K=130, stride=130, group=32, codes=512, scales=1024, ss=5, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), 1), (dict(K=-1), 1), (dict(stride=129), 1), (dict(group=16), 1), (dict(group=0), 1), (dict(ss=4), 1),
    (dict(codes=520), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(scales=1026), 1), (dict(w=None), 1),
    (dict(w=258), 1), (dict(dtype=3), 2), (dict(K=(1 << 31) - 1, stride=1 << 31, ss=1 << 27), 1), (dict(N=1 << 60), 1),
    (dict(N=0), 0), (dict(K=0, stride=0, ss=0), 0),
])
def test_quantize_arguments(lib, change, status):
    a = dict(QUANT, **change)
    assert lib.lse_quantize4(*a.values()) == status


PACK = dict(values=255, N=4, K=130, stride=130, codes=512, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), 1), (dict(K=-1), 1), (dict(stride=129), 1), (dict(codes=520), 1), (dict(codes=None), 1),
    (dict(values=None), 1), (dict(N=0), 0), (dict(K=0), 0),
])
def test_pack_arguments(lib, change, status):
    a = dict(PACK, **change)
    assert lib.lse_pack4(*a.values()) == status


DEQUANT = dict(codes=512, scales=1024, dtype=1, ss=5, N=4, K=130, group=32, out=256, stride=130, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), 1), (dict(stride=129), 1), (dict(out=None), 1), (dict(out=257), 1), (dict(dtype=3), 2), (dict(ss=4), 1),
    (dict(group=48), 1), (dict(codes=513), 1), (dict(N=0), 0),
])
def test_dequantize_arguments(lib, change, status):
    a = dict(DEQUANT, **change)
    assert lib.lse_dequantize4(*a.values()) == status


LINEAR = dict(x=256, dtype=1, T=3, K=130, xs=130, codes=512, scales=1024, sdt=0, ss=5, N=4, group=32, out=2048, odt=0,
              os=4, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 1), (dict(K=-1), 1), (dict(N=-1), 1), (dict(xs=129), 1), (dict(os=3), 1), (dict(ss=4), 1), (dict(group=8), 1),
    (dict(x=None), 1), (dict(x=257), 1), (dict(out=None), 1), (dict(out=2050), 1), (dict(codes=None), 1),
    (dict(codes=516), 1), (dict(scales=None), 1), (dict(scales=1026), 1), (dict(T=1 << 30), 1), (dict(dtype=9), 2),
    (dict(sdt=9), 2), (dict(odt=9), 2), (dict(odt=2), 2), (dict(T=0), 0), (dict(N=0), 0),
])
def test_linear_arguments(lib, change, status):
    a = dict(LINEAR, **change)
    assert lib.lse_linear4(*a.values()) == status


SETTINGS = dict(temperature_rows=None, top_k_rows=None, top_p_rows=None, min_p_rows=None, top_k=0, temperature=1.0,
                top_p=1.0, min_p=0.0)
SAMPLE = dict(x=256, dtype=0, B=4, N=8, stride=8, u=512, settings=None, token=1024, logprob=2048, stream=None)


@pytest.mark.parametrize("change,settings,status", [
    (dict(B=-1), {}, 1), (dict(N=-1), {}, 1), (dict(stride=7), {}, 1), (dict(x=None), {}, 1), (dict(x=258), {}, 1),
    (dict(u=None), {}, 1), (dict(u=514), {}, 1), (dict(token=None), {}, 1), (dict(token=1028), {}, 1),
    (dict(logprob=2050), {}, 1), (dict(dtype=4), {}, 2), (dict(N=(1 << 31) - 64, stride=1 << 31), {}, 1),
    (dict(B=1 << 31), {}, 1), ({}, dict(temperature=-1.0), 1), ({}, dict(temperature=float("nan")), 1),
    ({}, dict(temperature=2e20), 1), ({}, dict(top_k=-1), 1), ({}, dict(top_p=-0.5), 1), ({}, dict(top_p=float("nan")), 1),
    ({}, dict(min_p=-0.5), 1), ({}, dict(min_p=float("nan")), 1), ({}, dict(temperature_rows=258), 1),
    ({}, dict(top_k_rows=260), 1), ({}, dict(top_p_rows=258), 1), ({}, dict(min_p_rows=258), 1), (dict(B=0), {}, 0),
])
def test_sample_arguments(lib, change, settings, status):
    s = L.LseSampling(**dict(SETTINGS, **settings))
    a = dict(SAMPLE, **dict(change, settings=ctypes.byref(s)))
    assert lib.lse_sample(*a.values()) == status
    assert lib.lse_sample(*dict(a, settings=None).values()) in (1, 2)


def test_settings_layout(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "lse.h"\nint main(void){printf("%zu", '
                   "sizeof(lse_sampling));" + "".join(f'printf(" %zu", offsetof(lse_sampling, {f}));'
                                                      for f, _ in L.LseSampling._fields_) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", lse_build.INCLUDE, "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(L.LseSampling)] + [getattr(L.LseSampling, f).offset for f, _ in L.LseSampling._fields_]
    assert os.path.exists(exe)


def test_python_refusals_need_no_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros((3, 8))
    w = torch.ones(8)
    for call in (lambda: L.lse_residual_norm(x, x, w), lambda: L.residual_norm(x, x, w), lambda: L.lse_quantize4(x),
                 lambda: L.Weights4.from_values(x.to(torch.int8), w), lambda: L.lse_linear4(x, None),
                 lambda: L.lse_sample(x, w[:3])):
        with pytest.raises(ValueError):
            call()
