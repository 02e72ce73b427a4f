"""Kernels whose output may be their input must not load it through the read-only path
(ld.global.nc, __ldg): its promise is that nothing writes there while the kernel runs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "log_sum_exp_gb300", "csrc")


def body(source, name):
    """The text of function ``name``, up to the closing brace in column 0."""
    m = re.search(r"\b%s\(.*?\n}\n" % re.escape(name), source, flags=re.S)
    assert m, name
    return m.group(0)


@pytest.mark.parametrize("file,function,inputs", [
    ("lse_stats.cu", "grad_slots", r"x0|xr"),
    ("lse_stats.cu", "lse_stats_backward_kernel", r"xr"),
    ("lse_grads.cu", "chunk_scale", r"a0"),
])
def test_inputs_that_may_be_outputs(file, function, inputs):
    text = body(open(os.path.join(CSRC, file)).read(), function)
    assert not re.search(r"\b(ldg_stream16|load_elem<\w+>|__ldg)\(\s*(%s)\b" % inputs, text)
    assert re.search(r"\b(ld_stream16|load_own_elem<\w+>)\(\s*(%s)\b" % inputs, text)
