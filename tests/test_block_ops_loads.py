"""lse_residual_norm may write h over x and out over y: its rows are not loaded through the
read-only path, whose promise is that nothing writes there while the kernel runs."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "log_sum_exp_gb300", "csrc")


def test_rows_that_may_be_outputs():
    text = open(os.path.join(CSRC, "lse_norm.cuh")).read()
    load = re.search(r"\bload_slot\(.*?\n}\n", text, flags=re.S).group(0)
    assert "ld_stream16(" in load and not re.search(r"\b(ldg_stream16|load_elem<\w+>|__ldg)\(", load)
    kernel = re.search(r"\bnorm_kernel\(NormArgs a\).*?\n}\n", text, flags=re.S).group(0)
    assert not re.search(r"\b(ldg_stream16|load_elem<\w+>|__ldg)\(", kernel)
