"""lse_token_stats_pair and its gradient without a GPU: the arguments that the entry
points without lse_low check, and lse_low's own."""
import pytest

import log_sum_exp_gb300 as L
import test_model_ops_abi as base
from test_model_ops_abi import lib  # noqa: F401  (the fixture that builds and loads)


def _with(a, after, name, value):
    out = {}
    for k, v in a.items():
        out[k] = v
        if k == after:
            out[name] = value
    return out


STATS = _with(base.STATS, "lse", "lse_low", 32768)
BACK = _with(base.BACK, "lse", "lse_low", 768)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), 1), (dict(row_stride=7), 1), (dict(x=None), 1), (dict(dtype=3), 2), (dict(top_k=33), 1),
    (dict(target=None), 1), (dict(lse_low=32770), 1), (dict(lse=4098), 1), (dict(B=0), 0),
    (dict(target=None, logprob=None, entropy=None, lse=None, lse_low=None, top_k=0), 1),
])
def test_stats_arguments(lib, change, status):  # noqa: F811
    assert lib.lse_token_stats_pair(*dict(STATS, **change).values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), 1), (dict(dx_stride=7), 1), (dict(x=None), 1), (dict(dx=None), 1), (dict(lse=None), 1),
    (dict(lse_low=770), 1), (dict(target=None), 1), (dict(top_k=40), 1), (dict(B=0), 0),
    (dict(B=0, lse_low=None), 0),
])
def test_stats_backward_arguments(lib, change, status):  # noqa: F811
    assert lib.lse_token_stats_backward_pair(*dict(BACK, **change).values()) == status


def test_a_tuple_made_by_hand_has_no_second_part():
    s = L.TokenStats(1, 2, 3, 4, 5)
    assert tuple(s) == (1, 2, 3, 4, 5) and s.lse_low is None
    s.lse_low = 6
    assert s._replace(entropy=0).lse_low == 6 and s._replace(lse=0).lse_low is None
