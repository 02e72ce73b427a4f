"""Where lse_sample's search for a threshold or a column comes to no result -- a state that no known
row reaches -- the row is marked (-1, NaN) like one that is no distribution: it is not drawn with
nothing cut off, nor from what a failed search has left."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "log_sum_exp_gb300", "csrc")
TEXT = open(os.path.join(CSRC, "lse_sample.cuh")).read()


def body(start, end):
    at = TEXT.index(start)
    return TEXT[at:TEXT.index(end, at)]


def test_select_says_so():
    """Without a result from exact sums or counts select() sets `lost`; from fast sums it is not sure."""
    select = body(" select(bool by_mass", "\n};")
    returns = [m.group(0) for m in re.finditer(r"[^\n]*return (lost = true, )?base_key;[^\n]*", select)]
    assert len(returns) >= 5
    for line in returns:
        assert "lost = true, base_key" in line or "not sure" in line or line == "        return base_key;", line
    assert "lost = err == 0;  // (else it is not sure)\n        return base_key;" in select


def test_every_result_is_looked_at():
    row = body("__device__ void sample_row(", "\ntemplate <int TX> __host__ __device__ constexpr int sample_ctas")
    calls = re.findall(r"[^\n]*\br\.(?:locate|select|list_cut)\([^\n]*\n[^\n]*", row)
    assert len(calls) >= 7
    for call in calls:
        first, after = call.split("\n")
        if ".select(" in first:
            assert "if (r.lost) return mark();" in after, call
        else:
            assert "return mark();" in first or "const bool found = " in first, call
    assert row.count("!found) return mark();") == 1 and row.count("} else if (!found) {\n            return mark();") == 1
