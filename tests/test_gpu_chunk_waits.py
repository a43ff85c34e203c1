"""chunk_attention when its bounded waits run out: every row is right or NaN, and
the process goes on. SF_TEST_WAIT_POLLS makes the waits shorter than what they
wait for takes; it is read once, so the calls run in a process of their own."""

import os
import subprocess
import sys

import pytest
import torch

from test_gpu_chunk import call
from test_gpu_paged import BF, F4, FH, attn_case, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def cases():
    """Whole items and shared ones, one tile and two, several rounds' share of units, head dimensions and types."""
    yield attn_case(50, [900, 300, 5], [400, 300, 5], 14, 2, 64, 16, FH, FH)
    yield attn_case(51, [3000, 64, 0, 700], [2100, 64, 0, 130], 28, 4, 128, 64, BF, BF)
    yield attn_case(52, [30 + i % 40 for i in range(300)] + [600], [2 + i % 9 for i in range(300)] + [300], 8, 2, 128, 64, BF, BF)


CHILD = """
import sys
sys.path[:0] = [{here!r}, {root!r}]
import torch
import greedy_speculative_decoding_gb300 as pkg
import test_gpu_chunk_waits as t
res = []
for c in t.cases():
    for _ in range(3):
        res.append([x.cpu() for x in t.call(pkg, c, True)])
torch.cuda.synchronize()
c = t.after()
res.append([x.cpu() for x in t.call(pkg, c)])
torch.save(res, {out!r})
"""


def after():
    """A call of the kernels whose waits stay as they are."""
    return attn_case(53, [300], [90], 4, 2, 64, 64, F4, BF)


def right_or_nan(got, want, n):
    """Which (row, head) are NaN; all others are as they should be, bit by bit."""
    lost = got[0].isnan().all(-1) & got[1].isnan()
    assert torch.equal(got[0][~lost], want[0][~lost]) and torch.equal(got[1][~lost], want[1][~lost])
    assert not bool(lost[n:].any())            # (rows behind the last request)
    return lost


# Some polls end early, as what is waited for arrives in parts: with 1 every row is lost, with 40 few or none.
@pytest.mark.parametrize("polls", [1, 20, 26, 32, 40])
def test_waits_that_run_out(pkg, tmp_path, polls):
    out = str(tmp_path / "out.pt")
    code = CHILD.format(here=HERE, root=os.path.dirname(HERE), out=out)
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, SF_TEST_WAIT_POLLS=str(polls)),
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    res = torch.load(out)
    lost = 0
    for i, c in enumerate(cases()):
        want = [x.cpu() for x in call(pkg, c, True)]
        for got in res[3 * i:3 * i + 3]:
            lost += int(right_or_nan(got, want, c["starts"][-1]).sum())
    print(f"{polls} polls: {lost} rows of heads lost")
    assert lost > 0 or polls > 1
    want = [x.cpu() for x in call(pkg, after())]
    assert torch.equal(res[-1][0], want[0]) and torch.equal(res[-1][1], want[1])
