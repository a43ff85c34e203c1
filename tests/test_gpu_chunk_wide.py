"""chunk_attention in several rounds and in tables much wider than the lengths,
where the split and the number of rounds follow the tables: compared with the
oracle, with scores peaked enough that outputs are not small."""

import pytest
import torch

from test_gpu_chunk import call, check, reference
from test_gpu_paged import BF, FH, attn_case, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,nkv,group,lens,rows,dt", [
    (128, 4, 1, [40000], [3000], BF), (64, 16, 1, [40000], [2500], FH),
    (128, 2, 3, [30011, 7, 45000, 0, 25000], [3000, 7, 1500, 0, 2111], FH), (64, 8, 2, [30000, 41234], [2000, 1700], BF)])
def test_rounds_in_tight_and_wide_tables(pkg, hd, nkv, group, lens, rows, dt):
    """Some of the rows are compared: with them at the end of a shorter request."""
    c = attn_case(60, lens, rows, nkv * group, nkv, hd, 128, dt, dt, q_scale=3.0)
    runs = [call(pkg, c, wide) for wide in (False, True)]
    for b, m in enumerate(rows):
        s0 = c["starts"][b]
        for a, e in ((0, 3), (m // 2 + 50, m // 2 + 52), (m - 2, m)):
            if not 0 <= a < e <= m:
                continue
            part = dict(c, q=c["q"][s0 + a:s0 + e], tables=[c["tables"][b]], lens=[lens[b] - m + e], starts=[0, e - a])
            ref = reference(part)
            for out, lse in runs:
                assert float(out[s0 + a:s0 + e].float().abs().max()) > 0.3
                check(part, out[s0 + a:s0 + e], lse[s0 + a:s0 + e], ref=ref)
    for out, lse in runs:
        assert bool((out[c["starts"][-1]:] == 7).all() and (lse[c["starts"][-1]:] == 7).all())
        assert bool(torch.isfinite(out).all() and torch.isfinite(lse).all())
