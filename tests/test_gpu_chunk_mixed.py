"""chunk_attention over batches in which items of two query tiles have many
items of one tile behind them in a CTA's share: a long request among hundreds
of short ones. The second tile's warps pass over the short ones, and what they
still need of the long one's last item may not be overtaken.

Bounds as in test_gpu_chunk.py. Rows that do not see an odd value are compared
bit by bit with the run without it: a row's result in this kernel does not
depend on other rows' values."""

import random

import pytest
import torch

from test_gpu_chunk import call, check
from test_gpu_paged import BF, FH, attn_case, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

# query heads a KV head, KV heads, requests, long ones among them: 152 CTAs have up to 52, 31, 31 and 17 items of one
# tile in a row behind one of two.
BATCHES = [(4, 4, 2000, 12), (5, 8, 600, 6), (2, 2, 3000, 9), (7, 4, 900, 8)]


def mixed(seed, hd, dt, g, nkv, B, n_long):
    """Requests of 2 to 9 rows over at most 60 tokens, and long ones of one item (two tiles) a KV head."""
    r = random.Random(seed)
    lens = [r.randint(9, 60) for _ in range(B)]
    rows = [min(n, r.randint(2, 9)) for n in lens]
    at = [i * B // n_long + r.randint(0, B // n_long - 1) for i in range(n_long)]
    for b in at:
        rows[b] = 256 // g
        lens[b] = rows[b] + 200 + r.randint(0, 30)
    return attn_case(seed, lens, rows, nkv * g, nkv, hd, 64, dt, dt), at


def spoil(c, b, slot, value):
    pg = c["tables"][b][slot // 64]
    c["v"][pg, :, slot % 64, 3] = value


def rows_of(c, b):
    return slice(c["starts"][b], c["starts"][b + 1])


def same(a, b, rows):
    return torch.equal(a[0][rows], b[0][rows]) and torch.equal(a[1][rows], b[1][rows])


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
def test_short_requests_behind_long_ones(pkg, dt, hd, batch):
    g = batch[0]
    c, at = mixed(batch[2] + hd, hd, dt, *batch)
    clean = call(pkg, c)
    for _ in range(3):
        assert same(clean, call(pkg, c), slice(None))
    r = random.Random(0)
    for b in at + [b for b in r.sample(range(len(c["lens"])), 20) if b not in at]:
        part = dict(c, q=c["q"][rows_of(c, b)], tables=[c["tables"][b]], lens=[c["lens"][b]],
                    starts=[0, c["starts"][b + 1] - c["starts"][b]])
        check(part, *(x[rows_of(c, b)] for x in clean))

    # A value of the long ones that only rows of the second tile see: no finite number in all that do.
    odd = dict(c, v=c["v"].clone())
    j0 = 128 // g + 3
    seeing = torch.zeros(c["q"].shape[0], dtype=torch.bool, device="cuda")
    for i, b in enumerate(at):
        m = c["starts"][b + 1] - c["starts"][b]
        spoil(odd, b, c["lens"][b] - m + j0, [float("nan"), float("inf"), float("-inf")][i % 3])
        seeing[c["starts"][b] + j0:c["starts"][b + 1]] = True
    got = call(pkg, odd)
    assert not bool(got[0][seeing][..., 3].isfinite().any())
    assert same(got, clean, ~seeing)

    # Values of the short ones that their last two rows see: no other row changes, the long ones' least of all.
    odd = dict(c, v=c["v"].clone())
    seeing.fill_(False)
    for b in range(len(c["lens"])):
        if b not in at:
            spoil(odd, b, c["lens"][b] - 2, float("nan"))
            seeing[c["starts"][b + 1] - 2:c["starts"][b + 1]] = True
    got = call(pkg, odd)
    assert not bool(got[0][seeing][..., 3].isfinite().any())
    assert same(got, clean, ~seeing)
