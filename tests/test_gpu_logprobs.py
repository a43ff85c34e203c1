"""GPU parity of token_logprobs against the float64 oracle.

Ranks and orders are whole numbers: equal. With d_v = x_v - max x (rounded,
2^-24 |d_v|), an exponential e^(d_v) is off by 3 * 2^-24 |d_v| (the difference,
the factor log2 e and the product) and 2^-22 (the instruction), relatively; a
thread adds its n elements one after the other and may move its reference at
each (2^-22 and 3 * 2^-24 of the move, which the exponents count already): c =
(n + 32) 2^-21 with the joins. So with D = sum p |d| and D2 = sum p d^2, log s is
off by r = 3 * 2^-24 D + c, and 2^-23 of itself, and t / s by 3 * 2^-24 D2 + 2 c
max(D, 1) + 2 r D (the last for s). The differences round once more.
"""

import pytest
import torch

from oracle import logprobs as ol
from test_gpu_paged import BF, F4, FH, i32, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def check(pkg, x, tokens, top, rows=None, **kw):
    n, vocab = x.shape
    got = pkg.token_logprobs(x, i32(tokens), top=top, **kw)
    e = 2.0 ** -24
    c = (vocab / 512 + 32) * 2.0 ** -21
    for i in range(n) if rows is None else rows:
        if not 0 <= tokens[i] < vocab:
            continue
        logp, entropy, rank, first, D, D2 = ol.row(x[i].cpu(), tokens[i])
        assert int(got.rank[i]) == rank, i
        assert got.top_ids[i].tolist() == first[:top].tolist(), i
        r = 3 * e * D + c
        for want, have, bound in ([(logp[tokens[i]], got.logprob[i], None), (entropy, got.entropy[i], "H")]
                                  + [(logp[t], got.top_logprobs[i, j], None) for j, t in enumerate(first[:top].tolist())]):
            want, have = float(want), float(have)
            if want != want or abs(want) == INF:
                assert have == want or (have != have and want != want), (i, have, want)
                continue
            logs = -float(logp[first[0]])                       # log s
            tol = r + 2 * e * logs + e * (abs(want) + logs + 2 ** -20)
            tol += (3 * e * D2 + 2 * c * max(D, 1.0) + 2 * r * D + e * D) if bound else e * abs(want)
            assert abs(have - want) <= tol, (i, have, want, tol)
    return got


def rand(seed, n, vocab, dtype, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((n, vocab), device="cuda", generator=g) * scale).to(dtype)


def pick(seed, n, vocab):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, vocab, (n,), generator=g).tolist()


@pytest.mark.parametrize("dtype", [F4, BF, FH])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 31, 512, 1000, 1024, 2051, 4099, 16411])
@pytest.mark.parametrize("n", [1, 5, 40, 700])
def test_sizes(pkg, dtype, vocab, n):
    rows = range(n) if n < 100 else range(0, n, 97)
    check(pkg, rand(vocab + n, n, vocab, dtype), pick(vocab, n, vocab), min(vocab, 5), rows)


@pytest.mark.parametrize("dtype", [F4, BF, FH])
@pytest.mark.parametrize("vocab", [151936, 152064, 151665, 256003])
@pytest.mark.parametrize("n,top", [(1, 5), (2, 0), (9, 20), (33, 32), (80, 1), (200, 3), (700, 2)])
def test_vocabularies(pkg, dtype, vocab, n, top):
    check(pkg, rand(vocab + n, n, vocab, dtype), pick(n, n, vocab), top, range(0, n, max(1, n // 8)))


@pytest.mark.parametrize("dtype", [F4, BF, FH])
@pytest.mark.parametrize("top", [0, 1, 2, 31, 32])
def test_rows_apart_and_not_aligned(pkg, dtype, top):
    for off in (1, 3, 8):
        buf = rand(off, 7, 5000 + off, dtype)
        x = buf[:, off:off + 4097]
        check(pkg, x, pick(off, 7, 4097), top)
    x = rand(9, 1, 3001, dtype)[:, 1:].expand(6, 3000)          # one row for all
    check(pkg, x, pick(9, 6, 3000), top)


@pytest.mark.parametrize("dtype", [F4, BF, FH])
@pytest.mark.parametrize("vocab", [5, 1024, 50001])
@pytest.mark.parametrize("n", [4, 60, 400])
def test_ties(pkg, dtype, vocab, n):
    top = min(32, vocab)
    few = torch.randint(0, 3, (n, vocab), device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    rows = [0, 1, n - 1]
    check(pkg, few.to(dtype), pick(1, n, vocab), top, rows)
    check(pkg, torch.full((n, vocab), 2.5, device="cuda").to(dtype), pick(2, n, vocab), top, rows)
    zeros = torch.where(few == 1, -0.0, 0.0).to(dtype)          # -0 and 0 are equal
    check(pkg, zeros, pick(3, n, vocab), top, rows)


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("n", [1, 30, 300])
@pytest.mark.parametrize("vocab", [40000, 152064])
@pytest.mark.parametrize("period", [512, 2048, 4096])
def test_large_logits_that_recur(pkg, dtype, n, vocab, period):
    """The largest logits all in places that the same threads read."""
    x = rand(n, n, vocab, dtype, 1.0)
    v = torch.arange(vocab, device="cuda")
    for width in (4, 128):
        y = x + torch.where(v % period < width, 20.0, 0.0).to(dtype)
        check(pkg, y, pick(4, n, vocab), 32, [0, n - 1])


@pytest.mark.parametrize("dtype", [F4, BF, FH])
@pytest.mark.parametrize("n", [3, 90, 600])
@pytest.mark.parametrize("vocab", [40, 1000, 33333])
def test_masked_vocabularies(pkg, dtype, n, vocab):
    x = rand(5, n, vocab, dtype)
    g = torch.Generator(device="cuda").manual_seed(6)
    for share in (0.3, 0.99):
        y = x.masked_fill(torch.rand((n, vocab), device="cuda", generator=g) < share, -INF)
        check(pkg, y, pick(7, n, vocab), 20, [0, 1, n - 1])
    y = torch.full_like(x, -INF)                                # nothing is possible
    got = check(pkg, y, pick(8, n, vocab), 20, [0, n - 1])
    assert bool((got.entropy == 0).all())
    y[:, vocab // 2] = 3.0                                      # one token is
    got = check(pkg, y, [vocab // 2] * n, 20, [0, n - 1])
    assert bool((got.logprob == 0).all() and (got.entropy == 0).all() and (got.rank == 0).all())
    y = x.masked_fill(x < torch.finfo(dtype).max, torch.finfo(dtype).min)
    check(pkg, y, pick(9, n, vocab), 20, [0, n - 1])            # masks of the type's lowest value: all equal
    y[:, 3] = 0.5
    check(pkg, y, pick(10, n, vocab), 20, [0, n - 1])


@pytest.mark.parametrize("dtype", [F4, BF, FH])
@pytest.mark.parametrize("n", [3, 90, 600])
@pytest.mark.parametrize("vocab", [40, 1000, 33333])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_nan_and_infinity(pkg, dtype, n, vocab, bad):
    x = rand(11, n, vocab, dtype)
    tokens = pick(12, n, vocab)
    x[0, vocab // 3] = bad
    x[0, vocab - 1] = bad
    x[1] = bad
    x[2, ::2] = bad
    x[n - 1, 0] = bad
    x[n - 1, 1:] = -INF
    tokens[0] = vocab // 3
    got = check(pkg, x, tokens, 20, [0, 1, 2, n - 1])
    assert bool(torch.isnan(got.logprob[[0, 1, 2, n - 1]]).all() and torch.isnan(got.entropy[[0, 1, 2, n - 1]]).all())
    if n > 4:
        check(pkg, x[3:n - 1], tokens[3:n - 1], 20, [0, n - 5])


@pytest.mark.parametrize("n", [1, 50, 500])
def test_growing_rows(pkg, n):
    for sign in (1, -1):
        x = (torch.arange(30000, device="cuda") * (sign * 0.003)).expand(n, 30000)
        check(pkg, x, pick(13, n, 30000), 32, [0, n - 1])
    x = (torch.arange(30000, device="cuda") * 1.0e34).expand(n, 30000)
    check(pkg, x, pick(14, n, 30000), 32, [0, n - 1])


@pytest.mark.parametrize("n", [2, 64, 500])
def test_padding_rows_are_left(pkg, n):
    x = rand(15, n, 5000, BF)
    tokens = pick(16, n, 5000)
    for i, t in zip(range(0, n, 2), [-1, 5000, -2 ** 31, 2 ** 31 - 1] * n):
        tokens[i] = t
        x[i] = NAN
    f = lambda *s: torch.full(s, 7.0, device="cuda")
    kw = dict(logprob=f(n), entropy=f(n), rank=f(n).int(), top_ids=f(n, 5).int(), top_logprobs=f(n, 5))
    got = check(pkg, x, tokens, 5, range(1, min(n, 9), 2), **kw)
    for name, y in kw.items():
        assert getattr(got, name) is y
        assert bool((y[::2] == 7).all()) and not bool((y[1::2] == 7).any())


def test_same_result_in_every_run_and_on_another_stream(pkg):
    x, tokens = rand(17, 40, 152064, BF), i32(pick(18, 40, 152064))
    a = pkg.token_logprobs(x, tokens, top=32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    runs = [pkg.token_logprobs(x, tokens, top=32) for _ in range(4)] + [pkg.token_logprobs(x, tokens, top=32, stream=st)]
    torch.cuda.synchronize()
    for b in runs:
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    outs = [torch.zeros_like(y) for y in a]
    with torch.cuda.graph(graph):
        pkg.token_logprobs(x, tokens, 32, *outs)
    x.copy_(rand(19, 40, 152064, BF))
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(outs, pkg.token_logprobs(x, tokens, top=32)))


@pytest.mark.parametrize("n", [607, 609, 640, 700, 1300])
def test_passes_behind_one_another(pkg, n):
    """Logits written by the kernel before, results read by the one behind, at
    sizes that take whole waves of rows and a rest; padding in both."""
    tokens = i32(pick(23, n, 20011))
    tokens[::5] = -1
    outs = [torch.zeros_like(y) for y in pkg.token_logprobs(rand(24, n, 20011, BF), tokens, top=3)]   # (padding: left)
    xs = [rand(25 + i, n, 20011, BF) for i in range(6)]
    want = [[y.clone() for y in pkg.token_logprobs(x, tokens, 3, *outs)] for x in xs]
    torch.cuda.synchronize()
    x, got = torch.empty_like(xs[0]), []
    for src in xs:
        x.copy_(src)
        pkg.token_logprobs(x, tokens, 3, *outs)
        got.append([y.clone() for y in outs])
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_the_engines_verify_logits(pkg):
    """The target's choices are the logits' first ones; their log probabilities as
    the oracle has them from the same logits."""
    from synth import TINY_TARGET, make_weights
    shape, V = TINY_TARGET, TINY_TARGET.vocab
    eng = pkg.SpecEngine(shape, make_weights(shape, seed=11, device="cuda"), batch=2, K=4, s_max=128)
    eng.prefill([list(range(1, 30)), [5, 9, 5, 9, 5, 9, 5]])
    eng.set_drafter(pkg.SF_DRAFT_NGRAM, 2, 4)
    eng.ngram_draft(4)
    choice = torch.empty(2, 5, dtype=torch.int32, device="cuda")
    logits = torch.empty(2, 5, V, device="cuda")
    eng.verify(choice, logits)
    got = check(pkg, logits.view(10, V), choice.view(-1).tolist(), min(V, 8))
    assert bool((got.rank == 0).all()) and torch.equal(got.top_ids[:, 0], choice.view(-1))
    assert torch.equal(got.top_logprobs[:, 0], got.logprob)
    eng.accept_rollback()
    eng.close()


def test_outputs_left_out(pkg):
    import ctypes
    from greedy_speculative_decoding_gb300 import _lib as L
    lib = L.load()
    x, tokens = rand(20, 3, 1000, F4), i32([1, 2, 3])
    want = pkg.token_logprobs(x, tokens, top=4)
    outs = [torch.empty_like(y) for y in want]
    for keep in range(5):
        ptrs = [ctypes.c_void_p(o.data_ptr() if i == keep else None) for i, o in enumerate(outs)]
        L.check(lib.sf_token_logprobs(x.data_ptr(), L.SF_DT_F32, 1000, 3, 1000, tokens.data_ptr(), 4, *ptrs,
                                      torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert torch.equal(outs[keep], want[keep])


def test_no_rows_and_refusals(pkg):
    x, t = rand(21, 3, 100, F4), i32([1, 2, 3])
    assert pkg.token_logprobs(x[:0], t[:0], top=3).top_ids.shape == (0, 3)
    for kw in (dict(top=33), dict(top=101)):
        with pytest.raises(pkg.SFError):
            pkg.token_logprobs(x, t, **kw)
    for a in ((x.t(), i32([0] * 100)), (x.double(), t), (x, t.long()), (x, t[:2]), (x[0], t), (x.cpu(), t),
              (x.clone().requires_grad_(), t)):
        with pytest.raises(ValueError):
            pkg.token_logprobs(*a)
    with torch.no_grad():
        pkg.token_logprobs(x.clone().requires_grad_(), t)


def test_outputs_are_marked_as_changed(pkg):
    x, t = rand(22, 3, 100, F4), i32([1, 2, 3])
    out = pkg.token_logprobs(x, t, top=2)
    before = [o._version for o in out]
    pkg.token_logprobs(x, t, 2, *out)
    assert [o._version for o in out] == [v + 1 for v in before]
