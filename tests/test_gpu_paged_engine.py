"""The engine with its target's cache in pages (page plan, attention over the
pages) against the oracle and against the engine with one cache per sequence:
every drafter, ragged prompts, rewinds, a pool just large enough, a pool that
runs out. The plan and the lengths are integers; logits are compared with the
engine tests' tolerance (a share of each row's range).
"""

import numpy as np
import pytest
import torch

from oracle import model as om
from synth import TINY_DRAFT, TINY_TARGET, draft_from_target_layer0, make_weights, uniform_prompt
from synth.prompts import ngram_prompt

from gpu_helpers import LOGIT_TOL_BF16, logit_err, stream_report, to_cuda

pytestmark = pytest.mark.gpu
V = TINY_TARGET.vocab


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import greedy_speculative_decoding_gb300 as p
    return p


@pytest.fixture(scope="module", params=["bf16", "fp32"])
def tiny(request):
    dt = torch.float32 if request.param == "fp32" else torch.bfloat16
    tw = make_weights(TINY_TARGET, seed=0, dtype=dt)
    dw = draft_from_target_layer0(tw, TINY_DRAFT, 0.005, seed=1)
    gt, gd = to_cuda(tw), to_cuda(dw)
    gd["embed"], gd["norm"] = gt["embed"], gt["norm"]
    return om.Model(TINY_TARGET, tw), gt, gd


def engine(pkg, tiny, pages, batch=1, K=4, s_max=256, draft=True):
    _, gt, gd = tiny
    extra = (TINY_DRAFT, gd) if draft else (None, None)
    return pkg.SpecEngine(TINY_TARGET, gt, *extra, batch=batch, K=K, s_max=s_max, pages=pages)


def pages_for(tokens):
    return -(-tokens // 64)


def prompts_of(lens, seed=5):
    return [uniform_prompt(n, V, seed=seed + i).tolist() for i, n in enumerate(lens)]


@pytest.mark.parametrize("lens,K", [((32,), 4), ((70, 2, 129), 4), ((64, 64), 8), ((63, 65, 128, 30, 5), 3)])
@pytest.mark.parametrize("drafter", ["NEURAL", "NGRAM", "NONE", "TREE"])
def test_generates_the_oracles_stream(pkg, tiny, lens, K, drafter):
    m, _, _ = tiny
    n_new, B = 40, len(lens)
    prompts = [ngram_prompt(n, 0.8, V, seed=3 + i, base_len=64)[0].tolist() if drafter in ("NGRAM", "TREE") and n > 40
               else p for i, (n, p) in enumerate(zip(lens, prompts_of(lens)))]
    # Just the pages of the longest state the loop allows: two rounds ahead.
    pool = sum(pages_for(n - 1 + n_new + K + 2 * (K + 1)) for n in lens)
    eng = engine(pkg, tiny, pool, batch=B, K=K, draft=drafter == "NEURAL")
    eng.prefill(prompts)
    held, free = eng.pages_held()
    assert held.tolist() == [pages_for(n - 1) for n in lens] and free == pool - held.sum()
    eng.set_drafter(getattr(pkg, "SF_DRAFT_" + drafter), 2, 4)
    out, _ = eng.generate(n_new)
    held, free = eng.pages_held()
    assert free == pool - held.sum()
    eng.close()
    for b in range(B):
        stream_report(m, prompts[b], out[b].tolist(), LOGIT_TOL_BF16)


@pytest.mark.parametrize("drafter", ["NEURAL", "TREE"])
def test_rounds_agree_with_the_dense_engine(pkg, tiny, drafter):
    """Verify logits row by row within the tolerance of the dense engine's,
    accepted lengths equal wherever the choices are, pages as the lengths
    demand after every rewind."""
    lens, K = (100, 61, 7), 4
    prompts = prompts_of(lens)
    if drafter == "TREE":
        prompts = [ngram_prompt(100, 0.8, V, seed=1, base_len=64)[0].tolist()] + [[7] * 61, [3, 3, 3, 3, 3, 3, 3]]
    B, K1 = 3, K + 1
    dense, paged = (engine(pkg, tiny, p, batch=B, K=K, draft=drafter == "NEURAL") for p in (None, 12))
    for e in (dense, paged):
        e.prefill(prompts)
    for _ in range(5):
        res = []
        for e in (dense, paged):
            if drafter == "TREE":
                e.tree_draft(2, 2, 4)
            else:
                e.draft()
            logits = torch.zeros(B, K1, V, device="cuda")
            arg = torch.zeros(B, K1, dtype=torch.int32, device="cuda")
            e.verify(arg, logits)
            res.append((logits, arg, e.accept_rollback(), e.lengths()[0]))
        for b in range(B):
            for j in range(K1):
                assert logit_err(res[1][0][b, j], res[0][0][b, j]) < LOGIT_TOL_BF16
        if not torch.equal(res[0][1], res[1][1]):
            break   # a near tie: from here the two commit different tokens
        assert res[0][2][0].tolist() == res[1][2][0].tolist() and res[0][2][1] == res[1][2][1]
        assert res[0][3].tolist() == res[1][3].tolist()
    held, free = paged.pages_held()
    assert free == 12 - held.sum() and all(h >= pages_for(n) for h, n in zip(held, paged.lengths()[0]))
    dense.close()
    paged.close()


def test_rewound_rounds_and_reset_repeat_themselves(pkg, tiny):
    """sf_reset rewinds to the prompt: the same tokens again, from pages that
    went back and came again in another order."""
    eng = engine(pkg, tiny, 9, batch=2, K=4)
    eng.prefill(prompts_of((60, 120)))
    first, _ = eng.generate(50)
    eng.reset()
    again, _ = eng.generate(50)
    assert np.array_equal(first, again)
    eng.reset()
    steps = [[], []]
    for _ in range(6):
        for b, toks in enumerate(eng.step()):
            steps[b] += toks
    for b in range(2):
        n = min(50, len(steps[b]))
        assert steps[b][:n] == first[b].tolist()[:n]
    eng.prefill(prompts_of((5, 30), seed=40))
    held, free = eng.pages_held()
    assert held.tolist() == [1, 1] and free == 7
    eng.close()


def test_a_pool_that_runs_out(pkg, tiny):
    eng = engine(pkg, tiny, 3, batch=2, K=4)
    with pytest.raises(pkg.SFError) as e:
        eng.prefill(prompts_of((120, 70)))      # 2 + 2 pages
    assert e.value.status == 2
    eng.prefill(prompts_of((100, 40)))          # 2 + 1 pages
    with pytest.raises(pkg.SFError) as e:
        eng.generate(100)
    assert e.value.status == 2
    # What it has is still good: a step that fits, the same after a reset.
    eng.reset()
    a = eng.step()
    eng.reset()
    assert eng.step() == a
    eng.close()


def test_host_loop_gives_the_same_tokens(pkg, tiny, monkeypatch):
    prompts = prompts_of((50, 90))
    outs = []
    for host in ("0", "1"):
        monkeypatch.setenv("SF_HOST_LOOP", host)
        eng = engine(pkg, tiny, 8, batch=2, K=4)
        eng.prefill(prompts)
        outs.append(eng.generate(45)[0])
        eng.close()
    assert np.array_equal(*outs)


def test_nf4_target(pkg):
    tw = make_weights(TINY_TARGET.with_(ffn=704), seed=4)
    shape = TINY_TARGET.with_(ffn=704)
    q = pkg.quantize_model_nf4(shape, to_cuda(tw))
    outs = []
    prompt = prompts_of((90, 33))
    logits = []
    for pages in (None, 6):
        eng = pkg.SpecEngine(shape, q, batch=2, K=4, s_max=256, pages=pages)
        eng.prefill(prompt)
        eng.ngram_draft(4)
        lg = torch.zeros(2, 5, V, device="cuda")
        eng.verify(None, lg)
        eng.accept_rollback()
        logits.append(lg)
        outs.append(eng.generate(20)[0])
        eng.close()
    for b in range(2):
        for j in range(5):
            assert logit_err(logits[1][b, j], logits[0][b, j]) < LOGIT_TOL_BF16


def test_page_calls_of_an_engine_without_pages(pkg, tiny):
    eng = engine(pkg, tiny, None)
    with pytest.raises(pkg.SFError) as e:
        eng.pages_held()
    assert e.value.status == 5
    eng.close()
    with pytest.raises(pkg.SFError):
        engine(pkg, tiny, 0)


@pytest.mark.parametrize("drafter", ["NGRAM", "TREE", "NONE"])
def test_nf4_target_over_many_rounds(pkg, drafter):
    """NF4 weights: after every rewind the verify logits are the dense engine's
    (within the engine tests' tolerance), and what both then generate is the
    oracle's stream on the dequantised weights, up to the NF4 tolerance."""
    from test_gpu_nf4 import NF4_TOL, _oracle_nf4
    shape, K = TINY_TARGET.with_(ffn=768), 4
    gw, rw = _oracle_nf4(shape, make_weights(shape, seed=4))
    prompts = [ngram_prompt(90, 0.8, V, seed=2, base_len=40)[0].tolist(), [7, 9, 11] * 11]
    engines = [pkg.SpecEngine(shape, gw, batch=2, K=K, s_max=256, pages=p) for p in (None, 7)]
    for e in engines:
        e.prefill(prompts)
    rounds = 0
    for _ in range(12):
        res = []
        for e in engines:
            if drafter == "TREE":
                e.tree_draft(2, 1, 3)
            else:
                e.ngram_draft(4 if drafter == "NGRAM" else 1, 1, 3)
            logits, arg = torch.zeros(2, K + 1, V, device="cuda"), torch.zeros(2, K + 1, dtype=torch.int32, device="cuda")
            e.verify(arg, logits)
            res.append((logits, arg, e.accept_rollback()[0].tolist(), e.lengths()[0].tolist()))
        for b in range(2):
            for j in range(K + 1):
                assert logit_err(res[1][0][b, j], res[0][0][b, j]) < LOGIT_TOL_BF16
        rounds += 1
        if not torch.equal(res[0][1], res[1][1]):
            break   # a near tie: from here the two commit different tokens
        assert res[0][2:] == res[1][2:]
    assert rounds >= 3
    for e in engines:
        e.reset()
        e.set_drafter(getattr(pkg, "SF_DRAFT_" + drafter), 1, 3)
    outs = [e.generate(40)[0] for e in engines]
    m = om.Model(shape, rw)
    for out in outs:
        for b in range(2):
            stream_report(m, prompts[b], out[b].tolist(), NF4_TOL)
    for e in engines:
        e.close()


@pytest.mark.parametrize("pages", [None, 6])
@pytest.mark.parametrize("drafter", ["NEURAL", "NGRAM", "NONE", "TREE"])
@pytest.mark.parametrize("whole", [True, False])
def test_rounds_up_to_the_end_of_the_cache(pkg, tiny, pages, drafter, whole):
    """Every round that fits gives its tokens; the first that does not is
    refused, with everything as it was, and so is the one after it (with a
    cache per sequence, and in pages)."""
    m, _, _ = tiny
    K, s_max, prompts = 4, 128, [[5, 6, 7] * 20, ngram_prompt(90, 0.8, V, seed=3, base_len=64)[0].tolist()]
    eng = engine(pkg, tiny, pages, batch=2, K=K, s_max=s_max, draft=drafter == "NEURAL")
    eng.prefill(prompts)
    eng.set_drafter(getattr(pkg, "SF_DRAFT_" + drafter), 2, 4)

    def one_round():
        if whole:
            return eng.step()
        {"NEURAL": eng.draft, "TREE": lambda: eng.tree_draft(2, 2, 4)}.get(drafter, lambda: eng.ngram_draft(K, 2, 4))()
        eng.verify()
        return eng.accept_rollback()[1]

    got, committed = [[], []], [60, 90]
    for _ in range(s_max):
        fits = max(committed) + K + 1 <= s_max
        if not fits:
            break
        for b, t in enumerate(one_round()):
            got[b] += t
            committed[b] += len(t)
        assert [n + 1 for n in eng.lengths()[0].tolist()] == committed
    assert not fits
    for _ in range(2):
        with pytest.raises(pkg.SFError) as e:
            one_round()
        assert e.value.status == 2
        assert [n + 1 for n in eng.lengths()[0].tolist()] == committed
    for b in range(2):
        stream_report(m, prompts[b], got[b], LOGIT_TOL_BF16)
    eng.reset()
    first = one_round()
    assert all(t == g[:len(t)] for t, g in zip(first, got))
    eng.close()
