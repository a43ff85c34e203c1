"""Log probabilities of given tokens from rows of logits, as the engine's verify
leaves them. Argument marshalling over the C ABI."""

from typing import NamedTuple

import torch

from . import _lib as L
from . import paged
from .paged import _device, _empty


class TokenLogprobs(NamedTuple):
    """What token_logprobs leaves: the given tokens' log probabilities, the
    rows' entropies, the given tokens' ranks (0: the first choice), and the
    first choices with their log probabilities."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    rank: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor


def token_logprobs(logits, tokens, top: int = 0, logprob=None, entropy=None, rank=None, top_ids=None,
                   top_logprobs=None, stream=None) -> TokenLogprobs:
    """Log probabilities of tokens int32 [n] under logits [n, vocab] (fp32, bf16
    or fp16, rows any stride apart), with entropy, rank and the `top` (0..32)
    most probable tokens, larger logits first and of equal ones the lower token
    (sf_token_logprobs). Outputs fp32 [n], fp32 [n], int32 [n], int32 [n, top]
    and fp32 [n, top] are allocated unless given. Rows whose token lies outside
    the vocabulary (-1, say) are padding: nothing is written for them, so what
    is allocated here is undefined there. Work is enqueued on ``stream``
    (default: the current stream); there is no gradient."""
    call = (paged._native or paged._binding()).token_logprobs
    dev, st = _device(stream)
    if logprob is None:
        logprob = _empty(logits.shape[0], torch.float32, dev, stream)
    if entropy is None:
        entropy = _empty(logits.shape[0], torch.float32, dev, stream)
    if rank is None:
        rank = _empty(logits.shape[0], torch.int32, dev, stream)
    if top_ids is None:
        top_ids = _empty((logits.shape[0], top), torch.int32, dev, stream)
    if top_logprobs is None:
        top_logprobs = _empty((logits.shape[0], top), torch.float32, dev, stream)
    s = call(dev, st, top, logits, tokens, logprob, entropy, rank, top_ids, top_logprobs)
    if s:
        L.check(s)
    return TokenLogprobs(logprob, entropy, rank, top_ids, top_logprobs)
