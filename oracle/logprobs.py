"""Float64 reference of token log probabilities, row by row."""

import torch

F64 = torch.float64


def order(x):
    """Tokens of a row, larger logits first, of equal ones the lower token; a
    NaN counts as -infinity."""
    x = torch.where(torch.isnan(x), float("-inf"), x.to(F64))
    return torch.sort(x, descending=True, stable=True).indices


def row(x, token):
    """(log probabilities [vocab], entropy, rank of the token, order, sum of
    p |d| and of p d^2 with d the distance to the largest logit)."""
    first = order(x)
    rank = int(torch.nonzero(first == token)[0, 0])
    x = x.to(F64)
    if bool((x == float("-inf")).all()):
        return torch.full_like(x, float("-inf")), 0.0, rank, first, 0.0, 0.0
    if bool(torch.isnan(x).any()) or bool((x == float("inf")).any()):
        nan = float("nan")
        return torch.full_like(x, nan), nan, rank, first, 0.0, 0.0
    d = x - x.max()                                  # (first: -1e38 and the logarithm of a sum do not add up)
    logp = d - torch.log(torch.exp(d).sum())
    p = torch.exp(logp)
    d = torch.where(p > 0, d, 0.0)
    entropy = -float((p * torch.where(p > 0, logp, 0.0)).sum())
    return logp, entropy, rank, first, float((p * -d).sum()), float((p * d * d).sum())
