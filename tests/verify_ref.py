"""The verification of drafted trees on rows of any content, in 64 bits: NaN and negative probabilities, of the target and
of the draft, are taken as 0 before anything else, as include/ice.h states; the walk itself is tree_ref's, which is right on
rows of probabilities."""
import math

import torch

import tree_ref


def clean(x):
    return torch.where(x > 0, x, torch.zeros_like(x))


def verify(target, draft, tokens, parents, uniform, n):
    """As tree_ref.verify."""
    target = clean(target)
    if uniform is None:  # a row without probability has no likeliest token
        target = torch.where((target > 0).any(-1, keepdim=True), target, torch.full_like(target, math.nan))
        draft = None
    if draft is not None:  # beyond any other number, but 0 times it is 0
        draft = clean(draft).clamp(max=1e300)
    return tree_ref.verify(target, draft, tokens, parents, uniform, n)
