"""Attention of drafted trees at the ends of the number ranges: scores whose keys, queries or scale are near fp32's ends, values
near the largest that a sum holds, infinities and NaN of nodes that weigh nothing, elements far below their row's largest."""
import math

import pytest
import torch

import cache4_ref as ref4
import semantic_paged_kv_gb300 as ice
import tree_ref as ref
from test_gpu_tree import D, S, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ks,qs,scale", [
    (1e34, 1e-34, None), (1e35, 1e-35, None), (3e36, 1e-37, None), (1e-36, 1e36, None), (1e-30, 1e35, 1e-6),
    (1e36, 1.0, 1e-37), (1.0, 1e36, 1e-37), (1e18, 1e18, 1e-37), (1e-18, 1e-18, 1e35), (1e33, 1e-36, 1e2)])
def test_scores_at_the_ends_of_the_range(ks, qs, scale, dtype):
    """Keys, queries and scale far apart whose scores are ordinary: rows of cached tokens, of nodes, and of runs that are joined."""
    for lens in ([200, 33], [5000, 0]):
        c = Case(2, 9, 8, 2, dtype, True, lens, seed=7, k_scale=ks, q_scale=qs)
        if scale:
            c.scale = scale
        c.run()
        assert ice.ice_check(c.err) == ice.ICE_OK
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_keys_of_very_different_size(dtype):
    """A few keys beyond 2^112 among ordinary ones that are tiny beside them, with queries that make the large ones ordinary."""
    c = Case(2, 9, 8, 2, dtype, True, [300, 40], seed=11, q_scale=1e-34)
    big = torch.tensor([1e34 if i % 5 == 0 else 1.0 for i in range(c.recs.shape[0])], device="cuda")
    k, v = ref4.decode(c.recs.view(-1, 2304))
    fine = torch.isfinite(k).all(-1).all(-1) & torch.isfinite(v).all(-1).all(-1)
    k = (torch.nan_to_num(k).view(-1, c.hkv, S, D) * big[:, None, None, None]).view(-1, S, D)
    new = ref4.encode(k.bfloat16(), torch.nan_to_num(v).bfloat16())
    c.recs.copy_(torch.where(fine[:, None], new, c.recs.view(-1, 2304)).view_as(c.recs))
    c.k[:, ::3] *= 1e34
    c.run()
    assert ice.ice_check(c.err) == ice.ICE_OK
    c.check()
