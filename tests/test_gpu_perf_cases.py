"""The measured cases answer for the inputs as they are at each call, not as they were at the first one."""
import importlib.util
import pathlib

import pytest
import torch

pytestmark = pytest.mark.gpu


def _cases():
    spec = importlib.util.spec_from_file_location("more_operators", pathlib.Path(__file__).parents[1] / "perf/more_operators.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_commit_case_follows_its_inputs(dtype):
    """start, n_path, path, the block table, k and v change in place between two calls on one state (counts shrink, too)."""
    m = _cases()
    case = dict(next(c for c in m.listed() if c["op"] == "commit"), batch=3, layers=2, nodes=7, hkv=2, start=100, dtype=dtype)
    st = m.prepare(case, 1)
    st["n_path"].fill_(7)
    st["path"].copy_(torch.arange(7, device="cuda"))
    for i in range(4):
        if i:
            st["start"].copy_(torch.tensor([5 * i, 17, 40 + i], device="cuda"))
            st["n_path"].copy_(torch.tensor([7 - 2 * i, 1, 0], device="cuda"))
            st["path"].copy_(st["path"].flip(1))
            st["block_table"].copy_(st["block_table"].flip(0))
            st["k"].neg_()
            st["v"].mul_(2)
        m.own = False
        want = m.run(st)
        m.own = True
        got = m.run(st)
        for f in ("k", "v"):
            assert torch.equal(got[f], want[f]), (i, f)
        assert int(st["err"]) == 0
