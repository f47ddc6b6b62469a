"""The beam search example when the pool runs out of pages: what the beams hold stays as it is."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("prompt", [50, 64])
def test_a_step_without_pages_writes_nothing(prompt):
    """Beams that share a partly filled page, and ones that need a new one; a beam that is served goes on."""
    from mxfp4_beam_decode import Beams
    d = Beams(beams=3, longest=200, seed=3)
    d.prompt(prompt)
    free = (d.refs == 0).nonzero()[:, 0]
    d.refs[free[1:]] = 1                         # another table holds all but one
    before, table, lens = [c.clone() for c in d.cache], d.table.clone(), d.lens.clone()
    live = table[0, :-(-prompt // 32)].long()
    _, out, lse = d.step()
    assert d.stats.read()["status"] & 8
    assert d.lens.tolist() == [prompt + 1, prompt, prompt]
    for a, b in zip(d.cache, before):
        assert torch.equal(a[live], b[live])
    assert torch.equal(d.table[1:], table[1:])
    # the beam that got the page has its token; the others see nothing
    assert torch.isfinite(lse[0]).all() and (lse[1:] == -float("inf")).all() and (out[1:] == 0).all()
    new = int(d.table[0, prompt // 32])
    assert new == int(free[0]) and not torch.equal(d.cache[0][new, :, prompt % 32], before[0][new, :, prompt % 32])
    # with pages again, the next step serves them all
    d.refs[free[1:]] = 0
    d.step()
    assert d.lens.tolist() == [prompt + 2, prompt + 1, prompt + 1]
