"""The serving example end to end: prompts in pieces, graph-replayed steps and a fork from an 8-bit snapshot give what
whole prompts give.

Tolerances (relative 2-norm).  Pieces and steps recompute the same bf16 pipeline with other roundings of a few
intermediate results (each 2^-9 at most, amplified by the projections' sums of random signs by about 1): 2e-2.
A snapshot's values are off by up to half of 1/127 of their row's largest, some 0.3% of it for each, which the
readout's sum over the states averages: 3e-2."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("name", ["HeadBlock", "ChannelBlock"])
@pytest.mark.parametrize("lens", [(150, 37, 64), (5, 300, 2)])
def test_serving_example(name, lens):
    import decode
    r = decode.run(getattr(decode, name)(), lens=lens)
    torch.cuda.synchronize()
    assert r["pieces"] <= 2e-2 and r["steps"] <= 2e-2 and r["fork"] <= 3e-2, r
