"""The training-step example: it learns with states of either width, its balance loss evens the
experts out, and the problems that it hands to the solver get the oracle's plans."""
import os
import sys

import pytest

from memory_aware_device_gb300 import build as nbuild
from oracle import oracle as O

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("bits", [32, 8])
def test_example_learns_and_plans(bits):
    import moe_step
    nbuild.build()
    O.build()
    block, seen = moe_step.learn(bits, 60)
    assert block.opt.steps == 60
    assert seen[-1][0] < 0.9 * seen[0][0]                 # the task
    assert seen[-1][1] < seen[0][1] and seen[-1][2] < seen[0][2]   # balance, and the fullest expert's load
    assert block.opt.opt_factor == (6 if bits == 32 else 3)
    times = []
    for capacity in (seen[0][2], seen[-1][2]):
        x, r = moe_step.plan(capacity, block.opt)
        o = O.solve(x)
        assert (r["status"], r["t_batch"], r["plan"]) == (o["status"], o["t_batch"], o["plan"]) and r["status"] == 0
        times.append(r["t_batch"])
    assert times[1] <= times[0]      # less to move, no worse a plan
