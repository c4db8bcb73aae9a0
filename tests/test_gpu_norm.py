"""The gradient norm against a bound that follows its sums.

With u = 2^-24 and all terms positive, the sum of squares is off by at most 16 u for a thread's runs of
up to 16 products, 1 u for adding the runs up (the rounding errors of these additions are added up
beside them, which leaves the last rounding and a part of order n^2 u^2), 5 u for a tree over the
lanes and 5 u for one over the warps; the blocks' sums again 1 u, 5 u and 5 u.  Together 38 u: 19 u
of the norm, and 1 u for the root.  The clip scale adds one addition and one division: 22 u."""
import math

import numpy as np
import pytest
import torch

from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import train
from test_gpu_optim import LISTS, f64, make

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def check(norm, want):
    got, clip = norm.run(max_norm=0.7 * want).tolist(), min(1.0, 0.7 * want / (want + 1e-6))
    assert abs(got[0] - want) <= 20 * U * want, (got[0] / want - 1) / U
    assert abs(got[1] - clip) <= (22 + 1) * U * clip     # max_norm is rounded to 32 bits once


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("numels", LISTS + [[3000001, 5], [20_000_003, 77, 1_000_000]])
def test_norm_within_its_bound(numels, dtype):
    for shift in (0, 1, 7):
        g = make(numels, dtype, len(numels) + shift, shift=shift)
        check(train.GradNorm(g), math.sqrt(math.fsum((f64(t) ** 2).sum() for t in g)))


@pytest.mark.parametrize("value", [1.1502795219421387, 1.4765883684158325, 1.655121088027954])
def test_norm_of_many_equal_values(value):
    """About 215 runs to a thread, whose additions all round to one side: without the errors added up
    beside the sum the norm is off by 26 u."""
    v, n = np.float32(value), 2 ** 30 + 12345
    assert float(v) == value
    run = np.float32(0)
    for _ in range(16):
        run = np.float32(float(v) * float(v) + float(run))
    total = np.float32(0)
    for _ in range(215):
        total = np.float32(total + run)
    assert abs(math.sqrt(total / (215 * 16 * value * value)) - 1) > 25 * U
    check(train.GradNorm([torch.full((n,), value, device="cuda")]), math.sqrt(n) * value)
