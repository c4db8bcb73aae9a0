"""Routing of finite logits far from 0: rows whose largest logit is large in magnitude, and logits far
below it.  Bounds as in test_gpu_route: the exponent's error is relative to top - x alone, wherever top is."""
import itertools

import numpy as np
import pytest
import torch

import train_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import train
from test_gpu_route import f64, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


@pytest.mark.parametrize("E,k,top", list(itertools.product([30, 40, 100, 160, 256, 600], [3, 6, 12],
                                                           [1.0, 3e37, 4e37, 5e37, 7e37, 9e37, 1e38, 1.2e38, 3e38])))
def test_finite_logits_far_below_the_largest_are_chosen(E, k, top):
    """Fewer than k logits within the exponent's range of the largest: the next ones are chosen all the same."""
    low = np.array([-1.2e38, -1.3e38, -1.46e38, -1.5e38, -1.9e38, -2e38, -2.2e38, -3e38])
    x = logits(61, E, "fp32", E + k)
    for t in range(0, 61, 2):
        g = np.random.default_rng(t)
        at = g.permutation(E)
        x[t] = -float("inf")
        x[t, at[1:1 + t % 3]] = top * 0.9
        x[t, at[0]] = top
        few = low[:6] if t % 4 else g.permutation(low)[:2]
        x[t, at[5:5 + len(few)]] = torch.tensor(few, dtype=torch.float32)
    got, want = train.route(x.cuda(), k), ref.route(f64(x), k)
    np.testing.assert_array_equal(got.ids.cpu().numpy(), want["ids"])
    np.testing.assert_array_equal(got.counts.cpu().numpy(), want["counts"])
