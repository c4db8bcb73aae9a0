"""Routing of finite logits far from 0: rows whose largest logit is large in magnitude, and logits far
below it.  Bounds as in test_gpu_route: the exponent's error is relative to top - x alone, wherever top is."""
import itertools

import numpy as np
import pytest
import torch

import train_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import train
from test_gpu_route import both, f64, logits

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


LARGE = [1e5, 1e6, 1.1e6, 1e7, 1e8, 2e8, 1e9, 1e10, 1e20, 1e30, 9e37, 2e38]


@pytest.mark.parametrize("dtype,E,k", [("fp32", 40, 3), ("fp32", 100, 8), ("fp32", 160, 6), ("fp32", 256, 12),
                                       ("fp32", 600, 10), ("bf16", 40, 4), ("bf16", 190, 8), ("bf16", 300, 9)])
def test_rows_of_large_logits(dtype, E, k):
    """Whole rows of one large value of either sign, rows a few units in the last place around one,
    rows whose other logits hold a mask's -1e9, alone and among ordinary rows."""
    g = torch.Generator().manual_seed(E)
    rows = []
    for v in LARGE + [-v for v in LARGE]:
        rows += [torch.full((E,), v, dtype=torch.float64),
                 v * (1 + torch.randint(-4, 5, (E,), generator=g).double() * 2.0 ** (-23 if dtype == "fp32" else -8))]
        one = torch.full((E,), -abs(v), dtype=torch.float64)
        one[int(torch.randint(E, (1,), generator=g))] = 0.25
        rows.append(one)
        some = torch.randn(E, generator=g, dtype=torch.float64)
        some[torch.rand(E, generator=g) < 0.9] = -abs(v)
        rows.append(some)
    x = torch.stack(rows).to(torch.float32 if dtype == "fp32" else torch.bfloat16)
    for t in range(0, len(x), 7):
        both(x[t:t + 1].cuda(), k, normalize=t % 2 == 0, dtype=dtype)
    mixed = torch.cat([logits(len(x), E, dtype, E), x])[torch.randperm(2 * len(x), generator=g)]
    for normalize in (True, False):
        both(mixed.cuda(), k, normalize=normalize, dtype=dtype)
    assert torch.isfinite(train.route(mixed.cuda(), k).loss)
