"""Routing operators on the GPU against their 64-bit forms.

Tolerances.  A gate is exp(x - top) / sum.  The exponential's relative error is at most
(2 + 1.173 |x - top|) 2^-23 by the function's stated bound, plus 2^-24 |x - top| for the rounded
difference; the sum carries the mean error of its parts (the mean of |x - top| under the gates is
at most ln E < 7) and at most 40 roundings of a tree over lanes; the products after it three more.
Together below (32 + 2.4 |x - top|) 2^-23.  Means add at most 2^-24 per sequential addition."""
import itertools

import numpy as np
import pytest
import torch

import train_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import nest, train

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def logits(T, E, dtype, seed, spread=1.5, closed=0, ties=False):
    g = np.random.default_rng(seed)
    x = g.normal(size=(T, E)) * spread + g.normal(size=E) * 0.5
    if ties:
        x = np.round(x * 2) / 2
        x[x == 0] *= np.where(g.random((x == 0).sum()) < 0.5, -1, 1)   # -0 and +0
    if closed:
        x[:, g.permutation(E)[:closed]] = -np.inf
    return torch.tensor(x).to(TYPES[dtype])


def f64(x):
    return x.double().cpu().numpy()


def gate_bound(x):
    """Relative bound of the gates of x [T, E] (64-bit)."""
    with np.errstate(all="ignore"):
        top = np.nanmax(np.where(np.isnan(x), -np.inf, x), axis=1, keepdims=True, initial=-np.inf)
        d = np.where(np.isfinite(x - top), top - x, 0.0)
    return (32 + 2.4 * d) * U


def check_forward(got, x, k, mask=None, normalize=True):
    r = ref.route(x, k, mask, normalize)
    T, E = x.shape
    np.testing.assert_array_equal(got.ids.cpu().numpy(), r["ids"])
    np.testing.assert_array_equal(got.counts.cpu().numpy(), r["counts"])
    assert int(got.tokens[0]) == r["tokens"]
    rel = gate_bound(x)
    w, want = f64(got.weights), r["weights"]
    at = np.maximum(r["ids"], 0)
    wrel = np.take_along_axis(rel, at, 1) if T else np.zeros((0, k))
    if normalize:   # the sum's error is that of its parts
        wrel = wrel + wrel.max(axis=1, keepdims=True, initial=0.0) + 8 * U
    np.testing.assert_array_equal(np.isnan(w), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(w - want)[ok] <= (wrel * np.abs(want) + 1e-37)[ok]).all()
    mean, want = f64(got.mean_prob), r["mean_prob"]
    np.testing.assert_array_equal(np.isnan(mean), np.isnan(want))
    if not np.isnan(want).any():
        depth = (1024 + T / 512) * 2.0 ** -24
        tol = (r["p"] * rel)[r["live"]].sum(0) / max(1, r["tokens"]) + want * depth + 1e-37
        assert (np.abs(mean - want) <= tol).all()
        lt = E * float((r["counts"] * tol).sum()) / (k * max(1, r["tokens"])) + r["loss"] * 2 * U
        assert abs(float(got.loss) - r["loss"]) <= lt
    else:   # a NaN gate reaches the loss wherever its expert or any expert was chosen
        assert np.isnan(float(got.loss)) == bool(np.isnan(r["loss"]))
    return r


def check_backward(got, x, r, dw, dl, normalize, dtype):
    want, scale = ref.route_backward(x, r, dw, dl, normalize)
    got = f64(got)
    rounding = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype]
    with np.errstate(all="ignore"):
        # p (d - mean): p and the mean carry the gates' error, d that of u, a few gates deep
        tol = r["p"] * scale[:, None] * (4 * gate_bound(x) + 128 * U) + np.abs(want) * rounding
    tol = tol + (2.0 ** -25 if dtype == "fp16" else 1e-37)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= tol[ok]).all(), float(np.nanmax(np.abs(got - want) / tol))
    assert (got[~r["live"]] == 0).all()


def both(x_dev, k, mask=None, normalize=True, seed=0, dtype="fp32"):
    """Forward and backward of x_dev on the GPU against the 64-bit forms."""
    x = f64(x_dev)
    m = mask.cpu().numpy() if mask is not None else None
    got = train.route(x_dev, k, mask=mask, normalize=normalize)
    r = check_forward(got, x, k, m, normalize)
    g = np.random.default_rng(seed + 99)
    dw = torch.tensor(g.normal(size=(x.shape[0], k)), dtype=torch.float32, device="cuda")
    dl = torch.tensor(0.37, device="cuda")
    back = train.route_backward(x_dev, got, dw, dl, mask=mask, normalize=normalize)
    assert back.dtype == x_dev.dtype and back.shape == x_dev.shape
    check_backward(back, x, r, f64(dw), float(dl), normalize, dtype)
    return got, r


SIZES = [(0, 8, 2), (1, 1, 1), (1, 64, 2), (2, 2, 2), (3, 7, 7), (31, 8, 1), (33, 31, 4), (64, 32, 32), (5, 33, 32),
         (257, 64, 6), (100, 72, 5), (129, 100, 3), (77, 128, 8), (65, 129, 8), (300, 160, 6), (40, 255, 8),
         (2048, 256, 8), (19, 257, 10), (50, 512, 16), (9, 513, 4), (7, 1000, 32), (13, 1024, 32), (4099, 60, 4),
         (20011, 16, 2)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_sizes(T, E, k, dtype):
    both(logits(T, E, dtype, T + E).cuda(), k, normalize=(T + k) % 2 == 0, dtype=dtype)


@pytest.mark.parametrize("dtype,E,normalize", list(itertools.product(["fp32", "bf16"], [5, 64, 250], [True, False])))
def test_mask_closed_and_ties(dtype, E, normalize):
    """Padding rows full of NaN, closed experts (fewer than k open in the second call), equal logits."""
    x = logits(333, E, dtype, E, ties=True, closed=E // 4).cuda()
    mask = torch.rand(333, generator=torch.Generator().manual_seed(E)) < 0.7
    x[~mask.cuda()] = float("nan")
    k = min(E, 6)
    both(x, k, mask.cuda(), normalize, dtype=dtype)
    both(x, k, mask.to(torch.uint8).cuda(), normalize, dtype=dtype)
    x[:, 2:] = -float("inf")
    both(x, k, mask.cuda(), normalize, dtype=dtype)


@pytest.mark.parametrize("E,k", [(6, 2), (32, 8), (33, 3), (64, 1), (64, 8), (100, 5), (200, 16), (256, 7), (256, 8),
                                 (256, 12), (300, 8), (512, 16), (700, 6), (1024, 32),
                                 (129, 3), (160, 6), (190, 8), (192, 8), (192, 4)])
def test_logits_that_differ_in_their_last_bits(E, k):
    """32-bit logits a few units in the last place apart, alone, in pairs and in crowds, among the
    chosen and at their end; large and small ones, and ones near 0 beside a large one."""
    g = np.random.default_rng(E + k)
    T = 500
    x = g.normal(size=(T, E)).astype(np.float32) * np.exp(g.normal(size=(T, 1)) * 2).astype(np.float32)
    for t in range(T):
        for _ in range(g.integers(1, 6)):
            crowd = g.permutation(E)[:g.integers(1, min(E, 2 + t % 9) + 1)]
            v = np.sort(x[t])[-int(g.integers(1, min(E, k + 3) + 1))]
            x[t, crowd] = (v.view(np.int32) + g.integers(-3, 4, len(crowd))).astype(np.int32).view(np.float32)
        if t % 5 == 0:
            x[t, g.integers(E)] = 200.0
    both(torch.tensor(x).cuda(), k)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("E", [40, 64, 100, 128, 160, 190, 256, 300, 1000])
def test_chosen_experts_side_by_side(E, dtype):
    """The largest logits of a row are neighbours, or 4, 8, 16, 32 or 64 apart, in rising, falling and
    equal order: however a row is laid out, some rows draw all their experts from one part of it."""
    steps, T = [s for s in (1, 4, 8, 16, 32, 64) if s < E], 90
    x = logits(T, E, dtype, E, spread=1.0)
    for t in range(T):
        step = steps[t % len(steps)]
        at = (t + step * torch.arange(12)) % E
        x[t, at] = {0: 8.0 - 0.25 * torch.arange(12.0), 1: 5.0 + 0.25 * torch.arange(12.0),
                    2: torch.full((12,), 6.0)}[t // len(steps) % 3].to(x.dtype)
    for k in (1, 2, 3, 4, 5, 8, 9):
        both(x.cuda(), k, dtype=dtype)


def test_rows_that_leave_nothing():
    x = logits(40, 24, "fp32", 3).cuda()
    x[::3] = -float("inf")
    both(x, 4)
    got, _ = both(x, 4, torch.zeros(40, dtype=torch.bool, device="cuda"))
    assert int(got.tokens[0]) == 0 and float(got.loss) == 0 and (got.mean_prob == 0).all() and (got.ids == -1).all()
    x[:] = -float("inf")
    both(x, 4)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_lowest_and_largest_values(dtype):
    """Masks of the type's lowest value, alone and in whole rows; the largest value; rows of zeros."""
    info = torch.finfo(TYPES[dtype])
    x = logits(12, 40, dtype, 5)
    x[0] = info.min
    x[1] = info.max
    x[2] = 0
    x[3, 5:] = info.min
    x[4, ::2] = info.min
    x[5, 3] = info.max
    x[6, 0], x[6, 1:] = info.min, -float("inf")
    both(x.cuda(), 8, dtype=dtype)


def test_nan_and_infinity_in_live_rows():
    x = logits(10, 48, "fp32", 7)
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    x[5] = float("nan")
    x[6, :] = -float("inf")
    x[6, 3] = float("nan")
    got = train.route(x.cuda(), 4)
    r = check_forward(got, f64(x), 4)
    assert set(np.nonzero(np.isnan(r["p"]).any(1))[0]) == {2, 4, 5, 6}
    back = train.route_backward(x.cuda(), got, torch.ones(10, 4, device="cuda"), None)
    assert torch.isnan(back[[2, 4, 5, 6]]).all() and torch.isfinite(back[[0, 1, 3, 7, 8, 9]]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strides(dtype):
    """Columns of a wider matrix at every offset, transposed logits, every other column, one row for
    all tokens, and a gradient written into columns of a wider matrix."""
    wide = logits(150, 100, dtype, 11).cuda()
    for off in range(9):
        both(wide[:, off:off + 64], 4, dtype=dtype)
    both(wide.t(), 5, dtype=dtype)
    both(wide[:, ::2], 5, dtype=dtype)
    both(wide[3:4].expand(17, 100), 5, dtype=dtype)
    x = wide[:, 3:35]
    r = train.route(x, 3)
    dl = torch.tensor(1.0, device="cuda")
    room = torch.full((150, 50), 7.0, dtype=wide.dtype, device="cuda")
    train.route_backward(x, r, None, dl, out=room[:, 5:37])
    assert torch.equal(room[:, 5:37], train.route_backward(x, r, None, dl))
    assert (room[:, :5] == 7).all() and (room[:, 37:] == 7).all()


def test_offsets_beyond_32_bits():
    T, E, stride = 40, 64, 2 ** 27 + 8
    x = logits(T, E, "bf16", 13).cuda()
    far = torch.empty((T - 1) * stride + E, dtype=torch.bfloat16, device="cuda")
    view = far.as_strided((T, E), (stride, 1))
    view.copy_(x)
    a, b = train.route(x, 4), train.route(view, 4)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    dl = torch.tensor(1.0, device="cuda")
    want = train.route_backward(x, a, a.weights, dl)
    train.route_backward(view, a, a.weights, dl, out=view)      # in place, at the far addresses
    assert torch.equal(view, want)


def test_repeatable_and_out():
    x = logits(30000, 96, "bf16", 17).cuda()
    a = train.route(x, 6)
    out = train.Routing.empty(30000, 96, 6)
    for t in out:
        t.fill_(77)
    b = train.route(x, 6, out=out)
    assert b is out
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    dw = torch.randn(30000, 6, device="cuda")
    assert torch.equal(train.route_backward(x, a, dw), train.route_backward(x, b, dw))


def test_parts_of_the_gradient():
    """No gradients at all give zero; each part alone adds up to both; ids that are no experts are skipped."""
    x = logits(200, 32, "fp32", 19).cuda()
    r = train.route(x, 4)
    dw, dl = torch.randn(200, 4, device="cuda"), torch.tensor(3.0, device="cuda")
    assert (train.route_backward(x, r) == 0).all()
    whole = train.route_backward(x, r, dw, dl)
    parts = train.route_backward(x, r, dw) + train.route_backward(x, r, None, dl)
    assert (whole - parts).abs().max() <= 1e-5 * whole.abs().max()
    bad = r._replace(ids=torch.where(r.ids == r.ids[0, 0], 10 ** 6, r.ids))
    skip = r._replace(ids=torch.where(r.ids == r.ids[0, 0], -1, r.ids))
    assert torch.equal(train.route_backward(x, bad, dw, dl), train.route_backward(x, skip, dw, dl))


def test_gate_has_gradients():
    x = logits(64, 16, "fp32", 23).cuda().requires_grad_()
    mask = torch.arange(64, device="cuda") % 5 != 0
    r = train.gate(x, 2, mask=mask)
    dw = torch.randn(64, 2, device="cuda")
    ((r.weights * dw).sum() + 0.5 * r.loss).backward()
    plain = train.route(x.detach(), 2, mask=mask)
    want = train.route_backward(x.detach(), plain, dw, torch.tensor(0.5, device="cuda"), mask=mask)
    assert torch.equal(x.grad, want)
    y = x.detach().clone().requires_grad_()
    train.gate(y, 2, mask=mask).loss.backward()       # the weights unused
    assert torch.equal(y.grad, train.route_backward(x.detach(), plain, None, torch.tensor(1.0, device="cuda"), mask=mask))


def test_other_streams_and_graphs():
    """A call on another stream than the tensors' own, and one captured and replayed on new logits."""
    x = logits(5000, 64, "bf16", 29).cuda()
    want = train.route(x, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = train.route(x, 4, stream=side)
    back = train.route_backward(x, got, got.weights, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    assert torch.equal(back, train.route_backward(x, want, want.weights))
    out, grad, graph = train.Routing.empty(5000, 64, 4), torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train.route(x, 4, out=out)
        train.route_backward(x, out, out.weights, out=grad)
    x.copy_(logits(5000, 64, "bf16", 31))
    graph.replay()
    want = train.route(x, 4)
    for p, q in zip(want, out):
        assert torch.equal(p, q)
    assert torch.equal(grad, train.route_backward(x, want, want.weights))


@pytest.mark.parametrize("T,E,k,dtype", [(12000, 256, 8, "fp32"), (10500, 300, 10, "bf16"), (40000, 64, 8, "fp16"),
                                         (30011, 160, 6, "bf16"), (14000, 190, 8, "fp32"), (18000, 100, 4, "fp32"), (9000, 513, 12, "fp32")])
def test_many_rows(T, E, k, dtype):
    """Several passes of every block over the rows, and as many blocks as there are."""
    both(logits(T, E, dtype, T + E).cuda(), k, dtype=dtype)


def test_workspace_between_calls():
    """The head of the workspace is zero after a call, whatever the rest of it held."""
    x = logits(3000, 200, "fp32", 5).cuda()
    want = train.route(x, 4)
    out = train.Routing.empty(3000, 200, 4)
    for _ in range(3):
        out.call.workspace[256:] = 255
        train.route(x, 4, out=out)
        assert (out.call.workspace[:256] == 0).all()
        for p, q in zip(want, out):
            assert torch.equal(p, q)


def test_refusals():
    x = logits(8, 16, "fp32", 1).cuda()
    r = train.route(x, 2)
    with pytest.raises(nest.NestError):
        train.route(x, 17)
    with pytest.raises(nest.NestError):
        train.route(x, 0)
    with pytest.raises(TypeError):
        train.route(x.double(), 2)
    with pytest.raises(TypeError):
        train.route(x, 2, mask=torch.ones(8, device="cuda"))
    with pytest.raises(ValueError):
        train.route(x, 2, mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        train.route(x, 2, mask=torch.ones(8, dtype=torch.bool))
    with pytest.raises(ValueError):
        train.route(x, 3, out=r)
    with pytest.raises(ValueError):
        train.route_backward(x[:4], r)
    with pytest.raises(ValueError):
        train.route_backward(x, r, grad_weights=torch.zeros(8, 3, device="cuda"))
    with pytest.raises(ValueError):
        train.route_backward(x, r, grad_weights=torch.zeros(2, 8, device="cuda").t())
    with pytest.raises(ValueError):
        train.route_backward(x, r, grad_loss=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        train.route_backward(x, r, out=torch.empty(16, 8, device="cuda").t())
    with pytest.raises(ValueError):
        train.route_backward(x, r, out=x.bfloat16())
