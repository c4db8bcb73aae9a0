"""The output head's losses where the formulas meet infinities, extremes and long sums.  Bounds as in head_ref."""
import itertools

import pytest
import torch

import head_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import head
from test_gpu_head import INF, backward, forward, made, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


@pytest.mark.parametrize("T,V,D,first,count", [
    (*size, *columns) for size, columns in itertools.product(
        [(5, 600, 64), (70, 600, 64), (300, 1500, 72), (33, 40, 8)],
        [(0, 32), (32, 32), (64, 32), (0, 1), (31, 2), (256, 32), (0, 256), (512, 64)]) if sum(columns) < size[1]])
def test_nan_in_weights_reaches_every_loss(T, V, D, first, count):
    """Wherever the columns lie in a tile, and whatever the columns beside them hold."""
    for k in (0, 6):
        x = made(T, V, D, "bf16", k=k)
        x["labels" if not k else "ids"].fill_(V - 1)
        x["weight"][first:first + count] = float("nan")
        r = forward(x)
        assert torch.isnan(r.losses).all() and torch.isnan(r.lse).all() and torch.isnan(r.loss)
        assert int(r.tokens[0]) == T
        dh, dw = backward(x, r, torch.ones((), device="cuda"))
        assert torch.isnan(dh).all() and torch.isnan(dw[first:first + count]).all()


def closed(T, V, D, dtype, closed_columns, k=0, dead=0.0, seed=0):
    """(inputs whose logits of these columns are minus infinity, by a bias column; the same without those columns;
    the open columns)"""
    x = made(T, V, D, dtype, k=k, dead=dead, seed=seed)
    x["hidden"][:, D - 1] = torch.where(torch.isnan(x["hidden"][:, D - 1]), x["hidden"][:, D - 1], 1.0)
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    for a, b in closed_columns:
        keep[a:b] = False
    columns = keep.nonzero()[:, 0]
    name = "ids" if k else "labels"
    at = x[name] % len(columns)
    live = torch.ones_like(at, dtype=torch.bool) if k else x[name] >= 0
    y = x | {"weight": x["weight"][columns], name: torch.where(live, at, -100)}
    x[name] = torch.where(live, columns[at], -100)
    x["weight"][~keep, D - 1] = -INF
    return x, y, columns


@pytest.mark.parametrize("dtype,k", [("bf16", 0), ("bf16", 7), ("fp16", 0), ("fp16", 40)])
@pytest.mark.parametrize("T,V,ranges", [
    (5, 300, [(0, 32)]), (5, 300, [(32, 64)]), (90, 300, [(0, 32)]), (90, 300, [(32, 64)]), (90, 300, [(0, 64)]),
    (90, 300, [(64, 300)]), (90, 700, [(0, 256)]), (300, 2000, [(256, 1024)]), (300, 2000, [(0, 1999)]),
    (300, 2000, [(1, 2000)]), (12, 2000, [(0, 777), (778, 2000)]), (257, 2000, [(0, 777), (778, 2000)]),
    (40, 1000, [(i, i + 32) for i in range(0, 1000, 64)]), (40, 1000, [(i + 32, i + 64) for i in range(0, 960, 64)])])
def test_columns_of_minus_infinity_add_nothing(T, V, ranges, dtype, k):
    """As if they were not there: a part of the vocabulary that is closed by a bias.  (Of the bias itself the gradient
    of the hidden states is 0 * -inf.)"""
    D = 64
    x, y, columns = closed(T, V, D, dtype, ranges, k=k, dead=0.2)
    dl, r = torch.ones((), device="cuda"), forward(x)
    want = ref.loss(y, dl)
    assert int(r.tokens[0]) == want["tokens"]
    for name in ("losses", "lse", "loss"):
        near(getattr(r, name), want[name], want[name + "_off"], name)
    dh, dw = backward(x, r, dl)
    near(dh[:, :-1], want["dh"][:, :-1], want["dh_off"][:, :-1], "grad_hidden")
    near(dw[columns], want["dw"], want["dw_off"], "grad_weight")
    dw[columns] = 0
    assert not dw.any()


@pytest.mark.parametrize("T", [3, 80])
def test_labels_in_closed_columns_and_rows_that_are_closed(T):
    """A target that cannot be has an infinite loss; where nothing can be there is no loss."""
    for ranges, k in itertools.product(([(0, 32)], [(32, 64)], [(0, 256)], [(256, 300)]), (0, 4)):
        x, y, _ = closed(T, 300, 64, "bf16", ranges, k=k)
        want = ref.loss(y)
        name = "ids" if k else "labels"
        x[name] = x[name].clone()
        x[name][1] = ranges[0][0]
        r = forward(x)
        assert float(r.losses[1]) == INF and float(r.loss) == INF
        others = torch.arange(T, device="cuda") != 1
        near(r.losses[others], want["losses"][others], want["losses_off"][others], "losses")
        near(r.lse, want["lse"], want["lse_off"], "lse")
        x["weight"][:, 63] = -INF
        r = forward(x)
        assert torch.isnan(r.losses).all() and torch.isnan(r.loss) and (r.lse == -INF).all()
        dh, dw = backward(x, r, torch.ones((), device="cuda"))
        assert torch.isnan(dh).all() and torch.isnan(dw).all()


def test_temperatures_that_are_tensors():
    """A temperature that is changed in place counts as it is at each call, and at the forward call for its gradient."""
    x = made(50, 300, 64, "bf16", k=6)
    dl, heat = torch.ones((), device="cuda"), torch.tensor(2.0)
    for value in (2.0, 4.0, 0.5):
        heat.fill_(value)
        r, want = forward(x | {"temperature": heat}), forward(x | {"temperature": value})
        assert torch.equal(r.losses, want.losses) and torch.equal(r.lse, want.lse)
        grads = backward(x | {"temperature": value}, want, dl), backward(x | {"temperature": heat}, want, dl)
        assert all(torch.equal(p, q) for p, q in zip(*grads))
        h = x["hidden"].clone().requires_grad_()
        s = head.teacher_loss(h, x["weight"], x["ids"], x["teacher"], temperature=heat)
        heat.fill_(3.0)
        s.loss.backward()
        assert torch.equal(s.losses, want.losses) and torch.equal(h.grad, grads[0][0])


@pytest.mark.parametrize("k", [0, 5])
def test_losses_changed_in_place_before_the_backward_pass(k):
    """The backward pass reads lse alone: weighting the losses where they lie is no error, changing lse is."""
    x = made(40, 200, 64, "bf16", k=k)
    w = torch.rand(40, device="cuda")

    def losses():
        h = x["hidden"].clone().requires_grad_()
        if k:
            return h, head.teacher_loss(h, x["weight"], x["ids"], x["teacher"])
        return h, head.label_loss(h, x["weight"], x["labels"])
    h, r = losses()
    (r.losses * w).sum().backward()
    g, s = losses()
    s.losses.mul_(w)
    s.losses.sum().backward()
    assert torch.equal(g.grad, h.grad)
    h, r = losses()
    (r.loss * 0.5).backward()
    g, s = losses()
    s.loss.mul_(0.5)
    s.loss.backward()
    assert torch.equal(g.grad, h.grad)
    g, s = losses()
    s.lse.add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        s.loss.backward()


@pytest.mark.parametrize("k", [0, 4])
def test_results_over_inputs_are_refused(k):
    """Wherever in an input's memory they begin; a result between the rows of an input is not over it."""
    T, V, D = 24, 80, 16
    x = made(T, V, D, "bf16", k=k)
    room = torch.zeros(T + V, 2 * D, dtype=torch.bfloat16, device="cuda")
    hidden, weight = room[:T, :D], room[T:, :D]
    hidden.copy_(x["hidden"])
    weight.copy_(x["weight"])
    x |= {"hidden": hidden, "weight": weight, "mask": torch.ones(T, dtype=torch.bool, device="cuda")}
    name = "ids" if k else "labels"
    r, dl, dls = forward(x), torch.ones((), device="cuda"), torch.ones(T, device="cuda")
    dh, dw = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    want = [t.clone() for t in (*r, *backward(x, r, dl, dls))]
    flat, long = room.view(-1), torch.zeros(4000, dtype=torch.bfloat16, device="cuda")
    index = long[400:].view(x[name].dtype)[:x[name].numel()].view(x[name].shape).copy_(x[name])
    lse, rows, one = long.view(torch.float32)[100:100 + T], long.view(torch.float32)[200:200 + T], long.view(torch.float32)[300]
    for y, result, first, second in [
            (x, r, flat[D:D + T * D], dw), (x, r, dh, flat[3 * D:3 * D + V * D]), (x, r, dh, flat[(2 * T - 1) * D:][:V * D]),
            (x | {name: index}, r, long[300:300 + T * D], dw), (x, r, dw.view(-1)[8:8 + T * D], dw),
            (x | {"hidden": dw[-T:]}, r, dh, dw), (x, r._replace(lse=lse), long[190:190 + T * D], dw)]:
        with pytest.raises(ValueError, match="shares memory"):
            backward(y, result, dl, dls, out=(first.view(T, D), second.view(V, D)))
    for at in (dict(dl=dl, dls=rows), dict(dl=one, dls=dls), dict(dl=one)):
        with pytest.raises(ValueError, match="shares memory"):
            backward(x, r, out=(long[230:230 + T * D].view(T, D), dw), **at)
    good = head.HeadLoss(*(torch.empty_like(t) for t in r))
    places = [good._replace(lse=good.losses), good._replace(loss=good.losses[3]),
              good._replace(losses=flat.view(torch.float32)[2:2 + T]), good._replace(tokens=good.lse.view(torch.int32)[5:6])]
    if k:
        places += [good._replace(lse=x["teacher"].view(-1)[1:1 + T]), good._replace(losses=x["ids"].view(-1).view(torch.float32)[:T]),
                   good._replace(tokens=x["mask"].view(torch.int32)[3:4])]
    else:
        places.append(good._replace(losses=x["labels"].view(torch.float32)[T:]))
    for out in places:
        with pytest.raises(ValueError, match="shares memory"):
            forward(x, out=out)
    # one token: its gradient may lie beside it in its row
    y = {"hidden": hidden[:1], "weight": x["weight"], "labels": torch.zeros(1, dtype=torch.int64, device="cuda")}
    s = forward(y)
    plain = backward(y, s, dl)
    assert all(torch.equal(p, q) for p, q in zip(plain, backward(y, s, dl, out=(room[:1, D:], dw))))
    got = (*forward(x, out=good), *backward(x, good, dl, dls, out=(dh, dw)))
    assert all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.parametrize("temperature", [2.0 ** -10, 0.5, 0.7, 1.0, 3.0])
@pytest.mark.parametrize("teacher", [torch.float32, torch.bfloat16])
def test_extreme_teacher_logits_at_any_temperature(teacher, temperature):
    """Whether a slot counts goes by its logit, not by what dividing it gives; the largest logits share the mass."""
    low, high = torch.finfo(teacher).min, torch.finfo(teacher).max
    x = made(60, 300, 64, "bf16", k=6, teacher=teacher, temperature=temperature)
    dl = torch.ones((), device="cuda")

    def same(rows, slots):
        """The rows are as if their slots were those, of equal logits, and the others closed."""
        r, y = forward(x), x | {"teacher": x["teacher"].clone()}
        y["teacher"][rows] = -INF
        y["teacher"][rows, slots] = 0
        s = forward(y)
        assert int(r.tokens[0]) == 60 and torch.equal(r.losses, s.losses) and torch.equal(r.loss, s.loss)
        assert all(torch.equal(p, q) for p, q in zip(backward(x, r, dl), backward(y, s, dl)))
    x["teacher"][:20] = low                      # nothing but the lowest: all slots alike
    same(slice(0, 20), slice(0, 6))
    x["teacher"][20:30] = low
    x["teacher"][20:30, 2:4] = high              # two of the largest
    same(slice(20, 30), slice(2, 4))
    x["teacher"][30:40, 1] = high                # one, by more than any quotient holds
    same(slice(30, 40), slice(1, 2))
    x["teacher"][40] = -INF                      # closed at any temperature
    assert int(forward(x).tokens[0]) == 59


@pytest.mark.parametrize("T", [10, 90])
def test_listed_columns_of_share_zero_add_nothing(T):
    """Where the model's logit is minus infinity too: as if they were not listed."""
    x, _, columns = closed(T, 300, 64, "bf16", [(0, 40), (100, 290)], k=6)
    y = x | {"teacher": x["teacher"].clone()}
    x["ids"][:, 2], x["ids"][::2, 4] = 17, 288
    x["teacher"][:, 2], x["teacher"][::2, 4] = -1e9, -2000.0
    y["teacher"][:, 2], y["teacher"][::2, 4] = -INF, -INF
    r, s, dl = forward(x), forward(y), torch.ones((), device="cuda")
    assert torch.isfinite(r.losses).all()
    assert torch.equal(r.losses, s.losses) and torch.equal(r.loss, s.loss) and torch.equal(r.lse, s.lse)
    p, q = backward(x, r, dl), backward(y, s, dl)
    assert torch.equal(p[0][:, :-1], q[0][:, :-1]) and torch.equal(p[1], q[1])


@pytest.mark.parametrize("T,V,D", [(2 ** 21, 8300, 8), (2 ** 18 + 77, 24, 64)])
def test_long_sums_over_tokens(T, V, D):
    """All terms of the weights' gradient have one sign in columns that are no label, so that what each addition
    cuts off adds up.  Bound: half a step of 2^-10 for dz and for the result, and of a sum that grows evenly in
    parts of at most 2^17 tokens a step of 2^-23 of half the part for every 16 tokens."""
    g = torch.Generator(device="cuda").manual_seed(T)
    hidden = (1 + torch.rand(T, D, generator=g, device="cuda")).half()
    weight = (torch.rand(V, D, generator=g, device="cuda") * 0.01).half()
    labels = torch.randint(1, V - 1, (T,), generator=g, device="cuda")
    r = head.cross_entropy(hidden, weight, labels)
    dl = torch.tensor(1000.0, device="cuda")
    dw = head.cross_entropy_backward(hidden, weight, labels, r, dl, needs=(False, True))[1]
    assert torch.equal(dw, head.cross_entropy_backward(hidden, weight, labels, r, dl)[1])
    want, w = torch.zeros(2, D, dtype=torch.float64, device="cuda"), weight.double()
    for a in range(0, T, 2 ** 16):
        h = hidden[a:a + 2 ** 16].double()
        z = h @ w.T
        want += torch.exp(z[:, [0, V - 1]] - torch.logsumexp(z, 1)[:, None]).T @ h
    want *= 1000 / T
    bound = 2 * 2.0 ** -11 + min(T, 2 ** 17) / 16 * 2.0 ** -24 + 2.0 ** -16
    got = ((dw[[0, V - 1]].double() - want).abs() / want).max()
    assert got <= bound, (float(got), bound)


@pytest.mark.parametrize("dtype,per", [("bf16", 0.26), ("fp16", 0.30)])
@pytest.mark.parametrize("D", [64, 4096, 16384])
def test_logits_whose_sums_lose_nothing(D, dtype, per):
    """Rows of one number, and short rows padded with zeros: their logits are exact on the tensor cores, and get the
    factor of all logits, per * D / 16 steps of 2^-24."""
    T, V = 64, 40
    g = torch.Generator(device="cuda").manual_seed(D)
    kind = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    for width in (1, 8):
        hidden, weight = torch.zeros(T, D, device="cuda"), torch.zeros(V, D, device="cuda")
        at = torch.randint(0, D // 8, (1,), generator=g, device="cuda").item() * 8
        hidden[:, at:at + width] = torch.randint(-8, 9, (T, width), generator=g, device="cuda").float()
        weight[:, at:at + width] = torch.randint(-4, 5, (V, width), generator=g, device="cuda").float()
        x = {"hidden": hidden.to(kind), "weight": weight.to(kind),
             "labels": torch.randint(0, V, (T,), generator=g, device="cuda")}
        r, z = forward(x), hidden.double() @ weight.double().T
        lse, size = torch.logsumexp(z, 1), z.abs().amax(1)
        given = per * (D // 16) * 2.0 ** -24
        picked = z.gather(1, x["labels"][:, None])[:, 0]
        # the exponentials and the logarithm within 2^-19, the last operations within 2^-22 of their terms
        off = 2.0 ** -19 + 2.0 ** -22 * size
        near(r.lse, lse, size * given * 1.01 + off, "lse")
        near(r.losses, lse - picked, 2 * size * given * 1.01 + off, "losses")


@pytest.mark.parametrize("dtype,per", [("bf16", 0.26), ("fp16", 0.30)])
@pytest.mark.parametrize("D", [1024, 4096])
@pytest.mark.parametrize("signs", ["one", "both"])
def test_the_factor_of_logits_brings_dense_sums_nearer(D, dtype, per, signs):
    """One column, whose logit lse is: nearer to the sum, by the root of the mean square, than without the factor."""
    g = torch.Generator(device="cuda").manual_seed(D + 1)
    kind = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    if signs == "one":
        hidden, weight = (torch.rand(n, D, generator=g, device="cuda") for n in (2000, 1))
    else:   # rows that lean towards the column, as those of a model which has learnt its labels
        weight = torch.randn(1, D, generator=g, device="cuda") * 2 * D ** -0.5
        hidden = torch.randn(2000, D, generator=g, device="cuda") + 2 * weight * torch.rand(2000, 1, generator=g, device="cuda")
    x = {"hidden": hidden.to(kind), "weight": weight.to(kind), "labels": torch.zeros(2000, dtype=torch.int64, device="cuda")}
    z = (x["hidden"].double() @ x["weight"].double().T)[:, 0]
    got = forward(x).lse.double()
    with_, without = got - z, got / (1 + per * (D // 16) * 2.0 ** -24) - z
    assert float(with_.square().mean()) < float(without.square().mean())


def test_no_wait_gives_up():
    """NaN of the inputs is told from that of a wait that gave up."""
    x, dl = made(600, 3000, 128, "bf16"), torch.ones((), device="cuda")
    x["hidden"][5] = float("nan")
    for dtype in ("bf16", "fp16"):
        y = x | {n: x[n].to({"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]) for n in ("hidden", "weight")}
        r = forward(y)
        assert torch.isnan(r.loss) and torch.isnan(backward(y, r, dl)[1]).any()
    assert head.waits_given_up() == 0 and head.waits_given_up(x["hidden"].device, torch.cuda.Stream()) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = forward(x)
        with pytest.raises(RuntimeError, match="capture"):
            head.waits_given_up()
    graph.replay()
    assert head.waits_given_up() == 0 and torch.isnan(r.loss)


def test_the_gradient_of_a_broadcast_row_against_64_bits():
    """One hidden state for all tokens: autograd adds the rows' gradients in 32 bits and rounds once."""
    x = made(60, 200, 64, "bf16", k=6, temperature=2.0)
    x["ids"][:] = x["ids"][:1]                   # the rows' gradients point one way
    one = x["hidden"][:1].clone().requires_grad_()
    head.teacher_loss(one.expand(60, 64), x["weight"], x["ids"], x["teacher"], temperature=2.0).loss.backward()
    want = ref.loss(x | {"hidden": x["hidden"][:1].expand(60, 64)}, torch.ones((), device="cuda"))
    rows, sums = want["dh"], want["dh"].sum(0)
    off = want["dh_off"].sum(0) + 60 * 2.0 ** -23 * rows.abs().sum(0)
    off = off + 2.0 ** -9 * (sums.abs() + off)
    assert float(sums.abs().max()) > 8 * float(off.max())
    near(one.grad[0], sums, off, "gradient of the broadcast row")


@pytest.mark.parametrize("T,V,D,k", [(2 ** 24, 2, 1, 0), (2 ** 22, 5, 3, 2), (3, 2 ** 24, 8, 0), (2, 2 ** 24 - 1, 3, 4),
                                     (5, 40, 2 ** 16, 0), (300, 7, 2 ** 16 - 1, 5)])
def test_the_largest_sizes(T, V, D, k):
    x, dl = made(T, V, D, "bf16", k=k, dead=0.1), torch.ones((), device="cuda")
    r = forward(x)
    dh, dw = backward(x, r, dl)
    want = ref.loss(x, dl)
    assert int(r.tokens[0]) == want["tokens"]
    for name, got in (("losses", r.losses), ("lse", r.lse), ("loss", r.loss), ("dh", dh), ("dw", dw)):
        near(got, want[name], want[name + "_off"], name)
