"""The output head's losses and their gradients against a 64-bit form, within bounds that head_ref derives."""
import itertools

import pytest
import torch

import head_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import head, train

pytestmark = pytest.mark.gpu

INF = float("inf")
KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def made(T, V, D, dtype, k=0, seed=0, temperature=1.0, dead=0.0, spread=4.0, teacher=torch.float32, index=torch.int64):
    """Inputs whose softmax rests on a few columns, which lie anywhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x = {"hidden": normal(T, D).to(KINDS[dtype]), "weight": (normal(V, D) * spread * D ** -0.5).to(KINDS[dtype])}
    live = torch.rand(T, generator=g, device="cuda") >= dead
    x["hidden"][~live] = float("nan")
    if not k:
        x["labels"] = torch.where(live, torch.randint(0, V, (T,), generator=g, device="cuda"), -100).to(index)
        return x
    order = torch.rand(T, V, generator=g, device="cuda").argsort(1) if V <= 4096 else \
        torch.randint(0, V, (T, k), generator=g, device="cuda")
    ids = order[:, :k] if order.shape[1] >= k else order.repeat(1, -(-k // V))[:, :k]
    return x | {"ids": ids.contiguous().to(index), "teacher": (normal(T, k) * 2).to(teacher), "temperature": temperature,
                "mask": live if dead else None}


def forward(x, **kw):
    if "labels" in x:
        return head.cross_entropy(x["hidden"], x["weight"], x["labels"], **kw)
    return head.distill(x["hidden"], x["weight"], x["ids"], x["teacher"], temperature=x["temperature"], mask=x["mask"], **kw)


def backward(x, r, dl=None, dls=None, **kw):
    if "labels" in x:
        return head.cross_entropy_backward(x["hidden"], x["weight"], x["labels"], r, dl, dls, **kw)
    return head.distill_backward(x["hidden"], x["weight"], x["ids"], x["teacher"], r, dl, dls,
                                 temperature=x["temperature"], mask=x["mask"], **kw)


def near(got, want, off, what):
    bad = ~((got.double() - want).abs() <= off)
    # beyond the largest number by half a step, rounding gives infinity: 65504 + 16 in fp16
    big = torch.finfo(got.dtype).max * (1 + torch.finfo(got.dtype).eps / 4)
    bad &= ~((got.double() == want.sign() * INF) & (want.abs() + off >= big))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4], want[bad][:4], off[bad][:4])


def check(x, r, dl=None, dls=None, grads=None):
    want = ref.loss(x, dl, dls)
    assert int(r.tokens[0]) == want["tokens"]
    for name in ("losses", "lse", "loss"):
        near(getattr(r, name), want[name], want[name + "_off"], name)
    if grads is not None:
        near(grads[0], want["dh"], want["dh_off"], "grad_hidden")
        near(grads[1], want["dw"], want["dw_off"], "grad_weight")


def both(x, seed=0, parts="both"):
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    dl = torch.rand((), generator=g, device="cuda") + 0.5 if parts != "losses" else None
    dls = torch.randn(x["hidden"].shape[0], generator=g, device="cuda") * 0.1 if parts != "loss" else None
    r = forward(x)
    grads = backward(x, r, dl, dls)
    check(x, r, dl, dls, grads)
    return r, grads


SIZES = [(1, 1, 1), (1, 2, 8), (2, 31, 3), (3, 255, 7), (16, 256, 64), (31, 513, 200), (127, 257, 65), (128, 256, 64),
         (129, 512, 63), (255, 1000, 128), (256, 1, 64), (257, 300, 72), (300, 5000, 192), (513, 769, 321), (1, 40000, 96),
         (700, 33, 40), (64, 1024, 2048),
         # tiles of 224, 160 and 192 columns; rounds of several tiles for few tokens; split sums of either gradient
         (1, 17000, 4096), (40, 33000, 130), (300, 32000, 520), (9, 24000, 2048), (513, 20000, 1000), (8192, 1000, 64),
         (5000, 700, 41)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_labels(T, V, D, dtype):
    both(made(T, V, D, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_teacher(T, V, D, dtype):
    for k, temperature in ((1, 1.0), (7, 2.0)):
        both(made(T, V, D, dtype, k=k, temperature=temperature))


@pytest.mark.parametrize("k,teacher,index", [(2, torch.float32, torch.int32), (33, torch.bfloat16, torch.int64),
                                             (64, torch.float16, torch.int32), (100, torch.bfloat16, torch.int32),
                                             (255, torch.float32, torch.int64), (256, torch.float16, torch.int64)])
def test_lists_of_all_lengths(k, teacher, index):
    both(made(200, 700, 96, "bf16", k=k, teacher=teacher, index=index, temperature=1.5, dead=0.2))


@pytest.mark.parametrize("temperature", [2.0 ** -10, 0.3, 1.0, 17, 1024.0])
def test_temperatures(temperature):
    both(made(70, 600, 64, "bf16", k=20, temperature=temperature, spread=4 * min(temperature, 4)))


@pytest.mark.parametrize("dtype,index", [("bf16", torch.int64), ("fp16", torch.int32)])
@pytest.mark.parametrize("parts", ["loss", "losses", "both"])
def test_tokens_that_do_not_count(dtype, index, parts):
    """They hold NaN; the others are as in a batch of their own."""
    for k in (0, 9):
        x = made(777, 1500, 104, dtype, k=k, dead=0.4, index=index)
        r, grads = both(x, parts=parts)
        live = (r.losses != 0)
        assert not r.lse[~live].any() and not grads[0][~live].any()
        own = {n: v[live] if torch.is_tensor(v) and n != "weight" else v for n, v in x.items()}
        alone = forward(own)
        assert torch.equal(alone.losses, r.losses[live])


def test_no_token_counts():
    for k in (0, 5):
        for T in (0, 1, 300):
            x = made(T, 500, 64, "bf16", k=k, dead=1.1)
            if k:
                x["mask"] = torch.zeros(T, dtype=torch.uint8, device="cuda")
            r = forward(x)
            dh, dw = backward(x, r, torch.ones((), device="cuda"), torch.ones(T, device="cuda"))
            assert float(r.loss) == 0 and int(r.tokens[0]) == 0 and not r.losses.any() and not r.lse.any()
            assert not dh.any() and not dw.any() and dh.shape == (T, 64) and dw.shape == (500, 64)


def test_labels_outside_the_vocabulary():
    x = made(64, 300, 64, "bf16")
    x["labels"][:8] = torch.tensor([300, -1, 2 ** 40, -2 ** 40, 2 ** 32 + 5, -100, 299, 0], device="cuda")
    r, _ = both(x)
    assert (r.losses[:8] != 0).tolist() == [False] * 6 + [True] * 2


def test_lists_with_closed_slots_and_repeated_columns():
    x = made(90, 400, 64, "bf16", k=12)
    x["ids"][:, 3] = x["ids"][:, 7]             # a column listed twice, and three times
    x["ids"][::2, 9] = x["ids"][::2, 7]
    x["ids"][5:20, 2] = torch.tensor([-1, 400, 2 ** 40, -2 ** 33, 2 ** 32 + 1] * 3, device="cuda")
    x["teacher"][10:30, 4] = -INF
    x["teacher"][30] = -INF                     # nothing left
    x["ids"][31] = -1
    r, grads = both(x)
    assert float(r.losses[30]) == float(r.losses[31]) == 0 and not grads[0][30:32].any()
    # all slots one column: as that label
    x = made(40, 100, 64, "fp16", k=5)
    x["ids"][:] = x["ids"][:, :1]
    x["teacher"][:] = 0.25
    r, grads = both(x)
    y = {"hidden": x["hidden"], "weight": x["weight"], "labels": x["ids"][:, 0].contiguous()}
    assert torch.allclose(backward(y, forward(y), torch.ones((), device="cuda"))[0].float(),
                          backward(x, r, torch.ones((), device="cuda"))[0].float(), atol=2e-3)


def test_the_order_of_a_list_does_not_matter_to_the_gradient():
    x = made(130, 600, 64, "bf16", k=40)
    dl = torch.ones((), device="cuda")
    order = torch.rand(130, 40, device="cuda").argsort(1)
    y = x | {"ids": x["ids"].gather(1, order), "teacher": x["teacher"].gather(1, order)}
    r = forward(y)
    check(x, r, dl, None, backward(y, r, dl))


@pytest.mark.parametrize("teacher", [torch.float32, torch.bfloat16, torch.float16])
def test_lowest_values_of_a_type(teacher):
    x = made(50, 300, 64, "bf16", k=6, teacher=teacher)
    low = torch.finfo(teacher).min
    x["teacher"][:20, 1:4] = low                # closed by the lowest value, not by infinity
    r, _ = both(x)
    same = x | {"teacher": x["teacher"].clone()}
    same["teacher"][:20, 1:4] = -INF
    assert torch.equal(forward(same).losses, r.losses)
    x["teacher"][20:25] = low                   # a row of it: all slots alike
    x["teacher"][25:30] = 0
    r = forward(x)
    x["teacher"][20:25] = 0
    assert torch.equal(forward(x).losses, r.losses)


def test_large_logits():
    """No exponential overflows; the bound follows the logits' size."""
    for k in (0, 4):
        x = made(100, 500, 64, "bf16", k=k, spread=4000.0)
        r, _ = both(x)
        assert torch.isfinite(r.losses).all()


def test_nan_and_infinity_in_live_rows():
    for k, bad in itertools.product((0, 5), (float("nan"), INF, -INF)):
        x = made(300, 600, 64, "bf16", k=k)
        clean = forward(x)
        dl = torch.ones((), device="cuda")
        dh, _ = backward(x, clean, dl)
        x["hidden"] = x["hidden"].clone()
        x["hidden"][7, 3] = x["hidden"][280, 60] = bad
        r = forward(x)
        others = torch.ones(300, dtype=torch.bool, device="cuda")
        others[[7, 280]] = False
        assert not torch.isfinite(r.losses[~others]).any() and not torch.isfinite(r.loss)
        assert torch.equal(r.losses[others], clean.losses[others]) and int(r.tokens[0]) == 300
        got, dw = backward(x, r, dl)
        assert torch.equal(got[others], dh[others]) and not torch.isfinite(got[~others]).any()
        assert torch.isnan(dw).any()
    x = made(40, 100, 64, "bf16", k=5)
    x["teacher"][3, 2] = float("nan")
    x["teacher"][4, 1] = INF
    r = forward(x)
    assert torch.isnan(r.losses[3:5]).all() and torch.isfinite(r.losses[5:]).all()


def test_gradients_that_are_not_finite_stay_in_their_rows():
    x = made(80, 300, 64, "fp16")
    r, dls = forward(x), torch.ones(80, device="cuda")
    dh, _ = backward(x, r, None, dls)
    dls[9], dls[50] = INF, float("nan")
    got, dw = backward(x, r, None, dls)
    others = torch.ones(80, dtype=torch.bool, device="cuda")
    others[[9, 50]] = False
    assert torch.equal(got[others], dh[others]) and torch.isnan(got[50]).all() and torch.isnan(dw).any()


@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e-6, 3e4])
def test_scales_of_the_gradient(scale):
    """Loss scales, and rows whose gradients differ by orders of magnitude."""
    for dtype in ("bf16", "fp16"):
        x = made(150, 400, 64, dtype)
        r = forward(x)
        dl = torch.tensor(scale, device="cuda")
        dls = torch.exp(torch.randn(150, device="cuda", generator=torch.Generator("cuda").manual_seed(7)) * 3) * scale / 150 * 0.01
        check(x, r, dl, dls, backward(x, r, dl, dls))
        assert not backward(x, r)[1].any()      # no gradient given: zeros


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_strides(dtype):
    x = made(140, 520, 72, dtype)
    want = forward(x)
    dl = torch.ones((), device="cuda")
    grads = backward(x, want, dl)

    def wide(t, more, shift=0):
        room = torch.full((t.shape[0], t.shape[1] + more), float("nan"), dtype=t.dtype, device="cuda").reshape(-1)
        room = torch.cat([room, room[:64]])
        v = room.as_strided(t.shape, (t.shape[1] + more, 1), shift)
        v.copy_(t)
        return v
    ways = [lambda t: t.T.contiguous().T, lambda t: wide(t, 8), lambda t: wide(t, 5), lambda t: wide(t, 8, 1),
            lambda t: wide(t, 24, 8), lambda t: t.repeat_interleave(2, 1)[:, ::2]]
    for a, b in itertools.product(ways, ways):
        y = x | {"hidden": a(x["hidden"]), "weight": b(x["weight"])}
        got = forward(y)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(backward(y, got, dl), grads))
    y = x | {"hidden": x["hidden"][:1].expand(140, 72), "weight": x["weight"][:1].expand(520, 72)}
    both(y)


@pytest.mark.parametrize("k", [0, 30])
def test_pieces_of_the_vocabulary(k):
    """Tokens enough for a second and third piece; an odd hidden size."""
    for T, V, D in ((16384, 20001, 64), (13000, 24600, 37)):
        both(made(T, V, D, "bf16", k=k, dead=0.1))


def test_many_tiles_for_each_pair():
    both(made(2500, 9000, 640, "bf16"))
    both(made(1100, 3000, 2304, "fp16", k=50, temperature=2.0))


def test_one_gradient_alone():
    for k, (T, V, D) in itertools.product((0, 12), ((200, 900, 72), (3, 9000, 256), (3000, 600, 33), (16384, 9000, 64))):
        x = made(T, V, D, "bf16", k=k, dead=0.2)
        r, dl = forward(x), torch.ones((), device="cuda")
        dh, dw = backward(x, r, dl)
        one, none = backward(x, r, dl, needs=(True, False))
        assert none is None and (one.double() - dh.double()).abs().max() <= 2.0 ** -7 * dh.abs().max().double()
        none, one = backward(x, r, dl, needs=(False, True))
        assert none is None and torch.equal(one, dw)
        out = torch.empty_like(dw)
        assert backward(x, r, dl, out=(None, out), needs=(False, True))[1] is out and torch.equal(out, dw)
    h, w = x["hidden"].clone().requires_grad_(), x["weight"]
    h.data[~x["mask"]] = 0
    head.teacher_loss(h, w, x["ids"], x["teacher"], mask=x["mask"]).loss.backward()
    assert torch.equal(h.grad, backward(x, r, dl, needs=(True, False))[0]) and w.grad is None
    with pytest.raises(ValueError, match="neither"):
        backward(x, r, dl, needs=(False, False))


def test_weights_written_just_before():
    """The kernel that reads the weights may start before the one ahead of it ends: not before the weights are
    written, by an optimizer step whose kernels let the next start early too."""
    g = torch.Generator(device="cuda").manual_seed(11)
    for T, V, D in ((1, 30000, 512), (200, 20000, 256), (700, 8000, 128)):
        x = made(T, V, D, "bf16")
        w = [torch.nn.Parameter(x["weight"].clone()) for _ in range(2)]
        grads = [torch.randn(V, D, generator=g, device="cuda") for _ in range(3)]
        opts = [train.AdamW([t.detach()], [torch.empty_like(grads[0])]) for t in w]
        got, want = [], []
        for opt, t, losses, wait in ((opts[0], w[0], want, True), (opts[1], w[1], got, False)):
            y = x | {"weight": t.detach()}
            for n in range(6):
                opt.grads[0].copy_(grads[n % 3])
                opt.step(0.1)
                if wait:
                    torch.cuda.synchronize()
                r = forward(y)
                losses.append((r, backward(y, r, torch.ones((), device="cuda"))))
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        for (r, p), (s, q) in zip(want, got):
            assert torch.equal(r.losses, s.losses) and torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
        assert not torch.equal(want[0][0].losses, want[-1][0].losses)


def test_offsets_beyond_32_bits():
    """Weights of more than 2^31 numbers and hidden states that far apart."""
    V, D, T = 265000, 8192, 3
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 16384):
        w[a:a + 16384].normal_(std=D ** -0.5)
    room = torch.zeros(2 ** 31 * 2 + D, dtype=torch.bfloat16, device="cuda")
    hidden = room.as_strided((T, D), (2 ** 31, 1))
    hidden.copy_(torch.randn(T, D, device="cuda"))
    labels = torch.tensor([V - 1, 5, V - 70000], device="cuda")
    r = head.cross_entropy(hidden, w, labels)
    dl = torch.ones((), device="cuda")
    dh, dw = head.cross_entropy_backward(hidden, w, labels, r, dl)
    z = torch.cat([hidden.double() @ w[a:a + 16384].double().T for a in range(0, V, 16384)], 1)
    want = torch.logsumexp(z, 1) - z.gather(1, labels[:, None])[:, 0]
    assert (r.losses.double() - want).abs().max() < 1e-3
    dz = (torch.softmax(z, 1) - torch.zeros_like(z).scatter_(1, labels[:, None], 1.0)) / 3
    sums = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for a in range(0, V, 16384):
        part = w[a:a + 16384].double()
        sums += dz[:, a:a + 16384] @ part
        exact, size = dz[:, a:a + 16384].T @ hidden.double(), dz[:, a:a + 16384].abs().T @ hidden.double().abs()
        assert ((dw[a:a + 16384].double() - exact).abs() <= 2.0 ** -7 * size + 1e-30).all()
    assert (dh.double() - sums).abs().max() <= 2.0 ** -7 * sums.abs().max()


def test_repeatable_and_out():
    for k in (0, 20):
        x = made(1000, 3001, 130, "bf16", k=k, dead=0.3)
        dl = torch.ones((), device="cuda")
        r = forward(x)
        g = backward(x, r, dl)
        room = [torch.full((t.numel() + 40,), 7.0, dtype=t.dtype, device="cuda") for t in g]
        for shift in (0, 1, 8):
            out = head.HeadLoss(*(torch.empty_like(t) for t in r))
            assert forward(x, out=out) is out and all(torch.equal(p, q) for p, q in zip(r, out))
            for t in room:
                t.fill_(7.0)
            outs = tuple(t[shift:shift + p.numel()].view(p.shape) for t, p in zip(room, g))
            back = backward(x, out, dl, out=outs)
            for t, p, q in zip(room, g, back):
                assert torch.equal(p, q) and (t[:shift] == 7).all() and (t[shift + p.numel():] == 7).all()


def test_gradients_against_differences():
    """Inputs on a coarse grid, so that steps of a power of two are exact.  A central difference of the mean loss
    over e is off by e^2 / 6 of the third derivative, which for a log-sum of exponentials of slopes within s of
    each other is at most s^3 / 5, and by the losses' own error over e."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, V, D, e = 5, 60, 24, 2.0 ** -4
    for k in (0, 4):
        x = made(T, V, D, "fp16", k=k, temperature=1.0)
        x["hidden"] = (torch.randint(-16, 17, (T, D), generator=g, device="cuda") / 16).half()
        x["weight"] = (torch.randint(-16, 17, (V, D), generator=g, device="cuda") / 16).half()
        dl = torch.ones((), device="cuda")
        r = forward(x)
        grads = backward(x, r, dl)
        off = 2 * float(ref.loss(x)["losses_off"].max()) / e
        for name, grad in (("hidden", grads[0]), ("weight", grads[1])):
            for i, j in itertools.product(range(0, x[name].shape[0], 7 if name == "weight" else 2), range(0, D, 5)):
                up, down = x[name].clone(), x[name].clone()
                up[i, j] += e
                down[i, j] -= e
                d = (float(forward(x | {name: up}).loss) - float(forward(x | {name: down}).loss)) / (2 * e)
                s = 2.0
                assert abs(d - float(grad[i, j])) <= e * e / 6 * s ** 3 / 5 + off + 2.0 ** -9 * (abs(d) + 0.25), (name, i, j)


def test_differentiable():
    """Weights used by two heads and hidden states that are broadcast get the sums of their gradients."""
    a, b = made(60, 200, 64, "bf16"), made(60, 200, 64, "bf16", k=6, seed=1, temperature=2.0)
    w = a["weight"].clone().requires_grad_()
    x, one = a["hidden"].clone().requires_grad_(), b["hidden"][:1].clone().requires_grad_()
    r = head.label_loss(x, w, a["labels"])
    s = head.teacher_loss(one.expand(60, 64), w, b["ids"], b["teacher"], temperature=2.0)
    factors = torch.rand(60, device="cuda")
    ((r.losses * factors).sum() + 0.5 * r.loss + 2 * s.loss).backward()
    dh, dw = backward(a, forward(a), torch.tensor(0.5, device="cuda"), factors)
    b["hidden"], b["weight"] = b["hidden"][:1].expand(60, 64), a["weight"]
    eh, ew = backward(b, forward(b), torch.tensor(2.0, device="cuda"))
    assert torch.equal(x.grad, dh)
    assert torch.allclose(w.grad.float(), dw.float() + ew.float(), rtol=2.0 ** -7, atol=1e-6)
    # 60 rows of the same sizes, added in the type: half a step of the sums each
    assert (one.grad.float() - eh.float().sum(0)).abs().max() <= 60 * 2.0 ** -8 * float(eh.float().abs().max() * 60)
    assert not r.lse.requires_grad and not r.tokens.requires_grad
    x.grad = None
    head.label_loss(x, w.detach(), a["labels"]).loss.backward()
    assert torch.equal(x.grad, backward(a, forward(a), torch.ones((), device="cuda"))[0])
    y = (head.label_loss(x, w, a["labels"]).loss * x.float().sum())
    grad, = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.float().square().sum().backward()


def test_other_streams_and_graphs():
    side = [torch.cuda.Stream() for _ in range(2)]
    xs = [made(400, 1100, 96, "bf16", k=k, dead=0.2, seed=k) for k in (0, 8)]
    dl = torch.ones((), device="cuda")
    want = [(r := forward(x), backward(x, r, dl)) for x in xs]
    torch.cuda.synchronize()
    for _ in range(3):     # at the same time
        got = []
        for x, s in zip(xs, side):
            r = forward(x, stream=s)
            got.append((r, backward(x, r, dl, stream=s)))
        torch.cuda.synchronize()
        for (r, g), (p, q) in zip(got, want):
            assert all(torch.equal(m, n) for m, n in zip((*r, *g), (*p, *q)))
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = forward(x)
            g = backward(x, r, dl)
        graphs.append((graph, r, g))
    other = [made(400, 1100, 96, "bf16", k=k, dead=0.5, seed=k + 20) for k in (0, 8)]
    for x, y in zip(xs, other):
        for n in x:
            if torch.is_tensor(x[n]):
                x[n].copy_(y[n])
    torch.cuda.synchronize()
    for _ in range(2):     # replayed side by side, on other inputs and another number of live tokens
        for (graph, _, _), s in zip(graphs, side):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for x, (graph, r, g) in zip(xs, graphs):
        check(x, r, dl, None, g)


def test_a_captured_graph_of_autograd_is_refused():
    x = made(20, 50, 16, "bf16")
    w = x["weight"].requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="capture cross_entropy"):
            head.label_loss(x["hidden"], w, x["labels"])
        r = head.label_loss(x["hidden"], w.detach(), x["labels"])     # nothing to differentiate
    graph.replay()
    check(x, r)


def test_buffers_written_between_forward_and_backward_are_noticed():
    x = made(30, 70, 32, "bf16")
    out = forward(x)
    outs = backward(x, out, torch.ones((), device="cuda"))
    scale = torch.ones(30, device="cuda", requires_grad=True)
    ones = torch.ones(30, 32, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y, z = (scale * out.losses).sum(), (ones * outs[0]).sum()
    forward(x, out=out)
    backward(x, out, torch.ones((), device="cuda"), out=outs)
    for v in (y, z):
        with pytest.raises(RuntimeError, match="inplace"):
            v.backward()


def test_memory_freed_while_another_stream_uses_it():
    """The workspace of a call on another stream is not another tensor's before the call is done."""
    x, side = made(500, 3000, 128, "bf16"), torch.cuda.Stream()
    want = forward(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)      # about 50 ms
    got = forward(x, stream=side)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(40)]
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and len(junk) == 40


def test_a_training_step_of_a_small_model():
    """A router and experts, the output head's loss, the clip scale and the optimizer, as they are used together:
    gradients against the same step in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(0)
    T, D, V, E, k = 300, 64, 1000, 8, 2

    def normal(*s):
        return (torch.randn(*s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16()
    x, labels = normal(T, D) * 16, torch.randint(0, V, (T,), generator=g, device="cuda")
    labels[::5] = -100
    router, up = normal(D, E).requires_grad_(), normal(E, D, D).requires_grad_()
    out = (torch.randn(V, D, generator=g, device="cuda") * D ** -0.5).bfloat16().requires_grad_()
    leaves = [router, up, out]
    for t in leaves:
        t.grad = torch.zeros_like(t)
    opt = train.AdamW([t.detach() for t in leaves], [t.grad for t in leaves], state_bits=8)

    def hidden(gates, up):
        return sum(gates[:, e, None].to(up.dtype) * torch.tanh(x.to(up.dtype) @ up[e]) for e in range(E))
    r = train.gate(x @ router, k)
    h = hidden(torch.zeros(T, E, device="cuda").scatter(1, r.ids.long(), r.weights), up)
    loss = head.label_loss(h, out, labels)
    (loss.loss + 0.01 * r.loss).backward()
    norm = opt.grad_norm(1.0)
    before = [t.detach().clone() for t in leaves]
    opt.step(1e-2, grad_scale=norm[1])
    # the same loss of the same hidden states
    h64, w64 = h.detach().double().requires_grad_(), before[2].double().requires_grad_()
    live = labels >= 0
    want = torch.nn.functional.cross_entropy((h64 @ w64.T)[live], labels[live])
    want.backward()
    # dz and the result are rounded to half a step of 2^-8 each; errors of a row add up at random
    assert abs(float(loss.loss.detach()) - float(want.detach())) < 1e-4 * float(want.detach())
    assert (out.grad.double() - w64.grad).norm() < 2.0 ** -7 * w64.grad.norm()
    total = torch.cat([t.grad.double().reshape(-1) for t in leaves]).norm()
    assert abs(float(norm[0]) - float(total)) < 1e-5 * float(total)
    for t, b in zip(leaves, before):
        assert torch.isfinite(t).all() and not torch.equal(t, b)
    assert torch.equal(forward({"hidden": h.detach(), "weight": before[2], "labels": labels}).loss, loss.loss)


def test_refusals():
    x = made(8, 50, 16, "bf16")
    h, w, y = x["hidden"], x["weight"], x["labels"]
    ids, t = torch.zeros(8, 3, dtype=torch.int64, device="cuda"), torch.zeros(8, 3, device="cuda")
    for error, call in [
            (TypeError, lambda: head.cross_entropy(h.float(), w.float(), y)),
            (TypeError, lambda: head.cross_entropy(h, w.half(), y)),
            (TypeError, lambda: head.cross_entropy(h, w, y.short())),
            (ValueError, lambda: head.cross_entropy(h, w[:, :8], y)),
            (ValueError, lambda: head.cross_entropy(h[0], w, y)),
            (ValueError, lambda: head.cross_entropy(h, w, y[:7])),
            (ValueError, lambda: head.cross_entropy(h, w, y.cpu())),
            (ValueError, lambda: head.cross_entropy(h, w.cpu(), y)),
            (ValueError, lambda: head.cross_entropy(h.cpu(), w.cpu(), y.cpu())),
            (RuntimeError, lambda: head.cross_entropy(h[:, :0], w[:, :0], y)),
            (RuntimeError, lambda: head.cross_entropy(h, w[:0], y)),
            (ValueError, lambda: head.distill(h, w, y, t)),
            (ValueError, lambda: head.distill(h, w, ids[:, :2], t)),
            (ValueError, lambda: head.distill(h, w, ids.repeat(1, 100), t.repeat(1, 100))),
            (ValueError, lambda: head.distill(h, w, ids, t[:, ::2])),
            (TypeError, lambda: head.distill(h, w, ids, t.double())),
            (TypeError, lambda: head.distill(h, w, ids, t, mask=torch.ones(8, device="cuda"))),
            (RuntimeError, lambda: head.distill(h, w, ids, t, temperature=0.0)),
            (RuntimeError, lambda: head.distill(h, w, ids, t, temperature=-1.0)),
            (RuntimeError, lambda: head.distill(h, w, ids, t, temperature=float("nan"))),
            (RuntimeError, lambda: head.distill(h, w, ids, t, temperature=2048.0))]:
        with pytest.raises(error):
            call()
    r = head.cross_entropy(h, w, y)
    one = torch.ones((), device="cuda")
    for call in [lambda: head.cross_entropy_backward(h, w, y, r._replace(lse=r.lse[:7]), one),
                 lambda: head.cross_entropy_backward(h, w, y, r, torch.ones(2, device="cuda")),
                 lambda: head.cross_entropy_backward(h, w, y, r, one.double()),
                 lambda: head.cross_entropy_backward(h, w, y, r, None, torch.ones(7, device="cuda")),
                 lambda: head.cross_entropy_backward(h, w, y, r, one, out=(h.clone().half(), w.clone())),
                 lambda: head.cross_entropy_backward(h, w, y, r, one, out=(h.clone(), w.T.contiguous().T)),
                 lambda: head.cross_entropy_backward(h, w, y, r, one, out=(torch.empty_like(h), w)),
                 lambda: head.cross_entropy_backward(h, w, y, r, one, out=(h, torch.empty_like(w))),
                 lambda: head.cross_entropy(h, w, y, out=r._replace(tokens=r.loss))]:
        with pytest.raises(ValueError):
            call()
