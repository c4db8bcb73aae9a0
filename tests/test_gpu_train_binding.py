"""What the binding of the training-step operators keeps to: autograd's checks, streams, bound storage."""
import pytest
import torch

from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def test_second_derivatives_of_gate_are_refused():
    """Its gradient has no derivative: a penalty on it raises instead of adding nothing."""
    x = torch.randn(16, 8, device="cuda", requires_grad=True)
    y = (train.gate(x, 2).weights[:, 0] ** 2 * x[:, 0] ** 2).sum()
    grad, = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (grad ** 2).sum().backward()
    plain, = torch.autograd.grad((train.gate(x, 2).weights[:, 0] ** 2 * x[:, 0] ** 2).sum(), x)
    assert torch.equal(plain, grad.detach())


def small(bits=32, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(5)
    w = [torch.randn(n, generator=g, device="cuda").to(dtype) for n in (300, 7, 5000)]
    return train.AdamW(w, [torch.randn(t.shape, generator=g, device="cuda").to(dtype) for t in w], state_bits=bits)


def test_the_step_count_after_steps_on_another_stream():
    """Read and set behind a step that another stream has yet to run."""
    opt, side = small(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for n in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)      # about 50 ms
        opt.step(1e-3, stream=side)
        assert opt.steps == n + 1
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    opt.step(1e-3, stream=side)
    opt.set_step(100)
    assert opt.steps == 100
    with torch.cuda.stream(side):               # the stream that is current there
        torch.cuda._sleep(100_000_000)
        opt.step(1e-3)
    opt.set_step(200)
    assert opt.steps == 200
    opt.step(1e-3)
    assert opt.steps == 201 and not opt._state[24:28].any()


@pytest.mark.parametrize("step", [-1, -1000, 0.5])
def test_set_step_refuses(step):
    opt = small()
    opt.set_step(3)
    with pytest.raises(ValueError):
        opt.set_step(step)
    assert opt.steps == 3
    opt.set_step(0)
    opt.step(1e-3)
    assert opt.steps == 1 and all(torch.isfinite(w).all() for w in opt.weights)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_step_between_forward_and_backward_is_noticed(dtype):
    """Weights that autograd has saved are written: backward raises, as after any write in place."""
    base = torch.randn(40, device="cuda").to(dtype)
    leaf = torch.randn(30, device="cuda").to(dtype).requires_grad_()
    for bound, used in ((leaf.detach(), leaf), (leaf, leaf), (base[8:38], base[8:38]), (base[8:38].detach(), base)):
        opt = train.AdamW([bound, torch.zeros(5, device="cuda", dtype=dtype)],
                          [torch.ones(30, device="cuda", dtype=dtype), torch.ones(5, device="cuda", dtype=dtype)])
        x = torch.ones_like(used, requires_grad=True)
        y = (x * used).sum()
        opt.step(1e-2)
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
        (x * used).sum().backward()


def test_steps_of_inference_tensors():
    with torch.inference_mode():
        w, g = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    opt = train.AdamW([w], [g])
    opt.step(1e-2)
    assert (w < 1).all()


def test_buffers_written_between_forward_and_backward_are_noticed():
    logits = torch.randn(64, 16, device="cuda")
    kept, grad = train.Routing.empty(64, 16, 2), torch.ones(64, 16, device="cuda")
    for out in (kept, train.Routing(*kept)):
        train.route(logits, 2, out=out)
        x, z = torch.ones(64, 2, device="cuda", requires_grad=True), torch.ones(64, 16, device="cuda", requires_grad=True)
        y, z = (x * out.weights).sum(), (z * grad).sum()
        train.route(logits, 2, out=out)
        train.route_backward(logits, out, out.weights, out=grad)
        for v in (y, z):
            with pytest.raises(RuntimeError, match="inplace"):
                v.backward()
    with torch.inference_mode():
        out = train.Routing.empty(64, 16, 2)
        train.route(logits, 2, out=out)
    train.route(logits, 2, out=out)
    assert torch.equal(out.ids, kept.ids)


def test_bound_storage_stays():
    """Parameters that are given other storage: what was bound is neither freed nor reused."""
    w = torch.nn.Parameter(torch.ones(100_000, device="cuda"))
    w.grad = torch.ones_like(w)
    opt = train.AdamW([w], [w.grad], weight_decay=0.0)
    bound, w.data = w.data_ptr(), torch.full_like(w.data, 3.0)
    others = [torch.full_like(w.data, 7.0) for _ in range(8)]
    assert bound not in [t.data_ptr() for t in others]
    opt.step(1e-2)
    assert all((t == 7).all() for t in others) and (w == 3).all()
    at = [t.data_ptr() for t in (opt.m, opt.v)]
    opt.m = opt.v = None
    others += [torch.full((100_096,), 7.0, device="cuda") for _ in range(8)]
    assert not set(at) & {t.data_ptr() for t in others}
    opt.step(1e-2)
    assert all((t == 7).all() for t in others)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_bound_anew(bits):
    """The list goes on with new gradient tensors: same moments, count and results as one that kept its own;
    a captured step reads the new ones too."""
    a, b = small(bits), small(bits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(1e-3, grad_scale=b.grad_norm(1.0)[1])
    for n in range(4):
        new = [torch.randn_like(g) for g in a.grads]
        for g, x in zip(a.grads, new):
            g.copy_(x)
        b.bind_grads(new)
        assert all(p is q for p, q in zip(b.grads, new))
        del new
        norm = a.grad_norm(1.0)
        a.step(1e-3, grad_scale=norm[1])
        if n % 2:
            graph.replay()
        else:
            b.step(1e-3, grad_scale=b.grad_norm(1.0)[1])
        for p, q in zip((*a.weights, a.master, a.m, a.v), (*b.weights, b.master, b.m, b.v)):
            assert torch.equal(p, q)
    assert a.steps == b.steps == 4


def test_binding_refusals():
    opt = small()
    good = [torch.zeros_like(g) for g in opt.grads]
    before = opt.grads
    for bad in (good[:2], [], good[:2] + [good[2].float()], good[:2] + [good[2][1:]], good[:2] + [good[2].cpu()],
                good[:2] + [torch.zeros(10000, device="cuda", dtype=good[2].dtype)[::2]]):
        with pytest.raises(ValueError):
            opt.bind_grads(bad)
    assert opt.grads is before
    norm = train.GradNorm(good)
    norm.bind_grads([g + 1 for g in good])
    assert abs(float(norm.run()[0]) - 5307 ** 0.5) < 1e-3


def test_workspaces_are_clear_on_whichever_stream_the_first_call_is():
    """The clearing is late, on the stream where the buffers were made; the first call is elsewhere."""
    x = torch.randn(5000, 64, device="cuda")
    want, side = train.route(x, 4), torch.cuda.Stream()
    size = train.Routing.empty(5000, 64, 4).call.workspace.numel()
    torch.cuda.synchronize()
    for inside in (False, True):
        dirty = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del dirty
        torch.cuda._sleep(100_000_000)      # about 50 ms
        out = train.Routing.empty(5000, 64, 4)
        if inside:
            with torch.cuda.stream(side):
                train.route(x, 4, out=out)
        else:
            train.route(x, 4, out=out, stream=side)
        side.synchronize()
        for p, q in zip(want, out):
            assert torch.equal(p, q)
    grads = [torch.randn(100_000, device="cuda") for _ in range(3)]
    want = train.GradNorm(grads).run(1.0).clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    norm = train.GradNorm(grads)
    got = norm.run(1.0, stream=side)
    side.synchronize()
    assert torch.equal(want, got)


@pytest.mark.parametrize("given", [False, True])
def test_buffers_freed_while_another_stream_uses_them(given):
    """The memory of workspaces, tables and states is not another tensor's before the calls are done,
    whether the other stream is current or given."""
    x, side = torch.randn(5000, 64, device="cuda"), torch.cuda.Stream()
    out = train.Routing.empty(5000, 64, 4)
    weights = [torch.ones(100_000, device="cuda").bfloat16()]
    grads = [torch.ones(100_000, device="cuda")]
    opt, norm = train.AdamW(weights, grads, state_bits=8), train.GradNorm(grads)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)      # about 100 ms
        for t in (x, *out, *weights, *grads):
            t.record_stream(side)
        if not given:
            train.route(x, 4, out=out)
            norm.run()
            opt.step(1e-3, grad_scale=opt.grad_norm(1.0)[1])
            opt.state_values()
    if given:
        train.route(x, 4, out=out, stream=side)
        norm.run(stream=side)
        opt.step(1e-3, grad_scale=opt.grad_norm(1.0, stream=side)[1], stream=side)
        opt.state_values(stream=side)
    hidden = [out.call.workspace, *norm._table.own, *opt._table.own]
    at = {t.data_ptr(): t.numel() * t.element_size() for t in hidden}
    assert len(at) == len(hidden)
    del out, opt, norm, hidden
    others = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in at.values() for _ in range(4)]
    busy = not side.query()
    assert not at.keys() & {t.data_ptr() for t in others}
    assert busy     # else nothing was shown
