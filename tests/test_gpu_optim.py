"""Gradient norm and AdamW on the GPU against their 64-bit forms.

Tolerances.  With u = 2^-24: a 32-bit moment is two products and a sum with rounded coefficients,
at most 6 u of the magnitudes added; the gradient's scaling adds one u (two in its square).  A
master weight is off by 2 u of itself and by lr times the change's error, below 2^-20 of the
magnitudes of its two parts (sqrt, division and coefficients in 32 bits).  A norm's squares are
summed by threads over at most 64 values in 32 bits, then in 64: 40 u of the norm.  An 8-bit code
is the 64-bit form's unless the fraction and the noise are within 2^-10 of the next step, where it
may be one beside it: a moment's relative error of 8 u is 2^-17 of the 16 steps of a binade."""
import numpy as np
import pytest
import torch

import train_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import nest, train

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS_OF = {"fp32": 0.0, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
LISTS = [[1], [255, 256, 257], [0, 1, 0], [4096], [4095, 3, 4097, 8192, 511], [100003, 7, 65536], [31] * 300]


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def make(numels, dtype, seed, scale=1.0, shift=0):
    """Tensors of these sizes; with a shift, views that start that many elements off alignment."""
    g = np.random.default_rng(seed)
    out = []
    for n in numels:
        room = torch.zeros(n + shift, dtype=TYPES[dtype], device="cuda")
        room[shift:] = torch.tensor(g.normal(size=n) * scale).to(TYPES[dtype]).cuda()
        out.append(room[shift:])
    return out


def f64(t):
    return t.double().cpu().numpy()


def parts(opt, buffer):
    """The list's tensors out of one of its buffers."""
    return [buffer[a:a + t.numel()] for a, t in zip(opt.starts, opt.weights)]


# ---- norm -------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("numels", LISTS + [[3000001, 5]])
def test_norm(numels, dtype):
    for shift in (0, 1, 3):
        g = make(numels, dtype, len(numels) + shift, shift=shift)
        want = np.sqrt(sum((f64(t) ** 2).sum() for t in g))
        norm = train.GradNorm(g)
        got = norm.run(max_norm=2.0).clone()
        assert abs(float(got[0]) - want) <= 40 * U * want
        clip = min(1.0, 2.0 / (want + 1e-6))
        assert abs(float(got[1]) - clip) <= 44 * U * clip
        assert torch.equal(norm.run(max_norm=2.0), got)
        assert float(norm.run()[1]) == 1.0


def test_norm_of_nothing_and_of_too_much():
    assert train.GradNorm([torch.zeros(0, device="cuda")]).run(1.0).tolist() == [0.0, 1.0]
    assert train.GradNorm([torch.zeros(300, device="cuda")]).run(1.0).tolist() == [0.0, 1.0]
    for bad in (float("nan"), float("inf"), -float("inf"), 1e30):
        g = make([1000, 50], "fp32", 1)
        g[1][49] = bad
        out = train.GradNorm(g).run(1.0)
        assert not np.isfinite(float(out[0])) and np.isnan(float(out[1]))
    small = torch.full((100,), 1e-15, device="cuda")       # squares of 1e-30 are still normal
    assert abs(float(train.GradNorm([small]).run(1.0)[0]) - 1e-14) < 1e-19


def test_norm_workspace_between_calls():
    g = make([100003, 7, 65536], "bf16", 1)
    norm = train.GradNorm(g)
    want, ws = norm.run(1.0).clone(), norm._table.workspace
    for _ in range(3):
        ws[256:] = 255
        assert torch.equal(norm.run(1.0), want) and (ws[:256] == 0).all()


def test_parameters_that_require_gradients():
    w = torch.nn.Parameter(torch.randn(70, 30, device="cuda").bfloat16())
    w.grad = torch.randn_like(w)
    opt = train.AdamW([w], [w.grad])
    before = w.detach().clone()
    opt.step(1e-2)
    assert not opt.master.requires_grad and not torch.equal(w.detach(), before)


# ---- step -------------------------------------------------------------------------

def start(opt, seed, gscale):
    """Random moments, as after some steps."""
    g = np.random.default_rng(seed)
    n = opt.m.numel()
    m, v = g.normal(size=n) * gscale, g.normal(size=n) ** 2 * gscale ** 2
    live = np.zeros(n, bool)
    for a, t in zip(opt.starts, opt.weights):
        live[a:a + t.numel()] = True
    m, v = np.where(live, m, 0), np.where(live, v, 0)
    if opt.state_bits == 32:
        opt.m.copy_(torch.tensor(m))
        opt.v.copy_(torch.tensor(v))
    else:
        for x, signed, code, exp in ((m, True, opt.m, opt.m_exp), (v, False, opt.v, opt.v_exp)):
            x = x.reshape(-1, 256)
            s = ref.shared_exponent(x)
            c, _ = ref.to_codes(x, s, np.full(x.shape, 32768), signed)
            if signed:
                c = np.where(x < 0, c | 0x80, c)
            code.copy_(torch.tensor(c.reshape(-1).astype(np.uint8)))
            exp.copy_(torch.tensor(s.astype(np.int8)))


def moments(opt):
    if opt.state_bits == 32:
        return f64(opt.m), f64(opt.v)
    out = []
    for code, exp, signed in ((opt.m, opt.m_exp, True), (opt.v, opt.v_exp, False)):
        out.append(ref.code_value(code.cpu().numpy().reshape(-1, 256), exp.cpu().numpy(), signed).reshape(-1))
    return out


def check_step(opt, t, lr, decay, scale=None, lr_scale=None):
    """One step against the 64-bit form, from the state that the object holds."""
    eight = opt.state_bits == 8
    b1, b2 = opt.betas
    s = 1.0 if scale is None else float(scale)
    weight_type = {v: k for k, v in TYPES.items()}[opt.weights[0].dtype]
    p0 = [f64(x) for x in (opt.weights if opt.master is None else parts(opt, opt.master))]
    m0, v0 = moments(opt)
    grads = [f64(x) for x in opt.grads]
    untouched = opt.m.clone(), opt.v.clone()
    opt.step(lr, grad_scale=scale)
    masters = opt.weights if opt.master is None else parts(opt, opt.master)
    n = opt.m.numel()
    m1, v1, live = np.zeros(n), np.zeros(n), np.zeros(n, bool)
    for i, (a, w) in enumerate(zip(opt.starts, opt.weights)):
        at = slice(a, a + w.numel())
        live[at] = True
        step_lr = lr * (lr_scale[i] if lr_scale else 1.0)
        p, m1[at], v1[at], change = ref.adamw(p0[i], grads[i], m0[at], v0[at], t, step_lr, b1, b2, opt._args.eps,
                                              decay[i], s)
        gs = np.abs(grads[i] * s)
        with np.errstate(all="ignore"):
            part = np.abs(change - decay[i] * p0[i]) + decay[i] * np.abs(p0[i])
            # cancellation inside m: its error over the root
            root = np.sqrt(v1[at] / (1 - b2 ** t)) + opt._args.eps
            part = part + (b1 * np.abs(m0[at]) + (1 - b1) * gs) / (1 - b1 ** t) / root
        tol = 2 * U * np.abs(p) + step_lr * part * 2.0 ** -20 + 1e-37
        got = f64(masters[i])
        np.testing.assert_array_equal(np.isnan(got), np.isnan(p))
        ok = ~np.isnan(p)
        assert (np.abs(got - p) <= tol)[ok].all()
        if weight_type != "fp32":      # the weight is the master's rounding
            assert torch.equal(w, masters[i].to(w.dtype)) or np.isnan(got).any()
        if not eight:
            mt = 7 * U * (b1 * np.abs(m0[at]) + (1 - b1) * gs) + 1e-45
            vt = 9 * U * (b2 * v0[at] + (1 - b2) * gs ** 2) + 1e-45
            got_m, got_v = f64(opt.m[at]), f64(opt.v[at])
            ok = np.isfinite(m1[at])
            assert (np.abs(got_m - m1[at]) <= mt)[ok].all() and (np.abs(got_v - v1[at]) <= vt)[ok].all()
            np.testing.assert_array_equal(np.isnan(got_m), np.isnan(m1[at]))
    dead = torch.tensor(~live, device="cuda")
    assert torch.equal(opt.m[dead], untouched[0][dead]) and torch.equal(opt.v[dead], untouched[1][dead])
    if eight:
        noise = ref.noise(opt._args.seed, t, np.arange(n // 256))
        for x, code, exp, signed, r in ((m1, opt.m, opt.m_exp, True, noise[0]), (v1, opt.v, opt.v_exp, False, noise[1])):
            x, keep = x.reshape(-1, 256), live.reshape(-1, 256)
            want_s = ref.shared_exponent(x)
            got_s = exp.cpu().numpy().astype(np.int64)
            top = np.max(np.where(np.isfinite(x), np.abs(x), 0), 1)
            edge = np.abs(top / np.ldexp(1.75, np.clip(want_s - 1, -1000, 1000)) - 1) < 16 * U
            edge |= np.abs(top / np.ldexp(1.75, want_s) - 1) < 16 * U
            assert ((got_s == want_s) | edge).all()
            want, dist = ref.to_codes(x, got_s, r, signed)
            c = code.cpu().numpy().reshape(-1, 256).astype(np.int64)
            mag = c & 0x7F if signed else c
            off = np.abs(mag - want)
            assert ((off == 0) | ((off == 1) & (dist < 2.0 ** -10)))[keep].all()
            assert ((off > 0) & keep).mean() < 1e-3
            if signed:
                sure = keep & np.isfinite(x) & (mag > 0)
                assert ((c >> 7 == 1) == (x < 0))[sure].all()
        m, v = opt.state_values()
        for value, (code, exp, signed) in ((m, (opt.m, opt.m_exp, True)), (v, (opt.v, opt.v_exp, False))):
            want = ref.code_value(code.cpu().numpy().reshape(-1, 256), exp.cpu().numpy(), signed).reshape(-1)
            np.testing.assert_array_equal(f64(value), want)
    else:
        assert opt.state_values()[0] is opt.m
    assert opt.steps == t


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wtype,gtype", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"),
                                         ("fp32", "bf16"), ("fp16", "bf16"), ("fp32", "fp16"), ("bf16", "fp16"),
                                         ("fp16", "fp32")])
def test_step_types(wtype, gtype, bits):
    numels = [1000, 1, 4096, 333]
    w, g = make(numels, wtype, 1, 0.05), make(numels, gtype, 2, 1e-3)
    decay = [0.1, 0.0, 0.2, 0.0]
    opt = train.AdamW(w, g, state_bits=bits, betas=(0.9, 0.95), weight_decay=decay, seed=5)
    check_step(opt, 1, 1e-3, decay)
    start(opt, 3, 1e-3)
    opt.set_step(40)
    check_step(opt, 41, 1e-3, decay, torch.tensor(0.3, device="cuda"))
    check_step(opt, 42, 2e-3, decay)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("numels", LISTS + [[300007, 12]])
def test_step_sizes(numels, bits):
    decay, lr_scale = [0.05 * (i % 3) for i in range(len(numels))], [1.0 + i % 2 for i in range(len(numels))]
    for shift in (0, 1, 2, 4):
        w, g = make(numels, "bf16", 1, 0.05, shift), make(numels, "bf16", 2, 1e-4, (3 * shift) % 5)
        opt = train.AdamW(w, g, state_bits=bits, weight_decay=decay, lr_scale=lr_scale, seed=2 ** 31 + 9)
        opt.set_step(9)
        start(opt, 4, 1e-4)
        check_step(opt, 10, 1e-3, decay, lr_scale=lr_scale)


@pytest.mark.parametrize("bits,numels,wtype,gtype,shift", [
    (8, [5000001, 300], "bf16", "bf16", 0), (8, [5000001, 300], "bf16", "bf16", 1), (8, [5000100], "fp32", "fp32", 3),
    (8, [4000000, 1500003], "fp32", "fp16", 5), (8, [10100007, 5], "bf16", "bf16", 1),
    (32, [20000123, 777], "bf16", "bf16", 0), (32, [5000001], "fp32", "bf16", 7)])
def test_step_of_long_lists(bits, numels, wtype, gtype, shift):
    """Lists in which a warp takes several blocks, and several thread blocks share a worker; with
    gradients off alignment (and 32-bit weights with them)."""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def room(n, kind, scale, off):
        t = torch.zeros(n + off, dtype=TYPES[kind], device="cuda")
        t[off:] = (torch.randn(n, generator=gen, device="cuda") * scale).to(TYPES[kind])
        return t[off:]
    w = [room(n, wtype, 0.05, shift % 3) for n in numels]
    g = [room(n, gtype, 1e-3, shift) for n in numels]
    decay = [0.1, 0.0][:len(numels)]
    opt = train.AdamW(w, g, state_bits=bits, betas=(0.9, 0.95), weight_decay=decay, seed=77)
    opt.set_step(20)
    start(opt, 3, 1e-3)
    check_step(opt, 21, 1e-3, decay, torch.tensor(0.7, device="cuda"))
    want = np.sqrt(sum((f64(t) ** 2).sum() for t in g))
    assert abs(float(opt.grad_norm()[0]) - want) <= 40 * U * want


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_has_size_lr(bits):
    """From zero moments the first step is lr * sign(g), whatever the gradient's size."""
    w, g = make([5000], "fp32", 1), make([5000], "fp32", 2, 1e-2)
    before = w[0].clone()
    opt = train.AdamW(w, g, state_bits=bits, eps=0.0, weight_decay=0.0, betas=(0.9, 0.999))
    opt.step(0.5)
    # both corrections cancel the coefficients up to their roundings; the weight's own rounding
    assert ((before - w[0]) - 0.5 * g[0].sign()).abs().max() < 2 ** -21 + 5 * 2 ** -24


@pytest.mark.parametrize("bits", [32, 8])
def test_skipped_step(bits):
    w, g = make([700, 3], "bf16", 1), make([700, 3], "bf16", 2)
    opt = train.AdamW(w, g, state_bits=bits)
    start(opt, 1, 1.0)
    opt.set_step(3)
    held = [w[0], w[1], opt.master, opt.m, opt.v] + ([opt.m_exp, opt.v_exp] if bits == 8 else [])
    before = [t.clone() for t in held]
    g[1][2] = float("inf")
    opt.step(1e-2, grad_scale=opt.grad_norm(1.0)[1])
    opt.step(1e-2, grad_scale=torch.tensor(float("inf"), device="cuda"))
    assert opt.steps == 3 and all(torch.equal(a, b) for a, b in zip(held, before))
    g[1][2] = 0.5
    opt.step(1e-2, grad_scale=opt.grad_norm(1.0)[1])
    assert opt.steps == 4 and not torch.equal(w[0], before[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_values_that_are_not_finite(bits):
    """Without a scale that guards it, a NaN or infinite gradient stays in its own element."""
    w, g = make([600], "fp32", 1), make([600], "fp32", 2)
    g[0][3], g[0][300], g[0][599] = float("nan"), float("inf"), -float("inf")
    opt = train.AdamW(w, g, state_bits=bits, weight_decay=0.0)
    start(opt, 1, 1.0)
    opt.set_step(5)
    opt.step(1e-3)
    bad = torch.zeros(600, dtype=torch.bool, device="cuda")
    bad[[3, 300, 599]] = True
    assert torch.isfinite(w[0][~bad]).all() and torch.isnan(w[0][bad]).all()
    m, v = opt.state_values()
    for x in (m, v):
        assert torch.isfinite(x[:600][~bad]).all() and not torch.isfinite(x[:600][bad]).any()


@pytest.mark.parametrize("gscale", [0.0, 1e-30, 1e-20, 1e-12, 1.0, 1e4, 1e12])
def test_eight_bits_over_the_range(gscale):
    """Zero and tiny gradients (squares that vanish), and ones whose squares need the upper exponents."""
    w, g = make([2000], "fp32", 1), make([2000], "fp32", 2, gscale)
    opt = train.AdamW(w, g, state_bits=8, weight_decay=0.0, seed=3)
    check_step(opt, 1, 1e-3, [0.0])
    check_step(opt, 2, 1e-3, [0.0])
    assert torch.isfinite(w[0]).all()


def test_eight_bits_hold_small_changes_in_the_mean():
    """beta2 = 0.999 moves v by far less than a step of its code; the mean over many elements still
    follows: 200 steps with g^2 = 0 after v = 1 leave 0.999^200, to 5 standard deviations."""
    n = 256 * 400
    w, g = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]
    opt = train.AdamW(w, g, state_bits=8, betas=(0.9, 0.999), weight_decay=0.0, seed=1)
    opt.v.fill_((31 << 3) | 4)        # 0.75 * 2^(0 + 1)
    opt.v_exp.fill_(0)
    opt.set_step(1000)
    for _ in range(200):
        opt.step(0.0)
    v = opt.state_values()[1].double()
    want = 1.5 * 0.999 ** 200
    # a step's variance is at most (step / 2)^2 with steps of at most 1.5 / 8 on the way, mostly 1 / 8
    sd = (200 * 0.125 ** 2 / 4 / n) ** 0.5
    assert abs(float(v.mean()) - want) < 5 * sd + 200 * 0.125 * 2.0 ** -17
    assert opt.steps == 1200


@pytest.mark.parametrize("bits", [32, 8])
def test_repeatable_and_many_steps(bits):
    """The same steps twice give the same bits, and follow a 64-bit run of the formulas."""
    def go():
        w, g = make([5000, 77], "fp32", 1, 0.1), make([5000, 77], "fp32", 2, 0.1)
        opt = train.AdamW(w, g, state_bits=bits, betas=(0.9, 0.95), weight_decay=0.1, seed=8)
        for i in range(20):
            for t in g:
                t.mul_(0.9)
            opt.step(1e-2, grad_scale=opt.grad_norm(1.0)[1])
        return w
    a, b = go(), go()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ps, gs = [f64(t) for t in make([5000, 77], "fp32", 1, 0.1)], [f64(t) for t in make([5000, 77], "fp32", 2, 0.1)]
    m, v = [0.0, 0.0], [0.0, 0.0]
    for i in range(20):
        gs = [g * np.float32(0.9) for g in gs]
        scale = min(1.0, 1.0 / (np.sqrt(sum((g ** 2).sum() for g in gs)) + 1e-6))
        for j in range(2):
            ps[j], m[j], v[j], _ = ref.adamw(ps[j], gs[j], m[j], v[j], i + 1, 1e-2, 0.9, 0.95, 1e-8, 0.1, scale)
    for x, p in zip(a, ps):
        err = np.abs(f64(x) - p)
        # 32 bits: 20 steps of 2^-19 of lr and 2 u of the weight; 8 bits: each step's moments are
        # off by up to an eighth, 20 steps of lr at most a quarter off
        assert err.max() < (20 * (1e-2 * 2.0 ** -17 + 4 * U) if bits == 32 else 20 * 1e-2 * 0.25)


def test_beyond_31_bits_of_elements():
    """A list of 2.2e9 elements: addresses and element numbers past 32 bits."""
    n, tail = 2 ** 31 + 12345, 1000
    grad = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    weight = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    w, g = make([tail], "bf16", 1), make([tail], "bf16", 2)
    opt = train.AdamW([weight] + w, [grad] + g, state_bits=8, weight_decay=0.0, seed=4)
    norm = float(opt.grad_norm()[0])
    want = (0.25 * n + float((g[0].double() ** 2).sum())) ** 0.5
    assert abs(norm - want) <= 40 * U * want
    p0, noise = f64(parts(opt, opt.master)[1]), ref.noise(4, 1, [opt.starts[1] // 256])
    opt.step(1e-2)
    assert (weight.float() - weight[0].float()).abs().max() == 0 and abs(float(weight[0]) + 1e-2) < 1e-4
    p, m, v, _ = ref.adamw(p0, f64(g[0]), 0.0, 0.0, 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
    assert np.abs(f64(parts(opt, opt.master)[1]) - p).max() < 1e-7
    at = slice(opt.starts[1], opt.starts[1] + 256)
    s = opt.m_exp[opt.starts[1] // 256].item()
    want, dist = ref.to_codes(m[None, :256], np.array([s]), noise[0], True)
    got = opt.m[at].cpu().numpy().astype(np.int64)[None] & 0x7F
    assert ((got == want) | (dist < 2.0 ** -10)).all()


def test_streams_and_graphs():
    def new():
        w, g = make([3000, 17], "bf16", 1), make([3000, 17], "bf16", 2)
        return w, g, train.AdamW(w, g, state_bits=8, seed=6)
    w0, g0, a = new()
    for _ in range(3):
        a.step(1e-2, grad_scale=a.grad_norm(1.0)[1])
    w1, g1, b = new()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        scale = b.grad_norm(1.0, stream=side)[1]
        b.step(1e-2, grad_scale=scale, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    w2, g2, c = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step(1e-2, grad_scale=c.grad_norm(1.0)[1])
    for _ in range(3):
        graph.replay()
    assert c.steps == b.steps == a.steps == 3
    for x, y, z in zip(w0 + [a.m, a.v], w1 + [b.m, b.v], w2 + [c.m, c.v]):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_refusals():
    w, g = make([10, 20], "bf16", 1), make([10, 20], "bf16", 2)
    with pytest.raises(ValueError):
        train.AdamW(w, g[:1])
    with pytest.raises(ValueError):
        train.AdamW(w, [g[1], g[0]])
    with pytest.raises(ValueError):
        train.AdamW([w[0], w[1].float()], g)
    with pytest.raises(ValueError):
        train.AdamW(w, [g[0], g[1].cpu()])
    with pytest.raises(ValueError):
        train.AdamW(w, [g[0], torch.zeros(40, dtype=torch.bfloat16, device="cuda")[::2]])
    with pytest.raises(ValueError, match="overlap"):
        train.AdamW([w[1][:10], w[1][5:15]], [g[0], g[0]])
    with pytest.raises(TypeError):
        train.GradNorm([torch.zeros(4, dtype=torch.float64, device="cuda")])
    with pytest.raises(nest.NestError):
        train.AdamW(w, g, betas=(1.0, 0.9)).step(1e-3)
    opt = train.AdamW(w, g)
    with pytest.raises(nest.NestError):
        opt.step(float("nan"))
    with pytest.raises(nest.NestError):
        opt.grad_norm(0.0)
    with pytest.raises(ValueError):
        opt.step(1e-3, grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        opt.step(1e-3, grad_scale=torch.ones(1, dtype=torch.float64, device="cuda"))
    assert opt.steps == 0 and (train.AdamW(w, g).opt_factor, train.AdamW(w, g, state_bits=8).opt_factor) == (6, 3)
