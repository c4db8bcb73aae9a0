"""Host-side checks of the output head's losses that need no GPU: the ABI, refusals, workspace sizes, and the
64-bit form that the GPU tests compare against."""
import ctypes as C
import itertools
import os
import re

import pytest
import torch

import head_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import head, nest, train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 4096     # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "nest_head.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(nest_\w+)\s*\(", text, flags=re.M))
    assert names == set(head.EXPORTS)
    for n in names:
        assert hasattr(C.CDLL(nest.LIB_PATH), n), n


def desc(**kw):
    d = dict(tokens=4, vocab=100, hidden=64, hidden_row=64, hidden_col=1, weight_row=64, weight_col=1, dtype=train.BF16,
             index_type=head.I64, k=0, teacher_type=0, temperature=1.0, reserved=0)
    d.update(kw)
    return head.HeadDesc(*[d[n] for n, _ in head.HeadDesc._fields_])


def calls(d, hidden=FAKE, weight=FAKE, index=FAKE, teacher=None, mask=None, results=FAKE, ws=FAKE, more=0):
    L, ref_ = head.lib(), C.byref(d)
    sizes = [f(ref_, weight) + more for f in (L.nest_head_loss_workspace_size, L.nest_head_backward_workspace_size)]
    common = (ref_, hidden, weight, index, teacher, mask)
    return (L.nest_head_loss(*common, results, results, results, results, ws, max(0, sizes[0]), None),
            L.nest_head_loss_backward(*common, results, None, None, results, results, ws, max(0, sizes[1]), None))


INVALID = [dict(tokens=-1), dict(vocab=0), dict(hidden=0), dict(hidden_row=-1), dict(hidden_col=-1), dict(weight_row=-1),
           dict(weight_col=-1), dict(dtype=train.F32), dict(dtype=7), dict(index_type=2), dict(k=-1), dict(reserved=1),
           dict(temperature=2.0), dict(k=3, teacher_type=3), dict(k=3, temperature=0.0), dict(k=3, temperature=-1.0),
           dict(k=3, temperature=float("nan")), dict(k=3, temperature=float("inf")), dict(k=3, temperature=1025.0)]


@pytest.mark.parametrize("kw", INVALID)
def test_invalid_descriptions(kw):
    assert calls(desc(**kw)) == (nest.NEST_E_INVALID,) * 2
    assert head.lib().nest_head_loss_workspace_size(C.byref(desc(**kw)), FAKE) == 0


@pytest.mark.parametrize("kw", [dict(tokens=2 ** 24 + 1), dict(vocab=2 ** 24 + 1), dict(hidden=2 ** 16 + 1), dict(k=257),
                                dict(tokens=2 ** 24, vocab=2 ** 24)])
def test_limits(kw):
    assert calls(desc(**kw)) == (nest.NEST_E_LIMITS,) * 2
    assert head.lib().nest_head_backward_workspace_size(C.byref(desc(**kw)), FAKE) == 0


def test_missing_and_misaligned_buffers():
    bad = (nest.NEST_E_INVALID,) * 2
    for kw in (dict(hidden=None), dict(weight=None), dict(index=None), dict(hidden=FAKE + 1), dict(weight=FAKE + 1),
               dict(index=FAKE + 4), dict(teacher=FAKE), dict(mask=FAKE), dict(results=None)):
        assert calls(desc(), **kw) == bad, kw
    for kw in (dict(), dict(teacher=FAKE + 2), dict(teacher=FAKE, index=FAKE + 4)):
        assert calls(desc(k=3), **kw) == bad, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(more=-1)):
        assert calls(desc(), **kw) == (nest.NEST_E_WORKSPACE,) * 2, kw
    assert head.lib().nest_head_loss(None, *[None] * 10, 0, None) == nest.NEST_E_INVALID
    L, d = head.lib(), desc()
    size = L.nest_head_backward_workspace_size(C.byref(d), FAKE)
    for lse, dh, dw in ((None, FAKE, FAKE), (FAKE, None, None), (FAKE, FAKE + 1, FAKE), (FAKE, None, FAKE + 1)):
        assert L.nest_head_loss_backward(C.byref(d), FAKE, FAKE, FAKE, None, None, lse, None, None, dh, dw, FAKE, size,
                                         None) == nest.NEST_E_INVALID


def test_workspace_sizes():
    """Within a gigabyte of the inputs' copies whatever the vocabulary: the logits are not kept."""
    L = head.lib()
    for T, V, D in ((1, 32000, 4096), (2048, 32000, 4096), (8192, 128000, 8192), (131072, 256000, 1024)):
        d = desc(tokens=T, vocab=V, hidden=D, hidden_row=D, weight_row=D)
        pitch = -(-T // 256) * 256
        assert L.nest_head_loss_workspace_size(C.byref(d), FAKE) < 2 * pitch * D + 12 * pitch * (V // 256 + 2) + 2 ** 20
        back = L.nest_head_backward_workspace_size(C.byref(d), FAKE)
        assert back < 2 * pitch * D + 4 * pitch * D + max(2 ** 28, 2 * 8192 * pitch) + 64 * pitch + 2 ** 20
        # weights that have to be copied
        for odd, at in ((desc(tokens=T, vocab=V, hidden=D, hidden_row=D, weight_row=D + 1), FAKE),
                        (desc(tokens=T, vocab=V, hidden=D, hidden_row=D, weight_row=D, weight_col=2), FAKE), (d, FAKE + 2)):
            assert L.nest_head_backward_workspace_size(C.byref(odd), at) == back + -(-2 * V * D // 256) * 256


def test_tensors_on_the_cpu_are_refused():
    h, w = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        head.cross_entropy(h, w, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        head.distill(h, w, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))
    with pytest.raises(ValueError, match="CUDA"):
        head.label_loss(h, w.requires_grad_(), torch.zeros(3, dtype=torch.int64))


@pytest.mark.parametrize("k", [0, 4])
def test_the_64_bit_form_against_autograd(k):
    g = torch.Generator().manual_seed(k)
    T, V, D, heat = 9, 30, 6, 1.0 if not k else 1.7
    h, w = (torch.randn(n, D, generator=g, dtype=torch.float64).half() for n in (T, V))
    if k:
        x = dict(ids=torch.rand(T, V, generator=g).argsort(1)[:, :k], teacher=torch.randn(T, k, generator=g),
                 temperature=heat, mask=torch.arange(T) % 3 > 0)
    else:
        x = dict(labels=torch.where(torch.arange(T) % 3 > 0, torch.arange(T), -1))
    x |= dict(hidden=h, weight=w)
    dl, dls = torch.tensor(0.7), torch.randn(T, generator=g)
    got = ref.loss(x, dl, dls)
    a, b = h.double().requires_grad_(), w.double().requires_grad_()
    log_p = torch.log_softmax(a @ b.T / heat, 1)
    live = torch.arange(T) % 3 > 0
    if k:
        q = torch.softmax(x["teacher"].double() / heat, 1)
        losses = heat ** 2 * torch.nn.functional.kl_div(log_p.gather(1, x["ids"]), q, reduction="none").sum(1)
    else:
        losses = -log_p[torch.arange(T), x["labels"].clamp(min=0)]
    losses = torch.where(live, losses, 0.0)
    loss = losses.sum() / live.sum()
    (dl.double() * loss + (dls.double() * losses).sum()).backward()
    for p, q in ((got["losses"], losses), (got["loss"], loss), (got["dh"], a.grad), (got["dw"], b.grad)):
        assert torch.allclose(p, q, rtol=1e-10, atol=1e-12)


def test_a_temperature_is_taken_by_value():
    """Of a tensor too, which may be changed in place between two calls."""
    h, w = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    ids, teacher, heat = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), torch.tensor(2.0)
    for value in (2.0, 4.0, 0.5):
        heat.fill_(value)
        x = head._Inputs(h, w, ids, teacher, None, heat)
        assert C.cast(x.ref, C.POINTER(head.HeadDesc))[0].temperature == value


@pytest.mark.parametrize("strides", [(8, 1), (11, 1), (1, 5), (1, 9), (20, 2), (0, 1), (3, 1), (40, 0)])
def test_results_that_touch_an_input(strides):
    """Against the numbers of the input's rows one by one: what lies between two rows is free."""
    rows, cols = 5, 8
    room = torch.zeros(400, dtype=torch.bfloat16)
    t = room.as_strided((rows, cols), strides, 100)
    inner = min(strides)
    taken = set()
    for i in range(rows if strides[0] >= strides[1] else cols):
        n = cols if strides[0] >= strides[1] else rows
        taken |= set(range(100 + i * max(strides), 100 + i * max(strides) + (n - 1) * inner + 1))
    for at, n in itertools.product(range(60, 340), (1, 2, 7, 30)):
        try:
            head._apart((None, room[at:at + n]), ("first", "second"), (None, t))
            refused = False
        except ValueError as e:
            refused = "second shares memory" in str(e)
        assert refused == bool(taken & set(range(at, at + n))), (at, n)
    head._apart((room[120:120],), ("empty",), (t,))     # nothing is written, nothing read
    head._apart((room[120:130],), ("result",), (t[:0], t[:, :0]))
    with pytest.raises(ValueError, match="b shares memory"):
        head._apart((room[:10], room[9:12]), ("a", "b"), ())
    head._apart((room[:10], room[10:12]), ("a", "b"), ())


def test_the_count_of_waits_refuses():
    assert head.lib().nest_head_waits_given_up(None, None) == nest.NEST_E_INVALID
    with pytest.raises(ValueError, match="CUDA"):
        head.waits_given_up("cpu")


@pytest.mark.parametrize("T,V,D,k,loss,backward", [(1, 32000, 4096, 0, 2.5, 31.1), (64, 128000, 1024, 0, 2.1, 76.5),
                                                   (1777, 50021, 1000, 0, 8.4, 197.8), (2048, 32000, 4096, 0, 20.9, 147.9),
                                                   (2048, 32000, 4096, 64, 21.9, 148.9), (4096, 128000, 4096, 0, 58.2, 362.9),
                                                   (16384, 128000, 512, 0, 115.2, 319.0)])
def test_workspace_of_a_planner(T, V, D, k, loss, backward):
    """What a step at the head needs beside its inputs and results, in MB as it is documented."""
    L, d = head.lib(), desc(tokens=T, vocab=V, hidden=D, hidden_row=D, weight_row=D, k=k)
    assert round(L.nest_head_loss_workspace_size(C.byref(d), FAKE) / 1e6, 1) == loss
    assert round(L.nest_head_backward_workspace_size(C.byref(d), FAKE) / 1e6, 1) == backward
