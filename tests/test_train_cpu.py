"""Host-side checks of the training-step operators that need no GPU: the ABI, packing, refusals,
and the 64-bit forms that the GPU tests compare against."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import train_ref as ref
from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import nest, train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "nest_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(nest_\w+)\s*\(", text, flags=re.M))
    assert names == set(train.EXPORTS)
    L = C.CDLL(nest.LIB_PATH)
    for n in names:
        assert hasattr(L, n), n


def desc(**kw):
    d = dict(tokens=4, experts=8, k=2, row_stride=8, col_stride=1, dtype=train.F32, normalize=1)
    d.update(kw)
    return train.RouteDesc(*[d[n] for n, _ in train.RouteDesc._fields_])


@pytest.mark.parametrize("kw,rc", [
    (dict(tokens=-1), nest.NEST_E_INVALID), (dict(experts=0), nest.NEST_E_INVALID),
    (dict(k=0), nest.NEST_E_INVALID), (dict(k=9), nest.NEST_E_INVALID), (dict(dtype=3), nest.NEST_E_INVALID),
    (dict(row_stride=-1), nest.NEST_E_INVALID), (dict(col_stride=-1), nest.NEST_E_INVALID),
    (dict(normalize=2), nest.NEST_E_INVALID), (dict(experts=1025), nest.NEST_E_LIMITS),
    (dict(experts=64, k=33), nest.NEST_E_LIMITS), (dict(tokens=2**31), nest.NEST_E_LIMITS),
    (dict(tokens=2**30), nest.NEST_E_LIMITS), (dict(), nest.NEST_E_INVALID)])
def test_route_refusals(kw, rc):
    d = desc(**kw)
    L = train.lib()
    assert (L.nest_route_workspace_size(C.byref(d)) == 0) == bool(kw)
    assert L.nest_route(C.byref(d), None, None, None, None, None, None, None, None, None, 0, None) == rc
    assert L.nest_route_backward(C.byref(d), None, None, None, None, None, None, None, None, None, 8, None) == rc


def test_route_workspace_is_checked():
    d, L, fake = desc(), train.lib(), 4096
    need = L.nest_route_workspace_size(C.byref(d))
    args = [C.byref(d), fake, None, fake, fake, fake, fake, fake, fake]
    assert L.nest_route(*args, fake, need - 1, None) == nest.NEST_E_WORKSPACE
    assert L.nest_route(*args, fake + 16, need, None) == nest.NEST_E_WORKSPACE
    assert L.nest_route(*args, None, need, None) == nest.NEST_E_WORKSPACE
    args[1] = fake + 2   # not a float's address
    assert L.nest_route(*args, fake, need, None) == nest.NEST_E_INVALID


def test_route_backward_of_nothing_reads_nothing():
    d = desc(tokens=0)
    L = train.lib()
    assert L.nest_route_backward(C.byref(d), None, None, None, None, None, None, None, None, None, 8, None) == 0
    assert L.nest_route_backward(C.byref(d), None, None, None, None, None, None, None, None, None, 7, None) == \
        nest.NEST_E_INVALID


def tensors(numels):
    rec = np.zeros(len(numels), train.TENSOR_DT)
    rec["numel"], rec["grad"], rec["weight"] = numels, 4096, 8192
    return rec


def query(rec):
    info = train.TableInfo()
    rc = train.lib().nest_table_query(rec.ctypes.data, len(rec), C.byref(info))
    return rc, info


@pytest.mark.parametrize("numels", [[], [0], [1], [256], [257, 0, 1], [4096, 4097, 3], [10**6] * 3])
def test_table_counts_blocks(numels):
    rec = tensors(numels)
    rc, info = query(rec)
    assert rc == 0 and info.tensors == len(numels)
    assert info.blocks == sum(-(-n // 256) for n in numels)
    assert (info.items > 0) == (info.blocks > 0) and info.items <= info.blocks
    packed = np.full(info.table_bytes + 16, 0xAB, np.uint8)
    assert train.lib().nest_table_pack(rec.ctypes.data, len(rec), C.byref(info), packed.ctypes.data) == 0
    assert (packed[info.table_bytes:] == 0xAB).all()


def test_table_refusals():
    L = train.lib()
    assert query(tensors([-1]))[0] == nest.NEST_E_INVALID
    assert query(tensors([2**39]))[0] == nest.NEST_E_LIMITS
    assert query(tensors([2**38, 2**38, 2**38]))[0] == nest.NEST_E_LIMITS
    rec = tensors([5])
    rec["grad"] = 0
    assert query(rec)[0] == nest.NEST_E_INVALID
    info = train.TableInfo()
    assert L.nest_table_query(None, 1, C.byref(info)) == nest.NEST_E_INVALID
    assert L.nest_table_query(None, -1, C.byref(info)) == nest.NEST_E_INVALID
    rec = tensors([5, 7])
    rc, info = query(rec)
    info.items += 1
    buf = np.zeros(4096, np.uint8)
    assert L.nest_table_pack(rec.ctypes.data, 2, C.byref(info), buf.ctypes.data) == nest.NEST_E_INVALID


def adamw_args(**kw):
    d = dict(weight_type=train.BF16, grad_type=train.BF16, state_bits=8, seed=0, lr=1e-3, beta1=0.9, beta2=0.99,
             eps=1e-8, master=4096, m=4096, v=4096, m_exp=4096, v_exp=4096, state=4096, grad_scale=None)
    d.update(kw)
    return train.AdamWArgs(*[d[n] for n, _ in train.AdamWArgs._fields_])


@pytest.mark.parametrize("kw", [
    dict(weight_type=5), dict(grad_type=-1), dict(state_bits=16), dict(state=None), dict(state=4104), dict(beta1=1.0),
    dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1.0), dict(eps=float("inf")),
    dict(lr=float("nan")), dict(lr=float("inf")), dict(master=None), dict(weight_type=train.F32), dict(m=None),
    dict(v=None), dict(m_exp=None), dict(v_exp=None), dict(state_bits=32), dict(m=4096 + 16), dict(master=4100)])
def test_adamw_refusals(kw):
    _, info = query(tensors([300]))
    a = adamw_args(**kw)
    assert train.lib().nest_adamw(C.byref(info), 4096, C.byref(a), None) == nest.NEST_E_INVALID


def test_other_list_refusals():
    L = train.lib()
    _, info = query(tensors([300]))
    need = L.nest_grad_norm_workspace_size(C.byref(info))
    assert need > 0
    norm = lambda **kw: L.nest_grad_norm(C.byref(kw.get("info", info)), kw.get("table", 4096), kw.get("t", 0),
                                         kw.get("max_norm", 1.0), kw.get("out", 4096), kw.get("ws", 4096),
                                         kw.get("n", need), None)
    for kw in (dict(table=None), dict(table=4100), dict(t=9), dict(max_norm=0.0), dict(max_norm=-1.0),
               dict(max_norm=float("nan")), dict(out=None)):
        assert norm(**kw) == nest.NEST_E_INVALID, kw
    for kw in (dict(ws=None), dict(ws=4100), dict(n=need - 1)):
        assert norm(**kw) == nest.NEST_E_WORKSPACE, kw
    a = adamw_args()
    assert L.nest_adamw(None, 4096, C.byref(a), None) == nest.NEST_E_INVALID
    assert L.nest_adamw(C.byref(info), None, C.byref(a), None) == nest.NEST_E_INVALID
    assert L.nest_adamw(C.byref(info), 4096, None, None) == nest.NEST_E_INVALID
    bad = train.TableInfo(0, 2, 1, 1, 0)   # a table smaller than its entries
    assert L.nest_adamw(C.byref(bad), 4096, C.byref(a), None) == nest.NEST_E_INVALID
    assert L.nest_adamw_values(C.byref(info), 4096, 4096, 4096, None, 4096, 4096, None) == nest.NEST_E_INVALID
    assert L.nest_adamw_values(C.byref(info), 4096, 4096, 4096, 4096, 4100, 4096, None) == nest.NEST_E_INVALID


def test_python_refusals_on_the_cpu():
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="CUDA"):
        train.route(x, 2)
    with pytest.raises(ValueError, match="tokens, experts"):
        train.route(x[0], 2)
    with pytest.raises(TypeError):
        train.route(x.int(), 2)
    with pytest.raises(nest.NestError):
        train.route(x, 9)
    with pytest.raises(nest.NestError):
        train.route(torch.zeros(1, 2000), 2)
    with pytest.raises(ValueError):
        train.GradNorm([])
    with pytest.raises(ValueError, match="CUDA"):
        train.GradNorm([x])
    with pytest.raises(ValueError):
        train.AdamW([x], [x], state_bits=4)


def test_capacity():
    assert train.capacity_milli([2, 2, 2, 2], 4, 2) == 1000
    assert train.capacity_milli([5, 1, 1, 1], 4, 2) == 2500
    assert train.capacity_milli([3, 2, 2], 7, 1) == 1286       # 9/7 rounded up
    assert train.capacity_milli([1, 0], 4, 1) == 1000          # rows that chose nothing
    assert train.capacity_milli([0, 0], 0, 1) == 1000


# ---- the 64-bit forms ------------------------------------------------------------------

@pytest.mark.parametrize("normalize", [True, False])
def test_reference_gradient_against_differences(normalize):
    """Central differences of the 64-bit forward pass; the counts stay as they are, as long as no
    step changes an order (logits at least 0.02 apart, steps of 1e-5)."""
    rng = np.random.default_rng(1)
    T, E, k = 3, 7, 3
    x = np.stack([rng.permutation(E) * 0.3 + rng.uniform(-0.1, 0.1, E) for _ in range(T)])
    x[1, 2] = -np.inf
    dw, dl = rng.normal(size=(T, k)), 0.7
    r = ref.route(x, k, normalize=normalize)
    got, _ = ref.route_backward(x, r, dw, dl, normalize)

    def value(y):
        q = ref.route(y, k, normalize=normalize)
        assert (q["ids"] == r["ids"]).all()
        return float((dw * q["weights"]).sum()) + dl * q["loss"]
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(x[t, e]):
                assert got[t, e] == 0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            # third derivatives of order 1: h^2 = 1e-10; cancellation 1e-16 / h = 1e-11, times sums of order 10
            assert abs((value(up) - value(dn)) / (2 * h) - got[t, e]) < 2e-9


def test_reference_codes_round_trip():
    """Every code is its own rounding without noise, and rounding is monotone and unbiased."""
    for signed, codes in ((True, np.arange(0x7F)), (False, np.arange(0xFF))):
        c = np.zeros((1, 256), np.int64)
        c[0, :len(codes)] = codes
        exp = np.array([3])
        v = ref.code_value(c, exp, signed)
        assert (np.diff(v[0, :len(codes)]) > 0).all()
        back, _ = ref.to_codes(v, exp, np.zeros_like(c), signed)
        assert (back == c).all()
        assert (ref.to_codes(v, exp, np.full_like(c, 65535), signed)[0] == c).all()
    x = np.full((1, 256), 1.37)
    r = np.arange(65536).reshape(256, 256)
    got = np.mean([ref.code_value(*[np.asarray(q) for q in (ref.to_codes(x, np.array([0]), r[i:i + 1], True)[0],
                                                             np.array([0]))], True) for i in range(256)])
    assert abs(got - 1.37) <= 0.125 / 65536      # one part in 2^16 of a step


def test_noise_is_even():
    """Mean and correlation of the noise within 5 standard deviations of independent uniform words."""
    m, v = ref.noise(12345, 7, np.arange(4096))
    n = m.size
    sd = 65536 / 12 ** 0.5
    for x in (m, v):
        assert abs(x.mean() - 32767.5) < 5 * sd / n ** 0.5
        assert abs(np.mean(x[:, :-1] * 1.0 * x[:, 1:]) - 32767.5 ** 2) < 5 * 2 * 32767.5 * sd / n ** 0.5
        hist = np.bincount((x >> 8).ravel(), minlength=256)
        assert ((hist - n / 256) ** 2).sum() / (n / 256) < 255 + 5 * (2 * 255) ** 0.5
    c = np.corrcoef(m.ravel(), v.ravel())[0, 1]
    assert abs(c) < 5 / n ** 0.5
    m2, _ = ref.noise(12345, 8, np.arange(4096))
    assert abs(np.corrcoef(m.ravel(), m2.ravel())[0, 1]) < 5 / n ** 0.5


@pytest.mark.parametrize("numels", [[1], [31] * 300, [256 * 9 + 1, 0, 5], [10**6, 3, 2 * 10**6], [40000] * 70,
                                    [2**33, 7]])
def test_table_covers_every_block_once(numels):
    """The workers' segments are the tensors' blocks, each once; shares are even."""
    rec = tensors(numels)
    rc, info = query(rec)
    assert rc == 0
    packed = np.zeros(info.table_bytes, np.uint8)
    assert train.lib().nest_table_pack(rec.ctypes.data, len(rec), C.byref(info), packed.ctypes.data) == 0
    a, b = 48 * len(numels), 48 * len(numels) + 16 * info.items
    entries = packed[:a].view(np.int64).reshape(-1, 6)
    seg, starts = packed[a:b].view(np.int32).reshape(-1, 4), packed[b:].view(np.int32)
    blocks = [-(-n // 256) for n in numels]
    assert (entries[:, 2] == numels).all() and (entries[:, 3] == np.cumsum([0] + blocks[:-1])).all()
    assert len(starts) == info.workers + 1 and starts[0] == 0 and starts[-1] == info.items
    share = [seg[starts[w]:starts[w + 1], 2].sum() for w in range(info.workers)]
    assert max(share) - min(share) <= 1 and sum(share) == info.blocks
    runs = []
    for w in range(info.workers):
        before = 0
        for t, block, count, skip in seg[starts[w]:starts[w + 1]].astype(np.int64):
            assert count > 0 and skip == before and block + count <= blocks[t]
            before += count
            runs.append((entries[t, 3] + block, count))
    runs.sort()
    assert runs[0][0] == 0 and all(a + n == b for (a, n), (b, _) in zip(runs, runs[1:]))
    assert sum(runs[-1]) == info.blocks
