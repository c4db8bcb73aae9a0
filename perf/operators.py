"""The training-step operators beside the placement solver, as cases to be timed and compared.

Four operators of one training step of a mixture-of-experts block, whose results also feed the
solver's layer tables (the expert counts give the all-to-all volume, the optimizer states the bytes
per weight):

  route           softmax gates, the k chosen experts, expert counts and the balance loss
  route_backward  its gradient with respect to the logits
  grad_norm       the global norm of many gradient tensors and the scale that clips it
  adamw           one AdamW step over many tensors, with states in 32 or 8 bits

`own` false computes them in plain torch operations, true through memory_aware_device_gb300.train.
"""
import math
import random

import torch

own = False

BLOCK = 256          # elements that share a scale in the 8-bit states; tensors start at a multiple
WORD = 0xFFFFFFFF
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
BETA1, BETA2, EPS, LR = 0.9, 0.95, 1e-8, 3e-4
LARGEST_TOKENS = 262144


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------

def listed():
    def route(name, op, tokens, experts, k, dtype, normalize=True, padded=0.0, closed=0, wider=0):
        return {"name": name, "op": op, "tokens": tokens, "experts": experts, "k": k, "dtype": dtype,
                "normalize": normalize, "padded": padded, "closed": closed, "wider": wider}

    def weights(name, op, layout, size, count, grad, weight="bf16", bits=32, shift=0):
        return {"name": name, "op": op, "layout": layout, "size": size, "count": count, "grad": grad,
                "weight": weight, "bits": bits, "shift": shift}

    return [
        # serving: the router of one layer for the single token of a decoding step
        route("route 1 token", "route", 1, 64, 2, "fp32"),
        # the solver's own MoE block: 64 experts, 2 per token, a microbatch of 2048 tokens
        route("route microbatch", "route", 2048, 64, 2, "bf16"),
        # packed documents with padding, an odd expert count, some experts closed, logits that are
        # the first columns of a wider product
        route("route ragged", "route", 30011, 72, 5, "fp16", False, 0.2, 7, 9),
        # a global batch of a fine-grained mixture, routed in 32 bits
        route("route global batch", "route", 262144, 256, 8, "fp32"),
        # the gradient for the microbatch above
        route("route_backward microbatch", "route_backward", 2048, 64, 2, "bf16"),
        # and for half a global batch less one token
        route("route_backward half batch", "route_backward", 131071, 256, 8, "fp32"),
        # the small tensors alone: router and norms of a model, gradients kept in 32 bits
        weights("grad_norm small tensors", "grad_norm", "ragged", 5000, 67, "fp32"),
        # the gradients of one dense block of hidden size 4096 (the solver's 32-layer workload)
        weights("grad_norm dense block", "grad_norm", "block", 4096, 1, "bf16"),
        # routers, biases and norms, which stay in 32 bits
        weights("adamw small tensors", "adamw", "ragged", 60000, 130, "fp32", "fp32"),
        # one dense block of hidden size 4096 with the states that the solver's factor 6 stands for
        weights("adamw dense block", "adamw", "block", 4096, 1, "bf16"),
        # odd sizes with 8-bit states, gradients that start off alignment
        weights("adamw 8-bit ragged", "adamw", "ragged", 200000, 61, "fp16", "fp16", 8, 1),
        # the dense block with 8-bit states
        weights("adamw 8-bit dense block", "adamw", "block", 4096, 1, "bf16", "bf16", 8),
    ]


def log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "grad_norm", "adamw"])
    if op.startswith("route"):
        experts = log_between(rng, 8, 512)
        tokens = log_between(rng, 1, LARGEST_TOKENS)
        tokens = max(1, min(tokens, LARGEST_TOKENS * 128 // experts))
        return {"op": op, "tokens": tokens, "experts": experts, "k": rng.randint(1, min(16, experts)),
                "dtype": rng.choice(["fp32", "bf16", "fp16"]), "normalize": rng.random() < 0.7,
                "padded": rng.choice([0.0, 0.1, 0.4]), "closed": rng.choice([0, 0, experts // 6]),
                "wider": rng.choice([0, 0, rng.randint(1, 40)])}
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    case = {"op": op, "grad": dtype, "weight": rng.choice([dtype, "bf16"]), "bits": rng.choice([8, 32]),
            "shift": rng.choice([0, 0, 1])}
    if rng.random() < 0.3:
        return {**case, "layout": "block", "size": log_between(rng, 65, 3700), "count": 1}
    count = log_between(rng, 1, 300)
    return {**case, "layout": "ragged", "count": count, "size": log_between(rng, 16, 30_000_000 // count + 16)}


def numels(case):
    """Elements of each tensor: a transformer block's (four square products, the two of its
    feed-forward part, two norms), or odd sizes of up to `size` elements."""
    s = case["size"]
    if case["layout"] == "block":
        return [s * s] * 4 + [4 * s * s] * 2 + [s] * 2
    rng = random.Random(7 * case["count"] + s)
    return [log_between(rng, 1, s) for _ in range(case["count"])]


def places(case):
    """(start, elements) of each tensor in a buffer where each starts at a multiple of BLOCK, and
    the buffer's length."""
    at, got = 0, []
    for n in numels(case):
        got.append((at, n))
        at += -(-n // BLOCK) * BLOCK
    return got, at


def work(case):
    if case["op"].startswith("route"):
        t, e, k, s = case["tokens"], case["experts"], case["k"], BYTES[case["dtype"]]
        mask = t if case["padded"] else 0
        if case["op"] == "route":   # logits and mask in; ids and gates, counts and mean gates out
            return {"bytes": t * e * s + mask + 8 * t * k + 8 * e, "flops": 5 * t * e}
        # logits, mask, ids, gates, their gradients and the counts in; the logits' gradient out
        return {"bytes": 2 * t * e * s + mask + 12 * t * k + 4 * e, "flops": 8 * t * e}
    n, g, w = sum(numels(case)), BYTES[case["grad"]], BYTES[case["weight"]]
    if case["op"] == "grad_norm":
        return {"bytes": n * g, "flops": 2 * n}
    moved = g + (8 if case["weight"] == "fp32" else 8 + w)
    # moments in and out; with 8 bits also the values that they stand for, in 16 bits
    moved += 16 if case["bits"] == 32 else 4 + 4 / BLOCK + 4
    return {"bytes": n * moved, "flops": 15 * n}


# ---------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------

def router_inputs(case, seed):
    dev = device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    t, e, k = case["tokens"], case["experts"], case["k"]
    lean = torch.randn(e, generator=gen, device=dev) * 0.5      # some experts are liked more
    wide = torch.randn(t, e + case["wider"], generator=gen, device=dev) * 1.5
    wide[:, :e] += lean
    if case["closed"]:
        wide[:, torch.randperm(e, generator=gen, device=dev)[:case["closed"]]] = -math.inf
    mask = None
    if case["padded"]:
        mask = torch.rand(t, generator=gen, device=dev) >= case["padded"]
        wide[~mask] = math.nan                                  # what padding rows hold is anything
    state = {"case": case, "logits": wide.to(TYPES[case["dtype"]])[:, :e], "mask": mask}
    if case["op"] == "route_backward":
        state["routed"] = route_plain(state["logits"], mask, k, case["normalize"])
        state["grad_weights"] = torch.randn(t, k, generator=gen, device=dev) * 1e-3
        state["grad_loss"] = torch.rand((), generator=gen, device=dev) * 0.02 + 0.01
    return state


def tensor_inputs(case, seed):
    dev = device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    where, length = places(case)

    def per_block(values):
        return torch.repeat_interleave(torch.tensor(values, device=dev),
                                       torch.tensor([-(-n // BLOCK) for _, n in where], device=dev))

    filled = torch.arange(BLOCK, device=dev)[None, :] < per_block([n for _, n in where])[:, None] - \
        BLOCK * (torch.arange(length // BLOCK, device=dev) - per_block([a // BLOCK for a, _ in where]))[:, None]
    filled = filled.reshape(-1)

    def normal(scale):
        return torch.randn(length, generator=gen, device=dev).mul_(scale).mul_(filled)

    # gradients of single tensors differ in size by orders of magnitude
    sizes = torch.exp(torch.randn(len(where), generator=gen, device=dev) * 1.5 - 8)
    size = torch.repeat_interleave(sizes, torch.tensor([-(-n // BLOCK) for _, n in where], device=dev))
    grad = (normal(1.0).view(-1, BLOCK) * size[:, None]).reshape(-1)
    room = torch.zeros(length + case["shift"], dtype=TYPES[case["grad"]], device=dev)
    room[case["shift"]:] = grad
    state = {"case": case, "grads": room[case["shift"]:], "where": where}
    if case["op"] == "grad_norm":
        if own:
            from memory_aware_device_gb300 import train
            state["norm"] = train.GradNorm([state["grads"][a:a + n] for a, n in where])
        return state
    master = normal(0.02)
    m = grad * 0.5 + (normal(1.0).view(-1, BLOCK) * size[:, None]).reshape(-1) * 0.3
    v = ((normal(1.0).view(-1, BLOCK) * size[:, None]).square() + 0.3 * size[:, None] ** 2).reshape(-1) * filled
    weights = master.to(TYPES[case["weight"]])
    decay = [0.1 if n % 2 == 0 else 0.0 for _, n in where]      # some tensors are not decayed
    state |= {"weights": weights, "master": weights if case["weight"] == "fp32" else master,
              "m": m, "v": v, "step": 1000, "seed": seed & 0x7FFFFFFF, "decay": per_block(decay)[:, None],
              "scale": torch.rand((), generator=gen, device=dev) * 0.5 + 0.5}
    if case["bits"] == 8:
        half = torch.full((length // BLOCK, BLOCK), 1 << 15, dtype=torch.int64, device=dev)
        state["m"], state["m_exp"] = encode_m(m.view(-1, BLOCK), half)
        state["v"], state["v_exp"] = encode_v(v.view(-1, BLOCK), half)
    if own:
        from memory_aware_device_gb300 import train
        views = [[b[a:a + n] for a, n in where] for b in (weights, state["grads"])]
        opt = train.AdamW(*views, state_bits=case["bits"], betas=(BETA1, BETA2), eps=EPS, weight_decay=decay,
                          seed=state["seed"])
        opt.set_step(state["step"])
        for name in ("m", "v", "m_exp", "v_exp"):
            if name in state:
                getattr(opt, name).copy_(state.pop(name).view(-1))
        if opt.master is not None:
            opt.master.copy_(master)
        state.pop("master")
        state["opt"] = opt
    return state


def prepare(case, seed):
    if not case["op"].startswith("route"):
        return tensor_inputs(case, seed)
    state = router_inputs(case, seed)
    if own:
        from memory_aware_device_gb300 import train
        t, e, k = case["tokens"], case["experts"], case["k"]
        if case["op"] == "route":
            state["out"] = train.Routing.empty(t, e, k, device())
        else:
            state["routed"] = train.Routing(**state["routed"])
            state["out"] = torch.empty(t, e, dtype=state["logits"].dtype, device=device())
    return state


# ---------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------

def gates(logits, mask):
    """Softmax of the rows that count, 0 in the others; the logits by which experts are chosen."""
    x = logits.float()
    live = (x != -math.inf).any(1)
    if mask is not None:
        live = live & mask
    x = torch.where(live[:, None], x, 0.0)
    e = torch.exp(x - x.amax(1, keepdim=True))
    p = torch.where(live[:, None], e / e.sum(1, keepdim=True), 0.0)
    return p, live, torch.where(torch.isnan(x), -math.inf, x)


def route_plain(logits, mask, k, normalize):
    p, live, by = gates(logits, mask)
    experts = p.shape[1]
    by, order = torch.sort(by, dim=1, descending=True, stable=True)
    taken = (by[:, :k] > -math.inf) & live[:, None]
    order = order[:, :k]
    w = torch.where(taken, torch.gather(p, 1, order), 0.0)
    if normalize:
        w = torch.where(taken, w / w.sum(1, keepdim=True), 0.0)
    n = live.sum()
    counts = torch.zeros(experts + 1, dtype=torch.int32, device=p.device)
    counts.scatter_add_(0, torch.where(taken, order, experts).reshape(-1),
                        torch.ones(order.numel(), dtype=torch.int32, device=p.device))
    counts = counts[:experts]
    mean = p.sum(0) / n.clamp(min=1)
    loss = (counts.float() * mean).sum() * experts / (k * n.clamp(min=1).float())
    return {"ids": torch.where(taken, order, -1).int(), "weights": w, "counts": counts,
            "tokens": n.int().reshape(1), "mean_prob": mean, "loss": loss}


def route_backward_plain(logits, mask, routed, grad_weights, grad_loss, normalize):
    p, live, _ = gates(logits, mask)
    experts, k = p.shape[1], grad_weights.shape[1]
    n = routed["tokens"].clamp(min=1).float()
    taken = routed["ids"] >= 0
    at = routed["ids"].long().clamp(min=0)
    u = torch.where(taken, grad_weights, 0.0)
    if normalize:
        total = torch.where(taken, torch.gather(p, 1, at), 0.0).sum(1, keepdim=True)
        u = torch.where(taken, (u - (u * routed["weights"]).sum(1, keepdim=True)) / total, 0.0)
    # a constant in d drops out of the softmax's gradient: the counts enter by their distance from the mean
    d = (grad_loss * experts / (k * n * n)) * (routed["counts"].float() - k * n / experts)
    d = d.expand(p.shape).scatter_add(1, at, u)
    grad = p * (d - (p * d).sum(1, keepdim=True))
    return torch.where(live[:, None], grad, 0.0).to(logits.dtype)


def grad_norm_plain(grads):
    norm = grads.float().square().sum().sqrt()
    return torch.stack([norm, torch.clamp(1.0 / (norm + 1e-6), max=1.0)])


def mixed(x):
    """Spreads the bits of a 32-bit word."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & WORD
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & WORD
    return x ^ (x >> 16)


def noise(seed, step, blocks):
    """A word for each element: its upper 16 bits round the first moment, its lower ones the second."""
    dev = device()
    start = mixed(seed ^ mixed(step))
    block = mixed((start + torch.arange(blocks, device=dev) * 0x9E3779B1) & WORD)
    x = (block[:, None] + torch.arange(BLOCK, device=dev)[None, :] * 0x9E3779B1) & WORD
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & WORD
    return x ^ (x >> 16)


def power(e):
    """2 to the power of whole numbers in the normal range of 32 bits."""
    return ((e + 127).int() << 23).view(torch.float32)


def shared_exponent(x):
    """The exponent e of each block with every finite |x| < 1.75 * 2^e."""
    a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(1, keepdim=True)
    return (((a.view(torch.int32) + (1 << 21)) >> 23) - 127).clamp(-100, 120)


def rounded(a, r, lowest, offset, small):
    """Codes with 3 mantissa bits: the bits below them, with 16 random ones added, are cut off;
    under 2^lowest the code counts steps of 1/small."""
    code = ((a.view(torch.int32) + (r.int() << 4)) >> 20) - (offset << 3)
    return torch.where(a < 2.0 ** lowest, (a * small + r.float() * 2.0 ** -16).int(), code)


def encode_m(m, r):
    e = shared_exponent(m)
    y = m * power(8 - e)
    code = rounded(y.abs(), r, -6, 120, 512.0).clamp(max=0x7E)
    code = torch.where(torch.isfinite(m), code, 0x7F) | torch.where(y < 0, 0x80, 0)
    return code.to(torch.uint8), e.to(torch.int8)


def encode_v(v, r):
    e = shared_exponent(v)
    y = v * power(-1 - e)
    code = rounded(y, r, -31, 95, 2.0 ** 34).clamp(max=0xFE)
    return torch.where(torch.isfinite(v), code, 0xFF).to(torch.uint8), e.to(torch.int8)


def decode_m(code, e):
    return code.view(torch.float8_e4m3fn).float() * power(e.int() - 8)


def decode_v(code, e):
    y = (code.int() << 20).view(torch.float32) * 2.0 ** 95 * power(e.int() + 1)
    return torch.where(code == 0xFF, math.nan, y)


def adamw_plain(state):
    case = state["case"]
    state["step"] += 1
    t, eight = state["step"], case["bits"] == 8
    g = state["grads"].float().view(-1, BLOCK) * state["scale"]
    m, v = state["m"].view(-1, BLOCK), state["v"].view(-1, BLOCK)
    if eight:
        m, v = decode_m(m, state["m_exp"]), decode_v(v, state["v_exp"])
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    p = state["master"].view(-1, BLOCK)
    root = torch.sqrt(v) * (1 / math.sqrt(1 - BETA2 ** t)) + EPS
    p = p - (m * (1 / (1 - BETA1 ** t)) / root + p * state["decay"]) * LR
    state["master"].copy_(p.view(-1))
    if case["weight"] != "fp32":
        state["weights"].copy_(p.view(-1))
    if not eight:
        state["m"].copy_(m.view(-1))
        state["v"].copy_(v.view(-1))
        return {"weights": state["weights"], "master": state["master"], "m": state["m"], "v": state["v"]}
    r = noise(state["seed"], t, m.shape[0])
    state["m"], state["m_exp"] = encode_m(m, r >> 16)
    state["v"], state["v_exp"] = encode_v(v, r & 0xFFFF)
    # a code has four significant bits and a power of two: 16 bits hold its value exactly
    return {"weights": state["weights"], "master": state["master"],
            "m": decode_m(state["m"], state["m_exp"]).view(-1).bfloat16(),
            "v": decode_v(state["v"], state["v_exp"]).view(-1).bfloat16()}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from memory_aware_device_gb300 import train
        if op == "route":
            r = train.route(state["logits"], case["k"], mask=state["mask"], normalize=case["normalize"],
                            out=state["out"])
            return {"ids": r.ids, "weights": r.weights, "counts": r.counts, "tokens": r.tokens,
                    "mean_prob": r.mean_prob, "loss": r.loss}
        if op == "route_backward":
            return train.route_backward(state["logits"], state["routed"], state["grad_weights"], state["grad_loss"],
                                        mask=state["mask"], normalize=case["normalize"], out=state["out"])
        if op == "grad_norm":
            return state["norm"].run(max_norm=1.0)
        opt = state["opt"]
        opt.step(LR, grad_scale=state["scale"])
        m, v = opt.state_values()
        return {"weights": state["weights"], "master": state["weights"] if opt.master is None else opt.master,
                "m": m, "v": v}
    if op == "route":
        return route_plain(state["logits"], state["mask"], case["k"], case["normalize"])
    if op == "route_backward":
        return route_backward_plain(state["logits"], state["mask"], state["routed"], state["grad_weights"],
                                    state["grad_loss"], case["normalize"])
    if op == "grad_norm":
        return grad_norm_plain(state["grads"])
    return adamw_plain(state)


# ---------------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------------

def exact_softmax(logits, mask):
    x = logits.double()
    live = ~(x == -math.inf).all(1)
    if mask is not None:
        live &= mask
    z = x[live]
    return z, torch.exp(z - torch.logsumexp(z, 1, keepdim=True)), live


def exact_choice(z, k):
    """The k largest of each row, one after the other, the lower index where two are equal."""
    left = z.clone()
    index = torch.arange(z.shape[1], device=z.device).expand(z.shape)
    found = []
    for _ in range(k):
        best = left.amax(1, keepdim=True)
        at = torch.where(left == best, index, z.shape[1]).amin(1, keepdim=True)
        found.append(torch.where(best > -math.inf, at, -1))
        left.scatter_(1, at, -math.inf)
    return torch.cat(found, 1)


def exact_route(state, case):
    k, experts = case["k"], case["experts"]
    z, p, live = exact_softmax(state["logits"], state["mask"])
    t, n = live.shape[0], z.shape[0]
    pick = exact_choice(z, k)
    w = torch.where(pick >= 0, p.gather(1, pick.clamp(min=0)), 0.0)
    if case["normalize"] and n:
        w = w / w.sum(1, keepdim=True)
    counts = (torch.bincount(pick[pick >= 0], minlength=experts)).double()
    ids = torch.full((t, k), -1, dtype=torch.int32, device=z.device)
    ids[live] = pick.int()
    weights = torch.zeros(t, k, dtype=torch.float64, device=z.device)
    weights[live] = w
    mean = p.mean(0) if n else torch.zeros(experts, dtype=torch.float64, device=z.device)
    share = counts / max(1, k * n)
    return {"ids": ids, "weights": weights, "counts": counts.int(), "tokens": torch.tensor([n], dtype=torch.int32),
            "mean_prob": mean, "loss": experts * torch.dot(share, mean)}


def exact_route_backward(state, case):
    k, experts, routed = case["k"], case["experts"], state["routed"]
    z, p, live = exact_softmax(state["logits"], state["mask"])
    n = int(routed["tokens"][0])
    grad = torch.zeros(live.shape[0], experts, dtype=torch.float64, device=z.device)
    if not n:
        return grad
    pick = routed["ids"][live].long()
    chosen = torch.zeros_like(p, dtype=torch.bool)
    spare = torch.zeros(p.shape[0], experts + 1, dtype=torch.float64, device=z.device)
    spare.scatter_(1, torch.where(pick >= 0, pick, experts), state["grad_weights"][live].double())
    u = spare[:, :experts]
    chosen.scatter_(1, pick.clamp(min=0), True)
    if case["normalize"]:   # the gates are a softmax over the chosen experts alone
        q = torch.where(chosen, p, 0.0)
        q = q / q.sum(1, keepdim=True)
        through = q * (u - (q * u).sum(1, keepdim=True))
    else:
        through = p * (u - (p * u).sum(1, keepdim=True))
    f = float(state["grad_loss"]) * experts * routed["counts"].double() / (k * float(n) ** 2)
    grad[live] = through + p * (f - (p @ f)[:, None])
    return grad


def exact_words(seed, step, blocks):
    """The rounding words again, by remainders and quotients."""
    def spread(x):
        x ^= x >> 16
        x = x * 0x9E3779B1 % 2 ** 32
        x ^= x >> 15
        x = x * 0x6A09E667 % 2 ** 32
        return x ^ x >> 16
    start = spread(seed ^ spread(step))
    b = torch.arange(blocks, dtype=torch.int64, device=device())
    x = (start + b * 0x9E3779B1) % 2 ** 32
    x = x ^ x // 65536
    x = x * (0x9E3779B1 - 2 ** 32) % 2 ** 32
    x = x ^ x // 32768
    x = x * 0x6A09E667 % 2 ** 32
    x = x ^ x // 65536
    y = (x[:, None] + torch.arange(BLOCK, device=device()) * 0x9E3779B1 % 2 ** 32) % 2 ** 32
    y = y ^ y // 32768
    y = y * 0x6A09E667 % 2 ** 32
    return y ^ y // 65536


def exact_eight(x, r, lowest):
    """x rounded to three mantissa bits with the fraction r / 2^16; `lowest`: the binades under the block's
    top one after which the steps stay equal."""
    a = x.abs()
    top = a.amax(1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = e + (top >= 1.75 * torch.exp2(e))
    e = torch.where(top > 0, e, -100.0).clamp(-100, 120)
    binade = torch.floor(torch.log2(torch.where(a > 0, a, 2.0 ** -600)))
    step = torch.exp2(torch.maximum(binade, e - lowest) - 3)
    return torch.sign(x) * torch.floor(a / step + r.double() / 65536) * step


def exact_adamw(state, case):
    t, eight = state["step"] + 1, case["bits"] == 8
    g = state["grads"].double().view(-1, BLOCK) * state["scale"].double()
    m, v = state["m"].view(-1, BLOCK), state["v"].view(-1, BLOCK)
    if eight:   # a code's value from its fields
        c, e = m.int() & 0x7F, state["m_exp"].double()
        s = torch.where((c >> 3) > 0, 8 + (c & 7), c & 7).double()
        m = torch.where(m > 0x7F, -s, s) * torch.exp2((c >> 3).clamp(min=1).double() - 18 + e)
        c, e = v.int(), state["v_exp"].double()
        s = torch.where((c >> 3) > 0, 8 + (c & 7), c & 7).double()
        v = s * torch.exp2((c >> 3).clamp(min=1).double() - 34 + e)
    m = BETA1 * m.double() + (1 - BETA1) * g
    v = BETA2 * v.double() + (1 - BETA2) * g ** 2
    p = state["master"].double().view(-1, BLOCK)
    change = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS) + state["decay"].double() * p
    p = (p - LR * change).view(-1)
    del change, g
    if eight:
        r = exact_words(state["seed"], t, m.shape[0])
        m = exact_eight(m, r // 65536, 14)
        v = exact_eight(v, r % 65536, 30)
    return {"weights": p, "master": p, "m": m.view(-1), "v": v.view(-1)}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "route":
        return exact_route(state, case)
    if case["op"] == "route_backward":
        return exact_route_backward(state, case)
    if case["op"] == "grad_norm":
        norm = state["grads"].double().square().sum().sqrt()
        return torch.stack([norm, (1 / (norm + 1e-6)).clamp(max=1.0)])
    return exact_adamw(state, case)
