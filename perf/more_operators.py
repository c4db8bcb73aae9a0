"""The losses at a model's output head, as cases to be timed and compared.

The last stage of a placed model multiplies its hidden states with the output weights and compares the
logits with what the next token was, or with a teacher's largest logits.  Two operators and their gradients,
neither of which keeps the logits:

  cross_entropy   loss of the labels under the softmax over the vocabulary
  distill         divergence of a teacher's softmax over its largest logits from the model's

A case of kind "eval" is the loss alone (per token and its mean), one of kind "step" the loss and the
gradients of the hidden states and of the weights.

`own` false computes them in plain torch operations, true through memory_aware_device_gb300.head.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
LOGIT_STD = 2.0
# tokens * vocabulary * hidden size of the largest listed case, which a drawn one stays below
LARGEST = 4096 * 128000 * 4096


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------

def listed():
    def labels(name, kind, tokens, vocab, hidden, dtype, padded=0.0, wider=0):
        return {"name": name, "op": "cross_entropy", "kind": kind, "tokens": tokens, "vocab": vocab, "hidden": hidden,
                "dtype": dtype, "padded": padded, "wider": wider}

    def teacher(name, kind, tokens, vocab, hidden, dtype, k, temperature, logits="fp32", padded=0.0, wider=0):
        return {"name": name, "op": "distill", "kind": kind, "tokens": tokens, "vocab": vocab, "hidden": hidden,
                "dtype": dtype, "k": k, "temperature": temperature, "logits": logits, "padded": padded, "wider": wider}

    return [
        # scoring the one token of a decoding step at the hidden size of the solver's 32-layer workload
        labels("cross_entropy eval 1 token", "eval", 1, 32000, 4096, "bf16"),
        # perplexity of ragged documents under a small model with an odd vocabulary
        labels("cross_entropy eval ragged", "eval", 1777, 50021, 1000, "fp16", 0.3, 24),
        # a training step of a toy model: the calls' own time
        labels("cross_entropy step small", "step", 129, 1000, 256, "bf16"),
        # the solver's microbatch of 2048 tokens at hidden size 4096
        labels("cross_entropy step microbatch", "step", 2048, 32000, 4096, "bf16"),
        # instruction tuning: prompts and padding carry no label; rows off 16-byte alignment
        labels("cross_entropy step ragged", "step", 4099, 50021, 1003, "fp16", 0.4, 6),
        # two microbatches under a large vocabulary
        labels("cross_entropy step large", "step", 4096, 128000, 4096, "bf16"),
        # how far a small student is from its teacher on a few tokens
        teacher("distill eval few tokens", "eval", 16, 32000, 1024, "bf16", 8, 1.0),
        # the same on a microbatch, for early stopping
        teacher("distill eval microbatch", "eval", 2048, 32000, 4096, "bf16", 64, 2.0),
        # a student's training step on the microbatch
        teacher("distill step microbatch", "step", 2048, 32000, 4096, "bf16", 64, 2.0),
        # odd sizes, teacher logits stored in 16 bits, prompts without a target, lists that are not full
        teacher("distill step ragged", "step", 1031, 50021, 1003, "fp16", 37, 1.5, "bf16", 0.25, 6),
        # two microbatches under a large vocabulary, long lists
        teacher("distill step large", "step", 4096, 128000, 4096, "bf16", 128, 1.0, "bf16"),
    ]


def log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["cross_entropy", "distill"])
    hidden = log_between(rng, 64, 8192)
    if rng.random() < 0.6:
        hidden = -(-hidden // 64) * 64
    vocab = log_between(rng, 1000, 128000)
    if rng.random() < 0.5:
        vocab = -(-vocab // 64) * 64
    tokens = max(1, min(log_between(rng, 1, 16384), LARGEST // (vocab * hidden)))
    case = {"op": op, "kind": rng.choice(["eval", "step", "step"]), "tokens": tokens, "vocab": vocab, "hidden": hidden,
            "dtype": rng.choice(["bf16", "bf16", "fp16"]), "padded": rng.choice([0.0, 0.0, 0.2, 0.5]),
            "wider": rng.choice([0, 0, rng.randint(1, 40)])}
    if op == "distill":
        case |= {"k": log_between(rng, 1, 128), "temperature": rng.choice([1.0, 1.0, 2.0, 4.0, 0.7]),
                 "logits": rng.choice(["fp32", "bf16", "fp16"])}
    return case


def work(case):
    """Rows that carry no target need no work; a step has three products, an eval one."""
    t, v, d = case["tokens"], case["vocab"], case["hidden"]
    n = max(1, round(t * (1 - case["padded"])))
    step = case["kind"] == "step"
    moved = (n * d + v * d) * 2 + 8 * t
    if case["op"] == "distill":
        moved = (n * d + v * d) * 2 + n * case["k"] * (8 + (4 if case["logits"] == "fp32" else 2)) + 4 * t
    if step:
        moved += (t * d + v * d) * 2
    return {"bytes": moved, "flops": (6 if step else 2) * n * v * d}


# ---------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------

def prepare(case, seed):
    dev = device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    t, v, d, kind = case["tokens"], case["vocab"], case["hidden"], TYPES[case["dtype"]]
    weight = (torch.randn(v, d, generator=gen, device=dev) * (LOGIT_STD * d ** -0.5)).to(kind)
    labels = torch.randint(0, v, (t,), generator=gen, device=dev)
    # the model has learnt something: a label's logit is up to 12 above the others' mean
    lean = torch.rand(t, 1, generator=gen, device=dev) * (12 / LOGIT_STD ** 2)
    wide = torch.zeros(t, d + case["wider"], dtype=kind, device=dev)
    hidden = wide[:, :d]
    hidden.copy_(torch.randn(t, d, generator=gen, device=dev) + lean * weight[labels].float())
    live = torch.rand(t, generator=gen, device=dev) >= case["padded"]
    state = {"case": case, "hidden": hidden, "weight": weight,
             # the loss's own gradient (a loss scale or an accumulation's share), and one for each token
             "grad_loss": torch.rand((), generator=gen, device=dev) + 0.5}
    if case["op"] == "cross_entropy":
        state["labels"] = torch.where(live, labels, -100)
    else:
        # a teacher that agrees with the model in part
        other = hidden.float() * 0.7 + torch.randn(t, d, generator=gen, device=dev) * 0.7
        logits, ids = torch.topk(other.to(kind) @ weight.T, case["k"], dim=1)
        logits = logits.float() + torch.randn(t, case["k"], generator=gen, device=dev) * 0.1
        state |= {"ids": ids, "teacher": logits.to(TYPES[case["logits"]]), "mask": live if case["padded"] else None,
                  "temperature": case["temperature"]}
        if case["padded"]:   # lists are cut where the teacher's own mass was reached
            full = torch.randint(1, case["k"] + 1, (t, 1), generator=gen, device=dev)
            state["ids"] = torch.where(torch.arange(case["k"], device=dev)[None, :] < full, ids, -1)
    if case["padded"]:
        hidden[~live] = math.nan   # what rows without a target hold is anything
    return state


# ---------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------

def targets(state, vocab):
    """(rows that count, targets' columns, their probabilities, sum of q log q) of either operator."""
    if state["case"]["op"] == "cross_entropy":
        labels = state["labels"][:, None]
        live = ((labels >= 0) & (labels < vocab))[:, 0]
        return live, torch.where(live[:, None], labels, 0), live[:, None].float(), torch.zeros_like(labels[:, 0]).float()
    ids, x = state["ids"], state["teacher"].float() / state["temperature"]
    there = (ids >= 0) & (ids < vocab) & (x != -math.inf)
    if state["mask"] is not None:
        there = there & state["mask"][:, None]
    live = there.any(1)
    x = torch.where(there, x, -math.inf)
    top = torch.where(live, x.amax(1), 0.0)[:, None]
    e = torch.where(there, torch.exp(x - top), 0.0)
    total = torch.where(live[:, None], e.sum(1, keepdim=True), 1.0)
    q = e / total
    entropy = torch.where(there, q * (x - top - torch.log(total)), 0.0).sum(1)
    return live, torch.where(there, ids, 0), q, entropy


def run_plain(state):
    case, weight = state["case"], state["weight"].float()
    heat = state.get("temperature", 1.0)
    live, at, q, entropy = targets(state, weight.shape[0])
    hidden = torch.where(live[:, None], state["hidden"].float(), 0.0)
    z = hidden @ weight.T
    z = z / heat if heat != 1.0 else z
    top = z.amax(1, keepdim=True)
    picked = (q * torch.gather(z, 1, at)).sum(1)
    p = torch.exp(z - top)
    del z
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    losses = torch.where(live, heat * heat * (entropy + lse - picked), 0.0)
    n = live.sum()
    loss = losses.sum() / n.clamp(min=1)
    out = {"loss": loss, "losses": losses, "tokens": n.int().reshape(1)}
    if case["kind"] == "eval":
        return out
    # p - q, times the gradient of each row's loss
    p /= total
    p.scatter_add_(1, at, -q)
    p *= torch.where(live, heat * state["grad_loss"] / n.clamp(min=1), 0.0)[:, None]
    grad_hidden = (p @ weight).to(state["hidden"].dtype)
    del weight
    return out | {"grad_hidden": grad_hidden, "grad_weight": (p.T @ hidden).to(state["weight"].dtype)}


def run_own(state):
    from memory_aware_device_gb300 import head
    step = state["case"]["kind"] == "step"
    hidden, weight = state["hidden"], state["weight"]
    if state["case"]["op"] == "cross_entropy":
        r = head.cross_entropy(hidden, weight, state["labels"])
        if step:
            grads = head.cross_entropy_backward(hidden, weight, state["labels"], r, grad_loss=state["grad_loss"])
    else:
        how = {"temperature": state["temperature"], "mask": state["mask"]}
        r = head.distill(hidden, weight, state["ids"], state["teacher"], **how)
        if step:
            grads = head.distill_backward(hidden, weight, state["ids"], state["teacher"], r,
                                          grad_loss=state["grad_loss"], **how)
    out = {"loss": r.loss, "losses": r.losses, "tokens": r.tokens}
    return out | {"grad_hidden": grads[0], "grad_weight": grads[1]} if step else out


def run(state):
    return run_own(state) if own else run_plain(state)


# ---------------------------------------------------------------------------------
# The same in 64 bits, from the definitions
# ---------------------------------------------------------------------------------

def exact(case, seed):
    t, v, d = case["tokens"], case["vocab"], case["hidden"]
    if (6 if case["kind"] == "step" else 2) * t * v * d > 1.4e13:
        return None
    state = prepare(case, seed)
    heat = float(case.get("temperature", 1.0))
    if case["op"] == "cross_entropy":
        rows = torch.nonzero(state["labels"] >= 0)[:, 0]
        columns, share = state["labels"][rows][:, None], torch.ones(len(rows), 1, dtype=torch.float64, device=device())
    else:
        rows = torch.arange(t, device=device()) if state["mask"] is None else torch.nonzero(state["mask"])[:, 0]
        columns = state["ids"][rows]
        share = torch.softmax(torch.where(columns < 0, -math.inf, state["teacher"][rows].double() / heat), 1)
    n = len(rows)
    h, w = state["hidden"][rows].double(), state["weight"].double()
    log_p = torch.log_softmax(h @ w.T / heat, 1)
    cross = torch.where(share > 0, share * (torch.log(share) - torch.gather(log_p, 1, columns.clamp(min=0))), 0.0)
    each = heat ** 2 * cross.sum(1)
    losses = torch.zeros(t, dtype=torch.float64, device=h.device)
    losses[rows] = each
    out = {"loss": each.mean() if n else losses.sum(), "losses": losses, "tokens": torch.tensor([n], dtype=torch.int32)}
    if case["kind"] == "eval":
        return out
    grad = torch.exp(log_p)
    del log_p
    grad.scatter_add_(1, columns.clamp(min=0), -share)
    grad *= heat * float(state["grad_loss"]) / max(1, n)
    grad_hidden = torch.zeros(t, d, dtype=torch.float64, device=h.device)
    grad_hidden[rows] = grad @ w
    return out | {"grad_hidden": grad_hidden, "grad_weight": grad.T @ h}
