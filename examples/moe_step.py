"""Training steps of a mixture-of-experts block, and what they tell the placement solver.

A small block (a router and two-layer experts) learns a random target with the package's
training-step operators: gates and balance loss (`train.gate`), the gradients' clip scale and the
AdamW step (`train.AdamW`).  Two numbers of the run then replace assumptions of a placement
problem: the expert counts give the all-to-all volume (the load of the fullest expert), and the
optimizer's states give the bytes per weight.  The block is far smaller than the workload's, 16 experts
of width 64 against 64 of width 4096: the run shows where the numbers go, not that model's own load.

    python examples/moe_step.py [steps]
"""
import dataclasses
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from memory_aware_device_gb300 import nest, synth, train  # noqa: E402

TOKENS, HIDDEN, EXPERTS, TOP_K = 2048, 64, 16, 2


class Block:
    """Router and experts; weights in bfloat16, gradients in buffers that stay where they are."""

    def __init__(self, state_bits: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, scale):
            w = (torch.randn(*shape, generator=gen, device="cuda") * scale).bfloat16()
            w.requires_grad_().grad = torch.zeros_like(w)
            return w
        # a router that starts out liking some experts more
        self.router = weight(HIDDEN, EXPERTS, scale=HIDDEN ** -0.5)
        self.lean = weight(EXPERTS, scale=1.0)
        self.up = weight(EXPERTS, HIDDEN, 4 * HIDDEN, scale=HIDDEN ** -0.5)
        self.down = weight(EXPERTS, 4 * HIDDEN, HIDDEN, scale=(4 * HIDDEN) ** -0.5)
        weights = [self.router, self.lean, self.up, self.down]
        self.opt = train.AdamW([w.detach() for w in weights], [w.grad for w in weights], state_bits=state_bits,
                               betas=(0.9, 0.95), weight_decay=[0.1, 0.0, 0.1, 0.1], seed=seed)

    def forward(self, x):
        logits = x @ self.router + self.lean
        r = train.gate(logits, TOP_K)
        y = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        gates = torch.zeros(x.shape[0], EXPERTS, device=x.device).scatter(1, r.ids.long(), r.weights)
        for e in range(EXPERTS):    # every expert on every token: small enough here
            h = torch.nn.functional.gelu(x @ self.up[e]) @ self.down[e]
            y = y + gates[:, e, None] * h.float()
        return y, r

    def step(self, x, target, lr: float, balance: float):
        """One training step; returns (loss of the task, balance loss, Routing)."""
        for g in self.opt.grads:
            g.zero_()
        y, r = self.forward(x)
        task = torch.mean((y - target) ** 2)
        (task + balance * r.loss).backward()
        self.opt.step(lr, grad_scale=self.opt.grad_norm(max_norm=1.0)[1])
        return task.detach(), r.loss.detach(), r


def learn(state_bits: int, steps: int, seed: int = 0):
    """Trains a block; returns (block, [(task, balance, capacity factor in thousandths)] per step)."""
    block = Block(state_bits, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(TOKENS, HIDDEN, generator=gen, device="cuda").bfloat16()
    target = torch.randn(TOKENS, HIDDEN, generator=gen, device="cuda") * 0.5
    seen = []
    for _ in range(steps):
        task, balance, r = block.step(x, target, lr=3e-3, balance=0.05)
        seen.append((task, balance, r.counts, r.tokens))
    return block, [(float(t), float(b), train.capacity_milli(c.tolist(), int(n[0]), TOP_K)) for t, b, c, n in seen]


def plan(capacity: int, opt, instance: int = 0):
    """The mixture-of-experts workload's problem with this capacity factor and these optimizer states."""
    x = synth.config_instance(4, instance)
    even = np.where(x.moe == 1, synth.SEQ * 2 * 4096 * 2, 0)     # 2 experts per token, hidden size 4096, bf16
    budget = x.budget
    if opt.state_bits == 8:      # the codes' scales, for every weight of the model at most
        budget -= int(x.pd.sum() + x.pe.sum()) // 256
    x = dataclasses.replace(x, a2a=(even * capacity // 1000).astype(np.int64), opt_factor=opt.opt_factor, budget=budget)
    return x, nest.solve_instances([x])[0]


def main(steps: int = 200):
    for bits in (32, 8):
        block, seen = learn(bits, steps)
        print(f"states in {bits} bits, {block.opt.steps} steps: task loss {seen[0][0]:.4f} -> {seen[-1][0]:.4f}, "
              f"balance loss {seen[0][1]:.3f} -> {seen[-1][1]:.3f}, "
              f"capacity factor {seen[0][2] / 1000:.2f} -> {seen[-1][2] / 1000:.2f}")
        for what, capacity in (("as it started", seen[0][2]), ("as trained", seen[-1][2])):
            _, r = plan(capacity, block.opt)
            print(f"  plan with the experts' load {what}, optimizer {block.opt.opt_factor} bytes per weight byte: "
                  f"{r['t_batch'] / 1e9:.3f} s an iteration, {len(r['plan'])} stages")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
