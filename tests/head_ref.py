"""Plain 64-bit forms of the output head's losses (torch, from the definitions), and bounds on the errors of
the 32-bit sums and the 16-bit roundings that the kernels are documented to make."""
import torch

INF = float("inf")


def targets(x):
    """(live [T], columns [T, k], shares [T, k], entropies [T]) of the inputs `x`."""
    V, dev = x["weight"].shape[0], x["hidden"].device
    if "labels" in x:
        y = x["labels"].long()
        live = (y >= 0) & (y < V)
        return (live, torch.where(live, y, 0)[:, None], live.double()[:, None],
                torch.zeros(len(y), dtype=torch.float64, device=dev))
    ids, t = x["ids"].long(), x["teacher"].double() / x.get("temperature", 1.0)
    there = (ids >= 0) & (ids < V) & (t != -INF)
    if x.get("mask") is not None:
        there = there & x["mask"].bool()[:, None]
    q = torch.zeros_like(t)
    entropy = torch.zeros(len(t), dtype=torch.float64, device=dev)
    live = there.any(1) if ids.shape[0] else torch.zeros(0, dtype=torch.bool, device=dev)
    t = torch.where(there, t, -INF)[live]
    log_q = t - torch.logsumexp(t, 1, keepdim=True) if len(t) else t
    q[live] = torch.exp(log_q)
    entropy[live] = torch.where(there[live], torch.exp(log_q) * log_q, 0.0).sum(1)
    return live, torch.where(there, ids, 0), q, entropy


def loss(x, grad_loss=None, grad_losses=None):
    """The results and, where a gradient is given, both gradients; each with a bound on its error.

    z: a step of the tensor cores adds 16 products to a sum in 32 bits and cuts it off, so the sum of D products
    is off by at most (D / 16 + 16) 2^-23 of the sum of their sizes.  Exponentials, their sums and logarithms
    are within 2^-19 of 1, the last operations within 2^-22 of their terms.  dz is rounded once, to half
    a step of the type; in the products' sums it counts with the other factor's size."""
    h = float(x.get("temperature", 1.0))
    kind = x["hidden"].dtype
    u, steps = torch.finfo(kind).eps / 2, lambda n: (n / 16 + 16) * 2.0 ** -23
    V, D = x["weight"].shape
    T = x["hidden"].shape[0]
    live, at, q, entropy = targets(x)
    hid = torch.where(live[:, None], x["hidden"].double(), 0.0)
    w = x["weight"].double()
    z = hid @ w.T / h
    dz_z = steps(D) * (hid.abs() @ w.abs().T).amax(1) / h if T else torch.zeros(0, device=w.device)
    dz_z = dz_z + 2.0 ** -22 * z.abs().amax(1) if T else dz_z
    lse = torch.logsumexp(z, 1)
    picked = (q * z.gather(1, at)).sum(1)
    losses = torch.where(live, h * h * (entropy + lse - picked), 0.0)
    n = int(live.sum())
    out = dict(lse=torch.where(live, lse, 0.0), losses=losses, tokens=n,
               loss=losses.sum() / n if n else torch.zeros((), dtype=torch.float64, device=w.device))
    off = torch.where(live, 2 * dz_z + 2.0 ** -19 + 2.0 ** -22 * (lse.abs() + picked.abs() + 1), 0.0)
    if "teacher" in x:   # the teacher's shares: exponentials of rounded quotients
        big = torch.where(live, (x["teacher"].double().nan_to_num(0, 0, 0).abs().amax(1) / h), 0.0)
        share = 2.0 ** -21 * (big + 2)
        off = torch.where(live, off + share * (z.gather(1, at).abs().amax(1) + lse.abs() + entropy.abs() + 1), 0.0)
    else:
        share = torch.zeros(T, dtype=torch.float64, device=w.device)
    out["lse_off"], out["losses_off"] = off, h * h * off + 2.0 ** -22 * losses.abs()
    out["loss_off"] = out["losses_off"].sum() / max(n, 1) + 2.0 ** -22 * losses.abs().sum() / max(n, 1)
    if grad_loss is None and grad_losses is None:
        return out
    g = torch.zeros(T, dtype=torch.float64, device=w.device)
    if n and grad_loss is not None:
        g = g + grad_loss.double() / n
    if grad_losses is not None:
        g = g + grad_losses.double()
    g = torch.where(live, g * h, 0.0)
    p = torch.where(live[:, None], torch.exp(z - lse[:, None]), 0.0)
    shares = torch.zeros_like(p).scatter_add_(1, at, q)
    dz = g[:, None] * (p - shares)
    # of p, of q, of g, of the rounding, and below the smallest number of the type after scaling
    dz_off = g.abs()[:, None] * (p * (2 * dz_z + 2.0 ** -18 * (1 + lse.abs()))[:, None] + shares * (share + 2.0 ** -20)[:, None])
    dz_off = dz_off + (u + 2.0 ** -21) * (dz.abs() + dz_off)
    if kind == torch.float16 and T:
        dz_off = dz_off + torch.where(live, g.abs().amax(), 0.0)[:, None] * 2.0 ** -39
    out["dh"], out["dw"] = dz @ w, dz.T @ hid
    tiny = 2.0 ** -25 if kind == torch.float16 else 2.0 ** -134
    for name, got, sizes, offs in (("dh", out["dh"], dz.abs() @ w.abs(), dz_off @ w.abs()),
                                   ("dw", out["dw"], dz.abs().T @ hid.abs(), dz_off.T @ hid.abs())):
        length = V if name == "dh" else T
        bound = offs + (steps(length) + 2.0 ** -21) * (sizes + offs)
        out[name + "_off"] = (bound + u * (got.abs() + bound)) + tiny
    return out
