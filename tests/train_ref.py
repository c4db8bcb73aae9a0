"""Plain 64-bit forms of the training-step operators (numpy, from the definitions)."""
import numpy as np

BLOCK = 256


# ---- routing ---------------------------------------------------------------------

def route(x, k, mask=None, normalize=True):
    """x float64 [T, E].  Returns a dict; `p` are the gates of every expert (0 in rows that do not count)."""
    T, E = x.shape
    live = ~np.all(x == -np.inf, axis=1) if E else np.zeros(T, bool)
    if mask is not None:
        live &= mask.astype(bool)
    p = np.zeros((T, E))
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    with np.errstate(all="ignore"):
        z = x[live]
        e = np.exp(z - np.max(z, axis=1, keepdims=True, initial=-np.inf))   # NaN propagates
        p[live] = e / e.sum(1, keepdims=True)
    for t in np.nonzero(live)[0]:
        by = np.where(np.isnan(x[t]), -np.inf, x[t])
        order = [int(e) for e in np.argsort(-by, kind="stable")[:k] if by[e] > -np.inf]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        if normalize and order:
            w[t, :len(order)] /= w[t, :len(order)].sum()
    n = int(live.sum())
    counts = np.bincount(ids[ids >= 0], minlength=E)
    mean = p[live].sum(0) / n if n else np.zeros(E)
    loss = E / (k * n) * float((counts * mean).sum()) if n else 0.0
    return dict(p=p, ids=ids, weights=w, counts=counts, tokens=n, mean_prob=mean, loss=loss, live=live)


def route_backward(x, r, grad_weights, grad_loss, normalize=True):
    """Gradient of sum(grad_weights * weights) + grad_loss * loss, counts held constant; also
    `scale` [T], the largest |d| of a row that its rounding errors are relative to."""
    T, E = x.shape
    k, n, p = r["ids"].shape[1], r["tokens"], r["p"]
    grad, scale = np.zeros((T, E)), np.zeros(T)
    a = grad_loss * E * r["counts"] / (k * n * n) if n else np.zeros(E)
    for t in np.nonzero(r["live"])[0]:
        d = a.copy()
        ids = r["ids"][t][r["ids"][t] >= 0]
        u = grad_weights[t, :len(ids)].astype(np.float64)
        big = np.abs(u)
        if normalize and len(ids):
            w = r["weights"][t, :len(ids)]
            total = p[t, ids].sum()
            big = (np.abs(u) + np.sum(np.abs(u) * w)) / total
            u = (u - np.sum(u * w)) / total
        d[ids] += u
        grad[t] = p[t] * (d - np.sum(p[t] * d))
        scale[t] = np.max(np.abs(a)) + (big.max() if len(ids) else 0.0)
    return grad, scale


# ---- noise and codes ---------------------------------------------------------------

def mixed(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    x ^= x >> np.uint64(16)
    x = x * np.uint64(0x9E3779B1) & np.uint64(0xFFFFFFFF)
    x ^= x >> np.uint64(15)
    x = x * np.uint64(0x6A09E667) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def noise(seed, step, blocks):
    """16-bit noise (for m, for v), each [len(blocks), 256], of the blocks with these numbers."""
    M = np.uint64(0xFFFFFFFF)
    start = mixed(np.uint64(seed) ^ mixed(step & 0xFFFFFFFF))
    b = mixed((start + np.asarray(blocks, np.uint64) * np.uint64(0x9E3779B1)) & M)
    x = (b[:, None] + np.arange(BLOCK, dtype=np.uint64)[None, :] * np.uint64(0x9E3779B1)) & M
    x ^= x >> np.uint64(15)
    x = x * np.uint64(0x6A09E667) & M
    x ^= x >> np.uint64(16)
    return (x >> np.uint64(16)).astype(np.int64), (x & np.uint64(0xFFFF)).astype(np.int64)


def code_value(code, exp, signed):
    """Values of 8-bit codes [blocks, 256] with exponents [blocks]."""
    c = code.astype(np.int64)
    mag = c & 0x7F if signed else c
    f, frac = mag >> 3, mag & 7
    sig = np.where(f > 0, 8 + frac, frac).astype(np.float64)
    v = np.ldexp(sig, (np.maximum(f, 1) + exp.astype(np.int64)[:, None] - (18 if signed else 34)).astype(np.int64))
    if signed:
        v = np.where(c & 0x80, -v, v)
    return np.where(mag == (0x7F if signed else 0xFF), np.nan, v)


def shared_exponent(x):
    """s per block with every finite |x| < 1.75 * 2^s, clipped to [-100, 120]."""
    a = np.max(np.where(np.isfinite(x), np.abs(x), 0.0), axis=1)
    frac, e = np.frexp(a)                         # a = frac * 2^e, frac in [0.5, 1)
    s = np.where(frac * 2 >= 1.75, e, e - 1)
    return np.clip(np.where(a > 0, s, -127), -100, 120)


def to_codes(x, s, r, signed):
    """(codes, distance): the codes of x [blocks, 256] with exponents s and noise r, and how far the
    sum of the fraction cut off and the noise is from rounding the other way."""
    depth, top = (14, 0x7E) if signed else (30, 0xFE)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    _, e = np.frexp(a)
    lowest = s.astype(np.int64)[:, None] - depth
    binade = np.maximum(np.where(a > 0, e - 1, -10**6), lowest)
    q = np.ldexp(a, 3 - binade) + r / 65536.0      # in units of the last bit kept
    steps = np.floor(q).astype(np.int64)
    dist = np.minimum(q - steps, steps + 1 - q)
    mag = np.minimum(steps + 8 * (binade - lowest), top)    # steps >= 8 moves into the next binade
    nan = 0x7F if signed else 0xFF
    mag = np.where(np.isfinite(x), mag, nan)
    return mag, dist


# ---- AdamW -------------------------------------------------------------------------

def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay, scale=1.0):
    """One step on float64 arrays; t counts this step."""
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    with np.errstate(all="ignore"):
        change = m / (1 - beta1 ** t) / (np.sqrt(v / (1 - beta2 ** t)) + eps) + decay * p
    return p - lr * change, m, v, change
