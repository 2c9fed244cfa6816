"""The paged cache in numpy, from its definition: what written rows stand for, where their codes lie, and attention over them in
64 bits."""
import numpy as np

GROUP = 64


def bf16(x):
    """bf16 tensor -> float64 array."""
    return x.double().cpu().numpy()


def up(x):
    """The smallest bf16 not below x (fp32, >= 0)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return (((b + np.uint32(0xFFFF)) >> np.uint32(16)) << np.uint32(16)).view(np.float32)


def quantise(x, bits):
    """Rows [..., D] (float64 holding bf16 values) -> (codes int [..., D], scales [..., groups], lows [..., groups])."""
    n = x.shape[-1] if bits == 8 else GROUP
    g = x.reshape(*x.shape[:-1], x.shape[-1] // n, n)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        f = g.astype(np.float32)
        if bits == 8:
            low = np.zeros(g.shape[:-1], np.float32)
            span = np.abs(f).max(-1)
        else:
            low = f.min(-1)
            span = f.max(-1) - low
        fine = np.isfinite(g).all(-1) & np.isfinite(span)
        s = np.where(fine, up(np.where(fine, span, np.float32(0)) * (np.float32(1) / np.float32(127 if bits == 8 else 15))), np.float32("nan"))
        q = np.rint((f - low[..., None]) / np.where(s > 0, s, 1)[..., None])  # fp32 throughout
    q = np.where(fine[..., None] & (s > 0)[..., None], q, 0)
    return q.reshape(x.shape).astype(np.int64), s.astype(np.float64), np.where(fine, low, 0).astype(np.float64)


def stands_for(x, bits):
    """What rows [..., D] read back as, before the rounding to bf16."""
    if bits == 16:
        return x
    q, s, low = quantise(x, bits)
    n = x.shape[-1] if bits == 8 else GROUP
    return q * np.repeat(s, n, -1) + np.repeat(low, n, -1)


def k_units(q, bits):
    """Codes of one K row [D] -> its bytes."""
    if bits == 8:
        return (q + 128).astype(np.uint8)
    out = np.zeros(len(q) // 2, np.uint8)
    groups = len(q) // GROUP
    for e, u in enumerate(q):
        g, r = e // GROUP, e % GROUP
        part, word, i = r // 16, r % 16 // 8, r % 8
        nibble = i // 2 + 4 * (i % 2)
        out[part * 8 * groups + 8 * g + 4 * word + nibble // 2] |= u << (4 * (nibble % 2))
    return out


def v_pieces(q, bits):
    """Codes of one V row [D] -> [16, bytes of a piece]."""
    if bits == 8:
        return (q + 128).astype(np.uint8).reshape(16, -1)
    out = np.zeros((16, len(q) // 32), np.uint8)
    for e, u in enumerate(q):
        g, r = e // GROUP, e % GROUP
        out[r // 4, 2 * g + r % 4 // 2] |= u << (4 * (r % 2))
    return out


def v_block(dim, bits):
    return min(4, 16 // (dim * bits // 128))


def attend(q, keys, values, takes, scale):
    """One head: q [rows, D], keys, values [n, D], takes bool [rows, n] -> (O, sum p |v|, the probabilities) in 64 bits."""
    out, mag = np.zeros((len(q), values.shape[1])), np.zeros((len(q), values.shape[1]))
    probs = np.zeros(takes.shape)
    for r in range(len(q)):
        at = np.flatnonzero(takes[r])
        if len(at) == 0:
            continue
        s = keys[at] @ q[r] * scale
        p = np.exp(s - s.max())
        p /= p.sum()
        out[r], mag[r], probs[r, at] = p @ values[at], p @ np.abs(values[at]), p
    return out, mag, probs


def taken(n, new, q_len, tree=None):
    """bool [q_len, n]: which of a request's n keys (the last `new` being its new tokens) each new token takes."""
    t = np.zeros((q_len, n), bool)
    base = n - new
    for i in range(min(new, q_len)):
        t[i, :max(base, 0)] = True
        for j in range(new):
            if base + j >= 0 and (j <= i if tree is None else (int(tree[i]) >> j) & 1):
                t[i, base + j] = True
    return t
