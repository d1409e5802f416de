"""Plain definitions, in 64 bits, of the operators between two expert layers: short convolution, head norms with rotation
or gate, gated delta rule.  numpy only, a token at a time; no code of the library."""
import numpy as np


def sequences(T, offsets=None, slot=None, carry=None, slots=None):
    """(first row, end, slot, carries on) of each sequence that takes part."""
    n = T if offsets is None else len(offsets) - 1
    for s in range(n):
        lo, hi = (s, s + 1) if offsets is None else (int(offsets[s]), int(offsets[s + 1]))
        at = s if slot is None else int(slot[s])
        if hi > lo and at >= 0 and (slots is None or at < slots):
            yield lo, hi, at, True if carry is None else bool(carry[s])


def silu(x):
    return x / (1 + np.exp(-x))


def conv(x, w, bias, act, y, state, seqs):
    """y and state (or None) are replaced in place; also returns the sum of magnitudes of each output's terms."""
    W = w.shape[1]
    size = np.zeros_like(y)
    for lo, hi, at, carry in seqs:
        before = np.zeros((W - 1, x.shape[1])) if state is None or not carry else state[at]
        rows = np.concatenate([before, x[lo:hi]])
        for t in range(lo, hi):
            part = rows[t - lo:t - lo + W] * w.T
            total = part.sum(0) + (0 if bias is None else bias)
            size[t] = np.abs(part).sum(0) + (0 if bias is None else np.abs(bias))
            y[t] = silu(total) if act else total
        if state is not None:
            state[at] = rows[len(rows) - (W - 1):]
    return size


def head_norm(x, norm, eps, weight, offset, pos, inv_freq, rot, halves, gate):
    """x [T, H, D]; also returns the magnitudes that a value's rounding goes by."""
    D = x.shape[2]
    total = (x * x).sum(2, keepdims=True)
    with np.errstate(all="ignore"):
        z = x.copy() if norm == "none" else x / np.sqrt((total / D if norm == "rms" else total) + eps)
    if weight is not None:
        z = z * (offset + weight)
    size = np.abs(z)
    if rot:
        h = rot // 2
        i = np.arange(h)
        a, b = (i, i + h) if halves else (2 * i, 2 * i + 1)
        angle = pos.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        p, q = z[:, :, a], z[:, :, b]
        z = z.copy()
        z[:, :, a], z[:, :, b] = p * c - q * s, q * c + p * s
        size[:, :, a] = size[:, :, b] = np.abs(p) + np.abs(q)
    if gate is not None:
        z, size = z * silu(gate), size * np.abs(silu(gate))
    return z, size


def delta(q, k, v, g, beta, state, o, scale, seqs):
    """o and state (or None) are replaced in place; also returns, for each token and v head, the largest magnitude that
    the state has had."""
    Hk, Hv = q.shape[1], v.shape[1]
    largest = np.zeros((q.shape[0], Hv))
    for lo, hi, at, carry in seqs:
        S = np.zeros((Hv, v.shape[2], q.shape[2])) if state is None or not carry else state[at].copy()
        top = np.abs(S).max((1, 2))
        for t in range(lo, hi):
            kt, qt = (r[t].repeat(Hv // Hk, 0) for r in (k, q))
            S = np.where(np.isneginf(g[t])[:, None, None], 0, S) * np.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - np.einsum("hde,he->hd", S, kt))
            S = S + u[:, :, None] * kt[:, None, :]
            o[t] = scale * np.einsum("hde,he->hd", S, qt)
            top = np.maximum(top, np.abs(S).max((1, 2)))
            largest[t] = top
        if state is not None:
            state[at] = S
    return largest
