"""Plain implementations, in numpy and 64 bits, of the steps around the routed experts.

Written from the formulas, expert by expert and slot by slot; they share no code with the library.
"""
import numpy as np
import torch

EPS = 2.0 ** -24                                  # half an ulp of float32, relative
HALF_ULP = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12, torch.float32: 2.0 ** -25}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def f64(t):
    return t.detach().cpu().double().numpy()


def rounding(dtype, v):
    """What one rounding of v to dtype may change (half a unit in the last place, subnormals included)."""
    return 2 * HALF_ULP[dtype] * np.abs(v) + LEAST[dtype]


def sort(ids, first, experts):
    """offs, row_of, slot_of: the slots of expert first, then of first + 1, ..., each in order."""
    flat = np.asarray(ids).reshape(-1)
    found = [np.flatnonzero(flat == first + e) for e in range(experts)]
    order = np.concatenate(found) if found else np.zeros(0, np.int64)
    row_of = np.full(flat.size, -1, np.int32)
    slot_of = np.full(flat.size, -1, np.int32)
    row_of[order] = np.arange(order.size)
    slot_of[:order.size] = order
    return np.cumsum([f.size for f in found]).astype(np.int32), row_of.reshape(np.shape(ids)), slot_of


def combine(rows, row_of, weights=None):
    """Per token the weighted sum of its rows, and the sum of the terms' magnitudes."""
    tokens, top_k = row_of.shape
    total = np.zeros((tokens, rows.shape[1]))
    scale = np.zeros_like(total)
    for t in range(tokens):
        for j in range(top_k):
            r = row_of[t, j]
            if 0 <= r < rows.shape[0]:
                w = 1.0 if weights is None else float(weights[t, j])
                total[t] += w * rows[r]
                scale[t] += np.abs(w * rows[r])
    return total, scale


def combine_grads(grad, rows, row_of, weights):
    """Gradients of the rows and of the weights, and the sums of the magnitudes of the latter's terms."""
    grad_rows = np.zeros_like(rows)
    grad_weights = np.zeros(row_of.shape)
    scale = np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j in range(row_of.shape[1]):
            r = row_of[t, j]
            if 0 <= r < rows.shape[0]:
                grad_rows[r] = float(weights[t, j]) * grad[t]
                grad_weights[t, j] = np.dot(grad[t], rows[r])
                scale[t, j] = np.abs(grad[t] * rows[r]).sum()
    return grad_rows, grad_weights, scale


def quantize(x):
    """scale and q of rows of storage values, in float32: each row brought to a maximum near 1 by a power of two
    (exact), then one rounding of 127 x, one of the quotient, and one to an integer, ties to even."""
    amax = np.abs(x).max(1, keepdims=True)
    live = amax > 0
    e = np.frexp(np.where(live, amax, 1.0))[1]
    unit, most = np.ldexp(x, -e).astype(np.float32), np.ldexp(np.where(live, amax, 1.0), -e).astype(np.float32)
    q = np.rint(np.float32(127) * unit / most).astype(np.int8)
    return q, (amax[:, 0].astype(np.float32) / np.float32(127)).astype(np.float32)


def tie_rows(dtype):
    """Rows whose elements lie exactly between two integers: odd multiples of max / 254, where the reciprocal of the
    maximum is exact (254) and where it is not (254 * 3, 5 and 7, which bfloat16 does not hold)."""
    odd = 2 * np.arange(-127, 127) + 1
    return [np.concatenate([[254.0 * m], odd * m, [-254.0 * m]])
            for m in ((1,) if dtype == torch.bfloat16 else (1, 3, 5, 7))]


def bounds(offs, rows):
    """[start, end) of each expert's rows."""
    start = 0
    for end in offs:
        end = min(max(int(end), start), rows)
        yield start, end
        start = end


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def gate_up(a, a_scale, token_of, wg, sg, wu, su, offs, probs, limit):
    """y [rows, inter] and what float32 steps may change; token_of [rows], -1: a row of zeros."""
    rows, inter = len(token_of), wg.shape[1]
    y, slack = np.zeros((rows, inter)), np.zeros((rows, inter))
    for e, (r0, r1) in enumerate(bounds(offs, rows)):
        if r0 == r1:
            continue
        tok = np.asarray(token_of[r0:r1])
        x = np.where(tok[:, None] >= 0, a[tok].astype(np.float64), 0.0)
        sa = a_scale.astype(np.float64)[tok][:, None]
        g = (x @ wg[e].astype(np.float64).T) * sa * sg[e].astype(np.float64)
        u = (x @ wu[e].astype(np.float64).T) * sa * su[e].astype(np.float64)
        gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit)
        p = probs[r0:r1].astype(np.float64)[:, None]
        y[r0:r1] = silu(gc) * uc * p
        # gate and up each come from 3 roundings; silu passes a relative error on at most 1 + |gate|
        # times, and its own exponential and reciprocal add |gate| + 8; two products follow
        slack[r0:r1] = (4 * np.abs(gc) + 24) * EPS * np.abs(y[r0:r1]) + 1e-37
    return y, slack


def down(h, h_scale, w, s, offs, probs):
    """out [rows, hidden] and what the five roundings before the last may change."""
    rows = h.shape[0]
    out = np.zeros((rows, w.shape[1]))
    for e, (r0, r1) in enumerate(bounds(offs, rows)):
        out[r0:r1] = (h[r0:r1].astype(np.float64) @ w[e].astype(np.float64).T) * s[e].astype(np.float64)
        out[r0:r1] *= (h_scale[r0:r1].astype(np.float64) * probs[r0:r1].astype(np.float64))[:, None]
    return out, 5 * EPS * np.abs(out) + 1e-37
