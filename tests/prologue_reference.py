"""Plain implementations, in numpy and 64 bits, of the steps before the routed experts.

Written from the formulas, token by token where an order is chosen; they share no code with the library.
Each comes with what float32 steps may change (EPS is half an ulp of float32, relative).
"""
import numpy as np
import torch

from tests.routed_reference import EPS, f64, rounding  # noqa: F401


def to(dtype, v):
    """v rounded to a storage type."""
    return torch.from_numpy(np.ascontiguousarray(v)).to(dtype).double().numpy()


def chain(n):
    """Additions that one term of a sum of n may go through: n is shared by at least 16 lanes, whose sums are
    joined in at most 16 more steps."""
    return n / 16 + 16


# ---- norm -----------------------------------------------------------------------------

def norm(h, weight, eps):
    """y, n of rows h, and what float32 steps may change of each, relative: the sum of squares has positive terms,
    so its relative error is at most one rounding per addition (and one of the square), which the root halves; the
    mean, eps, root and reciprocal are four more; y is two products."""
    with np.errstate(all="ignore"):
        n = 1 / np.sqrt((h * h).mean(1) + eps)
        y = h * n[:, None] * weight
    slack_n = (chain(h.shape[1]) / 2 + 4) * EPS
    return y, n, slack_n + 2 * EPS, slack_n


def norm_grads(grad, h, weight, n, grad_h):
    """grad_x, grad_weight and what float32 steps may change of each. a = h n and g = grad weight have one rounding
    each; the mean's terms three, its sum chain() and the division one; grad_x is one fused step, one product and one
    sum after that. grad_weight's terms have two roundings and its sum one for each row and of each partial sum."""
    cols = h.shape[1]
    a, g = h * n[:, None], grad * weight
    mean, size = (g * a).mean(1, keepdims=True), np.abs(g * a).mean(1, keepdims=True)
    dx = n[:, None] * (g - a * mean)
    slack = EPS * n[:, None] * (4 * np.abs(g) + 5 * np.abs(a * mean) + (chain(cols) + 5) * np.abs(a) * size)
    if grad_h is not None:
        dx = dx + grad_h
    slack = slack + EPS * np.abs(dx) + 1e-42
    dw, dw_size = (grad * a).sum(0), np.abs(grad * a).sum(0)
    return dx, slack, dw, (h.shape[0] + 4) * EPS * dw_size + 1e-42


# ---- the router's product ---------------------------------------------------------------

def product(a, b, pieces=3):
    """a @ b and what its float32 sum may change, whatever the order: a rounding of each addition, doubled for an
    accumulator that truncates, and of each product what is left when float32 factors are cut into 8-bit pieces:
    2^-24 of it for each of the four smallest pairs of three, 2^-17 if only two are kept."""
    size = np.abs(a) @ np.abs(b)
    return a @ b, (2 * (a.shape[1] + 4) * EPS + (8 * EPS if pieces == 3 else 2.0 ** -16)) * size + 1e-37


# ---- choice of the experts ----------------------------------------------------------------

def scores(logits, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-logits))
        e = np.exp(logits - logits.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)


def route(logits, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_score="max"):
    """ids: the experts in the order of the choice, token by token; -1 where none remains."""
    tokens, experts = logits.shape
    size = experts // groups
    s = scores(logits, score)
    ids = np.full((tokens, top_k), -1, np.int32)
    for t in range(tokens):
        c = logits[t].copy() if bias is None else s[t] + bias
        ok = (c > -np.inf) & (logits[t] > -np.inf)         # False for NaN
        c[~ok] = -np.inf
        of = c if bias is not None or group_score == "max" else np.where(ok, s[t], -np.inf)
        value = []
        for g in range(groups):
            best = sorted(of[g * size:(g + 1) * size], reverse=True)
            value.append(best[0] + best[1] if group_score == "top2" and groups > 1 else best[0])
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        left = [e for g in kept for e in range(g * size, (g + 1) * size) if ok[e]]
        left = sorted(left, key=lambda e: (-c[e], e))[:top_k]
        ids[t, :len(left)] = left
    return ids


def log_scores(l, score):
    """Logarithms of one token's scores. Under softmax the largest logit is taken off first: the logarithm of a sum
    that is added to a logit of -3e38 would be lost."""
    if score == "sigmoid":
        return -np.logaddexp(0, -l)
    l = l - l.max()
    return l - np.logaddexp.reduce(l)


def parts(log_s):
    """Scores over their sum."""
    return np.exp(log_scores(log_s, "softmax"))


def weights(logits, ids, score="softmax", renormalise=True, scale=1.0):
    """Weights of the ids, and what float32 steps may change, relative: the difference of two logits is rounded
    once, which an exponential passes on as that many times its size; exponentials, reciprocals, quotients and the
    factor are below 24 roundings together, and a sum of positive terms adds one for each step."""
    tokens, experts = logits.shape
    out, slack = np.zeros(ids.shape), np.zeros(ids.shape)
    for t in range(tokens):
        ok = ids[t] >= 0
        if np.isnan(logits[t]).any() or (score == "softmax" and np.isposinf(logits[t]).any()):
            out[t] = np.nan
            continue
        l = logits[t, ids[t][ok]]
        if not l.size:
            continue
        with np.errstate(all="ignore"):
            log_s = log_scores(logits[t], score)[ids[t][ok]]
            far = np.abs(l - (min(l.max(), 0) if score == "sigmoid" else logits[t].max()))
            far[~np.isfinite(far)] = 0
            w = parts(log_s) if renormalise else np.exp(log_s)
        out[t, ok] = scale * w
        slack[t, ok] = (2 * far + 2 * far.min() + experts / 8 + 24) * EPS * np.abs(out[t, ok])
    return out, slack + 2.0 ** -126 * abs(scale)           # scores below the least normal number may be 0


def route_grad(grad, logits, ids, score="softmax", renormalise=True, scale=1.0):
    """grad_logits of finite rows, and what float32 steps may change, in units of the terms' sizes."""
    tokens, experts = logits.shape
    out, slack = np.zeros((tokens, experts)), np.zeros((tokens, experts))
    for t in range(tokens):
        slot = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < experts]
        if not slot:
            continue
        at, u, l = ids[t, slot], scale * grad[t, slot], logits[t]
        with np.errstate(all="ignore"):
            log_s = log_scores(l, score)
            far = np.abs(l - l.max()).max(initial=0, where=np.isfinite(l)) + np.abs(l).max(initial=0, where=np.isfinite(l))
            s, rest = np.exp(log_s), 1 / (1 + np.exp(l))
            if renormalise:
                v = parts(log_s[at]) if np.isfinite(log_s[at].max()) else 0 * u
            else:
                v = s[at]
        dot, size = (u * v).sum(), np.abs(u * v).sum()
        d = np.zeros(experts)
        e = np.zeros(experts)
        if renormalise:
            part, most = v * (u - dot), v * (np.abs(u) + size)
            if score == "sigmoid":
                part, most = part * rest[at], most * rest[at]
            np.add.at(d, at, part)
            np.add.at(e, at, most)
        elif score == "sigmoid":
            np.add.at(d, at, u * v * rest[at])
            np.add.at(e, at, np.abs(u * v * rest[at]))
        else:
            np.add.at(d, at, u)
            np.add.at(e, at, np.abs(u))
            d, e = s * (d - dot), s * (e + size)
        out[t] = d
        slack[t] = (4 * far + experts / 8 + 3 * ids.shape[1] + 48) * EPS * e
    return out, slack + 2.0 ** -120 * abs(scale)
