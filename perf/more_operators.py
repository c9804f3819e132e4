"""Measured cases of the steps before the routed experts: the norm that joins the residual stream, the router's
product, and the choice of experts, with their gradients.

Sizes: hidden 7168 and 2048 and 64 experts of which a token takes 8 are those of the package's own workloads;
the others are generic. "own" chooses between the plain forms below and the package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _norm(name, op, rows, cols, dtype="bf16", weight="bf16", residual=True, int8=False):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "weight": weight, "residual": residual, "int8": int8}


def _logits(name, op, rows, cols, experts, dtype="bf16", weight="bf16"):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "experts": experts, "dtype": dtype, "weight": weight}


def _route(name, op, rows, experts, top_k, score="softmax", bias=False, groups=1, top_groups=1, renormalise=True, dtype="f32"):
    return {"name": name, "op": op, "rows": rows, "experts": experts, "top_k": top_k, "score": score, "bias": bias,
            "groups": groups, "top_groups": top_groups, "renormalise": renormalise, "dtype": dtype}


def listed():
    return [
        # the norm before the experts in one serving step of 32 sequences
        _norm("norm_decode", "norm", 32, 7168),
        # the same for prompts, whose experts multiply 8-bit integers: the rows leave in both forms
        _norm("norm_prompt_int8", "norm", 16384, 7168, int8=True),
        # a ragged batch with an odd width in float16 storage, the weight kept in float32
        _norm("norm_ragged", "norm", 10007, 1001, dtype="f16", weight="f32"),
        # a training step's forward pass, which keeps the stream and the rows' factors
        _norm("norm_train", "norm", 65536, 7168),
        # and its gradients, with that of the stream added
        _norm("norm_grad", "norm_bwd", 32768, 7168, weight="f32"),
        # scores of a serving step
        _logits("logits_decode", "logits", 32, 7168, 64),
        # scores of a training step
        _logits("logits_train", "logits", 131072, 7168, 64),
        # scores of a prompt by a router kept in float32
        _logits("logits_f32", "logits", 8192, 2048, 128, weight="f32"),
        # gradients of the tokens and of the router's weight
        _logits("logits_grad", "logits_bwd", 65536, 7168, 64),
        # choice of the experts in a serving step
        _route("route_decode", "route", 32, 64, 8),
        # many experts in groups, balanced by a bias, for a long batch
        _route("route_groups", "route", 65536, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4),
        # gradient of every score from those of the chosen weights
        _route("route_grad", "route_bwd", 131072, 64, 8, renormalise=False),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm: odd, or a power of two."""
    if rng.random() < 0.3:
        return 2 ** rng.randint(math.ceil(math.log2(lo)), int(math.log2(hi)))
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) | 1


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "logits", "logits", "logits_bwd", "route", "route", "route_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    rows = _spread(rng, 1, 65536 if op in ("norm", "norm_bwd", "logits_bwd") else 131072)
    while True:
        if op in ("norm", "norm_bwd"):
            # rows that are to be 8-bit integers come from 16-bit activations
            case = _norm("", op, rows, _spread(rng, 64, 7168), dtype, rng.choice([dtype, "f32"]), rng.random() < 0.7,
                         op == "norm" and dtype != "f32" and rng.random() < 0.5)
        elif op in ("logits", "logits_bwd"):
            # rows of whole 16-byte pieces, as models have them, and others
            cols = _spread(rng, 64, 7168) if rng.random() < 0.3 else 16 * _spread(rng, 4, 448)
            case = _logits("", op, rows, cols, rng.choice([4, 8, 12, 60, 64, 128, 256]), dtype, rng.choice([dtype, "f32"]))
        else:
            experts = rng.choice([4, 8, 12, 60, 64, 128, 256])
            groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts // g >= 2 and experts % g == 0])
            top_groups = rng.randint((groups + 1) // 2, groups)
            top_k = rng.choice([n for n in (1, 2, 4, 5, 8) if n <= top_groups * (experts // groups)])
            case = _route("", op, rows, experts, top_k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, top_groups,
                          rng.random() < 0.6, rng.choice(["f32", "f32", "bf16"]))
        del case["name"]
        cost = work(case)
        if cost["bytes"] <= 3.5e9 and cost["flops"] <= 1.2e11:
            return case
        rows = max(1, rows // 2)


def work(case):
    t, op, e = case["rows"], case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_bwd"):
        n, w, joined = t * case["cols"], BYTES[case["weight"]], 2 if case["residual"] else 1
        if op == "norm":
            moved = joined * e + e + (joined - 1) * e + (1 if case["int8"] else 0)
            return {"bytes": n * moved + case["cols"] * w + t * (8 if case["int8"] else 4), "flops": 6 * n}
        # gradient, stream (and the stream's own gradient) in, one gradient out
        return {"bytes": n * e * (2 + joined) + 2 * case["cols"] * w + 4 * t, "flops": 10 * n}
    x = case["experts"]
    if op in ("logits", "logits_bwd"):
        h, w = case["cols"], BYTES[case["weight"]]
        if op == "logits":
            return {"bytes": t * h * e + x * h * w + t * x * 4, "flops": 2 * t * h * x}
        return {"bytes": 2 * t * h * e + 2 * x * h * w + t * x * 4, "flops": 4 * t * h * x}
    k = case["top_k"]
    if op == "route":
        return {"bytes": t * x * e + t * k * 8 + (4 * x if case["bias"] else 0), "flops": 4 * t * x}
    # where every score counts they are read, otherwise those of the chosen experts
    read = t * x * e if case["score"] == "softmax" and not case["renormalise"] else t * k * e
    return {"bytes": read + t * x * e + t * k * 8, "flops": 4 * t * k + (4 * t * x if read > t * k * e else 0)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, t, dt = case["op"], case["rows"], DTYPES[case["dtype"]]
    state = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def empty(*shape, dtype):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    if op in ("norm", "norm_bwd"):
        h, wt = case["cols"], DTYPES[case["weight"]]
        state["w"] = (1 + 0.1 * normal(h)).to(wt)
        x, r = normal(t, h).to(dt), (4 * normal(t, h)).to(dt) if case["residual"] else None
        if op == "norm":
            state |= {"x": x, "r": r, "out": empty(t, h, dtype=dt), "h": empty(t, h, dtype=dt) if case["residual"] else None,
                      "rstd": empty(t, dtype=torch.float32)}
            if case["int8"]:
                state |= {"q": empty(t, h, dtype=torch.int8), "scale": empty(t, dtype=torch.float32), "values": empty(t, h, dtype=dt)}
        else:
            # the stream that the forward pass left, and the factors of its rows
            stream = x if r is None else (x.float() + r.float()).to(dt)
            rstd = torch.rsqrt(stream.float().square().mean(1) + EPS)
            state |= {"h": stream, "rstd": rstd, "grad": normal(t, h).to(dt), "grad_h": normal(t, h).to(dt) if case["residual"] else None,
                      "grad_x": empty(t, h, dtype=dt), "grad_w": empty(h, dtype=wt), "workspace": _workspace("norm_bwd", t, h)}
    elif op in ("logits", "logits_bwd"):
        h, experts, wt = case["cols"], case["experts"], DTYPES[case["weight"]]
        state |= {"x": normal(t, h).to(dt), "w": (normal(experts, h) / math.sqrt(h)).to(wt), "workspace": _workspace(op, t, h, experts)}
        if op == "logits":
            state["logits"] = empty(t, experts, dtype=torch.float32)
        else:
            # as the choice gives them: of the size of a weight's gradient over the tokens
            state |= {"grad": normal(t, experts) / t, "grad_x": empty(t, h, dtype=dt), "grad_w": empty(experts, h, dtype=wt)}
    else:
        experts, k = case["experts"], case["top_k"]
        # some experts are liked more than others, and the bias works against that
        liked = 0.5 * normal(experts)
        state |= {"logits": (normal(t, experts) + liked).to(dt), "bias": -0.1 * liked if case["bias"] else None}
        if op == "route":
            state |= {"ids": empty(t, k, dtype=torch.int32), "weights": empty(t, k, dtype=torch.float32)}
        else:
            ids = normal(t, experts).argsort(1)[:, :k]
            state |= {"ids": ids.to(torch.int32), "grad": normal(t, k), "grad_logits": empty(t, experts, dtype=dt)}
    return state


def _workspace(op, *sizes):
    if not own:
        return None
    import moe_routed_expert_amd as epi
    need = {"norm_bwd": epi.rms_norm_bwd_workspace_bytes, "logits": epi.moe_router_logits_workspace_bytes,
            "logits_bwd": epi.moe_router_logits_bwd_workspace_bytes}[op](*sizes)
    return torch.empty(need, device="cuda", dtype=torch.uint8)


# ---- the plain forms ----------------------------------------------------------

SCALE = 2.5  # of the weights where the scores are sigmoids


def _factor(case):
    return SCALE if case["score"] == "sigmoid" else 1.0


def _chosen(s):
    """Ids in descending order of the scores, the lowest first where they are equal."""
    case, logits = s["case"], s["logits"].double()
    t, experts = logits.shape
    score = torch.softmax(logits, 1) if case["score"] == "softmax" else 1 / (1 + torch.exp(-logits))
    # without a bias the logits have the same order, and are exact
    order = logits if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        grouped = order.reshape(t, case["groups"], -1)
        top2 = grouped.sort(dim=2, descending=True).values[..., :2].sum(2) if case["bias"] else grouped.amax(2)
        best = top2.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros_like(top2, dtype=torch.bool).scatter_(1, best, True)
        order = torch.where(keep[..., None], grouped, -math.inf).reshape(t, experts)
    return order.sort(dim=1, descending=True, stable=True).indices[:, :case["top_k"]]


def _scores(s):
    logits = s["logits"].float()
    if s["case"]["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    shifted = torch.exp(logits - logits.amax(1, keepdim=True))
    return shifted / shifted.sum(1, keepdim=True)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op == "norm":
        h = s["x"]
        out = {}
        if s["r"] is not None:
            h = out["h"] = (h.float() + s["r"].float()).to(dt)
        h = h.float()
        rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
        y = h * rstd[:, None] * s["w"].float()
        out |= {"out": y.to(dt), "rstd": rstd}
        if case["int8"]:
            most = y.abs().amax(1, keepdim=True)
            q = torch.round(y * 127 / most)
            out |= {"values": (q * (most / 127)).to(dt), "scale": most[:, 0] / 127}
        return out
    if op == "norm_bwd":
        dy, a = s["grad"].float(), s["h"].float() * s["rstd"][:, None]
        g = dy * s["w"].float()
        dx = s["rstd"][:, None] * (g - a * (g * a).mean(1, keepdim=True))
        if s["grad_h"] is not None:
            dx = dx + s["grad_h"].float()
        return {"grad_x": dx.to(dt), "grad_w": (dy * a).sum(0).to(s["w"].dtype)}
    if op == "logits":
        return {"logits": s["x"].float() @ s["w"].float().T}
    if op == "logits_bwd":
        return {"grad_x": (s["grad"] @ s["w"].float()).to(dt), "grad_w": (s["grad"].T @ s["x"].float()).to(s["w"].dtype)}
    score = _scores(s)
    if op == "route":
        ids = _chosen(s)
        weights = score.gather(1, ids)
        if case["renormalise"]:
            weights = weights / weights.sum(1, keepdim=True)
        return {"ids": ids.to(torch.int32), "weights": weights * _factor(case)}
    ids, grad = s["ids"].long(), s["grad"] * _factor(case)
    chosen = score.gather(1, ids)
    if case["renormalise"]:
        part = chosen / chosen.sum(1, keepdim=True)
        grad = (grad - (grad * part).sum(1, keepdim=True)) / chosen.sum(1, keepdim=True)
    whole = torch.zeros_like(score).scatter_(1, ids, grad)
    if case["score"] == "sigmoid":
        return {"grad_logits": (whole * score * (1 - score)).to(dt)}
    return {"grad_logits": (score * (whole - (whole * score).sum(1, keepdim=True))).to(dt)}


# ---- the package's calls ------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import moe_routed_expert_amd as epi
    s, case, op = state, state["case"], state["case"]["op"]
    if op == "norm":
        out = {"h": s["h"]} if s["r"] is not None else {}
        if case["int8"]:
            epi.rms_norm_fwd(s["x"], s["w"], s["out"], EPS, residual=s["r"], residual_out=s["h"], rstd=s["rstd"], q=s["q"], scale=s["scale"])
            torch.mul(s["q"], s["scale"][:, None], out=s["values"])
            return out | {"out": s["out"], "rstd": s["rstd"], "values": s["values"], "scale": s["scale"]}
        epi.rms_norm_fwd(s["x"], s["w"], s["out"], EPS, residual=s["r"], residual_out=s["h"], rstd=s["rstd"])
        return out | {"out": s["out"], "rstd": s["rstd"]}
    if op == "norm_bwd":
        epi.rms_norm_bwd(s["grad"], s["h"], s["w"], s["rstd"], s["grad_x"], s["grad_w"], s["workspace"], grad_residual=s["grad_h"])
        return {"grad_x": s["grad_x"], "grad_w": s["grad_w"]}
    if op == "logits":
        epi.moe_router_logits_fwd(s["x"], s["w"], s["logits"], s["workspace"])
        return {"logits": s["logits"]}
    if op == "logits_bwd":
        epi.moe_router_logits_bwd(s["grad"], s["x"], s["w"], s["grad_x"], s["grad_w"], s["workspace"])
        return {"grad_x": s["grad_x"], "grad_w": s["grad_w"]}
    if op == "route":
        epi.moe_route_fwd(s["logits"], s["ids"], s["weights"], bias=s["bias"], score=case["score"], groups=case["groups"],
                          top_groups=case["top_groups"], group_score="top2" if case["bias"] else "max",
                          renormalise=case["renormalise"], scale=_factor(case))
        return {"ids": s["ids"], "weights": s["weights"]}
    epi.moe_route_bwd(s["grad"], s["logits"], s["ids"], s["grad_logits"], score=case["score"], renormalise=case["renormalise"],
                      scale=_factor(case))
    return {"grad_logits": s["grad_logits"]}


# ---- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        stream = s["x"] if s["r"] is None else (s["x"].double() + s["r"].double()).to(s["x"].dtype)
        h = stream.double()
        rstd = (torch.linalg.vecdot(h, h) / h.shape[1] + EPS).rsqrt()
        y = torch.einsum("th,t,h->th", h, rstd, s["w"].double())
        out = {} if s["r"] is None else {"h": stream.double()}
        out |= {"out": y, "rstd": rstd}
        if case["int8"]:
            step = torch.linalg.vector_norm(y, math.inf, dim=1) / 127
            out |= {"values": torch.round(y / step[:, None]).clamp(-127, 127) * step[:, None], "scale": step}
        return out
    if op == "norm_bwd":
        h, w, n, parts = s["h"].shape[1], s["w"].double(), s["rstd"].double(), []
        dw = torch.zeros(h, dtype=torch.float64, device="cuda")
        for at in torch.arange(s["h"].shape[0], device="cuda").split(8192):
            x, dy = s["h"][at].double(), s["grad"][at].double()
            dot = torch.linalg.vecdot(dy * w, x) * n[at] ** 3 / h
            dx = torch.addcmul(-x * dot[:, None], dy * w, n[at][:, None])
            parts.append(dx if s["grad_h"] is None else dx + s["grad_h"][at].double())
            dw += (n[at][None, :] @ (dy * x))[0]
        return {"grad_x": torch.cat(parts), "grad_w": dw}
    if op == "logits":
        return {"logits": torch.cat([torch.nn.functional.linear(x.double(), s["w"].double()) for x in s["x"].split(16384)])}
    if op == "logits_bwd":
        w, dw = s["w"].double(), 0
        dx = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for at in range(0, s["x"].shape[0], 16384):
            here = slice(at, at + 16384)
            torch.mm(s["grad"][here].double(), w, out=dx[here])
            dw = dw + torch.mm(s["grad"][here].double().T.contiguous(), s["x"][here].double())
        return {"grad_x": dx, "grad_w": dw}
    logits, factor = s["logits"].double(), _factor(case)
    t, experts = logits.shape
    log_score = torch.nn.functional.logsigmoid(logits) if case["score"] == "sigmoid" else torch.log_softmax(logits, 1)
    if op == "route":
        # the experts one at a time: the best that is left, the first of equal ones (argmax of a reversed row would take the last)
        value = logits.clone() if s["bias"] is None else log_score.exp() + s["bias"].double()
        lowest = torch.full_like(value[:, :1], -math.inf)
        size = experts // case["groups"]

        def first_best(v):
            best = v.max(1, keepdim=True).values
            place = torch.where(v == best, torch.arange(v.shape[1], device=v.device), v.shape[1])
            return place.min(1, keepdim=True).values
        if case["groups"] > 1:
            of = value.reshape(t, case["groups"], size)
            total = of.topk(2, 2).values.sum(2) if case["bias"] else of.max(2).values
            kept = torch.zeros(t, case["groups"], dtype=torch.bool, device="cuda")
            for _ in range(case["top_groups"]):
                at = first_best(total)
                kept.scatter_(1, at, True)
                total.scatter_(1, at, lowest)
            value[~kept.repeat_interleave(size, 1)] = -math.inf
        ids = []
        for _ in range(case["top_k"]):
            ids.append(first_best(value))
            value.scatter_(1, ids[-1], lowest)
        ids = torch.cat(ids, 1)
        part = log_score.gather(1, ids)
        weights = torch.softmax(part, 1) if case["renormalise"] else part.exp()
        return {"ids": ids.to(torch.int32), "weights": weights * factor}
    # the gradient of the weights' sum with the given ones, by differentiating the definition
    leaf = logits.clone().requires_grad_()
    part = torch.nn.functional.logsigmoid(leaf) if case["score"] == "sigmoid" else torch.log_softmax(leaf, 1)
    part = part.gather(1, s["ids"].long())
    weights = torch.softmax(part, 1) if case["renormalise"] else part.exp()
    (weights * factor * s["grad"].double()).sum().backward()
    return {"grad_logits": leaf.grad}
