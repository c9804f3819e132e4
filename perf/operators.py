"""Measured cases of the routed-expert operators: order of the rows, moves of the rows with their
gradients, and the experts' products in 8-bit integers.

Sizes: hidden 7168, inter 2048, top-8 of 64 experts with 8 on this GPU are those of the package's own
workloads; the others are generic. "own" chooses between the plain forms below and the package's calls.
"""
import math

import numpy as np
import torch

own = False

LIMIT = 10.0  # of the clamped SwiGLU, as the package's 2048-wide workloads have it
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    def case(name, op, tokens, top_k, experts, local, hidden=0, inter=0, dtype="bf16", out="bf16", ids="int32"):
        return {"name": name, "op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "local": local,
                "hidden": hidden, "inter": inter, "dtype": dtype, "out": out, "ids": ids}
    return [
        # the order of the rows for one step of a serving batch of 32 sequences, every expert on this GPU
        case("sort_decode", "sort", 32, 8, 64, 64, ids="int64"),
        # the order of the rows for a training step's share: 8 of 64 experts on this GPU
        case("sort_train", "sort", 131072, 8, 64, 8),
        # rows of a serving step, tokens repeated for each of their experts
        case("dispatch_decode", "dispatch_fwd", 32, 8, 64, 64, hidden=7168),
        # rows of a training step's share, about one row a token
        case("dispatch_train", "dispatch_fwd", 131072, 8, 64, 8, hidden=7168),
        # gradient of the tokens from the gradients of all their rows, every expert on this GPU
        case("dispatch_grad", "dispatch_bwd", 32768, 8, 64, 64, hidden=2048),
        # weighted sum of a serving step's rows
        case("combine_decode", "combine_fwd", 32, 8, 64, 64, hidden=7168),
        # a ragged prompt with an odd width in float16 storage, float32 out
        case("combine_ragged", "combine_fwd", 10007, 3, 12, 12, hidden=1001, dtype="f16", out="f32"),
        # gradients of the rows and of the routing weights in a training step's share
        case("combine_grad", "combine_bwd", 65536, 8, 64, 8, hidden=7168),
        # 8-bit gate and up products of a serving step: the weights are read for a few rows each
        case("gate_up_decode", "gate_up", 16, 2, 8, 8, hidden=7168, inter=2048),
        # the same of long prompts: every expert has thousands of rows
        case("gate_up_prefill", "gate_up", 32768, 2, 8, 8, hidden=7168, inter=2048),
        # 8-bit down product of a serving step, float32 rows for the sum that follows
        case("down_decode", "down", 16, 2, 8, 8, hidden=7168, inter=2048, out="f32"),
        # the same of long prompts, bfloat16 rows
        case("down_prefill", "down", 32768, 2, 8, 8, hidden=7168, inter=2048),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm: odd, or a power of two."""
    if rng.random() < 0.3:
        return 2 ** rng.randint(math.ceil(math.log2(lo)), int(math.log2(hi)))
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) | 1


def draw(rng):
    op = rng.choice(["sort", "dispatch_fwd", "dispatch_bwd", "combine_fwd", "combine_bwd", "gate_up", "down"])
    dtype, product = rng.choice(["bf16", "bf16", "f16", "f32"]), op in ("gate_up", "down")
    while True:
        experts = rng.choice([4, 8, 12, 64, 128])
        local = experts if rng.random() < 0.6 else experts // 4
        case = {"op": op, "top_k": rng.choice([n for n in (1, 2, 4, 5, 7, 8) if n <= experts]), "experts": experts, "local": local, "inter": 0,
                "hidden": 0, "dtype": dtype, "ids": rng.choice(["int32", "int64"]),
                "out": rng.choice([dtype, "f32"]) if op == "combine_fwd" else dtype}
        # with a share of the experts, as many tokens for each share
        shares = experts // local
        case["tokens"] = shares * _spread(rng, 1, (32768 if product else 131072) // shares)
        if product:
            case |= {"dtype": "bf16", "out": rng.choice(["bf16", "f32"]) if op == "down" else "bf16",
                     "hidden": 16 * _spread(rng, 16, 448), "inter": 16 * _spread(rng, 8, 128)}
            weights = local * case["hidden"] * case["inter"]
            if weights > 8 * 7168 * 2048:
                continue
        else:
            width = _spread(rng, 64, 7168)
            case["hidden"] = 0 if op == "sort" else width
        if work(case)["bytes"] <= 3.7e9 and work(case)["flops"] <= 3.5e12:
            return case


def _rows(case):
    """The rows that a case has on this GPU: all of its slots, or one share of them."""
    return case["tokens"] * case["top_k"] * case["local"] // case["experts"]


def work(case):
    t, k, h, i, rows = case["tokens"], case["top_k"], case["hidden"], case["inter"], _rows(case)
    slots, e, eo = t * k, BYTES[case["dtype"]], BYTES[case["out"]]
    # tokens that have a row here, and experts that have one, when the choice is an even one
    hit = t if case["local"] == case["experts"] else int(t * (1 - (1 - case["local"] / case["experts"]) ** k))
    used = case["local"] * (1 - (1 - k / case["experts"]) ** t)
    op = case["op"]
    if op == "sort":
        return {"bytes": slots * (8 if case["ids"] == "int64" else 4) + 8 * slots + 4 * case["local"], "flops": slots}
    if op == "dispatch_fwd":
        return {"bytes": hit * h * e + rows * h * e + 4 * rows, "flops": rows * h}
    if op == "dispatch_bwd":
        return {"bytes": rows * h * e + 4 * slots + t * h * e, "flops": rows * h}
    if op == "combine_fwd":
        return {"bytes": rows * h * e + 8 * slots + t * h * eo, "flops": 2 * rows * h}
    if op == "combine_bwd":
        return {"bytes": hit * h * e + 2 * rows * h * e + 12 * slots, "flops": 3 * rows * h}
    if op == "gate_up":
        return {"bytes": int(hit * h * 2 + used * 2 * i * (h + 4)) + 8 * rows + 4 * case["local"] + rows * i * 2,
                "flops": 4 * rows * h * i}
    return {"bytes": int(rows * i * 2 + used * h * (i + 4)) + 4 * case["local"] + rows * h * eo, "flops": 2 * rows * h * i}


def _routing(case, g):
    """Distinct experts for each token, some of them liked more than others, and weights that add up to 1.

    Where this GPU has one of several equal shares of the experts, each choice is made for as many tokens as
    there are shares, one share on from token to token, and the tokens are shuffled: every share then has
    tokens * top_k / shares rows whatever the seed, so that the buffers have one size."""
    t, k, experts, shares = case["tokens"], case["top_k"], case["experts"], case["experts"] // case["local"]
    scores = torch.randn(t // shares, experts, generator=g, device="cuda") + 0.3 * torch.randn(experts, generator=g, device="cuda")
    top = scores.topk(k, dim=1)
    on = case["local"] * torch.arange(shares, device="cuda")
    ids = ((top.indices[:, None] + on[None, :, None]) % experts).reshape(t, k)
    shuffled = torch.randperm(t, generator=g, device="cuda")
    return ids[shuffled], torch.softmax(top.values, dim=1).repeat_interleave(shares, 0)[shuffled]


def _channels(shape, g):
    """8-bit weights with a scale for each output channel, from normal weights of variance 1 / inputs."""
    w = torch.randn(*shape, generator=g, device="cuda") / math.sqrt(shape[-1])
    most = w.abs().amax(-1)
    q = torch.round(w * (127 / most)[..., None]).to(torch.int8)
    return q, most / 127


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, out_dt = DTYPES[case["dtype"]], DTYPES[case["out"]]
    t, k, h, i, local, op = (case[n] for n in ("tokens", "top_k", "hidden", "inter", "local", "op"))
    ids, weights = _routing(case, g)
    state = {"case": case, "first": 0}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def empty(*shape, dtype):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    if op == "sort":
        # the experts of this GPU sit in the middle of all
        state |= {"ids": ids.to(getattr(torch, case["ids"])), "first": (case["experts"] - local) // 2,
                  "offs": empty(local, dtype=torch.int32), "row_of": empty(t, k, dtype=torch.int32),
                  "slot_of": empty(t * k, dtype=torch.int32), "workspace": empty(_workspace(t, k, local), dtype=torch.uint8)}
        return state
    # what the sort gave: the order of the rows, and how many there are
    offs, row_of, slot_of = _sort(ids, 0, local)
    rows = int(offs[-1])
    slot_of = slot_of[:rows].clone()
    state |= {"offs": offs, "row_of": row_of, "slot_of": slot_of, "weights": weights, "rows": rows}
    if op == "dispatch_fwd":
        state |= {"x": normal(t, h).to(dt), "out": empty(rows, h, dtype=dt)}
    elif op == "dispatch_bwd":
        state |= {"grad": normal(rows, h).to(dt), "grad_x": empty(t, h, dtype=dt)}
    elif op == "combine_fwd":
        state |= {"rows_in": normal(rows, h).to(dt), "out": empty(t, h, dtype=out_dt)}
    elif op == "combine_bwd":
        state |= {"grad": normal(t, h).to(dt), "rows_in": normal(rows, h).to(dt),
                  "grad_rows": empty(rows, h, dtype=dt), "grad_weights": empty(t, k, dtype=torch.float32)}
    else:
        counts = torch.diff(offs, prepend=offs.new_zeros(1))
        at = torch.arange(rows, device="cuda", dtype=torch.int32)
        expert = torch.searchsorted(offs, at, right=True)
        # most rows of any expert, and each row's expert and its place there: the plain form's batches
        state |= {"most": int(counts.max()), "expert": expert, "place": (at - (offs - counts)[expert]).long()}
        if op == "gate_up":
            gate, gate_scale = _channels((local, i, h), g)
            up, up_scale = _channels((local, i, h), g)
            # inputs of about 4: gate and up reach the clamps as in the package's 2048-wide workloads
            state |= {"x": (4 * normal(t, h)).to(dt), "q": empty(t, h, dtype=torch.int8), "scale": empty(t, dtype=torch.float32),
                      "gate": gate, "gate_scale": gate_scale, "up": up, "up_scale": up_scale,
                      "probs": weights.reshape(-1)[slot_of.long()].contiguous(), "y": empty(rows, i, dtype=out_dt)}
        else:
            down, down_scale = _channels((local, h, i), g)
            state |= {"x": (0.5 * normal(rows, i)).to(dt), "q": empty(rows, i, dtype=torch.int8), "scale": empty(rows, dtype=torch.float32),
                      "down": down, "down_scale": down_scale, "out": empty(rows, h, dtype=out_dt)}
    return state


def _workspace(tokens, top_k, local):
    if not own:
        return 0
    import moe_routed_expert_amd as epi
    return epi.moe_sort_workspace_bytes(tokens, top_k, local)


# ---- the plain forms ----------------------------------------------------------

def _sort(ids, first, local):
    slots = ids.numel()
    e = ids.reshape(-1) - first
    key = torch.where((e >= 0) & (e < local), e, local)
    order = torch.argsort(key, stable=True)
    offs = (key[:, None] == torch.arange(local, device=key.device)).sum(0).cumsum(0).to(torch.int32)
    at = torch.arange(slots, device=key.device)
    here = at < offs[-1]
    slot_of = torch.where(here, order, -1).to(torch.int32)
    row_of = torch.empty(slots, dtype=torch.int32, device=key.device)
    row_of[order] = torch.where(here, at, -1).to(torch.int32)
    return offs, row_of.reshape(ids.shape), slot_of


def _sum_of_rows(rows, row_of, weights):
    if not rows.shape[0]:
        return torch.zeros(row_of.shape[0], rows.shape[1], device=rows.device)
    picked = rows[row_of.clamp(min=0).long()].float() * (row_of >= 0)[..., None]
    return picked.sum(1) if weights is None else (picked * weights[..., None]).sum(1)


def _quantize(x):
    x = x.float()
    most = x.abs().amax(1, keepdim=True)
    q = torch.where(most > 0, torch.round(x * 127 / most), 0.0)
    return q, most / 127


def _product(s, a, w, scale):
    """Rows times their expert's weights, as one batch of products padded to the largest expert."""
    batch = torch.zeros(w.shape[0], s["most"], a.shape[1], device=a.device)
    batch[s["expert"], s["place"]] = a
    return torch.bmm(batch, w.float().transpose(1, 2))[s["expert"], s["place"]] * scale[s["expert"]]


def _plain(s):
    op, k = s["case"]["op"], s["case"]["top_k"]
    dt, out_dt = DTYPES[s["case"]["dtype"]], DTYPES[s["case"]["out"]]
    if op == "sort":
        offs, row_of, slot_of = _sort(s["ids"], s["first"], s["case"]["local"])
        return {"offs": offs, "row_of": row_of, "slot_of": slot_of}
    if op == "dispatch_fwd":
        return {"out": s["x"][s["slot_of"].long() // k]}
    if op == "dispatch_bwd":
        return {"grad_x": _sum_of_rows(s["grad"], s["row_of"], None).to(dt)}
    if op == "combine_fwd":
        return {"out": _sum_of_rows(s["rows_in"], s["row_of"], s["weights"]).to(out_dt)}
    if op == "combine_bwd":
        slot = s["slot_of"].long()
        grad = s["grad"][slot // k].float()
        grad_weights = torch.zeros_like(s["weights"])
        grad_weights.view(-1)[slot] = (grad * s["rows_in"].float()).sum(1)
        return {"grad_rows": (grad * s["weights"].reshape(-1)[slot][:, None]).to(dt), "grad_weights": grad_weights}
    q, scale = _quantize(s["x"])
    if op == "down":
        return {"out": (_product(s, q, s["down"], s["down_scale"]) * scale).to(out_dt)}
    token = s["slot_of"].long() // k
    q, scale = q[token], scale[token]
    gate = (_product(s, q, s["gate"], s["gate_scale"]) * scale).clamp(max=LIMIT)
    up = (_product(s, q, s["up"], s["up_scale"]) * scale).clamp(-LIMIT, LIMIT)
    return {"y": (gate / (1 + torch.exp(-gate)) * up * s["probs"][:, None]).to(out_dt)}


# ---- the package's calls ------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import moe_routed_expert_amd as epi
    s, op, k = state, state["case"]["op"], state["case"]["top_k"]
    if op == "sort":
        epi.moe_sort_fwd(s["ids"], s["first"], s["offs"], s["row_of"], s["slot_of"], s["workspace"])
        return {"offs": s["offs"], "row_of": s["row_of"], "slot_of": s["slot_of"]}
    if op == "dispatch_fwd":
        epi.moe_dispatch_fwd(s["x"], s["slot_of"], k, s["out"])
        return {"out": s["out"]}
    if op == "dispatch_bwd":
        epi.moe_dispatch_bwd(s["grad"], s["row_of"], s["grad_x"])
        return {"grad_x": s["grad_x"]}
    if op == "combine_fwd":
        epi.moe_combine_weighted_fwd(s["rows_in"], s["row_of"], s["weights"], s["out"])
        return {"out": s["out"]}
    if op == "combine_bwd":
        epi.moe_combine_weighted_bwd(s["grad"], s["rows_in"], s["row_of"], s["weights"], s["grad_rows"], s["grad_weights"])
        return {"grad_rows": s["grad_rows"], "grad_weights": s["grad_weights"]}
    epi.quantize_rows_int8_fwd(s["x"], s["q"], s["scale"])
    if op == "down":
        epi.grouped_down_router_int8_fwd(s["q"], s["scale"], s["down"], s["down_scale"], s["offs"], None, s["out"])
        return {"out": s["out"]}
    epi.grouped_gate_up_swiglu_int8_fwd(s["q"], s["scale"], s["slot_of"], k, s["gate"], s["gate_scale"], s["up"], s["up_scale"],
                                        s["offs"], s["probs"], s["y"], LIMIT)
    return {"y": s["y"]}


# ---- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, k, t, h = case["op"], case["top_k"], case["tokens"], case["hidden"]
    if op == "sort":
        # numpy, expert by expert
        ids = s["ids"].cpu().numpy().reshape(-1) - s["first"]
        found = [np.flatnonzero(ids == e) for e in range(case["local"])]
        order = np.concatenate(found)
        row_of, slot_of = np.full(ids.size, -1, np.int32), np.full(ids.size, -1, np.int32)
        slot_of[:order.size], row_of[order] = order, np.arange(order.size)
        return {"offs": np.cumsum([f.size for f in found]).astype(np.int32), "row_of": row_of.reshape(t, k), "slot_of": slot_of}
    if op == "dispatch_fwd":
        return {"out": s["x"].double().repeat_interleave(k, 0)[s["slot_of"].long()] if t * k * h < 2 ** 28
                else torch.index_select(s["x"].double(), 0, torch.div(s["slot_of"], k, rounding_mode="floor"))}
    if op in ("dispatch_bwd", "combine_fwd"):
        rows = s["grad"] if op == "dispatch_bwd" else s["rows_in"]
        total = torch.zeros(t, h, dtype=torch.float64, device="cuda")
        for j in range(k):
            row = s["row_of"][:, j]
            token = torch.nonzero(row >= 0)[:, 0]
            add = rows[row[token].long()].double()
            total[token] += add if op == "dispatch_bwd" else add * s["weights"][token, j, None].double()
        return {"grad_x" if op == "dispatch_bwd" else "out": total}
    if op == "combine_bwd":
        grad_rows = torch.zeros(s["rows"], h, dtype=torch.float64, device="cuda")
        grad_weights = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            row = s["row_of"][:, j]
            token = torch.nonzero(row >= 0)[:, 0]
            row, grad = row[token].long(), s["grad"][token].double()
            grad_rows[row] = grad * s["weights"][token, j, None].double()
            grad_weights[token, j] = torch.linalg.vecdot(grad, s["rows_in"][row].double())
        return {"grad_rows": grad_rows, "grad_weights": grad_weights}
    x = s["x"].double()
    step = x.abs().max(1, keepdim=True).values / 127
    x = torch.where(step > 0, torch.round(x / step), 0.0) * step
    parts, start = [], 0
    for e, end in enumerate(s["offs"].tolist()):
        here, start = slice(start, end), end
        if op == "down":
            parts.append(x[here] @ (s["down"][e].double() * s["down_scale"][e].double()[:, None]).T)
            continue
        a = x[torch.div(s["slot_of"][here], k, rounding_mode="floor").long()]
        gate = torch.clamp(a @ (s["gate"][e].double() * s["gate_scale"][e].double()[:, None]).T, max=LIMIT)
        up = torch.clamp(a @ (s["up"][e].double() * s["up_scale"][e].double()[:, None]).T, -LIMIT, LIMIT)
        parts.append(gate * torch.sigmoid(gate) * up * s["probs"][here].double()[:, None])
    return {"out" if op == "down" else "y": torch.cat(parts)}
