"""The routed-expert layer put together from the package's calls, as a serving step and as a training step.

Serving, in 8-bit integers (weights quantised once, every buffer kept, the whole step captured in a graph):
  order of the rows -> rows of the tokens quantised -> gate and up products + clamped SwiGLU, reading the
  tokens in place -> the result quantised -> down product -> weighted sum back into the tokens.
Serving from the residual stream: norm of the stream with the last layer's output added, in bfloat16 for the
  router and in 8-bit integers for the experts -> router's product -> choice of the experts -> the step above.
Training, in bfloat16 with float32 sums (autograd), with the same steps before it:
  order of the rows -> dispatch -> expert products -> clamped SwiGLU -> expert products -> weighted combine,
  with gradients for the tokens, the routing weights and the experts. The expert products here are torch
  matrix products, one per expert, since the package's grouped products have a forward pass only.

  python examples/routed_experts.py            # both, on a small layer, checked against plain torch
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_routed_expert_amd as epi  # noqa: E402

LIMIT = 10.0
EPS = 1e-6


class Int8Experts:
    """Experts [first, first + n) of a layer, in 8-bit integers, with the buffers of a step of up to `tokens`
    tokens. Weights: gate, up [n, inter, hidden] and down [n, hidden, inter]."""

    def __init__(self, gate, up, down, tokens: int, top_k: int, first: int = 0):
        self.gate, self.up, self.down = (epi.quantize_rows_int8(w) for w in (gate, up, down))
        n, inter, hidden = gate.shape
        slots, dev = tokens * top_k, gate.device

        def new(*shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.first, self.top_k = first, top_k
        self.offs, self.slot_of = new(n, dtype=torch.int32), new(slots, dtype=torch.int32)
        self.row_of = new(tokens, top_k, dtype=torch.int32)
        self.workspace = new(epi.moe_sort_workspace_bytes(tokens, top_k, n), dtype=torch.uint8)
        self.q, self.scale = new(tokens, hidden, dtype=torch.int8), new(tokens, dtype=torch.float32)
        # every slot may have its expert here: as many rows as slots, of which offs says how many there are.
        # Rows past the last one are never written, so their buffer starts as zeros.
        self.y = torch.zeros((slots, inter), dtype=torch.bfloat16, device=dev)
        self.yq, self.y_scale = new(slots, inter, dtype=torch.int8), new(slots, dtype=torch.float32)
        self.rows = new(slots, hidden, dtype=torch.bfloat16)

    def step(self, x, expert_of, weights, out) -> None:
        """out [tokens, hidden] = the sum over a token's slots of weight * expert(x), for the experts held here."""
        epi.moe_sort_fwd(expert_of, self.first, self.offs, self.row_of, self.slot_of, self.workspace)
        epi.quantize_rows_int8_fwd(x, self.q, self.scale)
        self.products(weights, out)

    def products(self, weights, out) -> None:
        """The part of a step after the order of the rows and the tokens' 8-bit rows."""
        epi.grouped_gate_up_swiglu_int8_fwd(self.q, self.scale, self.slot_of, self.top_k, *self.gate, *self.up,
                                            self.offs, None, self.y, LIMIT)
        epi.quantize_rows_int8_fwd(self.y, self.yq, self.y_scale)
        epi.grouped_down_router_int8_fwd(self.yq, self.y_scale, *self.down, self.offs, None, self.rows)
        epi.moe_combine_weighted_fwd(self.rows, self.row_of, weights, out)


class Int8Layer:
    """Norm, router and experts of a layer, with the buffers of a step of `tokens` tokens. router [experts, hidden]
    and bias [experts] float32; scores are sigmoids, the bias counts for the choice alone."""

    def __init__(self, norm, router, bias, gate, up, down, tokens: int, top_k: int):
        self.norm, self.router, self.bias = norm, router, bias
        self.experts = Int8Experts(gate, up, down, tokens, top_k)
        n, hidden, dev = router.shape[0], router.shape[1], router.device
        self.normed = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=dev)
        self.logits = torch.empty((tokens, n), dtype=torch.float32, device=dev)
        self.ids = torch.empty((tokens, top_k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((tokens, top_k), dtype=torch.float32, device=dev)
        self.workspace = torch.empty(epi.moe_router_logits_workspace_bytes(tokens, hidden, n), dtype=torch.uint8, device=dev)

    def step(self, x, stream, out) -> None:
        """stream += x (the last layer's output), out = this layer's, both bfloat16 [tokens, hidden]."""
        e = self.experts
        epi.rms_norm_fwd(x, self.norm, self.normed, EPS, residual=stream, residual_out=stream, q=e.q, scale=e.scale)
        epi.moe_router_logits_fwd(self.normed, self.router, self.logits, self.workspace)
        epi.moe_route_fwd(self.logits, self.ids, self.weights, bias=self.bias, score="sigmoid")
        epi.moe_sort_fwd(self.ids, e.first, e.offs, e.row_of, e.slot_of, e.workspace)
        e.products(self.weights, out)


def train_layer(x, stream, norm, router, bias, gate, up, down, top_k: int):
    """(out, stream + x) of the same layer; parameters and inputs may need gradients, the bias has none."""
    normed, stream = epi.RmsNorm.apply(x, norm, EPS, stream)
    ids, weights = epi.MoeRoute.apply(epi.MoeRouterLogits.apply(normed, router), top_k, bias, "sigmoid")
    return train_step(normed, ids, weights, gate, up, down), stream


def train_step(x, expert_of, weights, gate, up, down, first: int = 0):
    """out [tokens, hidden] of a layer whose parameters and inputs may need gradients."""
    offs, row_of, slot_of = epi.moe_sort(expert_of, gate.shape[0], first)
    ends = offs.tolist()                                   # the expert products below need them on the host
    rows = epi.MoeDispatch.apply(x, row_of, slot_of[:ends[-1]])
    starts = [0] + ends[:-1]
    h = torch.cat([torch.cat([rows[a:b] @ gate[e].T, rows[a:b] @ up[e].T], 1)
                   for e, (a, b) in enumerate(zip(starts, ends))])
    y = epi.SwigluClamped.apply(h, torch.ones(h.shape[0], device=h.device), LIMIT)
    rows = torch.cat([y[a:b] @ down[e].T for e, (a, b) in enumerate(zip(starts, ends))])
    return epi.MoeCombineWeighted.apply(rows, row_of, weights)


def plain(x, expert_of, weights, gate, up, down):
    """The same layer in plain torch, expert by expert."""
    out = torch.zeros_like(x)
    for e in range(gate.shape[0]):
        t, j = torch.nonzero(expert_of == e, as_tuple=True)
        g = (x[t] @ gate[e].T).clamp(max=LIMIT)
        u = (x[t] @ up[e].T).clamp(-LIMIT, LIMIT)
        out = out.index_add(0, t, weights[t, j, None] * ((torch.nn.functional.silu(g) * u) @ down[e].T))
    return out


def main() -> None:
    tokens, top_k, hidden, inter, experts = 96, 3, 512, 256, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)

    def normal(*shape, sigma):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(torch.bfloat16)

    params = [normal(experts, inter, hidden, sigma=hidden ** -0.5),
              normal(experts, inter, hidden, sigma=hidden ** -0.5),
              normal(experts, hidden, inter, sigma=inter ** -0.5)]
    x, grad = normal(tokens, hidden, sigma=2.0), normal(tokens, hidden, sigma=1.0)
    scores, expert_of = torch.randn(tokens, experts, generator=gen, device="cuda").topk(top_k, dim=1)
    weights = torch.softmax(scores, 1)

    def error(a, b):
        a, b = a.detach().double(), b.detach().double()
        return float((a - b).norm() / b.norm())

    want = plain(x.float(), expert_of, weights, *(p.float() for p in params))

    # serving: warm up, capture the step, replay it
    layer, out = Int8Experts(*params, tokens, top_k), torch.empty_like(x)
    layer.step(x, expert_of, weights, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, expert_of, weights, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    print(f"serving step in 8-bit integers: relative error {error(out, want):.4f}", flush=True)
    assert error(out, want) < 0.03

    # training: outputs and every gradient against autograd of the plain form in float32
    mine = [t.detach().requires_grad_() for t in (x, weights, *params)]
    theirs = [t.detach().float().requires_grad_() for t in (x, weights, *params)]
    got = train_step(mine[0], expert_of, *mine[1:])
    got.backward(grad)
    ref = plain(theirs[0], expert_of, *theirs[1:])
    ref.backward(grad.float())
    errors = {"out": error(got, ref)}
    errors |= {n: error(a.grad, b.grad) for n, a, b in zip(("x", "weights", "gate", "up", "down"), mine, theirs)}
    print("training step in bfloat16: relative errors " + ", ".join(f"{n} {e:.4f}" for n, e in errors.items()),
          flush=True)
    assert max(errors.values()) < 0.02

    # the layer from the residual stream: a graph of the serving step, and every gradient of the training step
    stream = normal(tokens, hidden, sigma=3.0)
    norm = 1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")
    router = torch.randn(experts, hidden, generator=gen, device="cuda") * hidden ** -0.5
    bias = 0.05 * torch.randn(experts, generator=gen, device="cuda")
    served = Int8Layer(norm, router, bias, *params, tokens, top_k)
    kept = stream.clone()
    served.step(x, kept, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        served.step(x, kept, out)
    kept.copy_(stream)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()

    mine = [t.detach().requires_grad_() for t in (x, stream, norm, router, *params)]
    theirs = [t.detach().float().requires_grad_() for t in (x, stream, norm, router, *params)]
    got, summed = train_layer(*mine[:4], bias, *mine[4:], top_k)
    torch.autograd.backward([got, summed], [grad, grad])
    h = theirs[0] + theirs[1]
    normed = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * theirs[2]
    scores = torch.sigmoid(normed @ theirs[3].T).gather(1, served.ids.long())
    ref = plain(normed, served.ids, scores / scores.sum(1, keepdim=True), *theirs[4:])
    torch.autograd.backward([ref, h], [grad.float(), grad.float()])
    assert torch.equal(kept, summed)
    print(f"serving layer from the residual stream: relative error {error(out, ref):.4f}", flush=True)
    assert error(out, ref) < 0.03
    errors = {"out": error(got, ref)}
    errors |= {n: error(a.grad, b.grad)
               for n, a, b in zip(("x", "stream", "norm", "router", "gate", "up", "down"), mine, theirs)}
    print("training layer in bfloat16: relative errors " + ", ".join(f"{n} {e:.4f}" for n, e in errors.items()), flush=True)
    assert max(errors.values()) < 0.03


if __name__ == "__main__":
    main()
