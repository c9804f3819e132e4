"""The routed-expert layer put together from the package's calls, as a serving step and as a training step.

Serving, in 8-bit integers (weights quantised once, every buffer kept, the whole step captured in a graph):
  order of the rows -> rows of the tokens quantised -> gate and up products + clamped SwiGLU, reading the
  tokens in place -> the result quantised -> down product -> weighted sum back into the tokens.
Training, in bfloat16 with float32 sums (autograd):
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
        epi.grouped_gate_up_swiglu_int8_fwd(self.q, self.scale, self.slot_of, self.top_k, *self.gate, *self.up,
                                            self.offs, None, self.y, LIMIT)
        epi.quantize_rows_int8_fwd(self.y, self.yq, self.y_scale)
        epi.grouped_down_router_int8_fwd(self.yq, self.y_scale, *self.down, self.offs, None, self.rows)
        epi.moe_combine_weighted_fwd(self.rows, self.row_of, weights, out)


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


if __name__ == "__main__":
    main()
