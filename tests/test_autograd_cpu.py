"""The autograd wrappers of the epilogues refuse a second derivative, on the CPU: the kernel calls are replaced by plain
writes that autograd does not see, as it does not see the kernels'."""
import pytest
import torch

from moe_routed_expert_amd import binding

LIMIT = 1.0


def swiglu(x, probs):
    gate, up = x.chunk(2, 1)
    return torch.nn.functional.silu(gate.clamp(max=LIMIT)) * up.clamp(-LIMIT, LIMIT) * probs[:, None]


def router(x, probs):
    return x * probs[:, None]


@pytest.fixture(autouse=True)
def kernels(monkeypatch):
    def gradients(formula, grad, x, probs):
        with torch.enable_grad():
            leaf = [x.detach().requires_grad_(), probs.detach().requires_grad_()]
            return torch.autograd.grad(formula(*leaf), leaf, grad.detach())

    def write(formula, grad, x, probs, grad_x, grad_probs):
        got = gradients(formula, grad, torch.zeros_like(grad) if x is None else x, probs)
        with torch.no_grad():
            grad_x.copy_(got[0])
            if grad_probs is not None:
                grad_probs.copy_(got[1])

    def forward(formula):
        def f(x, probs, out, *limit):
            with torch.no_grad():
                out.copy_(formula(x, probs))
        return f

    monkeypatch.setattr(binding, "swiglu_clamped_fwd", forward(swiglu))
    monkeypatch.setattr(binding, "router_weight_mul_fwd", forward(router))
    monkeypatch.setattr(binding, "swiglu_clamped_bwd",
                        lambda x, probs, grad, gx, gp, limit: write(swiglu, grad, x, probs, gx, gp))
    monkeypatch.setattr(binding, "router_weight_mul_bwd",
                        lambda grad, x, probs, gx, gp: write(router, grad, x, probs, gx, gp))


def leaves(*shapes):
    torch.manual_seed(0)
    return [torch.randn(s).requires_grad_() for s in shapes]


OPS = {"swiglu": (lambda x, p: binding.SwigluClamped.apply(x, p, LIMIT), swiglu),
       "router": (lambda x, p: binding.RouterWeightMul.apply(x, p), router)}


@pytest.mark.parametrize("name", sorted(OPS))
@pytest.mark.parametrize("needs", [(True, True), (True, False), (False, True)])
def test_first_derivatives_are_the_formulas(name, needs):
    op, formula = OPS[name]
    inputs = [t.detach().requires_grad_(n) for t, n in zip(leaves((6, 8), (6,)), needs)]
    wanted = [t for t in inputs if t.requires_grad]
    got, want = (torch.autograd.grad(f(*inputs).pow(2).sum(), wanted) for f in (op, formula))
    for g, w in zip(got, want):
        assert torch.allclose(g, w, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("name", sorted(OPS))
@pytest.mark.parametrize("power", [1, 2])
def test_a_second_derivative_is_refused(name, power):
    op, _ = OPS[name]
    inputs = leaves((6, 8), (6,))
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(op(*inputs).pow(power).sum(), inputs, create_graph=True)
    if name == "swiglu":                           # not linear in x
        with pytest.raises(RuntimeError, match="first derivatives only"):
            torch.autograd.grad(op(inputs[0], inputs[1].detach()).sum(), inputs[0], create_graph=True)


@pytest.mark.parametrize("name,fixed", [("router", 0), ("router", 1), ("swiglu", 0)])
def test_gradients_that_depend_on_no_input_are_constants_of_a_graph(name, fixed):
    op, formula = OPS[name]
    inputs = leaves((6, 8), (6,))
    inputs[fixed] = inputs[fixed].detach()
    used = inputs[1 - fixed]
    got, want = (torch.autograd.grad(f(*inputs).sum() + used.pow(3).sum(), used, create_graph=True)[0]
                 for f in (op, formula))
    assert torch.allclose(got, want, rtol=1e-5, atol=1e-6)
    got, want = (torch.autograd.grad(g.pow(2).sum(), used)[0] for g in (got, want))
    assert torch.allclose(got, want, rtol=1e-5, atol=1e-5)
