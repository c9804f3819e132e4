"""Autograd wrappers of the steps before the experts on the CPU: the kernel calls are replaced by plain writes that
autograd does not see, as it does not see the kernels'. First derivatives are those of the formulas; a second
derivative, which the wrappers do not have, is an error."""
import pytest
import torch

from moe_routed_expert_amd import prologue

EPS = 1e-6


def norm(x, w, r=None):
    h = x if r is None else x + r
    return h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * w, h


def route(logits, ids, renormalise):
    p = torch.softmax(logits, 1).gather(1, ids.long())
    return p / p.sum(1, keepdim=True) if renormalise else p


def gradient(f, inputs, grads):
    with torch.enable_grad():
        leaves = [t.detach().clone().requires_grad_() for t in inputs]
        return torch.autograd.grad(f(*leaves), leaves, grads)


@pytest.fixture(autouse=True)
def kernels(monkeypatch):
    def norm_fwd(x, w, out, eps, residual=None, residual_out=None, q=None, scale=None, rstd=None):
        y, h = norm(x, w, residual)
        out.copy_(y)
        rstd.copy_((h.square().mean(1) + eps).rsqrt())
        if residual_out is not None:
            residual_out.copy_(h)

    def norm_bwd(grad_out, h, w, rstd, grad_x, grad_weight=None, workspace=None, grad_residual=None):
        assert grad_out.is_contiguous() and (grad_residual is None or grad_residual.is_contiguous())
        gx, gw = gradient(lambda h, w: norm(h, w)[0], (h, w), grad_out)
        grad_x.copy_(gx if grad_residual is None else gx + grad_residual)
        if grad_weight is not None:
            assert workspace.numel() == 4
            grad_weight.copy_(gw)

    def logits_fwd(x, w, logits, workspace=None):
        logits.copy_(x @ w.T)

    def logits_bwd(g, x, w, grad_x, grad_weight, workspace=None):
        assert g.is_contiguous()
        if grad_x is not None:
            grad_x.copy_(g @ w)
        if grad_weight is not None:
            grad_weight.copy_(g.T @ x)

    def route_fwd(logits, ids, weights, bias, score, groups, top_groups, group_score, renormalise, scale):
        ids.copy_(logits.argsort(1, descending=True)[:, :ids.shape[1]])
        weights.copy_(scale * route(logits, ids, renormalise))

    def route_bwd(g, logits, ids, grad_logits, score, renormalise, scale):
        assert g.is_contiguous()
        grad_logits.copy_(gradient(lambda l: scale * route(l, ids, renormalise), (logits,), g)[0])

    def quiet(f):
        return lambda *a, **k: torch.no_grad()(f)(*a, **k)

    for name, f in (("rms_norm_fwd", norm_fwd), ("rms_norm_bwd", norm_bwd), ("moe_router_logits_fwd", logits_fwd),
                    ("moe_router_logits_bwd", logits_bwd), ("moe_route_fwd", route_fwd), ("moe_route_bwd", route_bwd)):
        monkeypatch.setattr(prologue, name, quiet(f))
    for name in ("rms_norm_bwd", "moe_router_logits", "moe_router_logits_bwd"):
        monkeypatch.setattr(prologue, name + "_workspace_bytes", lambda *sizes: 4)


OPS = {
    "norm": (lambda x, w: prologue.RmsNorm.apply(x, w, EPS), lambda x, w: norm(x, w)[0], [(4, 6), (6,)]),
    "norm_residual": (lambda x, w, r: prologue.RmsNorm.apply(x, w, EPS, r), lambda x, w, r: norm(x, w, r), [(4, 6), (6,), (4, 6)]),
    "logits": (prologue.MoeRouterLogits.apply, lambda x, w: x @ w.T, [(4, 6), (5, 6)]),
    "route": (lambda l: prologue.MoeRoute.apply(l, 3)[1],
              lambda l: route(l, l.argsort(1, descending=True)[:, :3], True), [(4, 8)]),
    "route_scores": (lambda l: prologue.MoeRoute.apply(l, 3, None, "softmax", 1, 1, "max", False, 2.0)[1],
                     lambda l: 2 * route(l, l.argsort(1, descending=True)[:, :3], False), [(4, 8)]),
}


def leaves(shapes):
    torch.manual_seed(0)
    return [torch.randn(s, dtype=torch.float32).requires_grad_() for s in shapes]


def loss(out):
    return sum(o.pow(3).sum() for o in (out if isinstance(out, tuple) else (out,)))


@pytest.mark.parametrize("name", sorted(OPS))
def test_first_derivatives_are_the_formulas(name):
    op, formula, shapes = OPS[name]
    inputs = leaves(shapes)
    got, want = (torch.autograd.grad(loss(f(*inputs)), inputs) for f in (op, formula))
    for g, w in zip(got, want):
        assert torch.allclose(g, w, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("name", sorted(OPS))
def test_each_input_may_be_fixed_and_strided(name):
    """Gradients of sums have stride 0, and inputs may be transposed; an input that needs no gradient gets none."""
    op, formula, shapes = OPS[name]
    for only in range(len(shapes)):
        inputs = [t.detach() for t in leaves([s[::-1] for s in shapes])]
        inputs[only].requires_grad_()
        used = [t.t() if t.dim() == 2 else t for t in inputs]
        got, want = (torch.autograd.grad(sum(o.sum() for o in (r if isinstance(r, tuple) else (r,))), inputs[only])[0]
                     for r in (f(*used) for f in (op, formula)))
        assert torch.allclose(got, want, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("name", sorted(OPS))
def test_a_second_derivative_is_refused(name):
    op, _, shapes = OPS[name]
    inputs = leaves(shapes)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(loss(op(*inputs)), inputs, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        loss(op(*inputs)).backward(create_graph=True)


def test_a_sum_alone_passes_its_gradient_on():
    """The normed rows unused: the gradient of x + residual, which has every further derivative."""
    x, w, r = leaves([(4, 6), (6,), (4, 6)])
    h = prologue.RmsNorm.apply(x, w, EPS, r)[1]
    gx, gr = torch.autograd.grad(h.pow(2).sum(), (x, r), create_graph=True)
    assert torch.allclose(gx, 2 * h) and torch.allclose(gr, 2 * h)


def test_a_linear_products_gradient_may_be_part_of_a_graph():
    """With the weight fixed the gradient of x does not depend on x."""
    x, w = leaves([(4, 6), (5, 6)])
    out = prologue.MoeRouterLogits.apply(x, w.detach()).sum() + x.pow(3).sum()
    g, = torch.autograd.grad(out, x, create_graph=True)
    again, = torch.autograd.grad(g.pow(2).sum(), x)
    want = torch.autograd.grad((w.detach().sum(0) + 3 * x.pow(2)).pow(2).sum(), x)[0]
    assert torch.allclose(again, want, rtol=1e-4, atol=1e-4)


def test_the_ids_have_no_gradient():
    logits, = leaves([(4, 8)])
    ids, w = prologue.MoeRoute.apply(logits, 2)
    assert not ids.requires_grad and w.requires_grad and ids.dtype == torch.int32
