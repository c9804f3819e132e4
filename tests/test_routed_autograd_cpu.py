"""Autograd wrappers of the routed steps on the CPU: the kernel calls are replaced by plain writes that autograd does
not see, as it does not see the kernels'. First derivatives are those of the formulas; a second derivative, which the
wrappers do not have, is an error and not a gradient with its second-order terms missing."""
import pytest
import torch

from moe_routed_expert_amd import routed

ROW_OF = torch.tensor([[0, 3], [-1, 1], [2, -1], [-1, -1]], dtype=torch.int32)
SLOT_OF = torch.tensor([0, 3, 4, 1], dtype=torch.int32)


def dispatch(x):
    return x[SLOT_OF.long() // 2]


def dispatch_grad(g):
    return (g[ROW_OF.clamp(min=0).long()] * (ROW_OF >= 0)[..., None]).sum(1)


def combine(rows, weights):
    return (rows[ROW_OF.clamp(min=0).long()] * (weights * (ROW_OF >= 0))[..., None]).sum(1)


@pytest.fixture(autouse=True)
def kernels(monkeypatch):
    def dispatch_fwd(x, slot_of, top_k, out):
        with torch.no_grad():
            out.copy_(dispatch(x))

    def dispatch_bwd(grad_out, row_of, grad_x):
        with torch.no_grad():
            grad_x.copy_(dispatch_grad(grad_out))

    def combine_fwd(rows, row_of, weights, out):
        with torch.no_grad():
            out.copy_(combine(rows, weights))

    def combine_bwd(grad, rows, row_of, weights, grad_rows, grad_weights):
        with torch.no_grad():
            slot = SLOT_OF.long()
            grad_rows.copy_(grad[slot // 2] * weights.reshape(-1)[slot, None])
            if grad_weights is not None:
                grad_weights.zero_()
                grad_weights.view(-1)[slot] = (grad[slot // 2] * rows).sum(1)

    for name, f in (("moe_dispatch_fwd", dispatch_fwd), ("moe_dispatch_bwd", dispatch_bwd),
                    ("moe_combine_weighted_fwd", combine_fwd), ("moe_combine_weighted_bwd", combine_bwd)):
        monkeypatch.setattr(routed, name, f)


def leaves(*shapes):
    torch.manual_seed(0)
    return [torch.randn(s, dtype=torch.float32).requires_grad_() for s in shapes]


# what is applied, the formula, and the shapes of the inputs
OPS = {"dispatch": (lambda x: routed.MoeDispatch.apply(x, ROW_OF, SLOT_OF), dispatch, [(4, 5)]),
       "combine": (lambda r, w: routed.MoeCombineWeighted.apply(r, ROW_OF, w), combine, [(4, 5), (4, 2)])}


@pytest.mark.parametrize("name", sorted(OPS))
def test_first_derivatives_are_the_formulas(name):
    op, formula, shapes = OPS[name]
    inputs = leaves(*shapes)
    got, want = (torch.autograd.grad(f(*inputs).pow(2).sum(), inputs) for f in (op, formula))
    for g, w in zip(got, want):
        assert torch.allclose(g, w, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("name", sorted(OPS))
@pytest.mark.parametrize("strided", [False, True])
def test_a_second_derivative_is_refused(name, strided):
    op, _, shapes = OPS[name]
    inputs = leaves(*(s[::-1] if strided else s for s in shapes))
    used = [t.t() for t in inputs] if strided else inputs
    out = op(*used)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(out.pow(2).sum(), inputs, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        op(*used).pow(2).sum().backward(create_graph=True)


def test_gradients_that_depend_on_an_input_are_refused_and_others_are_right():
    """Of a sum: the combine's gradients depend on its inputs all the same, the dispatch's do not, nor does that of
    the rows alone; those may be part of a graph, as constants."""
    rows, weights = leaves((4, 5), (4, 2))
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(OPS["combine"][0](rows, weights).sum(), [rows, weights], create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad(OPS["combine"][0](rows, weights).sum(), [weights], create_graph=True)
    for name, used, fixed in (("dispatch", rows, ()), ("combine", rows, (weights.detach(),))):
        op, formula, _ = OPS[name]
        got, want = (torch.autograd.grad(f(used, *fixed).sum() + used.pow(3).sum(), used, create_graph=True)[0]
                     for f in (op, formula))
        assert torch.allclose(got, want, rtol=1e-5, atol=1e-6)
        got, want = (torch.autograd.grad(g.pow(2).sum(), used)[0] for g in (got, want))
        assert torch.allclose(got, want, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("tokens", [3, 5])
def test_a_dispatch_of_other_tokens_than_the_orders_is_refused(tokens):
    """Its backward pass would be refused; the forward pass alone must not answer with other tokens' rows."""
    x, = leaves((tokens, 5))
    with pytest.raises(ValueError, match=f"row_of.*{tokens}"):
        routed.MoeDispatch.apply(x, ROW_OF, SLOT_OF)
    with pytest.raises(ValueError, match="row_of"):
        routed.MoeDispatch.apply(x.detach(), ROW_OF, SLOT_OF)
