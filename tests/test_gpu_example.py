"""The example of the whole layer runs and checks itself: the 8-bit serving step replayed from a graph, and the
training step's outputs and gradients against autograd of a plain form."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("routed_experts", os.path.join(ROOT, "examples", "routed_experts.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    load().main()
    assert "serving step" in capsys.readouterr().out


@pytest.mark.parametrize("tokens", [1, 7, 200])
def test_serving_step_with_some_experts_elsewhere(tokens):
    """With half of the experts, the slots of the other half have no row and the rows here are the whole layer's,
    bit for bit; so is the output of a token whose experts are all here."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    m = load()
    torch.manual_seed(tokens)
    n, inter, hidden, top_k = 6, 64, 128, 2
    w = [(torch.randn(*s, device="cuda") * s[-1] ** -0.5).bfloat16()
         for s in ((n, inter, hidden), (n, inter, hidden), (n, hidden, inter))]
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    scores, ids = torch.randn(tokens, n, device="cuda").topk(top_k, 1)
    weights = torch.softmax(scores, 1)

    def step(first, last):
        layer = m.Int8Experts(*(p[first:last].contiguous() for p in w), tokens, top_k, first)
        out = torch.empty_like(x)
        layer.step(x, ids, weights, out)
        return layer, out

    whole, want = step(0, n)
    for first, last in ((0, 3), (3, 6)):
        half, out = step(first, last)
        here = (ids >= first) & (ids < last)
        assert torch.equal(half.row_of >= 0, here) and int(half.offs[-1]) == int(here.sum())
        assert torch.equal(half.rows[half.row_of[here].long()], whole.rows[whole.row_of[here].long()])
        assert torch.equal(out[here.all(1)], want[here.all(1)])
        assert bool((out[~here.any(1)] == 0).all())
