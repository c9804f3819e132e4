"""Refusals of the calls in include/moe_prologue.h, on the CPU: every call here fails validation (or has
nothing to do), so nothing is launched and the addresses are never used."""
import os
import re

import pytest
import torch

from moe_routed_expert_amd import binding, prologue
from tests.test_current_gpu_cpu import Stream, gpus  # noqa: F401
from tests.test_routed_abi_cpu import ALIAS, DTYPE, LIMIT, MISAL, NULLP, OK, SHAPE, P, Tensor, expect

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="host-only checks; a GPU is visible")
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from moe_routed_expert_amd import build
        build.build()
    return prologue._lib()


def calls(L):
    """name -> (function of keyword arguments, its defaults)."""
    def norm(x=P[0], r=P[1], dt=0, w=P[2], wdt=0, eps=1e-6, out=P[3], h=P[4], q=P[5], s=P[6], n=P[7], rows=16, cols=24):
        return L.rms_norm_fwd(x, r, dt, w, wdt, eps, out, h, q, s, n, rows, cols, None)

    def norm_bwd(g=P[0], h=P[1], dt=0, w=P[2], wdt=0, n=P[3], gh=P[4], gx=P[5], gw=P[6], ws=P[7], nbytes=1 << 30, rows=16,
                 cols=24):
        return L.rms_norm_bwd(g, h, dt, w, wdt, n, gh, gx, gw, ws, nbytes, rows, cols, None)

    def logits(x=P[0], dt=0, w=P[1], wdt=0, l=P[2], ws=P[3], nbytes=1 << 30, tokens=16, hidden=24, experts=8):  # noqa: E741
        return L.moe_router_logits_fwd(x, dt, w, wdt, l, ws, nbytes, tokens, hidden, experts, None)

    def logits_bwd(g=P[0], x=P[1], dt=0, w=P[2], wdt=0, gx=P[3], gw=P[4], ws=P[5], nbytes=1 << 30, tokens=16, hidden=24,
                   experts=8):
        return L.moe_router_logits_bwd(g, x, dt, w, wdt, gx, gw, ws, nbytes, tokens, hidden, experts, None)

    def route(l=P[0], dt=2, b=P[1], i=P[2], w=P[3], tokens=16, experts=24, top_k=4, groups=4, top_groups=2, score=0, group=0,  # noqa: E741
              renorm=1, scale=1.0):
        return L.moe_route_fwd(l, dt, b, i, w, tokens, experts, top_k, groups, top_groups, score, group, renorm, scale, None)

    def route_bwd(g=P[0], l=P[1], dt=2, i=P[2], gl=P[3], tokens=16, experts=24, top_k=4, score=0, renorm=1, scale=1.0):  # noqa: E741
        return L.moe_route_bwd(g, l, dt, i, gl, tokens, experts, top_k, score, renorm, scale, None)

    return locals()


TYPES = [{"dt": 3}, {"dt": -1}, {"wdt": 3}, {"dt": 0, "wdt": 1}, {"dt": 1, "wdt": 0}, {"dt": 2, "wdt": 0}]


def test_norm(L):
    f, b = calls(L)["norm"], calls(L)["norm_bwd"]
    shapes = [{"rows": -1}, {"cols": 0}, {"cols": 2 ** 30}, {"rows": 2 ** 61}]
    for g in (f, b):
        expect(g, DTYPE, *TYPES)
        expect(g, SHAPE, *shapes)
    expect(f, LIMIT, *({"eps": e} for e in (-1e-6, NAN, INF, -INF)))
    expect(f, NULLP, {"x": None}, {"w": None}, {"out": None, "q": None, "s": None}, {"q": None}, {"s": None}, {"r": None})
    expect(f, MISAL, {"x": P[0] + 1}, {"r": P[1] + 1}, {"w": P[2] + 1}, {"out": P[3] + 1}, {"h": P[4] + 1}, {"s": P[6] + 2},
           {"n": P[7] + 2}, {"wdt": 2, "w": P[2] + 2})
    expect(f, ALIAS, *({o: P[i] + 16} for o in ("out", "h", "q", "s", "n") for i in range(3)), {"h": P[0]}, {"out": P[1]},
           {"h": P[1] + 2}, {"out": P[4]}, {"q": P[3]}, {"s": P[5]}, {"n": P[6]}, {"h": P[1], "out": P[1]})
    expect(f, OK, {"rows": 0}, {"rows": 0, "x": None, "w": None, "out": None, "q": None, "s": None, "r": None, "h": None},
           {"rows": 0, "eps": 0.0})
    expect(b, NULLP, *({k: None} for k in ("g", "h", "w", "n", "gx", "ws")))
    need = prologue.rms_norm_bwd_workspace_bytes(16, 24)
    expect(b, SHAPE, {"nbytes": need - 1}, {"nbytes": 0})
    expect(b, MISAL, {"g": P[0] + 1}, {"h": P[1] + 1}, {"w": P[2] + 1}, {"n": P[3] + 2}, {"gh": P[4] + 1}, {"gx": P[5] + 1},
           {"gw": P[6] + 1}, {"ws": P[7] + 8}, {"wdt": 2, "gw": P[6] + 2})
    expect(b, ALIAS, *({o: P[i]} for o in ("gx", "gw", "ws") for i in range(5)), {"gw": P[5]}, {"ws": P[5]}, {"ws": P[6]})
    expect(b, OK, {"rows": 0, "gw": None}, {"rows": 0, "gw": None, "ws": None, "nbytes": 0, "g": None, "gx": None})
    assert prologue.rms_norm_bwd_workspace_bytes(0, 24) > 0
    for bad in ((-1, 4), (4, 0), (2 ** 61, 4), (1, 2 ** 30)):
        assert L.rms_norm_bwd_workspace_bytes(*bad) == -1
        with pytest.raises(ValueError):
            prologue.rms_norm_bwd_workspace_bytes(*bad)


def test_logits(L):
    f, b = calls(L)["logits"], calls(L)["logits_bwd"]
    for g in (f, b):
        expect(g, DTYPE, *TYPES)
        expect(g, SHAPE, {"tokens": -1}, {"tokens": 2 ** 31}, {"hidden": 0}, {"hidden": 2 ** 30}, {"experts": 0},
               {"experts": 1025})
    expect(f, NULLP, {"x": None}, {"w": None}, {"l": None})
    expect(f, MISAL, {"x": P[0] + 1}, {"w": P[1] + 1}, {"l": P[2] + 2}, {"wdt": 2, "w": P[1] + 2})
    expect(f, ALIAS, {"l": P[0]}, {"l": P[1] + 16})
    expect(f, OK, {"tokens": 0}, {"tokens": 0, "x": None, "l": None})
    expect(b, NULLP, {"g": None}, {"x": None}, {"w": None}, {"gx": None, "gw": None})
    expect(b, MISAL, {"g": P[0] + 2}, {"x": P[1] + 1}, {"w": P[2] + 1}, {"gx": P[3] + 1}, {"gw": P[4] + 1})
    expect(b, ALIAS, *({o: P[i] + 16} for o in ("gx", "gw") for i in range(3)), {"gw": P[3]})
    expect(b, OK, {"tokens": 0, "gw": None})
    # a call whose workspace is too small, absent, misaligned or something else's
    for g, need, sizes in ((f, prologue.moe_router_logits_workspace_bytes, (32, 7168, 64)),
                           (b, prologue.moe_router_logits_bwd_workspace_bytes, (4096, 2048, 64))):
        at = dict(zip(("tokens", "hidden", "experts"), sizes))
        n = need(*sizes)
        assert n >= 0
        if n:
            expect(g, SHAPE, {"nbytes": n - 1, **at})
            expect(g, NULLP, {"ws": None, **at})
            expect(g, MISAL, {"ws": P[5] + 8, **at})
            expect(g, ALIAS, {"ws": P[0], **at}, {"ws": P[1], **at}, {"ws": P[2], **at})
    for need in ("moe_router_logits_workspace_bytes", "moe_router_logits_bwd_workspace_bytes"):
        for bad in ((-1, 4, 4), (4, 0, 4), (4, 4, 0), (4, 4, 1025), (2 ** 31, 4, 4), (1, 2 ** 30, 4)):
            assert getattr(L, need)(*bad) == -1
            with pytest.raises(ValueError):
                getattr(prologue, need)(*bad)


def test_route(L):
    f, b = calls(L)["route"], calls(L)["route_bwd"]
    for g in (f, b):
        expect(g, DTYPE, {"dt": 3}, {"dt": -1}, {"score": 2}, {"score": -1})
        expect(g, SHAPE, {"tokens": -1}, {"tokens": 2 ** 31}, {"experts": 0}, {"experts": 1028}, {"top_k": 0}, {"top_k": 25},
               {"top_k": 65, "experts": 256})
        expect(g, LIMIT, {"scale": NAN}, {"scale": INF}, {"scale": -INF})
    expect(f, DTYPE, {"group": 2}, {"group": -1})
    expect(f, SHAPE, {"groups": 0}, {"groups": 5}, {"groups": 65, "experts": 130}, {"top_groups": 0}, {"top_groups": 5},
           {"top_k": 13}, {"groups": 24, "group": 1, "top_groups": 24})
    expect(f, NULLP, {"l": None}, {"i": None}, {"w": None})
    expect(f, MISAL, {"l": P[0] + 2}, {"b": P[1] + 2}, {"i": P[2] + 2}, {"w": P[3] + 2}, {"dt": 0, "l": P[0] + 1})
    expect(f, ALIAS, {"i": P[0]}, {"i": P[1]}, {"w": P[0] + 4}, {"w": P[1]}, {"w": P[2]})
    expect(f, OK, {"tokens": 0}, {"tokens": 0, "l": None, "i": None, "w": None, "b": None})
    expect(b, NULLP, *({k: None} for k in ("g", "l", "i", "gl")))
    expect(b, MISAL, {"g": P[0] + 2}, {"l": P[1] + 2}, {"i": P[2] + 2}, {"gl": P[3] + 2})
    expect(b, ALIAS, {"gl": P[0]}, {"gl": P[1]}, {"gl": P[2] + 4})
    expect(b, OK, {"tokens": 0})


def test_header_and_binding_name_the_same_calls(L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "moe_prologue.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert len(names) == 9
    for name in names:
        assert getattr(L, name).argtypes is not None and hasattr(prologue, name)


# ---- what the binding passes on ---------------------------------------------------------

I32, F32, I8, U8, BF16 = torch.int32, torch.float32, torch.int8, torch.uint8, torch.bfloat16
# call -> (its tensors by name, in order, and the other arguments)
TENSORS = {
    "rms_norm_fwd": ({"x": ((6, 16), BF16), "weight": ((16,), BF16), "out": ((6, 16), BF16), "residual": ((6, 16), BF16),
                      "residual_out": ((6, 16), BF16), "q": ((6, 16), I8), "scale": ((6,), F32), "rstd": ((6,), F32)},
                     {"eps": 1e-6}),
    "rms_norm_bwd": ({"grad_out": ((6, 16), BF16), "h": ((6, 16), BF16), "weight": ((16,), BF16), "rstd": ((6,), F32),
                      "grad_x": ((6, 16), BF16), "grad_weight": ((16,), BF16), "workspace": ((64,), U8),
                      "grad_residual": ((6, 16), BF16)}, {}),
    "moe_router_logits_fwd": ({"x": ((6, 16), BF16), "weight": ((4, 16), BF16), "logits": ((6, 4), F32),
                               "workspace": ((64,), U8)}, {}),
    "moe_router_logits_bwd": ({"grad_logits": ((6, 4), F32), "x": ((6, 16), BF16), "weight": ((4, 16), BF16),
                               "grad_x": ((6, 16), BF16), "grad_weight": ((4, 16), BF16), "workspace": ((64,), U8)}, {}),
    "moe_route_fwd": ({"logits": ((6, 8), BF16), "ids": ((6, 2), I32), "weights": ((6, 2), F32), "bias": ((8,), F32)}, {}),
    "moe_route_bwd": ({"grad_weights": ((6, 2), F32), "logits": ((6, 8), BF16), "ids": ((6, 2), I32),
                       "grad_logits": ((6, 8), BF16)}, {}),
}
OPTIONAL = {"rms_norm_fwd": {"residual_out", "rstd"}, "rms_norm_bwd": {"grad_weight", "workspace", "grad_residual"},
            "moe_router_logits_fwd": {"workspace"}, "moe_router_logits_bwd": {"grad_x", "grad_weight", "workspace"},
            "moe_route_fwd": {"bias"}, "moe_route_bwd": set()}
# sizes that only the tensor itself has
FREE = {("workspace", 0)}


@pytest.fixture
def reached(monkeypatch):
    found = []

    class Library:
        def __getattr__(self, call):
            return lambda *args: found.append((call, args)) or 0

    monkeypatch.setattr(prologue, "_fns", Library())
    monkeypatch.setattr(prologue, "_raw_stream", lambda device: 0)
    return found


def made(name):
    return {n: Tensor(*s) for n, s in TENSORS[name][0].items()}


@pytest.mark.parametrize("name", sorted(TENSORS))
def test_binding_passes_only_tensors_that_fit(name, reached):
    specs, others = TENSORS[name]
    call = getattr(prologue, name)
    call(**made(name), **others)
    assert [c for c, _ in reached] == [name]
    assert all(a == 4096 for a in reached[0][1] if isinstance(a, int) and a > 1000)
    assert sum(a == 4096 for a in reached[0][1] if isinstance(a, int)) == len(specs)
    for n, (shape, dtype) in specs.items():
        wrong = [Tensor(shape, torch.float64), Tensor(shape, dtype, device=1), Tensor(shape, dtype, device=-1),
                 Tensor(shape, dtype, contiguous=False), Tensor(shape + (1,), dtype)]
        wrong += [Tensor(shape[:d] + (shape[d] + 1,) + shape[d + 1:], dtype) for d in range(len(shape)) if (n, d) not in FREE]
        for bad in wrong:
            with pytest.raises((TypeError, ValueError)):
                call(**{**made(name), n: bad}, **others)
                raise AssertionError(f"{name}: {n} passed with {bad.shape} {bad.dtype} {bad.device}")
    tensors = made(name)
    for t in tensors.values():
        t.index = -1                               # all of them on the CPU
    with pytest.raises((TypeError, ValueError)):
        call(**tensors, **others)
    assert len(reached) == 1                       # the library was never reached again


@pytest.mark.parametrize("name", sorted(TENSORS))
def test_binding_names_a_tensor_that_is_missing(name, reached):
    for n in TENSORS[name][0]:
        args = {**made(name), n: None, **TENSORS[name][1]}
        if n in OPTIONAL[name]:
            getattr(prologue, name)(**args)
        elif name == "rms_norm_fwd" and n == "out":
            getattr(prologue, name)(**args)        # the 8-bit rows are there
            with pytest.raises(ValueError, match="out is required"):
                getattr(prologue, name)(**{**args, "q": None, "scale": None})
        elif name == "rms_norm_fwd" and n in ("q", "scale", "residual"):
            with pytest.raises(ValueError, match="go"):
                getattr(prologue, name)(**args)
        else:
            with pytest.raises(ValueError, match=f"{n} is required"):
                getattr(prologue, name)(**args)
    if name == "moe_router_logits_bwd":
        with pytest.raises(ValueError, match="grad_x or grad_weight"):
            prologue.moe_router_logits_bwd(**{**made(name), "grad_x": None, "grad_weight": None})


@pytest.mark.parametrize("name", sorted(TENSORS))
def test_tensors_of_another_gpu(name, gpus, monkeypatch):  # noqa: F811
    """The call makes the tensors' GPU the current one, and takes no stream of another."""
    monkeypatch.setattr(prologue, "_fns", binding._lib)
    monkeypatch.setattr(prologue, "_raw_stream", lambda device: 0)
    tensors = made(name)
    for t in tensors.values():
        t.index = 1
    getattr(prologue, name)(**tensors, **TENSORS[name][1])
    assert gpus.calls[-1][0] == 1 and gpus.current == 0
    with pytest.raises(ValueError, match="stream is on GPU 0"):
        getattr(prologue, name)(**tensors, **TENSORS[name][1], stream=Stream(0))


def test_words_that_are_no_score(reached):
    t = made("moe_route_fwd")
    for bad in ({"score": "tanh"}, {"score": 0}, {"group_score": "sum"}):
        with pytest.raises(ValueError, match="expected one of"):
            prologue.moe_route_fwd(**t, **bad)
    with pytest.raises(ValueError, match="expected one of"):
        prologue.moe_route_bwd(**made("moe_route_bwd"), score=None)
    assert not reached


def test_weights_of_another_type(reached):
    """A weight is of the rows' type or float32."""
    x, out = torch.zeros(4, 8, dtype=BF16), torch.zeros(4, 8, dtype=BF16)
    with pytest.raises(TypeError, match="weight"):
        prologue.rms_norm_fwd(x, torch.zeros(8, dtype=torch.float16), out, 1e-6)
    with pytest.raises(TypeError, match="weight"):
        prologue.moe_router_logits_fwd(x, torch.zeros(2, 8, dtype=torch.float16), torch.zeros(4, 2))
    with pytest.raises(TypeError):
        prologue.rms_norm_fwd(x.double(), torch.zeros(8), out, 1e-6)
    assert not reached


def test_helpers_take_rows_of_any_shape(monkeypatch):
    got = []
    monkeypatch.setattr(prologue, "rms_norm_fwd", lambda *a, **k: got.append((a, k)))
    x, r = torch.arange(48.0).view(2, 3, 8).transpose(0, 1), torch.ones(3, 2, 8)
    y, h = prologue.rms_norm(x, torch.ones(8), 1e-6, r)
    assert y.shape == h.shape == x.shape and got[0][0][0].is_contiguous() and torch.equal(got[0][0][0], x.reshape(6, 8))
    assert prologue.rms_norm(x, torch.ones(8), 1e-6).shape == x.shape
    q, scale = prologue.rms_norm_int8(x, torch.ones(8), 1e-6)
    assert q.shape == x.shape and scale.shape == (3, 2) and q.dtype == I8
    assert [t.shape for t in prologue.rms_norm_int8(x[0, 0], torch.ones(8), 1e-6, r[0, 0])] == [(8,), (), (8,)]
    for bad in (r[:1], r[..., :4]):
        with pytest.raises(ValueError, match="residual"):
            prologue.rms_norm(x, torch.ones(8), 1e-6, bad)
    with pytest.raises(ValueError):
        prologue.rms_norm(torch.tensor(1.0), torch.ones(1), 1e-6)
