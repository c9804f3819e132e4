"""Refusals of the calls in include/moe_routed.h, on the CPU: every call here fails validation (or has
nothing to do), so nothing is launched and the addresses are never used."""
import os

import pytest
import torch

from moe_routed_expert_amd import binding, routed

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="host-only checks; a GPU is visible")

OK, NULLP, SHAPE, LIMIT, ALIAS, LAUNCH, MISAL, DTYPE = range(8)
P = [i << 36 for i in range(1, 16)]               # far apart, aligned


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from moe_routed_expert_amd import build
        build.build()
    return routed._lib()


def calls(L):
    """name -> (function of keyword arguments, its defaults)."""
    def sort(ids=P[0], id_bytes=4, first=0, offs=P[1], row=P[2], slot=P[3], ws=P[4], nbytes=1 << 20, tokens=64,
             top_k=4, experts=8):
        return L.moe_sort_fwd(ids, id_bytes, first, offs, row, slot, ws, nbytes, tokens, top_k, experts, None)

    def dispatch(x=P[0], dt=0, slot=P[1], out=P[2], rows=32, tokens=16, top_k=2, hidden=24):
        return L.moe_dispatch_fwd(x, dt, slot, out, rows, tokens, top_k, hidden, None)

    def dispatch_bwd(g=P[0], dt=0, row=P[1], gx=P[2], rows=32, tokens=16, top_k=2, hidden=24):
        return L.moe_dispatch_bwd(g, dt, row, gx, rows, tokens, top_k, hidden, None)

    def combine(eo=P[0], dt=0, row=P[1], w=P[2], out=P[3], odt=0, rows=32, tokens=16, top_k=2, hidden=24):
        return L.moe_combine_weighted_fwd(eo, dt, row, w, out, odt, rows, tokens, top_k, hidden, None)

    def combine_bwd(go=P[0], gdt=0, eo=P[1], dt=0, row=P[2], w=P[3], ge=P[4], gw=P[5], rows=32, tokens=16, top_k=2,
                    hidden=24):
        return L.moe_combine_weighted_bwd(go, gdt, eo, dt, row, w, ge, gw, rows, tokens, top_k, hidden, None)

    def quantize(x=P[0], dt=0, q=P[1], s=P[2], rows=16, cols=24):
        return L.quantize_rows_int8_fwd(x, dt, q, s, rows, cols, None)

    def gate_up(a=P[0], sa=P[1], slot=P[2], wg=P[3], sg=P[4], wu=P[5], su=P[6], offs=P[7], p=P[8], y=P[9], rows=32,
                tokens=16, top_k=2, hidden=64, inter=24, experts=4, limit=7.0):
        return L.grouped_gate_up_swiglu_int8_fwd(a, sa, slot, wg, sg, wu, su, offs, p, y, rows, tokens, top_k, hidden,
                                                 inter, experts, limit, None)

    def down(h=P[0], sh=P[1], w=P[2], sw=P[3], offs=P[4], p=P[5], out=P[6], odt=0, rows=32, inter=64, hidden=24,
             experts=4):
        return L.grouped_down_router_int8_fwd(h, sh, w, sw, offs, p, out, odt, rows, inter, hidden, experts, None)

    return locals()


def expect(f, status, *changes):
    for kw in changes:
        assert f(**kw) == status, (f.__name__, kw)


def test_sort(L):
    f = calls(L)["sort"]
    expect(f, DTYPE, {"id_bytes": 2}, {"id_bytes": 0})
    expect(f, SHAPE, {"tokens": -1}, {"top_k": 0}, {"top_k": 1025}, {"experts": 0}, {"experts": 1025},
           {"tokens": 2 ** 31}, {"tokens": 2 ** 29, "top_k": 4}, {"tokens": 2 ** 62, "top_k": 1024},
           {"tokens": 9000, "nbytes": 0})
    expect(f, NULLP, {"ids": None}, {"offs": None}, {"row": None}, {"slot": None},
           {"ws": None, "tokens": 9000})
    expect(f, MISAL, {"ids": P[0] + 2}, {"id_bytes": 8, "ids": P[0] + 4}, {"offs": P[1] + 2}, {"row": P[2] + 1},
           {"slot": P[3] + 2}, {"ws": P[4] + 2})
    expect(f, ALIAS, {"offs": P[0]}, {"row": P[0] + 64}, {"slot": P[2]}, {"slot": P[1] + 16},
           {"ws": P[3], "tokens": 9000})
    assert L.moe_sort_workspace_bytes(16, 4, 8) == 0 and L.moe_sort_workspace_bytes(1 << 20, 8, 64) > 0
    for bad in ((-1, 4, 8), (16, 0, 8), (16, 4, 0), (16, 4, 5000), (2 ** 40, 8, 8)):
        assert L.moe_sort_workspace_bytes(*bad) == -1
        with pytest.raises(ValueError):
            routed.moe_sort_workspace_bytes(*bad)


def test_dispatch(L):
    f, b = calls(L)["dispatch"], calls(L)["dispatch_bwd"]
    shapes = [{"rows": -1}, {"tokens": -1}, {"top_k": 0}, {"top_k": 1025}, {"hidden": 0}, {"hidden": 2 ** 30},
              {"rows": 2 ** 31}, {"tokens": 2 ** 31}]
    for g in (f, b):
        expect(g, DTYPE, {"dt": 3}, {"dt": -1})
        expect(g, SHAPE, *shapes)
    expect(f, NULLP, {"x": None}, {"slot": None}, {"out": None})
    expect(f, MISAL, {"x": P[0] + 1}, {"out": P[2] + 1}, {"slot": P[1] + 2}, {"dt": 2, "x": P[0] + 2})
    expect(f, ALIAS, {"out": P[0] + 16}, {"out": P[1] - 2})
    expect(f, OK, {"rows": 0}, {"rows": 0, "x": None, "slot": None, "out": None})
    expect(b, NULLP, {"g": None}, {"row": None}, {"gx": None})
    expect(b, MISAL, {"g": P[0] + 1}, {"gx": P[2] + 1}, {"row": P[1] + 2})
    expect(b, ALIAS, {"gx": P[0] + 16}, {"gx": P[1] - 2})
    expect(b, OK, {"tokens": 0}, {"tokens": 0, "g": None, "row": None, "gx": None})


def test_combine(L):
    f, b = calls(L)["combine"], calls(L)["combine_bwd"]
    shapes = [{"rows": -1}, {"tokens": -1}, {"top_k": 0}, {"top_k": 1025}, {"hidden": 0}, {"rows": 2 ** 31}]
    expect(f, DTYPE, {"dt": 3}, {"odt": 3}, {"dt": 0, "odt": 1}, {"dt": 1, "odt": 0}, {"dt": 2, "odt": 0})
    expect(b, DTYPE, {"dt": 3}, {"gdt": 3}, {"dt": 0, "gdt": 1}, {"dt": 2, "gdt": 0})
    for g in (f, b):
        expect(g, SHAPE, *shapes)
    expect(f, NULLP, {"eo": None}, {"row": None}, {"w": None}, {"out": None})
    expect(f, MISAL, {"eo": P[0] + 1}, {"row": P[1] + 2}, {"w": P[2] + 2}, {"out": P[3] + 1},
           {"odt": 2, "out": P[3] + 2})
    expect(f, ALIAS, {"out": P[0]}, {"out": P[1]}, {"out": P[2] + 4})
    expect(f, OK, {"tokens": 0})
    expect(b, NULLP, {"go": None}, {"eo": None}, {"row": None}, {"w": None}, {"ge": None})
    expect(b, MISAL, {"go": P[0] + 1}, {"eo": P[1] + 1}, {"row": P[2] + 1}, {"w": P[3] + 2}, {"ge": P[4] + 1},
           {"gw": P[5] + 2})
    expect(b, ALIAS, {"ge": P[0]}, {"ge": P[1]}, {"ge": P[2]}, {"gw": P[3]}, {"gw": P[4] + 8}, {"gw": P[0] + 8})
    expect(b, OK, {"tokens": 0})


def test_quantize(L):
    f = calls(L)["quantize"]
    expect(f, DTYPE, {"dt": 5})
    expect(f, SHAPE, {"rows": -1}, {"cols": 0}, {"cols": 2 ** 30}, {"rows": 2 ** 61})
    expect(f, NULLP, {"x": None}, {"q": None}, {"s": None})
    expect(f, MISAL, {"x": P[0] + 1}, {"s": P[2] + 2}, {"dt": 2, "x": P[0] + 2})
    expect(f, ALIAS, {"q": P[0] + 3}, {"s": P[0]}, {"s": P[1]})
    expect(f, OK, {"rows": 0})


def test_products(L):
    f, d = calls(L)["gate_up"], calls(L)["down"]
    expect(f, SHAPE, {"rows": -1}, {"rows": 2 ** 31}, {"tokens": -1}, {"top_k": 0}, {"hidden": 0}, {"hidden": 72},
           {"hidden": 131072}, {"inter": 0}, {"inter": 20}, {"experts": 0}, {"experts": 2 ** 62},
           {"slot": None}, {"slot": None, "tokens": 32}, {"tokens": 2 ** 31}, {"tokens": 2 ** 30, "top_k": 2})
    for limit in (0.0, -1.0, float("inf"), float("nan")):
        assert f(limit=limit) == LIMIT
    expect(f, NULLP, *({k: None} for k in ("a", "sa", "wg", "sg", "wu", "su", "offs", "y")))
    expect(f, MISAL, {"a": P[0] + 8}, {"sa": P[1] + 2}, {"slot": P[2] + 2}, {"wg": P[3] + 4}, {"sg": P[4] + 1},
           {"wu": P[5] + 8}, {"su": P[6] + 2}, {"offs": P[7] + 2}, {"p": P[8] + 2}, {"y": P[9] + 2})
    expect(f, ALIAS, *({"y": P[i]} for i in range(9)))
    expect(f, OK, {"rows": 0}, {"rows": 0, "a": None, "y": None})
    expect(d, DTYPE, {"odt": 1}, {"odt": 3})
    expect(d, SHAPE, {"rows": -1}, {"inter": 72}, {"inter": 131072}, {"inter": 0}, {"hidden": 20}, {"hidden": 0},
           {"experts": 0}, {"experts": 2 ** 62})
    expect(d, NULLP, *({k: None} for k in ("h", "sh", "w", "sw", "offs", "out")))
    expect(d, MISAL, {"h": P[0] + 8}, {"sh": P[1] + 2}, {"w": P[2] + 4}, {"sw": P[3] + 1}, {"offs": P[4] + 2},
           {"p": P[5] + 1}, {"out": P[6] + 8})
    expect(d, ALIAS, *({"out": P[i]} for i in range(6)))
    expect(d, OK, {"rows": 0})


def test_gate_up_without_tokens_still_has_rows_to_write(L):
    """A call of no tokens writes rows of zeros: it needs its other tensors and takes no shortcut around their checks."""
    f = calls(L)["gate_up"]
    expect(f, NULLP, *({"tokens": 0, "a": None, "sa": None, k: None} for k in ("wg", "sg", "wu", "su", "offs", "y")))
    expect(f, MISAL, {"tokens": 0, "y": P[9] + 2})
    expect(f, ALIAS, {"tokens": 0, "y": P[3]})
    expect(f, OK, {"tokens": 0, "rows": 0})


def test_binding_refuses_tensors_the_calls_cannot_take():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    i = torch.zeros(8, dtype=torch.int32)
    r = torch.zeros(4, 2, dtype=torch.int32)
    f = torch.zeros(4, 2)
    w8, s8 = torch.zeros(2, 16, 32, dtype=torch.int8), torch.zeros(2, 16)
    with pytest.raises(ValueError):                # CPU tensors
        routed.moe_dispatch_fwd(x, i, 2, torch.zeros(8, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        routed.moe_sort_fwd(r, 0, i, r, i)
    with pytest.raises(ValueError):
        routed.moe_sort_fwd(i, 0, i, r, i)         # ids must be 2-D
    with pytest.raises(TypeError):
        routed.moe_sort_fwd(f, 0, i, r, i)         # ids must be whole numbers
    with pytest.raises(ValueError):
        routed.moe_combine_weighted_fwd(x, r, f, x)
    with pytest.raises(TypeError):
        routed.moe_combine_weighted_fwd(x.double(), r, f, x)
    with pytest.raises(ValueError):
        routed.moe_combine_weighted_bwd(x, x, r, f, x, f)
    with pytest.raises(ValueError):
        routed.moe_dispatch_bwd(x, r, x)
    with pytest.raises(ValueError):
        routed.quantize_rows_int8_fwd(x, torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError):
        routed.grouped_down_router_int8_fwd(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), w8[0], s8, i, None, x)
    with pytest.raises(TypeError):
        routed.grouped_down_router_int8_fwd(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), w8, s8, i, None,
                                            x.half())
    with pytest.raises(ValueError):
        routed.grouped_gate_up_swiglu_int8_fwd(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), i, 2, w8, s8, w8,
                                               s8, i, None, x, 7.0)


def test_header_and_binding_name_the_same_calls(L):
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "moe_routed.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert len(names) == 9
    for name in names:
        assert getattr(L, name).argtypes is not None and hasattr(routed, name)


class Tensor:
    """What the binding asks of a tensor, on GPU 0 unless told otherwise."""

    def __init__(self, shape, dtype, device=0, contiguous=True):
        self.shape, self.dtype, self.index, self.contiguous = torch.Size(shape), dtype, device, contiguous

    device = property(lambda self: torch.device("cuda", self.index) if self.index >= 0 else torch.device("cpu"))

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 4096


I32, F32, I8, BF16 = torch.int32, torch.float32, torch.int8, torch.bfloat16
# call -> (its tensors, in order, and the other arguments by position)
TENSORS = {
    "moe_sort_fwd": ([((6, 2), I32), ((4,), I32), ((6, 2), I32), ((12,), I32), ((64,), torch.uint8)], {1: 0}),
    "moe_dispatch_fwd": ([((6, 16), BF16), ((12,), I32), ((12, 16), BF16)], {2: 2}),
    "moe_dispatch_bwd": ([((12, 16), BF16), ((6, 2), I32), ((6, 16), BF16)], {}),
    "moe_combine_weighted_fwd": ([((12, 16), BF16), ((6, 2), I32), ((6, 2), F32), ((6, 16), BF16)], {}),
    "moe_combine_weighted_bwd": ([((6, 16), BF16), ((12, 16), BF16), ((6, 2), I32), ((6, 2), F32), ((12, 16), BF16),
                                  ((6, 2), F32)], {}),
    "quantize_rows_int8_fwd": ([((6, 16), BF16), ((6, 16), I8), ((6,), F32)], {}),
    "grouped_gate_up_swiglu_int8_fwd": ([((6, 16), I8), ((6,), F32), ((12,), I32), ((4, 8, 16), I8), ((4, 8), F32),
                                         ((4, 8, 16), I8), ((4, 8), F32), ((4,), I32), ((12,), F32), ((12, 8), BF16)],
                                        {3: 2, 11: 7.0}),
    "grouped_down_router_int8_fwd": ([((12, 8), I8), ((12,), F32), ((4, 16, 8), I8), ((4, 16), F32), ((4,), I32),
                                      ((12,), F32), ((12, 16), BF16)], {}),
}
# sizes that only the tensor itself has: experts and workspace of the sort, tokens that rows are taken from, rows
# that are summed, slots of a token
FREE = {("moe_sort_fwd", 1, 0), ("moe_sort_fwd", 4, 0), ("moe_dispatch_fwd", 0, 0), ("moe_dispatch_bwd", 0, 0),
        ("moe_dispatch_bwd", 1, 1), ("moe_combine_weighted_fwd", 0, 0)}


@pytest.mark.parametrize("name", sorted(TENSORS))
def test_binding_passes_only_tensors_that_fit(name, monkeypatch):
    reached = []

    class Library:
        def __getattr__(self, call):
            return lambda *args: reached.append((call, args)) or 0

    monkeypatch.setattr(routed, "_fns", Library())
    monkeypatch.setattr(routed, "_raw_stream", lambda device: 0)
    specs, others = TENSORS[name]

    def call(tensors):
        args = list(tensors)
        for at in sorted(others):
            args.insert(at, others[at])
        getattr(routed, name)(*args)

    def made():
        return [Tensor(*s) for s in specs]

    call(made())
    assert [c for c, _ in reached] == [name]
    assert all(a == 4096 for a in reached[0][1] if isinstance(a, int) and a > 1000)
    for i, (shape, dtype) in enumerate(specs):
        wrong = [Tensor(shape, torch.float64), Tensor(shape, dtype, device=1), Tensor(shape, dtype, device=-1),
                 Tensor(shape, dtype, contiguous=False), Tensor(shape + (1,), dtype)]
        wrong += [Tensor(shape[:d] + (shape[d] + 1,) + shape[d + 1:], dtype) for d in range(len(shape))
                  if (name, i, d) not in FREE]
        for bad in wrong:
            tensors = made()
            tensors[i] = bad
            with pytest.raises((TypeError, ValueError)):
                call(tensors)
                raise AssertionError(f"{name}: tensor {i} passed with {bad.shape} {bad.dtype} {bad.device} "
                                     f"contiguous={bad.contiguous}")
    tensors = made()
    for t in tensors:
        t.index = -1                               # all of them on the CPU
    with pytest.raises((TypeError, ValueError)):
        call(tensors)
    assert len(reached) == 1                       # the library was never reached again


OPTIONAL = {("moe_sort_fwd", 4), ("moe_combine_weighted_bwd", 5), ("grouped_gate_up_swiglu_int8_fwd", 2),
            ("grouped_gate_up_swiglu_int8_fwd", 8), ("grouped_down_router_int8_fwd", 5)}


@pytest.mark.parametrize("name", sorted(TENSORS))
def test_binding_names_a_tensor_that_is_missing(name, monkeypatch):
    """None in the place of a tensor that a call cannot do without is a ValueError, whichever one it is."""
    class Library:
        def __getattr__(self, call):
            return lambda *args: 0

    monkeypatch.setattr(routed, "_fns", Library())
    monkeypatch.setattr(routed, "_raw_stream", lambda device: 0)
    specs, others = TENSORS[name]
    for i in range(len(specs)):
        args = [Tensor(*s) for s in specs]
        args[i] = None
        for at in sorted(others):
            args.insert(at, others[at])
        if (name, i) in OPTIONAL:
            getattr(routed, name)(*args)
        else:
            with pytest.raises(ValueError, match="is required"):
                getattr(routed, name)(*args)


@pytest.mark.parametrize("strided", [lambda t: t.t(), lambda t: t[:, 1:5], lambda t: t.view(2, 4, 8).transpose(1, 2),
                                     lambda t: t.view(2, 4, 8)[:, :, ::2], lambda t: t[3]])
def test_quantize_helper_takes_any_strides(strided, monkeypatch):
    """The call gets contiguous rows with the same values, however the leading dimensions and the columns lie."""
    got = []
    monkeypatch.setattr(routed, "quantize_rows_int8_fwd", lambda x, q, scale: got.append((x, q, scale)))
    t = strided(torch.arange(64.0).view(8, 8))
    q, scale = routed.quantize_rows_int8(t)
    (x, q2, scale2), = got
    assert x.is_contiguous() and q2.is_contiguous() and torch.equal(x.view(t.shape), t)
    assert x.shape == q2.shape and scale2.shape == x.shape[:1]
    assert q.shape == t.shape and scale.shape == t.shape[:-1]
    assert q.data_ptr() == q2.data_ptr() and scale.data_ptr() == scale2.data_ptr()
