"""The steps around the routed experts on the GPU, against plain implementations in 64 bits.

Bars, from the arithmetic each call documents:
  - order of the rows, dispatch, 8-bit sums: equal;
  - the dispatch's gradient: the same binary32 additions in the same order, so equal;
  - combine: one float32 rounding per slot, then the output's rounding;
  - gradient of the rows: one product and one rounding, so equal; gradient of a weight: a sum of n
    float32 fused multiply-adds in some order, n * 2^-24 of the sum of the terms' magnitudes;
  - quantised rows: the quotient is rounded to float32 before it is rounded to an integer, which moves
    it by at most 127 * 2^-23 with the rounding of 127 x before it.
"""
import sys

import numpy as np
import pytest
import torch

import moe_routed_expert_amd as epi
from tests import routed_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SENTINEL = {torch.bfloat16: (torch.int16, 0x7FBF), torch.float16: (torch.int16, 0x7DAD),
            torch.float32: (torch.int32, 0x7FC0DEAD), torch.int32: (torch.int32, -77), torch.int8: (torch.int8, -128)}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    epi.binding.lib()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def say(request):
    print(f"\n[gpu-routed] {request.node.name}", flush=True)
    sys.stdout.flush()


def sentinel(shape, dtype, offset=0):
    """A contiguous tensor of NaNs (or out-of-the-way integers), its address `offset` elements past an aligned one."""
    view, value = SENTINEL[dtype]
    n = int(np.prod(shape))
    t = torch.empty(n + 64, dtype=dtype, device="cuda")
    t.view(view).fill_(value)
    return t[offset:offset + n].view(shape)


def placed(t, offset):
    """The same values at an address `offset` elements past an aligned one."""
    out = sentinel(t.shape, t.dtype, offset)
    out.copy_(t)
    return out


def normal(rng, shape, dtype, sigma=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).to(dtype).cuda()


def bits(t):
    return t.contiguous().view({2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def route(rng, tokens, top_k, experts, local, first=0):
    """Distinct experts per token, and the order of the rows of experts [first, first + local)."""
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :top_k].astype(np.int32)
    return (ids,) + ref.sort(ids, first, local)


def check(got, want, slack, dtype, what):
    got = ref.f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN positions differ"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = np.isfinite(want)
    err = np.abs(got[ok] - want[ok])
    bound = slack[ok] + ref.rounding(dtype, np.abs(want[ok]) + slack[ok])
    bad = int((err > bound).sum())
    assert bad == 0, f"{what}: {bad} beyond the bound, worst {float((err / bound).max()):.3g}"


# ---- order of the rows --------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,top_k,experts,first,local", [
    (1, 1, 1, 0, 1), (1, 8, 64, 0, 64), (3, 2, 5, 3, 2), (32, 8, 64, 0, 64), (63, 1, 7, 2, 3), (257, 3, 12, 0, 12),
    (512, 8, 64, 24, 8), (513, 8, 64, 24, 8), (1365, 3, 1024, 0, 1024), (4096, 1, 2, 0, 1), (4097, 1, 2, 1, 1),
    (5000, 7, 128, 32, 32), (20011, 8, 64, 0, 64), (3001, 8, 1024, 0, 1024), (8200, 8, 1024, 7, 1000),
    (60000, 7, 128, 0, 128), (128, 8, 64, 0, 64), (129, 8, 64, 8, 40), (293, 7, 1024, 0, 1024), (256, 8, 16, 0, 16),
    (2049, 1, 3, 1, 2), (50021, 7, 64, 0, 16), (40000, 8, 64, 0, 64), (70001, 8, 64, 3, 8)])
def test_sort(dtype, tokens, top_k, experts, first, local):
    rng = np.random.default_rng(tokens + local)
    ids, offs_w, row_w, slot_w = route(rng, tokens, top_k, experts, local, first)
    offs, row_of, slot_of = epi.moe_sort(torch.from_numpy(ids).to(dtype).cuda(), local, first)
    assert np.array_equal(offs.cpu(), offs_w)
    assert np.array_equal(row_of.cpu(), row_w)
    assert np.array_equal(slot_of.cpu(), slot_w)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,top_k,experts,first,local", [(131072, 8, 256, 0, 256), (75001, 8, 1024, 20, 1000),
                                                              (90007, 7, 300, 11, 60)])
def test_sort_of_long_calls_with_many_experts(dtype, tokens, top_k, experts, first, local):
    """Four groups a wavefront, and more counts than each block reads for itself: a launch of its own sums them."""
    rng = np.random.default_rng(tokens)
    ids = rng.integers(0, experts, (tokens, top_k)).astype(np.int32)
    want = ref.sort(ids, first, local)
    for got, w in zip(epi.moe_sort(torch.from_numpy(ids).to(dtype).cuda(), local, first), want):
        assert np.array_equal(got.cpu(), w)


@pytest.mark.parametrize("tokens", [40, 3000])
def test_sort_of_uneven_and_foreign_experts(tokens):
    """One expert for all; repeats within a token; ids that are negative, past the last or far out."""
    rng = np.random.default_rng(tokens)
    far = np.array([-1, 2 ** 31, -2 ** 63, 2 ** 63 - 1, 2 ** 32, 2 ** 32 + 3], np.int64)
    for first, ids in ((0, np.zeros((tokens, 4), np.int64)), (5, np.full((tokens, 4), 9, np.int64)),
                       (0, np.full((tokens, 4), -1, np.int64)), (2, rng.choice(far, (tokens, 4))),
                       (1, np.where(rng.random((tokens, 4)) < 0.2, rng.choice(far, (tokens, 4)),
                                    rng.integers(0, 6, (tokens, 4))))):
        want = ref.sort(ids, first, 5)
        for got, w in zip(epi.moe_sort(torch.from_numpy(ids).cuda(), 5, first), want):
            assert np.array_equal(got.cpu(), w)


def test_sort_of_nothing():
    offs, row_of, slot_of = epi.moe_sort(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6)
    assert offs.tolist() == [0] * 6 and row_of.shape == (0, 4) and slot_of.shape == (0,)


def test_sort_repeats_with_a_dirty_workspace():
    rng = np.random.default_rng(5)
    ids, *want = route(rng, 9000, 4, 16, 8, 4)
    t = torch.from_numpy(ids).cuda()
    ws = torch.full((epi.moe_sort_workspace_bytes(9000, 4, 8) + 64,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        out = [sentinel(w.shape, torch.int32) for w in want]
        epi.moe_sort_fwd(t, 4, *out, ws)
        for got, w in zip(out, want):
            assert np.array_equal(got.cpu(), w)


# ---- dispatch ---------------------------------------------------------------------------

WIDTHS = [1, 2, 3, 7, 8, 12, 40, 1000, 1001, 1024, 2052, 4100, 7168, 9001, 16384]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", WIDTHS)
def test_dispatch_and_its_gradient(dtype, hidden):
    rng = np.random.default_rng(hidden)
    for tokens, top_k, experts, local, offset in ((1, 1, 1, 1, 0), (5, 3, 4, 4, 1), (37, 8, 16, 4, 0),
                                                  (20, 2, 6, 3, 3)):
        _, offs, row_of, slot_of = route(rng, tokens, top_k, experts, local)
        rows = int(offs[-1])
        capacity = rows + 2                       # two rows without a slot
        x = placed(normal(rng, (tokens, hidden), dtype), offset)
        slots = ints(np.concatenate([slot_of, [-1, -1]])[:capacity])
        out = sentinel((capacity, hidden), dtype, offset)
        epi.moe_dispatch_fwd(x, slots, top_k, out)
        want = torch.zeros((capacity, hidden), dtype=dtype)
        want[:rows] = x.cpu()[torch.from_numpy(slot_of[:rows].astype(np.int64) // top_k)]
        assert torch.equal(bits(out), bits(want))
        g = placed(normal(rng, (capacity, hidden), dtype), offset)
        gx = sentinel((tokens, hidden), dtype, offset)
        epi.moe_dispatch_bwd(g, ints(row_of), gx)
        want = torch.zeros((tokens, hidden), dtype=torch.float32)
        gf = g.float().cpu()
        for t in range(tokens):
            for r in row_of[t]:
                if r >= 0:
                    want[t] += gf[r]              # binary32, slots ascending
        assert torch.equal(bits(gx), bits(want.to(dtype)))


def test_dispatch_leaves_out_wrong_indices():
    x = torch.randn(4, 32, device="cuda")
    slots = ints([0, 7, 8, -5, 2 ** 31 - 1, 3])
    out = sentinel((6, 32), torch.float32)
    epi.moe_dispatch_fwd(x, slots, 2, out)
    want = torch.stack([x[0], x[3], 0 * x[0].abs(), 0 * x[0].abs(), 0 * x[0].abs(), x[1]])
    assert torch.equal(bits(out), bits(want))
    row_of = ints([[0, 6], [-1, -2 ** 31], [2 ** 31 - 1, 5], [5, 5]])
    gx = sentinel((4, 32), torch.float32)
    epi.moe_dispatch_bwd(want, row_of, gx)
    assert torch.equal(bits(gx), bits(torch.stack([x[0], 0 * x[0].abs(), x[1], x[1] + x[1]])))


# ---- combine --------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                             (torch.float16, torch.float16), (torch.float16, torch.float32),
                                             (torch.float32, torch.float32)])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_combine_and_its_gradients(dtype, out_dtype, hidden):
    rng = np.random.default_rng(hidden + 1)
    for tokens, top_k, experts, local, offset in ((1, 1, 1, 1, 0), (9, 3, 4, 4, 1), (40, 8, 16, 4, 0),
                                                  (6, 20, 24, 24, 0)):
        _, offs, row_of, _ = route(rng, tokens, top_k, experts, local)
        rows = int(offs[-1])
        x = placed(normal(rng, (rows, hidden), dtype), offset)
        w = torch.from_numpy(rng.standard_normal((tokens, top_k)).astype(np.float32)).cuda()
        w[torch.from_numpy(row_of < 0).cuda()] = float("nan")   # weights of slots without a row are not used
        out = sentinel((tokens, hidden), out_dtype, offset)
        epi.moe_combine_weighted_fwd(x, ints(row_of), w, out)
        want, scale = ref.combine(ref.f64(x), row_of, ref.f64(w))
        check(out, want, top_k * ref.EPS * scale, out_dtype, "combine")
        assert bool((out[torch.from_numpy((row_of < 0).all(1)).cuda()] == 0).all())

        g = placed(normal(rng, (tokens, hidden), out_dtype), offset)
        gr = sentinel((rows, hidden), dtype, offset)
        gw = sentinel((tokens, top_k), torch.float32)
        epi.moe_combine_weighted_bwd(g, x, ints(row_of), w, gr, gw)
        gr_w, gw_w, scale = ref.combine_grads(ref.f64(g), ref.f64(x), row_of, ref.f64(w))
        t_of, j_of = np.nonzero(row_of >= 0)
        r = torch.from_numpy(row_of[t_of, j_of].astype(np.int64))
        product = w.cpu()[t_of, j_of][:, None] * g.float().cpu()[t_of]   # binary32
        assert torch.equal(bits(gr)[r], bits(product.to(dtype)))
        most = np.abs(gr_w).max()
        assert np.abs(ref.f64(gr) - gr_w).max() <= ref.rounding(dtype, most * (1 + 2 * ref.EPS)) + ref.EPS * most
        check(gw, gw_w, (hidden + 8) * ref.EPS * scale, torch.float32, "grad_weights")
        # without a gradient of the weights: the same rows
        gr2 = sentinel((rows, hidden), dtype, offset)
        epi.moe_combine_weighted_bwd(g, None, ints(row_of), w, gr2, None)
        assert torch.equal(bits(gr2), bits(gr))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden,top_k", [(264, 3), (1001, 9), (2048, 17)])
def test_a_tokens_sum_is_the_same_in_calls_of_all_sizes(dtype, hidden, top_k):
    rng = np.random.default_rng(hidden + top_k)
    tokens = 1200
    _, offs, row_of, _ = route(rng, tokens, top_k, 20, 18)
    x = normal(rng, (int(offs[-1]), hidden), dtype)
    w = torch.from_numpy(rng.standard_normal((tokens, top_k)).astype(np.float32)).cuda()
    rows = ints(row_of)
    whole, gx = sentinel((tokens, hidden), dtype), sentinel((tokens, hidden), dtype)
    epi.moe_combine_weighted_fwd(x, rows, w, whole)
    epi.moe_dispatch_bwd(x, rows, gx)
    for t0, n in ((0, 1), (tokens - 5, 5), (7, 300)):
        part, gpart = sentinel((n, hidden), dtype), sentinel((n, hidden), dtype)
        epi.moe_combine_weighted_fwd(x, rows[t0:t0 + n], w[t0:t0 + n], part)
        epi.moe_dispatch_bwd(x, rows[t0:t0 + n], gpart)
        assert torch.equal(bits(part), bits(whole[t0:t0 + n])) and torch.equal(bits(gpart), bits(gx[t0:t0 + n]))
    # and its gradients: the slots of few tokens are spread over several blocks
    g, gr, gw = normal(rng, (tokens, hidden), dtype), sentinel(x.shape, dtype), sentinel(w.shape, torch.float32)
    epi.moe_combine_weighted_bwd(g, x, rows, w, gr, gw)
    for t0, n in ((0, 1), (3, 33), (tokens - 5, 5), (7, 300)):
        gr2, gw2 = gr.clone(), sentinel((n, top_k), torch.float32)
        mine = torch.from_numpy(row_of[t0:t0 + n][row_of[t0:t0 + n] >= 0].astype(np.int64)).cuda()
        gr2[mine] = 7.0
        epi.moe_combine_weighted_bwd(g[t0:t0 + n], x, rows[t0:t0 + n], w[t0:t0 + n], gr2, gw2)
        assert torch.equal(bits(gr2), bits(gr)) and torch.equal(bits(gw2), bits(gw[t0:t0 + n]))


def test_combine_gradients_against_differences():
    """The combine is linear in the rows and in the weights: a central difference of any step is the
    derivative, up to the rounding of the two sums, 2 k eps of their size."""
    rng = np.random.default_rng(11)
    tokens, top_k, hidden = 12, 4, 96
    _, offs, row_of, _ = route(rng, tokens, top_k, 8, 6)
    rows, row_t = int(offs[-1]), ints(row_of)
    x, w = normal(rng, (rows, hidden), torch.float32), normal(rng, (tokens, top_k), torch.float32)
    g = normal(rng, (tokens, hidden), torch.float32)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    epi.MoeCombineWeighted.apply(xg, row_t, wg).backward(g)

    def loss(x, w):
        return float((epi.MoeCombineWeighted.apply(x, row_t, w).double() * g.double()).sum())

    size = float((ref.combine(np.abs(ref.f64(x)) + 3, row_of, np.abs(ref.f64(w)) + 3)[0] * np.abs(ref.f64(g))).sum())
    for _ in range(5):
        dx, dw = normal(rng, x.shape, torch.float32), normal(rng, w.shape, torch.float32)
        num = (loss(x + dx, w) - loss(x - dx, w)) / 2
        assert abs(num - float((xg.grad.double() * dx.double()).sum())) <= 4 * top_k * ref.EPS * size
        num = (loss(x, w + dw) - loss(x, w - dw)) / 2
        assert abs(num - float((wg.grad.double() * dw.double()).sum())) <= 4 * top_k * ref.EPS * size


def test_dispatch_gradient_against_differences():
    rng = np.random.default_rng(12)
    tokens, top_k, hidden = 15, 3, 64
    _, offs, row_of, slot_of = route(rng, tokens, top_k, 6, 4)
    slots, row_t = ints(slot_of[:int(offs[-1])]), ints(row_of)
    x = normal(rng, (tokens, hidden), torch.float32).requires_grad_()
    out = epi.MoeDispatch.apply(x, row_t, slots)
    g = normal(rng, out.shape, torch.float32)
    out.backward(g)
    d = normal(rng, x.shape, torch.float32)
    num = float((epi.MoeDispatch.apply(d, row_t, slots).double() * g.double()).sum())   # linear: f(d) is the derivative
    size = float((g.abs().double().sum() * d.abs().max().double()))
    assert abs(num - float((x.grad.double() * d.double()).sum())) <= 4 * top_k * ref.EPS * size


def test_combine_with_infinities_and_nans():
    """They reach the tokens that have the row and no other."""
    x = torch.ones(4, 24, device="cuda", dtype=torch.bfloat16)
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    row_of = ints([[0, -1], [1, 0], [2, 3], [-1, -1], [3, 9]])
    w = torch.tensor([[2.0, 0], [1, 1], [1, 1], [float("inf"), 1], [0.5, float("nan")]], device="cuda")
    out = sentinel((5, 24), torch.bfloat16)
    epi.moe_combine_weighted_fwd(x, row_of, w, out)
    want = torch.tensor([2.0, 2.0, 2.0, 0.0, 0.5])[:, None].repeat(1, 24)
    want[1, 3], want[2, 5] = float("inf"), float("nan")
    got = out.float().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", DTYPES)
def test_calls_with_no_rows_or_no_tokens(dtype):
    """No row here: sums and gradients of zeros. No token: nothing is written."""
    none, x = torch.empty((0, 40), dtype=dtype, device="cuda"), torch.ones((5, 40), dtype=dtype, device="cuda")
    row_of, weights = ints(np.full((5, 3), -1)), torch.ones((5, 3), device="cuda")
    for call in (lambda o: epi.moe_dispatch_bwd(none, row_of, o),
                 lambda o: epi.moe_combine_weighted_fwd(none, row_of, weights, o)):
        out = sentinel((5, 40), dtype)
        call(out)
        assert bool((out == 0).all())
    grad_weights = sentinel((5, 3), torch.float32)
    epi.moe_combine_weighted_bwd(x, none, row_of, weights, none, grad_weights)
    assert bool((grad_weights == 0).all())
    epi.moe_dispatch_fwd(x, ints([]), 3, none)
    out = sentinel((4, 40), dtype)
    epi.moe_dispatch_fwd(none, ints([0, 1, -1, 5]), 3, out)
    assert bool((out == 0).all())
    q, scale = epi.quantize_rows_int8(none)
    assert q.shape == (0, 40) and scale.shape == (0,)
    no_slots = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    epi.moe_dispatch_bwd(x, no_slots, none)
    epi.moe_combine_weighted_fwd(x, no_slots, weights[:0], none)
    xg, wg = x.clone().requires_grad_(), weights.clone().requires_grad_()
    rows = epi.MoeDispatch.apply(xg, row_of, ints([]))
    epi.MoeCombineWeighted.apply(rows, row_of, wg).sum().backward()
    assert bool((xg.grad == 0).all()) and bool((wg.grad == 0).all())


def shuffled(n):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


@pytest.mark.parametrize("hidden,tokens", [(264, 1_100_003), (1, 33_600_001), (8, 33_600_001)])
def test_moves_of_more_rows_than_a_grid_has_blocks(hidden, tokens):
    """2^20 blocks at most: each of them goes on to further rows or tokens, whole rows and narrow ones."""
    x = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda").normal_()
    row_of = shuffled(tokens).view(tokens, 1)
    weights = torch.rand((tokens, 1), device="cuda") + 0.5
    at = row_of[:, 0].long()
    out = sentinel((tokens, hidden), torch.bfloat16)
    epi.moe_dispatch_bwd(x, row_of, out)
    assert torch.equal(out, x[at])
    epi.moe_combine_weighted_fwd(x, row_of, weights, out)
    assert torch.equal(out, (x[at].float() * weights).bfloat16())
    rows, grad_w = sentinel((tokens, hidden), torch.bfloat16), sentinel((tokens, 1), torch.float32)
    epi.moe_combine_weighted_bwd(out, x, row_of, weights, rows, grad_w)
    assert torch.equal(rows[at], (out.float() * weights).bfloat16())
    for t0 in range(0, tokens, 1 << 22):
        here = slice(t0, t0 + (1 << 22))
        terms = out[here].double() * x[at[here]].double()
        assert bool(((grad_w[here, 0] - terms.sum(1)).abs() <= (hidden + 8) * ref.EPS * terms.abs().sum(1)).all())


@pytest.mark.parametrize("hidden,rows", [(264, 1_100_003), (1, 134_300_001)])
def test_dispatch_of_more_rows_than_a_grid_has_blocks(hidden, rows):
    x = torch.empty((1001, hidden), dtype=torch.bfloat16, device="cuda").normal_()
    slot_of = torch.randint(0, 1001, (rows,), dtype=torch.int32, device="cuda")
    out = sentinel((rows, hidden), torch.bfloat16)
    epi.moe_dispatch_fwd(x, slot_of, 1, out)
    assert torch.equal(out, x[slot_of])


# ---- 8-bit rows ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 7, 8, 16, 500, 512, 513, 520, 1001, 1024, 1032, 2048, 2049, 2056, 4096, 4099, 4104,
                                  7168, 8192, 8200, 20001])
def test_quantize_rows(dtype, cols):
    rng = np.random.default_rng(cols)
    rows = 23
    x = rng.standard_normal((rows, cols))
    x *= 10.0 ** rng.integers(-4, 4, (rows, 1))
    x[3] = 0.0
    x[4] = -0.0
    x[5, 1:] = 0.0
    t = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    least = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}[dtype]
    most = torch.finfo(dtype).max
    t[6] = t[6].sign() * least                    # subnormal and largest rows
    t[7] = t[7].sign() * most
    t[8] = t[8] / t[8].abs().max() * most
    for offset in (0, 1):
        src = placed(t, offset)
        q, scale = sentinel((rows, cols), torch.int8, offset), sentinel((rows,), torch.float32)
        epi.quantize_rows_int8_fwd(src, q, scale)
        v = ref.f64(src)
        amax = np.abs(v).max(1)
        with np.errstate(invalid="ignore", divide="ignore"):
            exact = np.where(amax[:, None] > 0, 127.0 * v / amax[:, None], 0.0)
        want_scale = (amax.astype(np.float32) / np.float32(127)).astype(np.float32)
        assert np.array_equal(scale.cpu().numpy().view(np.uint32), want_scale.view(np.uint32))
        got = q.cpu().numpy().astype(np.float64)
        off = np.abs(got - exact)
        assert off.max() <= 0.5 + 127 * 2.0 ** -23, off.max()
        assert np.abs(got).max() <= 127


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [100, 520, 1001, 1032, 2056, 4099, 8192, 9001])
def test_quantize_gives_a_row_the_same_in_calls_of_all_sizes(dtype, cols):
    rng = np.random.default_rng(cols + 7)
    x = rng.standard_normal((700, cols)) * 10.0 ** rng.integers(-4, 4, (700, 1))
    t = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    q, scale = epi.quantize_rows_int8(t)
    v = ref.f64(t)
    amax = np.abs(v).max(1)
    assert np.abs(q.cpu().numpy() - 127.0 * v / amax[:, None]).max() <= 0.5 + 127 * 2.0 ** -23
    assert torch.equal(bits(scale), bits(torch.from_numpy(amax.astype(np.float32) / np.float32(127))))
    for r0, n in ((0, 1), (3, 512), (187, 513), (693, 7)):
        part = epi.quantize_rows_int8(t[r0:r0 + n].clone())
        assert torch.equal(part[0], q[r0:r0 + n]) and torch.equal(bits(part[1]), bits(scale[r0:r0 + n]))


def test_quantize_ties_to_even_and_rows_that_are_not_finite():
    # 127 * 0.5 / 1 = 63.5 and its like: the integer is the even neighbour
    x = torch.tensor([[1.0, 0.5, -0.5, 0.25], [2.0, 1.0, -1.0, 0.0], [float("inf"), 1, 2, 3],
                      [1, float("nan"), 2, 3], [-float("inf"), float("nan"), 0, 0]], device="cuda",
                     dtype=torch.bfloat16)
    q, scale = epi.quantize_rows_int8(x)
    assert q[0].tolist() == [127, 64, -64, 32] and q[1].tolist() == [127, 64, -64, 0]
    assert q[2:].abs().max() == 0 and bool(torch.isnan(scale[2:]).all()) and bool(torch.isfinite(scale[:2]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [256, 264, 271, 520, 1032, 2056, 4104, 9001, 16392])
def test_quantize_rounds_as_the_division_does(dtype, cols):
    """Every integer is that of the division in float32, ties to even among them, in vectors and in a row's last
    elements, aligned or not, with the lanes of few rows and of many."""
    rng = np.random.default_rng(cols + 13)
    rows = 600
    x = rng.standard_normal((rows, cols)) * 10.0 ** rng.integers(-3, 3, (rows, 1))
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    for i, tie in enumerate(ref.tie_rows(dtype)):
        tie = torch.from_numpy(tie).to(dtype)
        t[i, :256] = tie
        t[i, 256:] = tie.repeat(cols // 256 + 1)[:cols][256:]
        t[8 + i] = t[i].roll(cols - 256)          # the ties at the end of the row
    want_q, want_scale = ref.quantize(ref.f64(t))
    t = t.cuda()
    for offset in (0, 1):
        for n in (23, rows):                      # up to 512 rows take more lanes each
            q, scale = sentinel((n, cols), torch.int8, offset), sentinel((n,), torch.float32)
            epi.quantize_rows_int8_fwd(placed(t[:n], offset), q, scale)
            assert np.array_equal(q.cpu().numpy(), want_q[:n])
            assert np.array_equal(scale.cpu().numpy().view(np.uint32), want_scale[:n].view(np.uint32))


@pytest.mark.parametrize("cols,rows", [(8, 16_800_003), (4104, 1_050_007)])
def test_quantize_more_rows_than_a_grid_has_blocks(cols, rows):
    """2^20 blocks at most: each goes on to further rows, within a wavefront and with a block for a row."""
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_()
    q, scale = epi.quantize_rows_int8(x)
    for r0 in range(0, rows, 1 << 16):
        v = x[r0:r0 + (1 << 16)].float()
        most = v.abs().amax(1)
        assert torch.equal(bits(scale[r0:r0 + (1 << 16)]), bits(most / torch.full_like(most, 127)))
        assert torch.equal(q[r0:r0 + (1 << 16)], torch.round(127 * v / most[:, None]).to(torch.int8))


# ---- products in 8-bit integers -----------------------------------------------------------------

def int8_of(rng, shape):
    return torch.from_numpy(rng.integers(-127, 128, shape).astype(np.int8)).cuda()


def scales(rng, shape, size):
    return torch.from_numpy((rng.random(shape) + 0.5).astype(np.float32) * np.float32(size)).cuda()


# rows per expert, K, N: single rows, tiles of one row more or less, empty experts, short and odd K and N
PRODUCTS = [([1], 16, 8), ([1], 128, 128), ([1, 0, 3], 48, 24), ([0, 16, 17, 0], 112, 136), ([5, 40, 2], 144, 264),
            ([64, 65, 1, 63], 256, 128), ([255, 256, 257], 272, 72), ([700], 128, 520), ([3, 130, 0, 200], 1040, 200),
            ([2] * 33, 400, 40), ([0, 0, 0], 64, 16), ([129, 31, 33, 500], 2064, 48),
            ([0] * 30 + [100] + [3] * 70, 528, 56),
            ([1, 90, 0, 2, 7], 7184, 40)]
# enough rows and columns for the small, the middle and the large tiles, partial ones among them; K below,
# at and past one step and with odd numbers of steps
PRODUCTS += [(counts * 7, k, n) for counts, n in (([30, 0, 25, 31, 64, 17], 520), ([100, 128, 1, 0, 140, 129], 520),
                                                  ([300, 256, 257, 1, 512, 0], 776)) for k in (16, 112, 128, 272, 384)]
PRODUCTS += [([100, 128, 1, 0, 140, 129] * 7, k, n) for n in (264, 1032) for k in (16, 256, 272, 640)]


@pytest.mark.parametrize("counts,k,n", PRODUCTS)
@pytest.mark.parametrize("extra", [0, 3])
def test_down_product(counts, k, n, extra):
    rng = np.random.default_rng(k + n)
    offs = np.cumsum(counts).astype(np.int32)
    rows = int(offs[-1]) + extra                  # rows past the last expert's: not written
    h, w = int8_of(rng, (rows, k)), int8_of(rng, (len(counts), n, k))
    sh, sw = scales(rng, rows, 0.01), scales(rng, (len(counts), n), 0.01)
    p = torch.from_numpy(rng.random(rows).astype(np.float32)).cuda()
    for probs in (None, p):
        pw = np.ones(rows, np.float32) if probs is None else p.cpu().numpy()
        want, slack = ref.down(h.cpu().numpy(), sh.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(), offs, pw)
        for dtype in (torch.bfloat16, torch.float32):
            out = sentinel((rows, n), dtype)
            kept = bits(out[rows - extra:].clone())
            epi.grouped_down_router_int8_fwd(h, sh, w, sw, ints(offs), probs, out)
            live = rows - extra
            check(out[:live], want[:live], slack[:live], dtype, f"down {dtype}")
            assert torch.equal(bits(out[live:]), kept)


@pytest.mark.parametrize("counts,k,n", PRODUCTS)
@pytest.mark.parametrize("gathered", [False, True])
def test_gate_up_product(counts, k, n, gathered):
    rng = np.random.default_rng(k + 2 * n)
    offs = np.cumsum(counts).astype(np.int32)
    rows, extra = int(offs[-1]), 2
    top_k = 3 if gathered else 1
    tokens = 50 if gathered else rows + extra
    if tokens == 0:
        return
    a = int8_of(rng, (tokens, k))
    sa = scales(rng, tokens, 8.0 / (5400 * np.sqrt(k)))
    wg, wu = int8_of(rng, (len(counts), n, k)), int8_of(rng, (len(counts), n, k))
    sg, su = scales(rng, (len(counts), n), 1.0), scales(rng, (len(counts), n), 1.0)
    slots, token_of = None, np.arange(rows + extra)
    if gathered:
        s = rng.integers(0, tokens * top_k, rows + extra)
        if rows > 4:
            s[[1, 3]] = [-1, tokens * top_k]      # no slot: zeros
        token_of = np.where((s >= 0) & (s < tokens * top_k), s // top_k, -1)
        slots = ints(s)
    p = torch.from_numpy(rng.random(rows + extra).astype(np.float32)).cuda()
    for probs in (None, p):
        pw = np.ones(rows + extra, np.float32) if probs is None else p.cpu().numpy()
        y = sentinel((rows + extra, n), torch.bfloat16)
        kept = bits(y[rows:].clone())
        epi.grouped_gate_up_swiglu_int8_fwd(a, sa, slots, top_k, wg, sg, wu, su, ints(offs), probs, y, 7.0)
        want, slack = ref.gate_up(a.cpu().numpy(), sa.cpu().numpy(), token_of, wg.cpu().numpy(), sg.cpu().numpy(),
                                  wu.cpu().numpy(), su.cpu().numpy(), offs, pw, 7.0)
        check(y[:rows], want[:rows], slack[:rows], torch.bfloat16, "gate_up")
        assert torch.equal(bits(y[rows:]), kept)


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_sums_are_exact_integers(rows):
    """Unit scales, float32 out: sums below 2^24 come out exactly; the longest K of largest values does not wrap."""
    rng = np.random.default_rng(rows)
    k, n = 1040, 40
    h, w = torch.from_numpy(rng.integers(-20, 21, (rows, k)).astype(np.int8)).cuda(), int8_of(rng, (1, n, k))
    one = torch.ones(max(rows, n), device="cuda")
    out = sentinel((rows, n), torch.float32)
    epi.grouped_down_router_int8_fwd(h, one[:rows], w, one[:n].view(1, n), ints([rows]), None, out)
    want = h.cpu().numpy().astype(np.int64) @ w[0].cpu().numpy().astype(np.int64).T
    assert np.array_equal(out.cpu().numpy().astype(np.int64), want)
    k = 131056
    for a, b in ((-128, -128), (127, -128), (127, 127)):
        h = torch.full((rows, k), a, dtype=torch.int8, device="cuda")
        w = torch.full((1, n, k), b, dtype=torch.int8, device="cuda")
        epi.grouped_down_router_int8_fwd(h, one[:rows], w, one[:n].view(1, n), ints([rows]), None, out)
        assert bool((out == float(np.float32(a * b * k))).all())


def test_products_of_rows_that_are_not_finite_stay_in_their_rows():
    rng = np.random.default_rng(3)
    x = normal(rng, (40, 64), torch.float32)
    x[7, 3], x[30, 0] = float("inf"), float("nan")
    q, s = epi.quantize_rows_int8(x)
    w, sw = epi.quantize_rows_int8(normal(rng, (2, 24, 64), torch.bfloat16))
    out = sentinel((40, 24), torch.bfloat16)
    epi.grouped_down_router_int8_fwd(q, s, w, sw, ints([10, 40]), None, out)
    nan = torch.isnan(out).cpu()
    assert bool(nan[[7, 30]].all()) and int(nan.sum()) == 2 * 24


def test_offs_out_of_order_or_past_the_rows_are_clamped():
    rng = np.random.default_rng(4)
    h, w = int8_of(rng, (50, 32)), int8_of(rng, (4, 16, 32))
    sh, sw = scales(rng, 50, 0.1), scales(rng, (4, 16), 0.1)
    for offs in ([20, 10, 500, 600], [-5, 0, 30, 50], [2 ** 31 - 1, 0, 0, 0]):
        out = sentinel((50, 16), torch.float32)
        epi.grouped_down_router_int8_fwd(h, sh, w, sw, ints(offs), None, out)
        want, slack = ref.down(h.cpu().numpy(), sh.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(), offs,
                               np.ones(50, np.float32))
        check(out, want, slack, torch.float32, "down")


@pytest.mark.parametrize("counts,n", [([7], 16), ([40, 0, 35], 16), ([30, 0, 25, 31, 64, 17] * 7, 520),
                                      ([100, 128, 1, 0, 140, 129] * 7, 520), ([300, 256, 257, 1, 512, 0] * 7, 776)])
def test_gate_up_of_no_tokens_gives_rows_of_zeros(counts, n):
    """Without tokens every slot is out of range: y = 0 * probs below the last expert's end, by every kernel."""
    rng = np.random.default_rng(n)
    offs, k, top_k = np.cumsum(counts).astype(np.int32), 144, 2
    rows, extra = int(offs[-1]), 2
    w, s = int8_of(rng, (len(counts), n, k)), scales(rng, (len(counts), n), 1.0)
    p = torch.from_numpy(rng.random(rows + extra).astype(np.float32)).cuda()
    p[3] = float("inf")
    none, no_scale = torch.empty((0, k), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    for probs in (None, p):
        y = sentinel((rows + extra, n), torch.bfloat16)
        kept = bits(y[rows:].clone())
        epi.grouped_gate_up_swiglu_int8_fwd(none, no_scale, ints(rng.integers(-2, 50, rows + extra)), top_k, w, s, w, s,
                                            ints(offs), probs, y, 7.0)
        zeros = y[:rows].float()
        if probs is not None:
            assert bool(torch.isnan(zeros[3]).all())
            zeros[3] = 0.0
        assert bool((zeros == 0).all())
        assert torch.equal(bits(y[rows:]), kept)


def test_tokens_past_two_and_four_gigabytes():
    """Rows read in place from a tensor whose byte offsets pass 2^31 and 2^32, moved and multiplied, with
    few rows and with small, middle and large tiles."""
    tokens, k = 600_000, 7200
    a = torch.zeros((tokens, k), dtype=torch.int8, device="cuda")
    picks = np.array([0, 1, 298_261, 298_262, 596_523, 596_524, tokens - 1])
    rng = np.random.default_rng(6)
    values = int8_of(rng, (len(picks), k))
    a[torch.from_numpy(picks).cuda()] = values
    one = torch.ones(tokens, device="cuda")
    for rows, n in ((7, 16), (2048, 264), (4096, 264), (8192, 776)):
        w = int8_of(rng, (1, n, k))
        y = sentinel((rows, n), torch.bfloat16)
        which = np.arange(rows) % len(picks)
        epi.grouped_gate_up_swiglu_int8_fwd(a, one * 1e-4, ints(picks[which]), 1, w, one[:n].view(1, n) * 0.01, w,
                                            one[:n].view(1, n) * 0.01, ints([rows]), None, y, 7.0)
        s = np.full((1, n), 0.01, np.float32)
        want, slack = ref.gate_up(values.cpu().numpy(), np.full(len(picks), 1e-4, np.float32), np.arange(len(picks)),
                                  w.cpu().numpy(), s, w.cpu().numpy(), s, [len(picks)],
                                  np.ones(len(picks), np.float32), 7.0)
        check(y, want[which], slack[which], torch.bfloat16, "gate_up")
    x = a.view(torch.bfloat16)                    # the same bytes, moved as 16-bit rows
    out = sentinel((len(picks), k // 2), torch.bfloat16)
    epi.moe_dispatch_fwd(x, ints(picks), 1, out)
    assert torch.equal(bits(out), bits(values.view(torch.bfloat16)))


# ---- streams and graphs -------------------------------------------------------------------------

class Chain:
    """A serving step in 8-bit integers and a training step's moves, on static buffers."""

    def __init__(self, seed, tokens=96, hidden=256, inter=128, experts=8, top_k=3):
        rng = np.random.default_rng(seed)
        self.top_k = top_k
        self.ids = torch.from_numpy(np.argsort(rng.random((tokens, experts)), 1)[:, :top_k].astype(np.int64)).cuda()
        self.weights = torch.softmax(normal(rng, (tokens, top_k), torch.float32), 1)
        self.x = normal(rng, (tokens, hidden), torch.bfloat16, 4.0)
        self.grad = normal(rng, (tokens, hidden), torch.bfloat16)
        w = np.random.default_rng(0)
        self.gate = epi.quantize_rows_int8(normal(w, (experts, inter, hidden), torch.bfloat16, 0.06))
        self.up = epi.quantize_rows_int8(normal(w, (experts, inter, hidden), torch.bfloat16, 0.06))
        self.down = epi.quantize_rows_int8(normal(w, (experts, hidden, inter), torch.bfloat16, 0.09))
        rows, bf, f32, i32, i8 = tokens * top_k, torch.bfloat16, torch.float32, torch.int32, torch.int8
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")
        self.outs = {"offs": e(experts, i32), "row_of": e((tokens, top_k), i32), "slot_of": e(rows, i32),
                     "q": e((tokens, hidden), i8), "scale": e(tokens, f32), "y": e((rows, inter), bf),
                     "hq": e((rows, inter), i8), "hs": e(rows, f32), "rows": e((rows, hidden), bf),
                     "out": e((tokens, hidden), bf), "moved": e((rows, hidden), bf), "grad_x": e((tokens, hidden), bf),
                     "grad_rows": e((rows, hidden), bf), "grad_w": e((tokens, top_k), f32)}

    def step(self):
        o = self.outs
        epi.moe_sort_fwd(self.ids, 0, o["offs"], o["row_of"], o["slot_of"])
        epi.quantize_rows_int8_fwd(self.x, o["q"], o["scale"])
        epi.grouped_gate_up_swiglu_int8_fwd(o["q"], o["scale"], o["slot_of"], self.top_k, *self.gate, *self.up,
                                            o["offs"], None, o["y"], 7.0)
        epi.quantize_rows_int8_fwd(o["y"], o["hq"], o["hs"])
        epi.grouped_down_router_int8_fwd(o["hq"], o["hs"], *self.down, o["offs"], None, o["rows"])
        epi.moe_combine_weighted_fwd(o["rows"], o["row_of"], self.weights, o["out"])
        epi.moe_combine_weighted_bwd(self.grad, o["rows"], o["row_of"], self.weights, o["grad_rows"], o["grad_w"])
        epi.moe_dispatch_fwd(self.x, o["slot_of"], self.top_k, o["moved"])
        epi.moe_dispatch_bwd(o["grad_rows"], o["row_of"], o["grad_x"])

    def reset(self):
        for t in self.outs.values():
            t.view(torch.uint8).fill_(0x5A)

    def snapshot(self):
        return {k: v.clone() for k, v in self.outs.items()}


def same(a, b):
    return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


def test_chain_replayed_from_a_graph_equals_eager():
    c, other = Chain(1), Chain(2)
    c.reset()
    c.step()
    torch.cuda.synchronize()
    want = c.snapshot()
    assert bool(torch.isfinite(want["out"].float()).all()) and bool(torch.isfinite(want["grad_w"]).all())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same(c.outs, want)                     # the same on another stream
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step()
    noise = torch.randn(256, 256, device="cuda")
    for _ in range(3):
        c.reset()
        noise = noise @ noise.t() / 256
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(c.outs, want)
    for name in ("ids", "weights", "x", "grad"):
        getattr(c, name).copy_(getattr(other, name))
    other.step()
    c.reset()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert same(c.outs, other.snapshot()) and not torch.equal(want["row_of"], c.outs["row_of"])
