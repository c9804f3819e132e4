"""The steps before the routed experts on the GPU, against plain implementations in 64 bits.

Bars are the float32 steps that each call documents, counted in tests/prologue_reference.py, and the
output's own rounding; the choice of the experts is equal.
"""
import sys

import numpy as np
import pytest
import torch

import moe_routed_expert_amd as epi
from tests import prologue_reference as ref
from tests.test_gpu_routed import DTYPES, bits, check, normal, placed, sentinel

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    epi.binding.lib()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def say(request):
    print(f"\n[gpu-prologue] {request.node.name}", flush=True)
    sys.stdout.flush()


def space(nbytes):
    """A workspace that holds what another call may have left: NaNs."""
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


# ---- norm -------------------------------------------------------------------------------

COLS = [1, 2, 7, 8, 24, 128, 136, 250, 512, 1001, 1024, 2048, 2056, 4100, 7168, 8192, 9001, 16384, 20008, 40000]


def check_norm(x, r, w, eps, offset, with_q=True, in_place=False):
    rows, cols = x.shape
    dt = x.dtype
    h = x.float() if r is None else (x.float() + r.float()).to(dt).float()
    out, rstd = sentinel((rows, cols), dt, offset), sentinel((rows,), F32)
    q = sentinel((rows, cols), torch.int8, offset) if with_q else None
    scale = sentinel((rows,), F32) if with_q else None
    stream = None if r is None else (placed(r, offset) if in_place else sentinel((rows, cols), dt, offset))
    epi.rms_norm_fwd(placed(x, offset), placed(w, offset), out, eps,
                     residual=None if r is None else (stream if in_place else placed(r, offset)), residual_out=stream,
                     q=q, scale=scale, rstd=rstd)
    if r is not None:
        assert torch.equal(bits(stream), bits(h.to(dt)))
    y, n, slack_y, slack_n = ref.norm(ref.f64(h), ref.f64(w), eps)
    check(rstd, n, slack_n * np.abs(n), F32, "rstd")
    check(out, y, slack_y * np.abs(y), dt, "out")
    if with_q:
        most = np.abs(y).max(1)
        check(scale, most / 127, (slack_y + 2 * ref.EPS) * most / 127, F32, "scale")
        live = most > 0
        # the nearest whole number, but for what y and the quotient's three roundings may be off
        want = np.where(live[:, None], 127 * y / np.where(live, most, 1)[:, None], 0)
        off = np.abs(ref.f64(q) - want)
        assert off.max() <= 0.5 + 127 * (2 * slack_y + 3 * ref.EPS), off.max()
    return out, q, scale, stream


@pytest.mark.parametrize("dtype,weight", PAIRS)
@pytest.mark.parametrize("cols", COLS)
def test_norm(dtype, weight, cols):
    rng = np.random.default_rng(cols)
    for rows, offset, residual in ((1, 0, True), (3, 1, True), (5, 0, False), (37, 0, True), (530, 3, False)):
        x = normal(rng, (rows, cols), dtype)
        r = normal(rng, (rows, cols), dtype, 4.0) if residual else None
        w = (1 + 0.2 * normal(rng, (cols,), F32)).to(weight)
        first = check_norm(x, r, w, 1e-6, offset)
        again = check_norm(x, r, w, 1e-6, 0, in_place=True)
        for a, b in zip(first, again):                     # other addresses, and in place: the same bits
            assert a is None or torch.equal(a.cpu().view(torch.uint8), b.cpu().view(torch.uint8))
        plain = check_norm(x, r, w, 1e-6, offset, with_q=False)
        assert torch.equal(bits(plain[0]), bits(first[0]))


@pytest.mark.parametrize("rows,cols", [(600, 7168), (2000, 256), (1025, 1024), (4099, 128)])
def test_norm_of_many_rows_equals_that_of_few(rows, cols):
    rng = np.random.default_rng(rows)
    x, r, w = normal(rng, (rows, cols), BF16), normal(rng, (rows, cols), BF16), normal(rng, (cols,), BF16)

    def call(a, b):
        o, h, q = torch.empty_like(a), torch.empty_like(a), torch.empty(a.shape, dtype=torch.int8, device="cuda")
        s, n = (torch.empty(a.shape[0], device="cuda") for _ in range(2))
        epi.rms_norm_fwd(a, w, o, 1e-5, residual=b, residual_out=h, q=q, scale=s, rstd=n)
        return o, h, q, s, n

    whole = call(x, r)
    check_norm(x, r, w, 1e-5, 0)
    for at, n in ((0, rows), (5, 700 if rows > 705 else 300), (rows - 520, 520)):
        part = call(x[at:at + n], r[at:at + n])
        for a, b in zip(part, whole):
            assert torch.equal(a, b[at:at + n])


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_of_rows_that_are_zero_or_not_finite(dtype):
    x = torch.ones(6, 40, dtype=dtype, device="cuda")
    x[1] = 0
    x[2, 7], x[3, 0] = float("inf"), float("nan")
    x[4] = torch.finfo(dtype).tiny
    w = torch.ones(40, dtype=dtype, device="cuda")
    out, q, scale = torch.empty_like(x), torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    epi.rms_norm_fwd(x, w, out, 1e-6, q=q, scale=scale)
    got = out.float().cpu()
    assert bool((got[[1]] == 0).all()) and bool(scale[1] == 0) and bool((q[1] == 0).all())
    assert torch.isnan(got[2, 7]) and bool((got[2, :7] == 0).all())   # inf / inf, and 1 / inf
    assert bool(torch.isnan(got[3]).all())
    for r in (2, 3):
        assert torch.isnan(scale[r]) and bool((q[r] == 0).all())
    one = float(torch.tensor(1 / np.sqrt(1 + 1e-6)).to(dtype))
    for r in (0, 5):
        assert bool((got[r] == one).all() if dtype != F32 else ((got[r] - one).abs() < 4e-7).all())
        assert bool((q[r] == 127).all())
    epi.rms_norm_fwd(x[1:2], w, out[1:2], 0.0)             # 0 / 0
    assert bool(torch.isnan(out[1]).all())


@pytest.mark.parametrize("dtype,weight", PAIRS)
@pytest.mark.parametrize("cols", COLS)
def test_norm_gradients(dtype, weight, cols):
    rng = np.random.default_rng(cols + 1)
    for rows, offset, with_h, with_w in ((1, 0, True, True), (3, 1, False, True), (70, 0, True, True), (5, 0, True, False),
                                         (300, 0, False, True), (300, 1, True, True)):
        h, g = normal(rng, (rows, cols), dtype, 3.0), normal(rng, (rows, cols), dtype)
        gh = normal(rng, (rows, cols), dtype) if with_h else None
        w = (1 + 0.2 * normal(rng, (cols,), F32)).to(weight)
        n = ref.norm(ref.f64(h), ref.f64(w), 1e-6)[1].astype(np.float32)
        gx = sentinel((rows, cols), dtype, offset)
        gw = sentinel((cols,), weight, offset) if with_w else None
        ws = space(epi.rms_norm_bwd_workspace_bytes(rows, cols)) if with_w else None
        epi.rms_norm_bwd(placed(g, offset), placed(h, offset), placed(w, offset), torch.from_numpy(n).cuda(), gx, gw, ws,
                         grad_residual=None if gh is None else placed(gh, offset))
        dx, slack, dw, slack_w = ref.norm_grads(ref.f64(g), ref.f64(h), ref.f64(w), n.astype(np.float64),
                                                None if gh is None else ref.f64(gh))
        check(gx, dx, slack, dtype, "grad_x")
        if with_w:
            check(gw, dw, slack_w, weight, "grad_weight")


def test_norm_gradients_of_no_rows():
    w = torch.ones(24, device="cuda")
    none, gw = torch.empty(0, 24, device="cuda"), sentinel((24,), F32)
    epi.rms_norm_bwd(none, none, w, none[:, 0].contiguous(), torch.empty_like(none), gw,
                     space(epi.rms_norm_bwd_workspace_bytes(0, 24)))
    assert bool((gw == 0).all())
    epi.rms_norm_fwd(none, w, torch.empty_like(none), 1e-6)


@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradients_against_differences(residual):
    """Along a direction d of unit-size entries, a central difference of step s of the loss L = sum y g + sum h gh is
    its derivative up to s^2 |L'''| / 6 and what float32 changes of L over s. The third derivative along d is below
    60 |g| |w| |d|^3 / |h|^2 summed over entries of about 1; with s = 2^-7 both errors are below 2e-3 of
    sum |g| + |gh|."""
    rng = np.random.default_rng(3)
    rows, cols, s = 6, 200, 2.0 ** -7
    x, r, w = normal(rng, (rows, cols), F32), normal(rng, (rows, cols), F32), 1 + 0.2 * normal(rng, (cols,), F32)
    g, gh = normal(rng, (rows, cols), F32), normal(rng, (rows, cols), F32)
    leaves = [t.clone().requires_grad_() for t in ((x, w, r) if residual else (x, w))]

    def loss(x, w, r=None):
        if r is None:
            return (epi.RmsNorm.apply(x, w, 1e-6).double() * g).sum()
        y, h = epi.RmsNorm.apply(x, w, 1e-6, r)
        return (y.double() * g).sum() + (h.double() * gh).sum()

    loss(*leaves).backward()
    size = float(g.abs().sum() + gh.abs().sum())
    for i, leaf in enumerate(leaves):
        d = torch.sign(normal(rng, leaf.shape, F32))
        moved = [[t.detach() + sign * s * d if j == i else t.detach() for j, t in enumerate(leaves)] for sign in (1, -1)]
        num = float(loss(*moved[0]) - loss(*moved[1])) / (2 * s)
        assert abs(num - float((leaf.grad.double() * d).sum())) <= 2e-3 * size


def test_norm_helpers_and_autograd_take_any_strides():
    rng = np.random.default_rng(4)
    x, r = normal(rng, (5, 6, 48), BF16).transpose(0, 1), normal(rng, (6, 5, 48), BF16)
    w = normal(rng, (48,), F32)
    y, h = epi.rms_norm(x, w, 1e-6, r)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    q, scale, h2 = epi.rms_norm_int8(x, w, 1e-6, r)
    assert torch.equal(h, h2) and q.shape == x.shape and scale.shape == (6, 5)
    a = x.reshape(30, 48).t().contiguous().t().requires_grad_()
    b, c = r.reshape(30, 48).clone().requires_grad_(), w.clone().requires_grad_()
    y2, h3 = epi.RmsNorm.apply(a, c, 1e-6, b)
    assert torch.equal(y2.view(y.shape), y) and torch.equal(h3.view(h.shape), h)
    (y2.sum() + h3.sum()).backward()                       # gradients of sums: stride 0
    one = torch.ones_like(h3)
    gx, gw = torch.empty_like(one), torch.empty_like(w)
    n = torch.empty(30, device="cuda")
    epi.rms_norm_fwd(h3.detach(), w, gx, 1e-6, rstd=n)
    epi.rms_norm_bwd(one, h3.detach(), w, n, gx, gw, space(epi.rms_norm_bwd_workspace_bytes(30, 48)), grad_residual=one)
    assert torch.equal(a.grad, gx) and torch.equal(b.grad, gx) and torch.equal(c.grad, gw)
    a.grad = b.grad = None
    epi.RmsNorm.apply(a, c, 1e-6, b)[1].backward(one)      # the sum alone
    assert torch.equal(a.grad, one) and torch.equal(b.grad, one)


# ---- the router's product ------------------------------------------------------------------

SIZES = [(1, 1, 1), (1, 7168, 64), (2, 64, 8), (3, 100, 5), (16, 1001, 60), (31, 512, 64), (33, 2048, 256), (64, 128, 1024),
         (65, 40, 12), (127, 7168, 64), (130, 32, 4), (257, 1056, 128), (300, 16, 33), (1000, 72, 65), (2050, 264, 16)]


@pytest.mark.parametrize("dtype,weight", PAIRS)
@pytest.mark.parametrize("tokens,hidden,experts", SIZES)
def test_router_logits(dtype, weight, tokens, hidden, experts):
    rng = np.random.default_rng(tokens + hidden)
    x, w = normal(rng, (tokens, hidden), dtype), normal(rng, (experts, hidden), weight)
    want, slack = ref.product(ref.f64(x), ref.f64(w).T)
    ws = space(epi.moe_router_logits_workspace_bytes(tokens, hidden, experts))
    found = []
    for offset in (0, 1):
        logits = sentinel((tokens, experts), F32)
        epi.moe_router_logits_fwd(placed(x, offset), placed(w, offset), logits, ws)
        check(logits, want, slack, F32, "logits")
        found.append(logits)
    logits = sentinel((tokens, experts), F32)
    epi.moe_router_logits_fwd(x, w, logits, ws)            # the workspace as the last call left it
    assert torch.equal(bits(logits), bits(found[0]))


@pytest.mark.parametrize("dtype,weight", PAIRS)
def test_router_logits_of_whole_numbers_are_exact(dtype, weight):
    """Sums of small whole numbers need no rounding in any order, so every product is counted once."""
    rng = np.random.default_rng(7)
    for tokens, hidden, experts in ((5, 333, 7), (40, 4096, 64), (200, 2056, 100), (513, 160, 64)):
        x = torch.from_numpy(rng.integers(-8, 9, (tokens, hidden))).to(dtype).cuda()
        w = torch.from_numpy(rng.integers(-8, 9, (experts, hidden))).to(weight).cuda()
        g = torch.from_numpy(rng.integers(-8, 9, (tokens, experts))).float().cuda()
        assert torch.equal(epi.moe_router_logits(x, w).double().cpu(), x.double().cpu() @ w.double().cpu().T)
        gx, gw = sentinel(x.shape, dtype), sentinel(w.shape, weight)
        epi.moe_router_logits_bwd(g, x, w, gx, gw, space(epi.moe_router_logits_bwd_workspace_bytes(tokens, hidden, experts)))
        assert torch.equal(gx.cpu(), (g.double().cpu() @ w.double().cpu()).to(dtype))
        assert torch.equal(gw.cpu(), (g.double().cpu().T @ x.double().cpu()).to(weight))


@pytest.mark.parametrize("dtype,weight", [(BF16, F32), (F16, F32), (F32, F32)])
def test_router_products_keep_all_bits_of_float32(dtype, weight):
    """One product per sum: what is off is at most four of the smallest pairs of pieces, and a rounding."""
    rng = np.random.default_rng(8)
    x, w = normal(rng, (300, 1), dtype), normal(rng, (64, 1), weight)
    want = ref.f64(x) @ ref.f64(w).T
    check(epi.moe_router_logits(x, w), want, 6 * ref.EPS * np.abs(want), F32, "logits")
    if dtype == F32:
        g, gx = normal(rng, (300, 1), F32), sentinel((300, 64), F32)
        epi.moe_router_logits_bwd(g, normal(rng, (300, 64), F32), w.T.contiguous(), gx, None)
        want = ref.f64(g) @ ref.f64(w).T
        check(gx, want, 6 * ref.EPS * np.abs(want), F32, "grad_x")


@pytest.mark.parametrize("dtype,weight", PAIRS)
@pytest.mark.parametrize("tokens,hidden,experts", SIZES)
def test_router_logits_gradients(dtype, weight, tokens, hidden, experts):
    rng = np.random.default_rng(tokens + hidden + 1)
    x, w = normal(rng, (tokens, hidden), dtype), normal(rng, (experts, hidden), weight)
    g = normal(rng, (tokens, experts), F32, 1e-3)
    ws = space(epi.moe_router_logits_bwd_workspace_bytes(tokens, hidden, experts))
    want_x, slack_x = ref.product(ref.f64(g), ref.f64(w), 3 if dtype == F32 else 2)
    want_w, slack_w = ref.product(ref.f64(g).T, ref.f64(x), 3 if weight == F32 else 2)
    for offset in (0, 1):
        gx, gw = sentinel(x.shape, dtype, offset), sentinel(w.shape, weight, offset)
        epi.moe_router_logits_bwd(g, placed(x, offset), placed(w, offset), gx, gw, ws)
        check(gx, want_x, slack_x, dtype, "grad_x")
        check(gw, want_w, slack_w, weight, "grad_weight")
        gx2, gw2 = sentinel(x.shape, dtype, offset), sentinel(w.shape, weight, offset)
        epi.moe_router_logits_bwd(g, placed(x, offset), placed(w, offset), gx2, None)
        epi.moe_router_logits_bwd(g, placed(x, offset), placed(w, offset), None, gw2, ws)
        assert torch.equal(bits(gx), bits(gx2)) and torch.equal(bits(gw), bits(gw2))


@pytest.mark.parametrize("dtype,weight", PAIRS)
@pytest.mark.parametrize("hidden", [1, 2, 3, 5])
def test_router_weight_gradient_of_short_rows(dtype, weight, hidden):
    """Rows shorter than a lane's load, in numbers around a step's and a part's."""
    rng = np.random.default_rng(33)
    for tokens in (31, 32, 33, 34, 65, 66, 97, 130, 161, 290):
        x, g = normal(rng, (tokens, hidden), dtype), normal(rng, (tokens, 6), F32)
        gw = sentinel((6, hidden), weight)
        epi.moe_router_logits_bwd(g, x, normal(rng, (6, hidden), weight), None, gw,
                                  space(epi.moe_router_logits_bwd_workspace_bytes(tokens, hidden, 6)))
        check(gw, *ref.product(ref.f64(g).T, ref.f64(x)), weight, "grad_weight")


def test_router_logits_of_no_tokens():
    w, none = torch.ones(8, 16, device="cuda"), torch.empty(0, 16, device="cuda")
    assert epi.moe_router_logits(none, w).shape == (0, 8)
    gw = sentinel((8, 16), F32)
    epi.moe_router_logits_bwd(torch.empty(0, 8, device="cuda"), none, w, torch.empty_like(none), gw,
                              space(epi.moe_router_logits_bwd_workspace_bytes(0, 16, 8)))
    assert bool((gw == 0).all())


@pytest.mark.parametrize("dtype,weight", PAIRS)
def test_router_logits_with_infinities_and_nans(dtype, weight):
    """They reach the token or the expert that has them, and no other."""
    rng = np.random.default_rng(9)
    x, w = normal(rng, (40, 160), dtype), normal(rng, (20, 160), weight)
    clean = epi.moe_router_logits(x, w)
    x[3, 5], x[17, 100], w[6, 7] = float("inf"), float("nan"), float("inf")
    got = epi.moe_router_logits(x, w)
    bad = torch.zeros(40, 20, dtype=torch.bool)
    bad[[3, 17]] = True
    bad[:, 6] = True
    assert not bool(torch.isfinite(got.cpu()[bad]).any())
    assert torch.equal(got.cpu()[~bad], clean.cpu()[~bad])


def test_router_logits_gradients_against_differences():
    """The product is linear in either input: a difference of any step is the derivative, up to rounding."""
    rng = np.random.default_rng(10)
    tokens, hidden, experts = 37, 200, 12
    x, w, g = normal(rng, (tokens, hidden), F32), normal(rng, (experts, hidden), F32), normal(rng, (tokens, experts), F32)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    epi.MoeRouterLogits.apply(xg, wg).backward(g)

    def loss(x, w):
        return float((epi.MoeRouterLogits.apply(x, w).double() * g.double()).sum())

    size = float(((x.abs() + 3).double() @ (w.abs() + 3).double().T * g.abs()).sum())
    for _ in range(3):
        dx, dw = normal(rng, x.shape, F32), normal(rng, w.shape, F32)
        for num, grad, d in (((loss(x + dx, w) - loss(x - dx, w)) / 2, xg.grad, dx),
                             ((loss(x, w + dw) - loss(x, w - dw)) / 2, wg.grad, dw)):
            assert abs(num - float((grad.double() * d.double()).sum())) <= 4 * (hidden + 16) * ref.EPS * size


@pytest.mark.parametrize("dtype,weight", PAIRS)
def test_router_gradients_keep_all_bits_where_terms_cancel(dtype, weight):
    """Sums of two terms that cancel to 2^-12 of their size: a 16-bit result is rounded to 2^-20 of the terms or less, so
    factors of fewer bits than float32 has would show. The other terms are products with 0, which round nothing."""
    rng = np.random.default_rng(31)
    for tokens, hidden, experts in ((3, 40, 5), (200, 264, 40), (70, 136, 100), (40, 72, 300)):
        u = 16 * rng.standard_normal((2, max(tokens, experts)))
        u[1] = -u[0] * (1 + 2.0 ** -12 * u[1])
        # two experts whose rows of the weight are equal
        w, g = normal(rng, (experts, hidden), weight), np.zeros((tokens, experts), np.float32)
        w[experts - 1] = w[1]
        g[:, [1, experts - 1]] = u[:, :tokens].T
        gx, gd = sentinel((tokens, hidden), dtype), torch.from_numpy(g).cuda()
        epi.moe_router_logits_bwd(gd, sentinel((tokens, hidden), dtype), w, gx, None)
        check(gx, *ref.product(g[:, [1, experts - 1]].astype(np.float64), ref.f64(w[[1, experts - 1]])), dtype, "grad_x")
        # two tokens of equal rows
        x, g = normal(rng, (tokens, hidden), dtype), np.zeros((tokens, experts), np.float32)
        x[tokens - 1] = x[1]
        g[[1, tokens - 1]] = u[:, :experts]
        gw, gd = sentinel((experts, hidden), weight), torch.from_numpy(g).cuda()
        epi.moe_router_logits_bwd(gd, x, w, None, gw, space(epi.moe_router_logits_bwd_workspace_bytes(tokens, hidden, experts)))
        check(gw, *ref.product(g[[1, tokens - 1]].astype(np.float64).T, ref.f64(x[[1, tokens - 1]])), weight, "grad_weight")


@pytest.mark.parametrize("dtype,weight", [(BF16, F32), (F16, F32), (F32, F32)])
def test_router_products_of_the_largest_float32(dtype, weight):
    """Finite float32 factors above the largest bfloat16, which round to an infinite one, have finite products."""
    rng = np.random.default_rng(32)
    tokens, hidden, experts = 150, 200, 20
    largest = np.finfo(np.float32).max
    beyond = np.array([largest, -largest, 3.395e38, -3.397e38, 3.39e38, 3.3895314e38, -3.38e38], np.float32)

    def put(shape):
        """One of them in each row, zeros in the rest."""
        a = np.zeros(shape, np.float32)
        a[np.arange(shape[0]), rng.integers(0, shape[1], shape[0])] = rng.choice(beyond, shape[0])
        return torch.from_numpy(a).cuda()

    def small(shape, to):
        return normal(rng, shape, to).clamp(-3, 3) * 2.0 ** -6

    x, w = small((tokens, hidden), dtype), put((experts, hidden))
    check(epi.moe_router_logits(x, w), *ref.product(ref.f64(x), ref.f64(w).T), F32, "logits")
    if dtype == F32:
        x, w = put((tokens, hidden)), small((experts, hidden), F32)
        check(epi.moe_router_logits(x, w), *ref.product(ref.f64(x), ref.f64(w).T), F32, "logits")
    g, x = put((tokens, experts)), small((tokens, hidden), dtype)
    gw = sentinel((experts, hidden), weight)
    g[1:] *= 2.0 ** -6                                     # a sum over the tokens has one of the largest
    g[1:, 3] = 0
    epi.moe_router_logits_bwd(g, x, w, None, gw, space(epi.moe_router_logits_bwd_workspace_bytes(tokens, hidden, experts)))
    check(gw, *ref.product(ref.f64(g).T, ref.f64(x)), weight, "grad_weight")
    if dtype != F16:                                       # whose results would be infinite
        g, w, gx = put((tokens, experts)), small((experts, hidden), weight), sentinel((tokens, hidden), dtype)
        epi.moe_router_logits_bwd(g, x, w, gx, None)
        check(gx, *ref.product(ref.f64(g), ref.f64(w)), dtype, "grad_x")
        g, w = small((tokens, experts), F32), put((experts, hidden)) * 2.0 ** -3
        w[1] = float(largest)
        epi.moe_router_logits_bwd(g, x, w, gx, None)
        check(gx, *ref.product(ref.f64(g), ref.f64(w)), dtype, "grad_x")


@pytest.mark.parametrize("dtype,weight", PAIRS)
def test_router_gradients_with_infinities_and_nans(dtype, weight):
    """They reach the sums that have them among their factors, and no other."""
    rng = np.random.default_rng(34)
    tokens, hidden, experts = 70, 200, 20
    x, w, g = normal(rng, (tokens, hidden), dtype), normal(rng, (experts, hidden), weight), normal(rng, (tokens, experts), F32)

    def call():
        gx, gw = sentinel(x.shape, dtype), sentinel(w.shape, weight)
        epi.moe_router_logits_bwd(g, x, w, gx, gw, space(epi.moe_router_logits_bwd_workspace_bytes(tokens, hidden, experts)))
        return gx.cpu(), gw.cpu()

    clean = call()
    g[3, 5], g[69, 7], x[17, 100], w[6, 9] = float("inf"), float("nan"), -float("inf"), float("inf")
    bad = torch.zeros(tokens, hidden, dtype=torch.bool), torch.zeros(experts, hidden, dtype=torch.bool)
    bad[0][[3, 69]] = bad[0][:, 9] = True
    bad[1][[5, 7]] = bad[1][:, 100] = True
    for got, want, of in zip(call(), clean, bad):
        assert not bool(torch.isfinite(got[of]).any())
        assert torch.equal(got[~of], want[~of])


# ---- choice of the experts ----------------------------------------------------------------------

FORMS = [dict(score=s, bias=b, groups=g) for s in ("softmax", "sigmoid") for b in (False, True)
         for g in ((1, 1, "max"), (4, 2, "max"), (4, 3, "top2"))]
SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 2), (7, 12, 3), (40, 64, 8), (33, 60, 6), (65, 128, 8), (50, 256, 8), (20, 300, 17),
          (9, 1024, 64), (5, 1000, 33), (300, 16, 4)]


def run_route(logits, top_k, bias, form, renormalise=True, scale=1.0):
    groups, top_groups, group_score = form["groups"]
    ids, weights = sentinel((logits.shape[0], top_k), torch.int32), sentinel((logits.shape[0], top_k), F32)
    epi.moe_route_fwd(logits, ids, weights, bias=bias, score=form["score"], groups=groups, top_groups=top_groups,
                      group_score=group_score, renormalise=renormalise, scale=scale)
    return ids, weights


def check_route(logits, top_k, bias, form, renormalise, scale):
    groups, top_groups, group_score = form["groups"]
    want = ref.route(ref.f64(logits), top_k, None if bias is None else ref.f64(bias), form["score"], groups, top_groups,
                     group_score)
    ids, weights = run_route(logits, top_k, bias, form, renormalise, scale)
    assert np.array_equal(ids.cpu().numpy(), want)
    w, slack = ref.weights(ref.f64(logits), want, form["score"], renormalise, scale)
    check(weights, w, slack, F32, "weights")
    return ids, weights


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f['score']}-{'bias' if f['bias'] else 'plain'}-{f['groups']}")
@pytest.mark.parametrize("tokens,experts,top_k", SHAPES)
def test_route(form, tokens, experts, top_k):
    groups, top_groups, group_score = form["groups"]
    if experts % groups or (groups > 1 and (experts // groups < 2 or top_k > top_groups * (experts // groups))):
        pytest.skip("no such groups")
    rng = np.random.default_rng(tokens + experts)
    for dtype in DTYPES:
        for renormalise, scale, spread in ((True, 1.0, 1.0), (False, 2.5, 6.0)):
            logits = normal(rng, (tokens, experts), dtype, spread)
            bias = normal(rng, (experts,), F32, 0.1) if form["bias"] else None
            check_route(logits, top_k, bias, form, renormalise, scale)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f['score']}-{'bias' if f['bias'] else 'plain'}-{f['groups']}")
def test_route_at_ties_masks_and_borders(form):
    """Equal logits, all equal, neighbouring float32 values, masked experts, tokens with few or none left, NaN and
    infinite logits."""
    rng = np.random.default_rng(12)
    experts, top_k = 32, 5
    base = rng.standard_normal((80, experts)).astype(np.float32)
    base[0] = 0
    base[1] = 3
    base[2:12] = rng.integers(-1, 2, (10, experts))                     # many ties
    base[12:22] = np.float32(0.5) + rng.integers(0, 3, (10, experts)).astype(np.float32) * np.float32(2 ** -24)
    base[22:32][rng.random((10, experts)) < 0.7] = -np.inf
    base[32] = -np.inf
    base[33] = -np.inf
    base[33, 9] = 1
    base[34, 3] = np.nan
    base[35] = np.nan
    base[36, [4, 20]] = np.inf
    base[37] = -120 - np.arange(experts, dtype=np.float32)              # sigmoids that underflow
    base[38] = np.finfo(np.float32).min                                 # a mask of the type's lowest value for all
    base[39, 1:] = np.finfo(np.float32).min
    base[40:50] = np.float32(10) + rng.integers(0, 4, (10, experts)).astype(np.float32) * np.float32(2 ** -20)
    base[50] *= 1e4
    for bias in ([None] if not form["bias"] else
                 [rng.standard_normal(experts) * 0.1, np.zeros(experts), np.where(np.arange(experts) % 3 == 0, -np.inf, 0.25),
                  np.where(np.arange(experts) == 7, np.nan, 0.0)]):
        b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
        for renormalise, scale in ((True, 1.0), (False, 1.0)):
            logits = torch.from_numpy(base).cuda()
            fine = [t for t in range(80) if t not in (34, 35, 36)]
            check_route(logits[fine], top_k, b, form, renormalise, scale)
            ids, weights = run_route(logits, top_k, b, form, renormalise, scale)
            bad = [34, 35] + ([36] if form["score"] == "softmax" else [])
            assert bool(torch.isnan(weights[bad]).all())
            for t in (34, 35, 36):
                found = [e for e in ids[t].tolist() if e != -1]
                assert len(set(found)) == len(found) and all(0 <= e < experts for e in found)
            if form["score"] == "sigmoid" and b is None:
                check_route(logits[36:37], top_k, b, form, renormalise, scale)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f['score']}-{'bias' if f['bias'] else 'plain'}-{f['groups']}")
def test_a_tokens_choice_is_the_same_in_calls_of_all_sizes(form):
    rng = np.random.default_rng(13)
    logits, bias = normal(rng, (5000, 64), F32), normal(rng, (64,), F32, 0.1) if form["bias"] else None
    ids, weights = run_route(logits, 8, bias, form)
    for at, n in ((0, 1), (4999, 1), (7, 33), (100, 1025)):
        a, b = run_route(logits[at:at + n], 8, bias, form)
        assert torch.equal(a, ids[at:at + n]) and torch.equal(b, weights[at:at + n])


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f['score']}-{'bias' if f['bias'] else 'plain'}-{f['groups']}")
@pytest.mark.parametrize("experts,top_k", [(16, 5), (64, 8), (256, 8), (320, 12)])
def test_route_with_experts_that_finite_values_switch_off(form, experts, top_k):
    """Biases and logits far below all others leave the others' order as it is, also that of near ones; so does a
    bias far above."""
    rng = np.random.default_rng(experts)
    base = rng.standard_normal((300, experts)).astype(np.float32)
    base[:, 9] = base[:, 4] + rng.integers(-1, 2, 300).astype(np.float32) * np.float32(2 ** -21)
    base[:, [4, 9]] += 2
    off = rng.choice(experts, 3, replace=False)
    for value in (-1e4, -1e9, -3.4e38, 1e9):
        logits, bias = base.copy(), None
        if form["bias"]:
            bias = rng.standard_normal(experts).astype(np.float32) * np.float32(0.01)
            bias[9] = bias[4]
            bias[off] = value
            bias = torch.from_numpy(bias).cuda()
        else:
            logits[:, off] = -abs(value)
        check_route(torch.from_numpy(logits).cuda(), top_k, bias, form, True, 1.0)


@pytest.mark.parametrize("offset", [0.02, 1.02, 16.02, 17.0, 33.0, 64.1, 130.0, 513.0])
@pytest.mark.parametrize("experts,top_k", [(16, 8), (16, 11), (200, 8)])
def test_route_by_scores_that_a_common_bias_makes_coarse(offset, experts, top_k):
    """With a large part in common float32's biased scores are an ulp of that part apart, and each of two is off by up to
    half of it. A token's first two experts are within 2^-25 of a border between two float32 values, where what their
    scores are off decides to which side each goes: they keep the order of 64 bits."""
    rng = np.random.default_rng(int(offset) + experts + top_k)
    tokens = 1500
    for spread in (0.05, 0.2, 0.4):
        bias = (offset + rng.uniform(0, spread, experts)).astype(np.float32)
        bias[[2, experts - 1]] = np.float32(offset + spread), np.float32(offset + 1.01 * spread)
        logits = rng.uniform(-0.3, 0.3, (tokens, experts))
        ulp = float(np.spacing(np.float32(offset + spread + 0.6)))
        border = (np.floor((offset + spread + rng.uniform(0.6, 0.7, tokens)) / ulp) + 0.5) * ulp
        for e in (2, experts - 1):
            s = border - float(bias[e]) + rng.uniform(-1, 1, tokens) * 2.0 ** -25
            logits[:, e] = np.log(s / (1 - s))
        check_route(torch.from_numpy(logits.astype(np.float32)).cuda(), top_k, torch.from_numpy(bias).cuda(),
                    dict(score="sigmoid", groups=(1, 1, "max")), True, 1.0)


@pytest.mark.parametrize("size", [2, 3, 4])
@pytest.mark.parametrize("offset", [0.5, 4.0, 16.0, 32.0, 100.0])
def test_route_by_groups_whose_biases_cancel(offset, size):
    """A group's two best have biases of opposite sign: the roundings of both stay in their sum, which is small. Groups
    that are nearer than those keep the order of 64 bits."""
    rng = np.random.default_rng(int(offset) + size)
    groups, tokens = 4, 1500
    bias = np.full((groups, size), -4 * offset) + rng.uniform(-0.05, 0.05, (groups, size))
    bias[:, 0] += 5 * offset
    bias[:, 1] += 3 * offset
    bias = bias.astype(np.float32)
    logits = rng.uniform(-0.3, 0.3, (tokens, groups, size)).astype(np.float32)
    s = ref.scores(logits.astype(np.float64), "sigmoid") + bias
    for g in (1, 2, 3):                                    # the sum of the first group, by the second expert's score
        want = s[:, 0, :2].sum(1) - s[:, g, 0] - float(bias[g, 1]) + rng.uniform(-1, 1, tokens) * 2.0 ** -22
        logits[:, g, 1] = np.log(want / (1 - want))
    logits = torch.from_numpy(logits.reshape(tokens, groups * size)).cuda()
    check_route(logits, 4, torch.from_numpy(bias.reshape(-1)).cuda(), dict(score="sigmoid", groups=(groups, 2, "top2")), True,
                1.0)


@pytest.mark.parametrize("size", [2, 3])
def test_route_by_groups_whose_sums_are_beyond_float32(size):
    """Sums of two finite biases that float32 does not hold, an infinite bias, and groups with fewer than two experts."""
    rng = np.random.default_rng(size)
    tokens = 40
    for best in ([2.0e38, 2.5e38, 3e38, 1e38], [3e38, 3e38, 3.1e38, 3e38], [np.inf, 1.0, 3e38, np.inf],
                 [-np.inf, 1.0, 2.0, -np.inf], [-3e38, -2e38, -2.5e38, -3.1e38]):
        bias = np.array(best)[:, None] * np.linspace(1, 0.9, size)
        for score in ("sigmoid", "softmax"):
            check_route(normal(rng, (tokens, 4 * size), F32), 4, torch.from_numpy(bias.reshape(-1).astype(np.float32)).cuda(),
                        dict(score=score, groups=(4, 2, "top2")), True, 1.0)


GRADS = [(s, r) for s in ("softmax", "sigmoid") for r in (False, True)]


@pytest.mark.parametrize("score,renormalise", GRADS)
@pytest.mark.parametrize("tokens,experts,top_k", SHAPES)
def test_route_gradient(score, renormalise, tokens, experts, top_k):
    rng = np.random.default_rng(tokens + experts + 1)
    for dtype in DTYPES:
        logits = normal(rng, (tokens, experts), dtype, 2.0)
        ids = np.argsort(rng.random((tokens, experts)), 1)[:, :top_k].astype(np.int32)
        ids[rng.random(ids.shape) < 0.1] = -1
        ids[0, 0] = experts                                # no expert
        if top_k > 1:
            ids[-1, 1] = ids[-1, 0] = 0                    # the same one twice
        grad = normal(rng, (tokens, top_k), F32)
        got = sentinel((tokens, experts), dtype)
        epi.moe_route_bwd(grad, logits, torch.from_numpy(ids).cuda(), got, score=score, renormalise=renormalise, scale=1.7)
        want, slack = ref.route_grad(ref.f64(grad), ref.f64(logits), ids, score, renormalise, float(np.float32(1.7)))
        check(got, want, slack, dtype, "grad_logits")


@pytest.mark.parametrize("score,renormalise", GRADS)
def test_route_gradient_of_masked_experts_and_empty_tokens(score, renormalise):
    rng = np.random.default_rng(14)
    base = rng.standard_normal((9, 24)).astype(np.float32)
    base[1:5][rng.random((4, 24)) < 0.6] = -np.inf
    base[5] = -np.inf
    base[6] = np.finfo(np.float32).min
    base[7] = -120 - np.arange(24)
    base[8] = 100 + np.arange(24)
    logits = torch.from_numpy(base).cuda()
    ids, _ = epi.moe_route(logits, 6, score=score)
    assert bool((ids[5] == -1).all())
    grad = normal(rng, (9, 6), F32)
    grad[ids < 0] = float("nan")                           # of slots without an expert, not used
    got = sentinel((9, 24), F32)
    epi.moe_route_bwd(grad, logits, ids, got, score=score, renormalise=renormalise)
    want, slack = ref.route_grad(ref.f64(grad), base.astype(np.float64), ids.cpu().numpy(), score, renormalise)
    check(got, want, slack, F32, "grad_logits")
    assert bool((got[torch.from_numpy(np.isneginf(base)).cuda()] == 0).all())


@pytest.mark.parametrize("score,renormalise", GRADS)
def test_route_gradient_against_differences(score, renormalise):
    """With the ids fixed, a central difference of step s = 2^-6 along a direction of entries +-1 is the derivative up
    to s^2 / 6 of the third derivative, which is below 26 |g| times the weights' sum, and what float32 changes of the
    loss over s: below 2e-3 of sum |g| together."""
    rng = np.random.default_rng(15)
    tokens, experts, top_k, s = 20, 16, 4, 2.0 ** -6
    logits, g = normal(rng, (tokens, experts), F32), normal(rng, (tokens, top_k), F32)
    leaf = logits.clone().requires_grad_()
    ids, w = epi.MoeRoute.apply(leaf, top_k, None, score, 1, 1, "max", renormalise, 1.0)
    w.backward(g)
    assert not ids.requires_grad
    fixed = ids.long()

    def loss(l):
        # the same experts, whatever their order now: the scores of all of them, then those of the ids
        every, weights = epi.moe_route(l, experts, score=score, renormalise=False)
        p = torch.zeros_like(l).scatter_(1, every.long(), weights).gather(1, fixed).double()
        if renormalise:
            p = p / p.sum(1, keepdim=True)
        return float((p * g).sum())

    d = torch.sign(normal(rng, logits.shape, F32))
    num = (loss(logits + s * d) - loss(logits - s * d)) / (2 * s)
    assert abs(num - float((leaf.grad.double() * d).sum())) <= 2e-3 * float(g.abs().sum())


def test_route_of_no_tokens():
    ids, weights = epi.moe_route(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == weights.shape == (0, 4)
    none = torch.empty(0, 16, device="cuda")
    epi.moe_route_bwd(weights, none, ids, torch.empty_like(none))


# ---- together -----------------------------------------------------------------------------------

def layer(hidden, inter, experts, seed):
    rng = np.random.default_rng(seed)
    return {"norm": (1 + 0.1 * normal(rng, (hidden,), F32)), "router": normal(rng, (experts, hidden), F32, hidden ** -0.5),
            "gate": normal(rng, (experts, inter, hidden), BF16, hidden ** -0.5),
            "up": normal(rng, (experts, inter, hidden), BF16, hidden ** -0.5),
            "down": normal(rng, (experts, hidden, inter), BF16, inter ** -0.5)}


@pytest.mark.parametrize("tokens", [1, 5, 96])
def test_a_whole_layer_in_a_graph(tokens):
    """Norm into 8-bit rows, router, choice, order, products, weighted sum: captured once and replayed on other
    inputs, equal to the eager calls, and near the layer in float64."""
    hidden, inter, experts, top_k = 256, 128, 12, 3
    p = layer(hidden, inter, experts, tokens)
    rng = np.random.default_rng(tokens + 100)
    gate, up, down = (epi.quantize_rows_int8(p[n]) for n in ("gate", "up", "down"))
    slots, new = tokens * top_k, lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    x, stream, normed, out = new(tokens, hidden), new(tokens, hidden), new(tokens, hidden), new(tokens, hidden)
    q, scale = new(tokens, hidden, dtype=torch.int8), new(tokens, dtype=F32)
    logits, ids, weights = new(tokens, experts, dtype=F32), new(tokens, top_k, dtype=torch.int32), new(tokens, top_k, dtype=F32)
    ws = space(epi.moe_router_logits_workspace_bytes(tokens, hidden, experts))
    offs, row_of, slot_of = (new(*s, dtype=torch.int32) for s in ((experts,), (tokens, top_k), (slots,)))
    sort_ws = space(epi.moe_sort_workspace_bytes(tokens, top_k, experts))
    y, yq, ys, rows = torch.zeros(slots, inter, dtype=BF16, device="cuda"), new(slots, inter, dtype=torch.int8), \
        new(slots, dtype=F32), new(slots, hidden)

    def step():
        epi.rms_norm_fwd(x, p["norm"], normed, 1e-6, residual=stream, residual_out=stream, q=q, scale=scale)
        epi.moe_router_logits_fwd(normed, p["router"], logits, ws)
        epi.moe_route_fwd(logits, ids, weights, score="sigmoid", scale=2.0)
        epi.moe_sort_fwd(ids, 0, offs, row_of, slot_of, sort_ws)
        epi.grouped_gate_up_swiglu_int8_fwd(q, scale, slot_of, top_k, *gate, *up, offs, None, y, 10.0)
        epi.quantize_rows_int8_fwd(y, yq, ys)
        epi.grouped_down_router_int8_fwd(yq, ys, *down, offs, None, rows)
        epi.moe_combine_weighted_fwd(rows, row_of, weights, out)
        return [t.clone() for t in (stream, q, scale, logits, ids, weights, row_of, out)]

    def inputs(seed):
        g = np.random.default_rng(seed)
        x.copy_(normal(g, (tokens, hidden), BF16))
        stream.copy_(normal(g, (tokens, hidden), BF16, 2.0))

    inputs(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        found = step()
    for seed in (1, 2, 3):
        inputs(seed)
        want = step()
        inputs(seed)
        first = (x.float() + stream.float()).bfloat16()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(found, want):
            assert torch.equal(a, b)
        assert torch.equal(want[0], first)
        h = ref.f64(first)
        n = ref.norm(h, ref.f64(p["norm"]), 1e-6)[0]
        l = ref.to(BF16, n) @ ref.f64(p["router"]).T
        # ids that differ must be those of two experts within what the normed rows' rounding changes of a logit
        picked = ids.cpu().numpy()
        assert np.abs(ref.f64(want[3]) - l).max() < 2e-2
        w, _ = ref.weights(ref.f64(want[3]), picked, "sigmoid", True, 2.0)
        total = np.zeros((tokens, hidden))
        for t in range(tokens):
            for j, e in enumerate(picked[t]):
                g_, u_ = ref.f64(p["gate"][e]) @ n[t], ref.f64(p["up"][e]) @ n[t]
                g_, u_ = min_max(g_, None, 10.0), min_max(u_, -10.0, 10.0)
                total[t] += w[t, j] * (ref.f64(p["down"][e]) @ (g_ / (1 + np.exp(-g_)) * u_))
        assert np.linalg.norm(ref.f64(want[7]) - total) < 0.03 * np.linalg.norm(total)


def min_max(v, lo, hi):
    return np.clip(v, lo, hi)


def test_gradients_through_norm_router_and_choice():
    """The three autograd wrappers in a row, against torch's gradients of the plain forms in float64. Every step is
    float32: 1e-5 of each gradient's size covers the sums of up to 200 terms."""
    rng = np.random.default_rng(20)
    tokens, hidden, experts, top_k = 50, 200, 16, 4
    leaves = [normal(rng, s, F32) for s in ((tokens, hidden), (tokens, hidden), (hidden,), (experts, hidden))]
    leaves[2] = 1 + 0.1 * leaves[2]
    g, gy, gh = normal(rng, (tokens, top_k), F32), normal(rng, (tokens, hidden), F32), normal(rng, (tokens, hidden), F32)
    mine = [t.clone().requires_grad_() for t in leaves]
    y, h = epi.RmsNorm.apply(mine[0], mine[2], 1e-6, mine[1])
    ids, w = epi.MoeRoute.apply(epi.MoeRouterLogits.apply(y, mine[3]), top_k)
    ((w * g).sum() + (y * gy).sum() + (h * gh).sum()).backward()
    x, r, nw, rw = theirs = [t.double().cpu().requires_grad_() for t in leaves]
    h = x + r
    y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * nw
    part = torch.log_softmax(y @ rw.T, 1).gather(1, ids.long().cpu())
    loss = (torch.softmax(part, 1) * g.double().cpu()).sum() + (y * gy.double().cpu()).sum() + (h * gh.double().cpu()).sum()
    loss.backward()
    for a, b in zip(mine, theirs):
        a, b = a.grad.double().cpu(), b.grad
        assert float((a - b).norm() / b.norm()) < 1e-5


def test_calls_on_another_stream_and_two_at_once():
    """Each call runs on the stream it is given or the current one; two streams with workspaces of their own."""
    rng = np.random.default_rng(21)
    x, w = normal(rng, (64, 4096), BF16), normal(rng, (64, 4096), BF16)
    g = normal(rng, (64, 64), F32)
    sizes = (64, 4096, 64)
    want = epi.moe_router_logits(x, w)
    gw = torch.empty_like(w)
    epi.moe_router_logits_bwd(g, x, w, None, gw, space(epi.moe_router_logits_bwd_workspace_bytes(*sizes)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    found = [(torch.zeros_like(want), torch.zeros_like(gw)) for _ in streams]
    spaces = [(space(epi.moe_router_logits_workspace_bytes(*sizes)), space(epi.moe_router_logits_bwd_workspace_bytes(*sizes)))
              for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (a, b), (wa, wb) in zip(streams, found, spaces):
            epi.moe_router_logits_fwd(x, w, a, wa, stream=s)
            with torch.cuda.stream(s):
                epi.moe_router_logits_bwd(g, x, w, None, b, wb)
    torch.cuda.synchronize()
    for a, b in found:
        assert torch.equal(a, want) and torch.equal(b, gw)


# ---- large calls ------------------------------------------------------------------------------------

def test_calls_past_2_32_bytes_and_of_several_launches():
    """The last rows of tensors beyond 2^32 bytes, and calls of more rows than one launch has: the same as those rows in
    a call of their own."""
    rows, cols = 330_000, 7168
    x = torch.empty((rows, cols), dtype=BF16, device="cuda")
    x.view(torch.int16).fill_(0x3F80)                      # ones
    tail = slice(rows - 300, rows)
    x[tail] = torch.randn(300, cols, device="cuda").to(BF16)
    w = torch.randn(cols, device="cuda").to(BF16)
    out = torch.empty_like(x)
    epi.rms_norm_fwd(x, w, out, 1e-6)
    part = torch.empty((300, cols), dtype=BF16, device="cuda")
    epi.rms_norm_fwd(x[tail], w, part, 1e-6)
    assert torch.equal(out[tail], part)
    router = torch.randn(8, cols, device="cuda").to(BF16)
    logits = torch.empty((rows, 8), device="cuda")
    epi.moe_router_logits_fwd(x, router, logits, space(epi.moe_router_logits_workspace_bytes(rows, cols, 8)))
    check(logits[tail], *ref.product(ref.f64(x[tail]), ref.f64(router).T), F32, "logits")
    g = torch.randn(rows, 8, device="cuda")
    epi.moe_router_logits_bwd(g, x, router, out, None)
    check(out[tail], *ref.product(ref.f64(g[tail]), ref.f64(router), 2), BF16, "grad_x")
    # the tail alone counts: all other gradients are 0
    g[:rows - 300] = 0
    gw = torch.empty_like(router)
    epi.moe_router_logits_bwd(g, x, router, None, gw, space(epi.moe_router_logits_bwd_workspace_bytes(rows, cols, 8)))
    check(gw, *ref.product(ref.f64(g[tail]).T, ref.f64(x[tail]), 2), BF16, "grad_weight")
    del x, out, logits, g

    rows = (1 << 20) + 77
    x, w = torch.randn(rows, 24, device="cuda"), torch.randn(24, device="cuda")
    out, q, scale = torch.empty_like(x), torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    epi.rms_norm_fwd(x, w, out, 1e-6, q=q, scale=scale)
    few = torch.empty((100, 24), device="cuda")
    epi.rms_norm_fwd(x[-100:], w, few, 1e-6)
    assert torch.equal(out[-100:], few)
    logits = torch.randn(rows, 4, device="cuda")
    ids, weights = epi.moe_route(logits, 2, score="sigmoid", bias=torch.zeros(4, device="cuda"))
    ids2, weights2 = epi.moe_route(logits[-100:], 2, score="sigmoid", bias=torch.zeros(4, device="cuda"))
    assert torch.equal(ids[-100:], ids2) and torch.equal(weights[-100:], weights2)
    gw, gl, gl2 = torch.randn(rows, 2, device="cuda"), torch.empty_like(logits), torch.empty(100, 4, device="cuda")
    epi.moe_route_bwd(gw, logits, ids, gl)
    epi.moe_route_bwd(gw[-100:], logits[-100:], ids[-100:], gl2)
    assert torch.equal(gl[-100:], gl2)
    rows = (1 << 24) + 40
    x, w = torch.randn(rows, 2, device="cuda").to(BF16), torch.randn(3, 2, device="cuda").to(BF16)
    logits = epi.moe_router_logits(x, w)
    for part in (slice(0, 50), slice((1 << 24) - 20, rows)):
        check(logits[part], *ref.product(ref.f64(x[part]), ref.f64(w).T), F32, "logits")


def test_norm_gradients_of_more_columns_than_a_grid_of_blocks():
    """2^28 columns and some: one launch of a block for each 64 of them would have 2^32 work-items."""
    cols = (1 << 28) + 72
    h = torch.randn(1, cols, device="cuda").to(BF16)
    g, w = h.flip(1), torch.ones(cols, dtype=BF16, device="cuda")
    rstd = torch.full((1,), 0.75, device="cuda")
    gx, gw = torch.empty_like(h), sentinel((cols,), BF16)
    epi.rms_norm_bwd(g, h, w, rstd, gx, gw, space(epi.rms_norm_bwd_workspace_bytes(1, cols)))
    assert torch.equal(gw, (g[0].float() * (h[0].float() * 0.75)).to(BF16))   # one row: one product, rounded


@pytest.mark.parametrize("dtype,weight", PAIRS)
def test_router_products_of_small_values(dtype, weight):
    """Factors whose pieces or products leave the normal range of their type: a value that a matrix instruction takes
    for 0 is below 2^-126 in bfloat16 and float32 and 2^-14 in float16, so the sums are right to hidden times that of
    the other factor."""
    rng = np.random.default_rng(30)
    sigma = 2.0 ** -16 if dtype == F16 else 2.0 ** -110
    x, w = normal(rng, (40, 64), dtype, sigma), normal(rng, (16, 64), weight)
    want, slack = ref.product(ref.f64(x), ref.f64(w).T)
    least = 2.0 ** -14 if dtype == F16 and weight == F16 else 2.0 ** -126
    check(epi.moe_router_logits(x, w), want, slack + least * np.abs(ref.f64(w)).sum(1)[None], F32, "logits")


def test_router_products_take_the_least_factors():
    """One product per sum: factors of 16 bits down to their least are taken as they are, float32 ones to 2^-134."""
    for dtype, weight, values in ((BF16, BF16, [2.0 ** -133, 5 * 2.0 ** -133, 2.0 ** -126]),
                                  (F16, F16, [2.0 ** -24, 3 * 2.0 ** -24, 2.0 ** -14]), (F16, F32, [2.0 ** -24, 5 * 2.0 ** -24]),
                                  (F32, F32, [1.2345678e-38, 1.2345678e-36, -7.654321e-40, 1.2345678e-33, 2.0 ** -149])):
        v = torch.tensor(values, device="cuda").to(dtype)
        x, w = torch.zeros(len(values), 72, dtype=dtype, device="cuda"), torch.zeros(5, 72, dtype=weight, device="cuda")
        x[:, 67], w[2, 67], w[3, 67] = v, 1.0, -0.5
        want = ref.f64(x) @ ref.f64(w).T
        check(epi.moe_router_logits(x, w), want, (2.0 ** -134 if dtype == F32 else 0) * np.abs(ref.f64(w)).sum(1)[None] +
              2 * ref.EPS * np.abs(want), F32, "logits")
