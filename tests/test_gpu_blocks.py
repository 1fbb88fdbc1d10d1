"""The operators of a block on the GPU against plain forms in 64 bits on the same
rounded inputs.

Tolerances, all worst cases by arithmetic.  A stored result is off by at most half a
step of its type: u |want| (bf16 2^-8, fp32 2^-24).  What is computed in fp32 before that
is off by at most (number of roundings in a row) u32 times the sum of the magnitudes
of the terms, u32 = 2^-24; each test states that number and forms that sum.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


import gated_deltanet_chunked_delta_amd as gdn  # noqa: E402
from gated_deltanet_chunked_delta_amd import GDNError, blocks  # noqa: E402


def rn(seed, *s, std=1.0, dt=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda", dtype=torch.float64) * std).to(dt)


def ru(seed, lo, hi, *s):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lo + (hi - lo) * torch.rand(*s, generator=g, device="cuda")


def within(name, got, want, scale=None, n=0.0, u=None):
    """|got - want| <= u |want| + n u32 scale, element by element."""
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if want.numel() == 0:
        return
    u = U[got.dtype] if u is None else u
    bound = u * want.abs() + n * U32 * (want.abs() if scale is None else scale) + 1e-37
    off = (got.detach().double() - want).abs() / bound
    worst = float(off.detach().max())
    print(f"    {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, (name, worst)


def rms(got, want):
    return float((got.detach().double() - want).norm() / want.norm())


# ------------------------------------------------------------------ residual norm
def ref_norm(x, w, r, eps):
    s = x.double() if r is None else (x.double() + r.double()).to(r.dtype).double()
    return s, s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps) * w.double()


NORMS = [(1, 1, "bf16", ""), (3, 8, "bf16", "bf16"), (5, 7, "f32", "f32"), (64, 2048, "bf16", "bf16"), (2000, 1024, "bf16", "f32"),
         (1500, 2304, "bf16", "f32"), (1030, 3001, "bf16", "bf16"), (130, 129, "bf16", "f32"), (1100, 515, "f32", "f32"),
         (70, 4096, "f32", ""), (1025, 4095, "bf16", ""), (9, 8191, "bf16", "bf16"), (3, 20001, "bf16", "f32"),
         (2, 9000, "f32", "f32"), (4, 16384, "bf16", ""), (1, 131073, "bf16", "bf16")]


@pytest.mark.parametrize("R,D,dt,res", NORMS)
def test_norm_and_gradients(R, D, dt, res):
    dt = DT[dt]
    x, w = rn(1, R, D, dt=dt), (1 + rn(2, D, std=.2)).to(dt)
    r = rn(3, R, D, std=2., dt=DT[res]) if res else None
    dy = rn(4, R, D, dt=dt)
    ds = rn(5, R, D, dt=r.dtype) if res else None
    s, y = ref_norm(x, w, r, 1e-5)
    rs = 1 / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-5)
    n = s * rs
    dn = dy.double() * w.double()
    c = (dn * n).mean(-1, keepdim=True)
    dv = (dn - n * c) * rs + (0 if ds is None else ds.double())
    dw = (dy.double() * n).sum(0)
    leaves = [t.requires_grad_(True) for t in (x, w, r) if t is not None]
    gy, gs = gdn.add_rms_norm(x, w, r, eps=1e-5)
    if res:
        # (an fp32 sum rounded to bf16: off by another fp32 rounding in front of the tie)
        within("s", gs, x.detach().double() + r.detach().double(), n=1)
        assert torch.equal(gs.double(), s)
    else:
        assert gs is x
    # roundings of an element: square, sum (64 in a thread, 8 steps, 4 waves), mean, sqrt, quotient, two products
    within("y", gy, y, n=100)
    outs, gouts = ([gy, gs], [dy, ds]) if res else ([gy], [dy])
    grads = torch.autograd.grad(outs, leaves, gouts)
    many = 160 + D / 256       # (rows past the registers: a thread's part of a row)
    S = (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True)) * rs + (0 if ds is None else ds.double().abs())
    within("dx", grads[0], dv, S, many)
    within("dw", grads[1], dw, (dy.double() * n).abs().sum(0), 200)
    if res:
        within("dr", grads[2], dv, S, many)
        if dt == r.dtype:
            assert torch.equal(grads[0], grads[2])


def test_norm_gradient_by_differences():
    x, w, r = rn(1, 3, 40), 1 + rn(2, 40, std=.1), rn(3, 3, 40)
    dy, ds = rn(4, 3, 40), rn(5, 3, 40)
    f = lambda a, b, c: ((ref_norm(a, b, None, 1e-5)[1] if c is None else
                          ((a + c) / torch.sqrt((a + c).square().mean(-1, keepdim=True) + 1e-5) * b)) * dy.double()).sum() + ((a + c) * ds.double()).sum()
    leaves = [t.requires_grad_(True) for t in (x, w, r)]
    y, s = gdn.add_rms_norm(x, w, r, eps=1e-5)
    for k, g in enumerate(torch.autograd.grad([y, s], leaves, [dy, ds])):
        d = rn(9 + k, *leaves[k].shape, dt=torch.float64)
        p = [t.detach().double() for t in leaves]
        a, b = [q + (1e-5 * d if j == k else 0) for j, q in enumerate(p)], [q - (1e-5 * d if j == k else 0) for j, q in enumerate(p)]
        want = float((f(*a) - f(*b)) / 2e-5)
        assert abs(float((g.double() * d).sum()) - want) <= 1e-5 * (1 + abs(want))


def test_norm_only_the_gradients_asked_for():
    x, w, r = rn(1, 9, 64), rn(2, 64), rn(3, 9, 64)
    dy = rn(4, 9, 64)
    full = blocks.gdn_addnorm_bwd(x, w, dy)
    for k in range(3):
        need = tuple(j == k for j in range(3))
        part = blocks.gdn_addnorm_bwd(x, w, dy, need=need)
        assert [p is not None for p in part] == list(need) and torch.equal(part[k], full[k])
    y, s = gdn.add_rms_norm(x.requires_grad_(True), w, r)   # the sum's gradient alone
    (g,) = torch.autograd.grad(s, x, dy)
    assert torch.equal(g, dy)


@pytest.mark.parametrize("shape", [(0, 40), (3, 0, 40)])
def test_norm_without_rows(shape):
    x, w, r = torch.zeros(shape, device="cuda"), rn(1, 40), torch.zeros(shape, device="cuda")
    leaves = [t.requires_grad_(True) for t in (x, w, r)]
    y, s = gdn.add_rms_norm(x, w, r)
    dx, dw, dr = torch.autograd.grad([y, s], leaves, [torch.zeros_like(y), torch.zeros_like(s)])
    assert y.shape == s.shape == dx.shape == dr.shape == shape and not dw.any()
    with torch.no_grad():
        q, scale, _ = gdn.add_rms_norm_8bit(x, w, r)
    assert q.shape == shape and scale.shape == shape[:-1]


def test_calls_with_more_dimensions():
    """[..., D] in, [..., N] out, as the same rows flattened."""
    x, w, r, W = rn(1, 2, 3, 5, 48), rn(2, 48), rn(3, 2, 3, 5, 48), rn(4, 20, 48, std=.2)
    flat = lambda t: t.reshape(30, -1)
    for a, b in zip(gdn.add_rms_norm(x, w, r), gdn.add_rms_norm(flat(x), w, flat(r))):
        assert a.shape == (2, 3, 5, 48) and torch.equal(flat(a), b)
    q, s = gdn.quantize_rows(x)
    q2, s2 = gdn.quantize_rows(flat(x))
    assert s.shape == (2, 3, 5) and torch.equal(flat(q.view(torch.uint8)), q2.view(torch.uint8)) and torch.equal(s.reshape(30), s2)
    p, t = gdn.quantize_rows(W)
    y = gdn.linear_8bit(q, s, p, t, out_dtype=torch.float32)
    assert y.shape == (2, 3, 5, 20) and torch.equal(flat(y), gdn.linear_8bit(q2, s2, p, t, out_dtype=torch.float32))
    assert torch.equal(flat(gdn.linear(x, W, None, "gelu")), gdn.linear(flat(x), W, None, "gelu"))


def test_training_step_by_backward():
    """.backward() with a summed loss (an expanded gradient), one leaf used twice."""
    x, w = rn(1, 70, 64, dt=torch.bfloat16).requires_grad_(True), (1 + rn(2, 64, std=.1)).to(torch.bfloat16).requires_grad_(True)
    W = rn(3, 64, 64, std=.1, dt=torch.bfloat16).requires_grad_(True)
    y, s = gdn.add_rms_norm(x, w, x)
    z = gdn.linear(y, W, None, "silu", s)
    h = gdn.gated_recurrence(z[None], z[None], z[None], scale=ru(4, .1, .2, 64))
    h.sum().backward()
    X, w_, W_ = (t.detach().double().requires_grad_(True) for t in (x, w, W))
    S = 2 * X
    Y = S / torch.sqrt(S.square().mean(-1, keepdim=True) + 1e-6) * w_
    v = Y @ W_.t()
    Z = v * torch.sigmoid(v) + S
    ref_rec(Z, Z, Z, ru(4, .1, .2, 64).double(), None, [(0, 70)])[0].sum().backward()
    for a, b in ((x, X), (w, w_), (W, W_)):   # some ten roundings of bf16 along the way, of 1.7e-3 (rms) each
        assert rms(a.grad, b.grad) <= 3e-2


def test_norm_takes_slices_and_leaves_its_inputs():
    wide, wr = rn(1, 33, 500, dt=torch.bfloat16), rn(2, 33, 301)
    x, r, w = wide[:, 3:252], wr[:, 5:254], rn(3, 249, dt=torch.bfloat16)
    keep = wide.clone(), wr.clone()
    a = gdn.add_rms_norm(x, w, r)
    b = gdn.add_rms_norm(x.contiguous(), w, r.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and torch.equal(wide, keep[0]) and torch.equal(wr, keep[1])
    q1, s1, _ = gdn.add_rms_norm_8bit(x, w, r)
    q2, s2, _ = gdn.add_rms_norm_8bit(x.contiguous(), w, r.contiguous())
    assert torch.equal(q1.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s1, s2)


# ------------------------------------------------------------------ 8 bits
def nearest8(v):
    e = torch.clamp(torch.frexp(v).exponent - 1, min=-6)
    step = ((e.to(torch.int64) - 3 + 1023) << 52).view(torch.float64)   # (torch.ldexp is off by a rounding)
    return torch.clamp(torch.round(v / step) * step, -448., 448.)


ROWS8 = [(1, 1), (3, 5), (64, 2048), (1000, 1001), (1100, 2048), (7, 513), (1030, 3001), (5, 20011), (1025, 100)]


@pytest.mark.parametrize("R,D", ROWS8)
def test_rows_of_bf16_in_8_bits_are_exact(R, D):
    """Every quotient rounded to its nearest value, ties to even: no difference allowed."""
    x = rn(1, R, D, std=3., dt=torch.bfloat16)
    x[:, ::3] = x[:, ::3] * 0.01
    q, s = gdn.quantize_rows(x)
    top = x.double().abs().amax(1).clamp(min=2.0 ** -100)
    assert torch.equal(q.double(), nearest8(x.double() * 448 / top[:, None]))
    within("scale", s, top / 448)


@pytest.mark.parametrize("R,D", ROWS8)
@pytest.mark.parametrize("res", ["", "f32", "same"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_in_8_bits(R, D, res, dt):
    dt = DT[dt]
    x, w = rn(1, R, D, dt=dt), (1 + rn(2, D, std=.2)).to(dt)
    r = None if not res else rn(3, R, D, dt=dt if res == "same" else torch.float32)
    q, sc, s = gdn.add_rms_norm_8bit(x, w, r, eps=1e-5)
    rs, y = ref_norm(x, w, r, 1e-5)
    assert torch.equal(s.double(), rs)
    top = y.abs().amax(1)
    within("scale", sc, top / 448, n=104)
    # half a step (2^-4 of the value, 2^-10 below the smallest normal) and the fp32 form's error
    v = y * 448 / top[:, None]
    assert bool(((q.double() - v).abs() <= (2.0 ** -4 + 210 * U32) * v.abs() + 2.0 ** -10).all())
    # and the nearest value but where the quotient lies within that error of a border
    near = nearest8(v * (1 + 210 * U32)) != nearest8(v * (1 - 210 * U32))
    assert bool(((q.double() == nearest8(v)) | near).all())


def test_rows_in_8_bits_at_the_ends():
    x = torch.zeros(8, 40, device="cuda")
    x[1, 3] = 2.0 ** -110
    x[2] = 3e38
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    x[5, :] = torch.linspace(-1, 1, 40)
    x[6, 0], x[6, 1] = 1.0, 2.0 ** -30
    x[7] = float("nan")
    q, s = gdn.quantize_rows(x)
    v = q.float() * s[:, None]
    assert bool((s[[0, 1, 2, 4, 5, 6, 7]].isfinite() & (s[[0, 1, 2, 4, 5, 6, 7]] > 0)).all())
    assert bool((v[:2].abs() <= 2.0 ** -110).all()) and bool((q[2].float() == 448).all())
    assert bool(v[3].isnan().all())
    assert bool(v[4, 9].isnan()) and bool((v[4, :9] == 0).all())
    assert float(v[6, 0]) == 1.0 and float(v[6, 1]) == 0.0 and bool(v[7].isnan().all())
    assert gdn.quantize_rows(torch.zeros(0, 5, device="cuda"))[0].shape == (0, 5)


# ------------------------------------------------------------------ projections
def ref_act(v, act):
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    return v, torch.ones_like(v)


LINEAR = [(1, 1, 1), (1, 33, 17), (2, 64, 64), (16, 2048, 512), (17, 40, 129), (33, 4099, 48), (64, 128, 100), (65, 8, 8),
          (66, 40, 33), (128, 512, 4096), (255, 130, 257), (300, 72, 270), (333, 1000, 777), (513, 64, 1025), (1000, 2048, 512),
          (257, 6144, 130), (129, 33, 2000)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", LINEAR)
def test_linear_and_gradients(M, K, N, dt):
    dt, k = DT[dt], M + K + N
    act = (None, "silu", "gelu")[k % 3]
    x, w = rn(1, M, K, dt=dt), rn(2, N, K, std=K ** -.5, dt=dt)
    b = rn(3, N, dt=dt) if k % 2 else None
    r = rn(4, M, N, dt=dt) if k % 5 < 3 else None
    dy = rn(5, M, N, dt=dt)
    X, W = x.double(), w.double()
    v = X @ W.t() + (0 if b is None else b.double())
    y, d = ref_act(v, act)
    want = y + (0 if r is None else r.double())
    leaves = [t.requires_grad_(True) for t in (x, w, b, r) if t is not None]
    got = gdn.linear(x, w, b, act, r)
    # a sum of K products in fp32: K roundings at most (and a few more around them); |act'| < 1.13
    Sv = X.abs() @ W.abs().t() + (0 if b is None else b.double().abs())
    S = 1.13 * Sv + y.abs() + (0 if r is None else r.double().abs())
    within("y", got, want, S, K + 24)
    with torch.no_grad():
        assert torch.equal(gdn.linear(x, w, b, act, r), got)
    grads = dict(zip([n for n, t in zip("xwbr", (x, w, b, r)) if t is not None], torch.autograd.grad(got, leaves, dy)))
    dv = dy.double() * d
    # bf16's dv is rounded once more before its products; v's error moves act' by at most 0.5 of itself
    ua = (U[dt] if act else 0.0) / U32
    dd = dy.double().abs() * 0.5 * Sv * (K + 24) if act else 0.0
    within("dx", grads["x"], dv @ W, (dv.abs() * (N + 24 + ua) + dd) @ W.abs(), 1)
    within("dw", grads["w"], dv.t() @ X, (dv.abs() * (M + 24 + ua) + dd).t() @ X.abs(), 1)
    if b is not None:  # 64 rows to an fp32 sum
        within("db", grads["b"], dv.sum(0), (dv.abs() * 90 + dd).sum(0), 1)
    if r is not None:
        assert torch.equal(grads["r"], dy)


@pytest.mark.parametrize("act,most", [(None, 1.9e-3), ("silu", 2.7e-3), ("gelu", 2.7e-3)])
def test_linear_rounds_once_or_twice(act, most):
    """rms of bf16 results: their own rounding is at most 2^-8 / sqrt(3) / ~1.3 = 1.7e-3 for spread
    mantissas; dv's before the products adds as much in quadrature."""
    M, K, N = 1024, 768, 1280
    x, w, dy = rn(1, M, K, dt=torch.bfloat16), rn(2, N, K, std=K ** -.5, dt=torch.bfloat16), rn(3, M, N, dt=torch.bfloat16)
    v = x.double() @ w.double().t()
    y, d = ref_act(v, act)
    got = gdn.linear(x.requires_grad_(True), w.requires_grad_(True), None, act)
    assert rms(got, y) <= 1.9e-3
    dx, dw = torch.autograd.grad(got, [x, w], dy)
    dv = dy.double() * d
    assert rms(dx, dv @ w.detach().double()) <= most and rms(dw, dv.t() @ x.detach().double()) <= most


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(1, 5, 3), (16, 2048, 130), (64, 100, 70), (65, 16, 16), (70, 100, 90), (300, 2048, 512),
                                   (257, 1027, 333), (1000, 640, 1030)])
def test_linear_8bit(M, K, N, out):
    out, act = DT[out], (None, "silu", "gelu")[(M + N) % 3]
    q, s = gdn.quantize_rows(rn(1, M, K))
    p, t = gdn.quantize_rows(rn(2, N, K, std=K ** -.5))
    b, r = rn(3, N, dt=out), rn(4, M, N, dt=out)
    X, W = q.double() * s.double()[:, None], p.double() * t.double()[:, None]
    y, _ = ref_act(X @ W.t() + b.double(), act)
    got = gdn.linear_8bit(q, s, p, t, b, act, r, out_dtype=out)
    S = 1.13 * (X.abs() @ W.abs().t() + b.double().abs()) + y.abs() + r.double().abs()
    # bf16 results: the 8-bit matrix instructions' sums carry 16 bits at least
    within("y", got, y + r.double(), S, K + 24 + (256 if out == torch.bfloat16 else 0))


def test_linear_takes_slices_and_any_alignment():
    wide = rn(1, 200, 700, dt=torch.bfloat16)
    flat = rn(2, 90 * 256 + 1, std=.1, dt=torch.bfloat16)
    res = rn(3, 200, 333, dt=torch.bfloat16)
    for M in (5, 200):
        for off in (0, 3, 8):
            x, r = wide[:M, off:off + 256], res[:M, 7:97]
            for w in (flat[1:].view(90, 256), flat[:-1].view(90, 256)):
                want = gdn.linear(x.contiguous(), w.clone(), None, "silu", r.contiguous())
                assert torch.equal(gdn.linear(x, w, None, "silu", r), want)
                dy = rn(5, M, 90, dt=torch.bfloat16)
                v = blocks.gdn_linear_fwd(x, w, None, "silu", save=True)[1]
                a = blocks.gdn_linear_bwd(x, w, dy, "silu", v)
                b = blocks.gdn_linear_bwd(x.contiguous(), w.clone(), dy, "silu", v)
                assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("act", [None, "gelu"])
@pytest.mark.parametrize("K", [64, 37])
def test_linear_only_the_gradients_asked_for(act, K):
    x, w, b, dy = (rn(k, *s, dt=torch.bfloat16) for k, s in enumerate([(90, K), (50, K), (50,), (90, 50)]))
    v = blocks.gdn_linear_fwd(x, w, b, act, save=True)[1]
    full = blocks.gdn_linear_bwd(x, w, dy, act, v)
    for bits in range(8):
        need = tuple(bool(bits >> k & 1) for k in range(3))
        part = blocks.gdn_linear_bwd(x, w, dy, act, v, need=need)
        assert all((p is None) if not n else torch.equal(p, q) for p, q, n in zip(part, full, need))


def test_linear_without_rows():
    x, w, b = torch.zeros(0, 24, device="cuda"), rn(1, 10, 24), rn(2, 10)
    for t in (x, w, b):
        t.requires_grad_(True)
    y = gdn.linear(x, w, b, "silu")
    dx, dw, db = torch.autograd.grad(y, [x, w, b], torch.zeros(0, 10, device="cuda"))
    assert y.shape == (0, 10) and dx.shape == (0, 24) and not dw.any() and not db.any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_at_the_types_ends(act, dt):
    """A bias of the type's lowest value (a mask) gives 0 and no gradient, its largest passes through."""
    dt = DT[dt]
    top = torch.finfo(dt).max
    b = torch.tensor([-top, -1e19, -100., -20., 20., 100., 1e19, top], device="cuda").to(dt)
    for M in (3, 70):
        x, w = torch.zeros(M, 16, device="cuda", dtype=dt), torch.zeros(8, 16, device="cuda", dtype=dt)
        leaves = [t.requires_grad_(True) for t in (x, w, b)]
        y = gdn.linear(x, w, b, act)
        g = torch.autograd.grad(y, leaves, torch.ones_like(y))
        assert bool((y[:, :3].abs() < 1e-30).all()) and torch.equal(y[:, 4:], b[4:].expand(M, 4)) and bool((y[:, 3].abs() < 1e-7).all())
        assert all(bool(t.isfinite().all()) for t in g)
        # (silu'(-20) = -19 e^-20 = -3.92e-8 a row, gelu's less)
        assert bool((g[2][:4].abs() < M * 4e-8).all()) and bool(((g[2][4:] - M).abs() < 1e-5).all())


def test_linear_keeps_what_is_not_finite_to_its_row():
    for M in (20, 300):
        x, w = rn(1, M, 72, dt=torch.bfloat16), rn(2, 130, 72, dt=torch.bfloat16)
        clean = gdn.linear(x, w)
        x[3, 71], x[7, 0] = float("nan"), float("inf")
        y = gdn.linear(x, w)
        keep = [m for m in range(M) if m not in (3, 7)]
        assert bool(y[3].isnan().all()) and not bool(y[7].isfinite().any()) and torch.equal(y[keep], clean[keep])


# ------------------------------------------------------------------ gated recurrence
def bounds_of(lens, B, T):
    if lens is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    out, at = [], 0
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def ref_rec(x, g, i, scale, h0, spans):
    """Token by token in 64 bits over flat [tokens, D], differentiable."""
    L = g if scale is None else -scale * torch.sigmoid(g)
    u = x if i is None else x * torch.sigmoid(i)
    if scale is not None:
        u = u * torch.sqrt(-torch.expm1(2 * L))
    ys, hT = [], []
    for n, (lo, hi) in enumerate(spans):
        h = h0[n] if h0 is not None else x.new_zeros(x.shape[1])
        for t in range(lo, hi):
            h = torch.exp(L[t]) * h + u[t]
            ys.append(h)
        hT.append(h)
    return (torch.stack(ys) if ys else x[:0]), torch.stack(hT)


REC = [("bf16", None, 1, 1, 5, 1, 1, 0, 1), ("bf16", None, 3, 16, 1, 1, 1, 0, 1), ("f32", [3, 0, 1, 0, 0, 64, 7], 0, 0, 33, 1, 1, 0, 1),
       ("bf16", [0, 0, 5, 128, 127, 129, 1, 1, 1, 0], 0, 0, 130, 1, 0, 1, 1), ("f32", None, 3, 65, 64, 0, 1, 0, 0),
       ("bf16", None, 2, 300, 257, 0, 0, 1, 1), ("f32", None, 1, 257, 129, 1, 1, 0, 0), ("bf16", None, 1, 600, 2, 1, 1, 1, 0),
       ("f32", [128, 128, 64, 1, 15, 16, 17], 0, 0, 65, 1, 0, 0, 1), ("bf16", [2049, 1], 0, 0, 6, 1, 1, 0, 1), ("bf16", [1300, 3, 200], 0, 0, 1030, 1, 1, 0, 1)]


@pytest.mark.parametrize("dt,lens,B,T,D,scaled,inp,g32,init", REC)
def test_recurrence_and_gradients(dt, lens, B, T, D, scaled, inp, g32, init):
    dt = DT[dt]
    if lens:
        B, T = 1, sum(lens)
    spans = bounds_of(lens, B, T)
    N = len(spans)
    gdt = torch.float32 if g32 else dt
    x = rn(1, B, T, D, dt=dt)
    # decays of 0.995 at most: a state remembers 1 / (1 - 0.995) = 200 tokens
    g = rn(2, B, T, D, dt=gdt) if scaled else (-0.005 - rn(2, B, T, D).abs() * .1).to(gdt)
    scale = ru(3, .02, .2, D) if scaled else None
    i = rn(4, B, T, D, dt=dt) if inp else None
    h0 = rn(5, N, D, std=2.) if init else None
    dy, dh = rn(6, B, T, D, dt=dt), rn(7, N, D)
    cu = torch.tensor([0] + [hi for _, hi in spans], dtype=torch.int32) if lens else None
    d = [t.double().reshape(-1, D).requires_grad_(True) if t is not None and t.dim() == 3 else
         t.double().requires_grad_(True) if t is not None else None for t in (x, g, i, scale, h0)]
    y, hT = ref_rec(*d, spans)
    live = [(t, q) for t, q in zip((x, g, i, scale, h0), d) if t is not None]
    want = torch.autograd.grad([y, hT], [q for _, q in live], [dy.double().reshape(-1, D), dh.double()], allow_unused=True)
    leaves = [t.requires_grad_(True) for t, _ in live]
    seqs = dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu) if lens else {}
    gy, gh = gdn.gated_recurrence(x, g, i, scale, h0, output_final_state=True, **seqs)
    got = torch.autograd.grad([gy, gh], leaves, [dy, dh])
    # of the largest entry: a chain of 200 tokens' roundings (four each: decay, gate, product,
    # sum), the sums of gradients 64 tokens and the tokens' parts in 64 bits
    n = 4 * 200 + 100
    most = lambda t: t.abs().max().expand_as(t) if t.numel() else t
    within("y", gy.reshape(-1, D), y, most(y), n)
    within("hT", gh, hT, most(hT), n)
    for (t, _), a, b in zip(live, got, want):
        b = torch.zeros_like(a, dtype=torch.float64) if b is None else b.reshape(a.shape)
        # (gradients multiply the state's chain with the gradient's)
        within(str(tuple(t.shape)), a, b, most(b), 4 * n * (8 if a.dim() == 1 else 1))
    with torch.no_grad():
        y2, h2 = gdn.gated_recurrence(x, g, i, scale, h0, output_final_state=True, **seqs)
    assert torch.equal(y2, gy) and torch.equal(h2, gh)
    # states recomputed, and a second run: the same bits
    kept = [t.detach() if t is not None else None for t in (x, g, i, scale, h0)]
    for states in (None, blocks.gdn_rec_fwd(*kept, save_states=True, **seqs)[2]):
        again = blocks.gdn_rec_bwd(kept[0], kept[1], dy, kept[2], kept[3], kept[4], dh, states=states, **seqs)
        assert all(torch.equal(p, q) for p, q in zip([t for t in again if t is not None], got))


def test_recurrence_gradient_by_differences():
    x, g, i, sc, h0 = rn(1, 1, 40, 3), rn(2, 1, 40, 3), rn(3, 1, 40, 3), ru(4, .1, .5, 3), rn(5, 1, 3)
    dy, dh = rn(6, 1, 40, 3), rn(7, 1, 3)
    f = lambda a, b, c, s, h: sum((p * q.double().reshape(p.shape)).sum() for p, q in
                                  zip(ref_rec(a[0], b[0], c[0], s, h, [(0, 40)]), (dy, dh)))
    leaves = [t.requires_grad_(True) for t in (x, g, i, sc, h0)]
    y, hT = gdn.gated_recurrence(*leaves[:4], initial_state=h0, output_final_state=True)
    for k, got in enumerate(torch.autograd.grad([y, hT], leaves, [dy, dh])):
        d = rn(9 + k, *leaves[k].shape, dt=torch.float64)
        p = [t.detach().double() for t in leaves]
        a, b = ([q + (e * d if j == k else 0) for j, q in enumerate(p)] for e in (1e-6, -1e-6))
        want = float((f(*a) - f(*b)) / 2e-6)
        assert abs(float((got.double() * d).sum()) - want) <= 2e-5 * (1 + abs(want))


def test_recurrence_long_chain():
    """Many chunks and groups of them against blocks joined in 64 bits; the mean error does not drift."""
    T, D = 20011, 130
    x, g, i, sc = rn(1, 1, T, D, dt=torch.bfloat16), rn(2, 1, T, D, dt=torch.bfloat16), rn(3, 1, T, D, dt=torch.bfloat16), ru(4, .01, .1, D)
    L = (-sc.double() * torch.sigmoid(g[0].double())).cpu()
    u = (x[0].double() * torch.sigmoid(i[0].double())).cpu() * torch.sqrt(-torch.expm1(2 * L))
    a, h, want = torch.exp(L), torch.zeros(D, dtype=torch.float64), torch.empty(T, D, dtype=torch.float64)
    for t in range(T):
        h = a[t] * h + u[t]
        want[t] = h
    y, hT = gdn.gated_recurrence(x, g, i, sc, output_final_state=True)
    within("y", y[0].cpu(), want, want.abs().max().expand_as(want), 4 * 400)
    assert rms(hT[0].cpu(), h) <= 5e-6


def test_recurrence_gates_at_their_ends():
    """Sigmoids that vanish or reach one, scale 0: m = 0 has derivative 0, nothing is NaN."""
    D = 8
    x, g = rn(1, 1, 70, D), torch.full((1, 70, D), -200., device="cuda")
    g[:, :, 4:] = 200.
    sc = torch.tensor([0., 1e-3, 1., 30.] * 2, device="cuda")
    leaves = [t.requires_grad_(True) for t in (x, g, sc)]
    y, hT = gdn.gated_recurrence(x, g, scale=sc, initial_state=torch.ones(1, D, device="cuda"), output_final_state=True)
    grads = torch.autograd.grad(y.sum() + hT.sum(), leaves)
    assert all(bool(t.isfinite().all()) for t in (y, hT, *grads))
    assert bool((y[0, :, :4] == 1).all()) and bool((y[0, :, 4] == 1).all())   # nothing decays, nothing enters
    assert bool((grads[0][0, :, :5] == 0).all())


def test_recurrence_keeps_what_is_not_finite_to_its_sequence():
    lens = [200, 61, 300, 1]
    cu = torch.tensor([0, 200, 261, 561, 562], dtype=torch.int32)
    x, g, sc = rn(1, 1, 562, 40), rn(2, 1, 562, 40), ru(3, .1, .5, 40)
    seqs = dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
    dy = rn(4, 1, 562, 40)
    clean = gdn.gated_recurrence(x, g, scale=sc, output_final_state=True, **seqs)
    cg = blocks.gdn_rec_bwd(x, g, dy, None, sc, **seqs)
    x[0, 230, 5], g[0, 231, 6] = float("inf"), float("nan")
    y, hT = gdn.gated_recurrence(x, g, scale=sc, output_final_state=True, **seqs)
    bg = blocks.gdn_rec_bwd(x, g, dy, None, sc, **seqs)
    own = torch.zeros(562, 40, dtype=torch.bool, device="cuda")
    own[200:261, 5:7] = True
    assert torch.equal(y[0][~own], clean[0][0][~own]) and not bool(y[0, 230:261, 5].isfinite().any())
    assert torch.equal(y[0, 200:230], clean[0][0, 200:230])
    assert not bool(hT[1, 5:7].isfinite().any()) and bool(hT[[0, 2, 3]].isfinite().all())
    for p, q in zip(bg[:2], cg[:2]):
        assert torch.equal(p[0][~own], q[0][~own])


def test_recurrence_rows_behind_the_last_sequence():
    """Without the host copy the lengths may end early: those rows hold zeros, of gradients too, and
    the library itself leaves them as they were."""
    x, g, dy = rn(1, 1, 300, 20), -rn(2, 1, 300, 20).abs(), rn(3, 1, 300, 20)
    cu = torch.tensor([0, 100, 250], dtype=torch.int32, device="cuda")
    y, hT = gdn.gated_recurrence(x, g, cu_seqlens=cu, output_final_state=True)
    want, wT = gdn.gated_recurrence(x[:, :250].contiguous(), g[:, :250].contiguous(), cu_seqlens=cu, output_final_state=True)
    assert torch.equal(y[:, :250], want) and not y[:, 250:].any() and torch.equal(hT, wT)
    grads = blocks.gdn_rec_bwd(x, g, dy, cu_seqlens=cu)
    wg = blocks.gdn_rec_bwd(x[:, :250].contiguous(), g[:, :250].contiguous(), dy[:, :250].contiguous(), cu_seqlens=cu)
    assert all(torch.equal(a[:, :250], b) and not a[:, 250:].any() for a, b in zip(grads[:2], wg[:2]))


@pytest.mark.parametrize("lens", [None, [0, 0, 0]])
def test_recurrence_without_tokens(lens):
    N = 3
    x, g, sc, h0, dh = torch.zeros(1 if lens else N, 0, 70, device="cuda"), None, ru(1, .1, .2, 70), rn(2, N, 70), rn(3, N, 70)
    g = torch.zeros_like(x)
    cu = torch.zeros(4, dtype=torch.int32)
    leaves = [t.requires_grad_(True) for t in (x, g, sc, h0)]
    y, hT = gdn.gated_recurrence(x, g, scale=sc, initial_state=h0, output_final_state=True,
                                 **(dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu) if lens else {}))
    dx, dg, ds, d0 = torch.autograd.grad([y, hT], leaves, [torch.zeros_like(y), dh])
    assert y.shape == x.shape and torch.equal(hT, h0) and torch.equal(d0, dh) and not ds.any()


def test_recurrence_of_many_sequences():
    """A thousand sequences of up to 40 tokens, a third of them empty, against each alone."""
    g0 = torch.Generator().manual_seed(5)
    lens = (torch.randint(0, 41, (1000,), generator=g0) * (torch.rand(1000, generator=g0) > .33)).tolist()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    T, D = int(cu[-1]), 66
    x, g, h0, dy, dh = rn(1, 1, T, D), -rn(2, 1, T, D).abs() * .1, rn(3, 1000, D), rn(4, 1, T, D), rn(5, 1000, D)
    seqs = dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
    y, hT = gdn.gated_recurrence(x, g, initial_state=h0, output_final_state=True, **seqs)
    dx, dg, _, _, d0 = blocks.gdn_rec_bwd(x, g, dy, h0=h0, dhT=dh, **seqs)
    for n in list(range(0, 1000, 37)) + [999]:
        lo, hi = int(cu[n]), int(cu[n + 1])
        q = [t.double().requires_grad_(True) for t in (x[0, lo:hi], g[0, lo:hi], h0[n:n + 1])]
        wy, wT = ref_rec(q[0], q[1], None, None, q[2], [(0, hi - lo)])
        wx, wg, w0 = torch.autograd.grad([wy, wT], q, [dy[0, lo:hi].double(), dh[n:n + 1].double()], allow_unused=True)
        pairs = [(hT[n:n + 1], wT), (d0[n:n + 1], w0)] + ([(y[0, lo:hi], wy), (dx[0, lo:hi], wx), (dg[0, lo:hi], wg)] if hi > lo else [])
        for a, b in pairs:   # forty tokens' roundings, four each
            within(str(n), a, b, b.abs().max().expand_as(b), 400)


def test_recurrence_takes_slices():
    wide = rn(1, 2, 90, 400, dt=torch.bfloat16)
    x, g, i = wide[..., 1:64], wide[..., 100:163], wide[..., 301:364]
    sc = ru(2, .1, .4, 63)
    a = gdn.gated_recurrence(x, g, i, sc)
    assert torch.equal(a, gdn.gated_recurrence(x.contiguous(), g.contiguous(), i.contiguous(), sc))


@pytest.mark.parametrize("dt,D,scaled,inp", [("bf16", 130, 1, 1), ("f32", 33, 0, 1), ("bf16", 1, 1, 0), ("f32", 1, 1, 1)])
def test_recurrence_steps_continue_a_prompt(dt, D, scaled, inp):
    dt = DT[dt]
    B, T, slots = 5, 24, 9
    x, g = rn(1, B, T, D, dt=dt), (rn(2, B, T, D) if scaled else -rn(2, B, T, D).abs() * .2).to(dt)
    i = rn(3, B, T, D, dt=dt) if inp else None
    sc = ru(4, .1, .6, D) if scaled else None
    cut = lambda a, lo, hi: None if a is None else a[:, lo:hi].contiguous()
    y, hT = gdn.gated_recurrence(x, g, i, sc, output_final_state=True)
    _, h = gdn.gated_recurrence(cut(x, 0, 20), cut(g, 0, 20), cut(i, 0, 20), sc, output_final_state=True)
    idx = torch.tensor([7, 2, 100, 0, -1], dtype=torch.int32, device="cuda")    # the third and the last: padding
    real = [0, 1, 3]
    state = rn(9, slots, D)
    state[idx[real].long()] = h[real]
    before = state.clone()
    out = torch.full((B, D), 7.0, device="cuda", dtype=dt)
    for t in range(20, 24):
        got = gdn.gdn_rec_step(x[:, t], g[:, t], state, None if i is None else i[:, t], sc, state_idx=idx, y=out)
        assert bool((got[[2, 4]] == 7).all())
        within("y", got[real], y[real, t].double(), y.double().abs().max().expand(3, D), 100)
    within("state", state[idx[real].long()], hT[real].double(), hT.double().abs().max().expand(3, D), 100)
    others = [s for s in range(slots) if s not in (7, 2, 0)]
    assert torch.equal(state[others], before[others])


# ------------------------------------------------------------------ a block
def block(x, stream, p, n8=None):
    """One block's forward pass: norm, projections, recurrence, projection back onto the stream."""
    y, s = gdn.add_rms_norm(x, p["nw"], stream)
    u = gdn.linear(y, p["w_in"], p["b_in"], "silu")
    D = u.shape[-1] // 3
    h = gdn.gated_recurrence(u[..., :D], u[..., D:2 * D], u[..., 2 * D:], p["scale"])
    return gdn.linear(h, p["w_out"]), s


def block_params(W, D, dt):
    return dict(nw=(1 + rn(11, W, std=.1)).to(dt), w_in=rn(12, 3 * D, W, std=W ** -.5, dt=dt), b_in=rn(13, 3 * D, std=.1, dt=dt),
                scale=ru(14, .02, .2, D), w_out=rn(15, W, D, std=D ** -.5, dt=dt))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_block_in_one_run(dt):
    """A block's loss and gradients against the same block in 64 bits: roundings at each stage in bf16
    (half a step each, some ten of them along the longest way), none that matters in fp32."""
    dt, W, D, T = DT[dt], 72, 40, 150
    p = block_params(W, D, dt)
    x, stream = rn(1, 2, T, W, dt=dt), rn(2, 2, T, W)
    d1, d2 = rn(3, 2, T, W, dt=dt), rn(4, 2, T, W)
    leaves = [t.requires_grad_(True) for t in (x, stream, *p.values())]
    out, s = block(x, stream, p)
    got = torch.autograd.grad([out, s], leaves, [d1, d2])
    q = [t.detach().double().requires_grad_(True) for t in leaves]
    P = dict(zip(p, q[2:]))
    S = q[0] + q[1]
    Y = S / torch.sqrt(S.square().mean(-1, keepdim=True) + 1e-6) * P["nw"]
    v = Y @ P["w_in"].t() + P["b_in"]
    u = v * torch.sigmoid(v)
    y, _ = ref_rec(u[..., :D].reshape(-1, D), u[..., D:2 * D].reshape(-1, D), u[..., 2 * D:].reshape(-1, D), P["scale"], None,
                   [(0, T), (T, 2 * T)])
    want_out = y.reshape(2, T, D) @ P["w_out"].t()
    want = torch.autograd.grad([want_out, S], q, [d1.double(), d2.double()])
    tol = 3e-2 if dt == torch.bfloat16 else 2e-5
    for name, a, b in zip(["out", "x", "stream", *p], [out, *got], [want_out.detach(), *want]):
        e = rms(a, b)
        print(f"    {name} {e:.1e}", flush=True)
        assert e <= tol, name


def test_block_in_8_bits_prefill_and_steps():
    """Serving: the 8-bit block over a prompt, then token by token from its state, equals one long prompt
    but for the bf16 rounding of what the products read."""
    W, D, T = 128, 96, 80
    p = block_params(W, D, torch.bfloat16)
    wq, ws = gdn.quantize_rows(p["w_in"])
    oq, os_ = gdn.quantize_rows(p["w_out"])
    x, stream = rn(1, 3, T, W, dt=torch.bfloat16), rn(2, 3, T, W)

    def front(a, r):
        q, sc, s = gdn.add_rms_norm_8bit(a, p["nw"], r)
        return gdn.linear_8bit(q, sc, wq, ws, p["b_in"], "silu"), s

    def back(h, s):
        q, sc = gdn.quantize_rows(h)
        return gdn.linear_8bit(q, sc, oq, os_, residual=s, out_dtype=torch.float32)

    u, s = front(x, stream)
    h, _ = gdn.gated_recurrence(u[..., :D], u[..., D:2 * D], u[..., 2 * D:], p["scale"], output_final_state=True)
    whole = back(h, s)
    assert whole.dtype == torch.float32 and bool(whole.isfinite().all())
    u, s = front(x[:, :70].contiguous(), stream[:, :70].contiguous())
    _, state = gdn.gated_recurrence(u[..., :D], u[..., D:2 * D], u[..., 2 * D:], p["scale"], output_final_state=True)
    for t in range(70, T):
        u, s = front(x[:, t], stream[:, t])
        h = gdn.gdn_rec_step(u[:, :D], u[:, D:2 * D], state, u[:, 2 * D:], p["scale"])
        # both ways read the same 8-bit rows; the products' tiles differ in the order of their sums, so a value
        # on a border may round to its neighbour: steps of 2^-3 of a row's entry, averaged over D of them
        assert rms(back(h, s), whole[:, t].double()) <= 5e-3


# ------------------------------------------------------------------ streams, graphs, sizes
def calls(seed=0):
    """{name: function of no arguments that returns tensors}"""
    bf = torch.bfloat16
    x, r, w = rn(seed + 1, 300, 520, dt=bf), rn(seed + 2, 300, 520), rn(seed + 3, 520, dt=bf)
    W = rn(seed + 4, 777, 520, std=.05, dt=bf)
    q, s = gdn.quantize_rows(x)
    p, t = gdn.quantize_rows(W)
    a, g, i, sc = rn(seed + 5, 1, 3000, 200, dt=bf), rn(seed + 6, 1, 3000, 200, dt=bf), rn(seed + 7, 1, 3000, 200, dt=bf), ru(seed + 8, .1, .4, 200)
    dy, du = rn(seed + 9, 300, 777, dt=bf), rn(seed + 10, 1, 3000, 200, dt=bf)
    v = blocks.gdn_linear_fwd(x, W, None, "gelu", save=True)[1]
    deep, wide = rn(seed + 11, 70, 8192, dt=bf), rn(seed + 12, 100, 8192, std=.01, dt=bf)
    return dict(norm8=lambda: gdn.add_rms_norm_8bit(x, w, r), norm=lambda: gdn.add_rms_norm(x, w, r),
                norm_bwd=lambda: blocks.gdn_addnorm_bwd(r, w, x), quant=lambda: gdn.quantize_rows(x),
                linear=lambda: gdn.linear(x, W, None, "gelu"), few=lambda: gdn.linear(x[:9], W),
                split=lambda: gdn.linear(deep, wide), linear8=lambda: gdn.linear_8bit(q, s, p, t),
                linear_bwd=lambda: blocks.gdn_linear_bwd(x, W, dy, "gelu", v),
                rec=lambda: gdn.gated_recurrence(a, g, i, sc, output_final_state=True),
                rec_bwd=lambda: blocks.gdn_rec_bwd(a, g, du, i, sc))


NAMES = ["norm8", "norm", "norm_bwd", "quant", "linear", "few", "split", "linear8", "linear_bwd", "rec", "rec_bwd"]


def tup(o):
    return [t.view(torch.uint8) if t.dtype == F8 else t for t in (o if isinstance(o, (tuple, list)) else (o,)) if t is not None]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(tup(a), tup(b)))


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(name):
    f, g = calls()[name], calls(100)[name]
    want = f(), g()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            a = f()
        with torch.cuda.stream(s2):
            b = g()
        got.append((a, b))
    torch.cuda.synchronize()
    assert all(same(a, want[0]) and same(b, want[1]) for a, b in got)


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """Two graphs of the same call on different inputs, replayed in turn with eager work between."""
    fs = calls()[name], calls(100)[name]
    want = [f() for f in fs]
    torch.cuda.synchronize()
    graphs = []
    for f in fs:
        G = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G):
            out = f()
        graphs.append((G, out))
    for k in range(3):
        for (G, out), f, w in zip(graphs, fs, want):
            for t in tup(out):
                t.zero_()
            G.replay()
            assert same(f(), w)
            torch.cuda.synchronize()
            assert same(out, w), k


def test_captured_training_step():
    p = block_params(64, 48, torch.bfloat16)
    x, stream = rn(1, 1, 400, 64, dt=torch.bfloat16), rn(2, 1, 400, 64)
    d1 = rn(3, 1, 400, 64, dt=torch.bfloat16)
    leaves = [t.requires_grad_(True) for t in (x, stream, *p.values())]

    def step():
        out, s = block(x, stream, p)
        return [out.detach(), *torch.autograd.grad([out, s], leaves, [d1, stream.detach()])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    G = torch.cuda.CUDAGraph()
    with torch.cuda.graph(G):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        G.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows against the same rows alone."""
    bf = torch.bfloat16
    R, D = (1 << 20) + 3, 2048
    x = torch.zeros(R, D, device="cuda", dtype=bf)
    x[-3:] = rn(1, 3, D, dt=bf)
    x[0] = x[-1]
    w = rn(2, D, dt=bf)
    q, s, _ = gdn.add_rms_norm_8bit(x, w)
    assert torch.equal(q[0].view(torch.uint8), q[-1].view(torch.uint8)) and torch.equal(s[0], s[-1])
    _, want = ref_norm(x[-3:], w, None, 1e-6)
    within("scale", s[-3:], want.abs().amax(1) / 448, n=104)
    assert bool(((q[-3:].double() * s[-3:, None].double() - want).abs() <= (2.0 ** -4 + 210 * U32) * want.abs() + s[-3:, None] * 2.0 ** -10).all())
    W = rn(3, 64, D, std=.02, dt=bf)
    y = gdn.linear(x, W)
    assert torch.equal(y[-1], y[0]) and rms(y[-3:], x[-3:].double() @ W.double().t()) <= 2e-3
    g = torch.full((1, R, D), -1.0, device="cuda", dtype=bf)
    h = gdn.gated_recurrence(x.view(1, R, D), g)
    want = torch.zeros(D, dtype=torch.float64, device="cuda")
    for k in range(3):
        want = want * math.exp(-1) + x[R - 3 + k].double()
        within("h", h[0, R - 3 + k], want, x[-3:].double().abs().max().expand(D), 100)
    del g, y, q
    wide = rn(4, 40000, 32, std=.2, dt=bf)
    out = gdn.linear(x[:60000, :32], wide)          # 2.4e9 outputs
    assert torch.equal(out[0, -40:], gdn.linear(x[:70, :32], wide[-40:])[0])
    last = x[59999:60000, :32].copy_(x[-1:, :32])
    out = gdn.linear(x[:60000, :32], wide)
    within("out", out[-1:], last.double() @ wide.double().t(), last.double().abs() @ wide.double().abs().t(), 56)


def test_refusals_on_the_gpu():
    x, w = rn(1, 4, 8), rn(2, 8)
    with pytest.raises(GDNError, match="residual"):
        gdn.add_rms_norm(x, w, rn(3, 4, 8, dt=torch.bfloat16))
    with pytest.raises(GDNError, match="eps"):
        gdn.add_rms_norm(x, w, eps=0.0)
    with pytest.raises(GDNError, match="contiguous"):
        gdn.linear(x.t(), rn(3, 5, 4))
    with pytest.raises(GDNError, match="out_dtype"):
        gdn.linear_8bit(x.to(F8), torch.ones(4, device="cuda"), x.to(F8), torch.ones(4, device="cuda"), out_dtype=torch.float16)
    for f in (lambda: gdn.add_rms_norm_8bit(x.requires_grad_(True), w), lambda: gdn.quantize_rows(x),
              lambda: gdn.gdn_rec_step(x, x, torch.zeros(4, 8, device="cuda"))):
        with pytest.raises(GDNError, match="no gradient"):
            f()
