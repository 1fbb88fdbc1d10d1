"""Projections where their sums, scales, sizes and tiles could go wrong, against plain forms
in 64 bits.  Tolerances are worst cases by arithmetic, as in the tests of the operators
themselves: half a step of the stored type, and (roundings in a row) u32 times the sum of
the magnitudes of the terms before it, u32 = 2^-24."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


import gated_deltanet_chunked_delta_amd as gdn  # noqa: E402
from gated_deltanet_chunked_delta_amd import GDNError, binding, blocks  # noqa: E402


def rn(seed, *s, std=1.0, dt=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda", dtype=torch.float64) * std).to(dt)


def rows8(x):
    """8-bit rows, their scales, and what they stand for."""
    q, s = gdn.quantize_rows(x)
    return q, s, q.double() * s.double()[:, None]


def within(got, want, S, n):
    """|got - want| <= u |want| + n u32 S + half a step of the type's subnormals (they lie
    2^-126 2^-7 = 2^-133 apart in bf16 and 2^-126 2^-23 = 2^-149 in fp32)."""
    assert got.shape == want.shape
    tiny = 2.0 ** -126 * U[got.dtype]
    worst = float(((got.double() - want).abs() / (U[got.dtype] * want.abs() + n * U32 * S + tiny)).max())
    print(f"    {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0


# ------------------------------------------------------------------ scales of 8-bit rows
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 70])
@pytest.mark.parametrize("a,b", [(1e-19, 1.25e-19), (1e-12, 1e-25), (1e30, 1e-30), (1e-25, 1e25), (1e-28, 1e35), (1e35, 1e-28), (1e18, 1e18)])
def test_scales_whose_product_leaves_the_range(M, a, b, out):
    """Results near 1e-37 (normal numbers) come from scales whose product is subnormal: it may not
    be formed alone."""
    K, N, out = 64, 70, DT[out]
    q, s, X = rows8(rn(1, M, K, std=a))
    p, t, W = rows8(rn(2, N, K, std=b))
    y = gdn.linear_8bit(q, s, p, t, out_dtype=out)
    # bf16: the 8-bit matrix instructions' sums carry 16 bits at least
    within(y, X @ W.t(), X.abs() @ W.abs().t(), K + 24 + (256 if out == torch.bfloat16 else 0))


@pytest.mark.parametrize("M", [5, 70])
def test_scales_whose_product_is_infinite(M):
    """Rows that share no column give 0, whatever their scales."""
    x, w = rn(1, M, 64, std=1e25), rn(2, 70, 64, std=1e25)
    x[:, :32], w[:, 32:] = 0, 0
    (q, s, _), (p, t, _) = rows8(x), rows8(w)
    for out in DT.values():
        assert not gdn.linear_8bit(q, s, p, t, out_dtype=out).any()
    s[1], t[3] = float("nan"), float("inf")     # and scales that are no numbers stay that
    q[0, :32] = q[2, 40]
    y = gdn.linear_8bit(q, s, p, t, out_dtype=torch.float32)
    assert bool(y[1].isnan().all()) and not bool(y[:, 3].isfinite().any())


# ------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 70, 700])
def test_8bit_rows_that_are_not_finite_stay_rows(M, out):
    """Rows and weights that hold an infinity or a NaN (NaN in 8 bits): their outputs, and no others."""
    out = DT[out]
    x, w = rn(1, M, 200), rn(2, 330, 200)
    clean = gdn.linear_8bit(*rows8(x)[:2], *rows8(w)[:2], out_dtype=out)
    x[1, 3], x[4, 199], w[7, 0], w[329, 130] = float("inf"), float("nan"), float("nan"), -float("inf")
    y = gdn.linear_8bit(*rows8(x)[:2], *rows8(w)[:2], out_dtype=out)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[[1, 4]] = True
    bad[:, [7, 329]] = True
    assert bool(y[bad].isnan().all()) and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("M", [5, 70, 700])
def test_fp32_rows_that_are_not_finite_stay_rows(M):
    x, w, dy = rn(1, M, 72), rn(2, 330, 72), rn(3, M, 330)
    clean, cx = gdn.linear(x, w), blocks.gdn_linear_bwd(x, w, dy, need=(True, False, False))[0]
    x[1, 71], x[4, 0] = float("inf"), float("nan")
    dy[2, 329] = float("nan")
    y, dx = gdn.linear(x, w), blocks.gdn_linear_bwd(x, w, dy, need=(True, False, False))[0]
    rest = [m for m in range(M) if m not in (1, 4)]
    assert not bool(y[[1, 4]].isfinite().any()) and torch.equal(y[rest], clean[rest])
    rest = [m for m in range(M) if m != 2]
    assert bool(dx[2].isnan().all()) and torch.equal(dx[rest], cx[rest])


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("M,N", [(131077, 131103), ((1 << 30) + 130, 17), (5, (1 << 30) + 71)])
def test_products_of_1e10_outputs(M, N):
    """Each of them checked (more than 2^22 workgroups in the last two): small whole numbers, whose
    products every type holds."""
    K = 8
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randint(-5, 6, (n, K), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16) for n in (M, N))
    y = gdn.linear(x, w)
    step = max(1, (1 << 29) // N)
    for m in range(0, M, step):
        want = torch.zeros_like(y[m:m + step])
        for k in range(K):          # (whole numbers up to 8 x 25 = 200 fit bf16's 8 bits)
            want.addcmul_(x[m:m + step, k, None], w[None, :, k])
        assert torch.equal(y[m:m + step], want), m


@pytest.mark.parametrize("act", [None, "silu"])
def test_gradients_of_more_rows_than_the_weights_takes(act):
    """x's and the bias's gradients of 2^22 rows and more, row by row those of the same rows alone;
    the weight's is refused."""
    M, K, N = (1 << 22) + 77, 16, 24
    x, w, dy = rn(1, M, K, dt=torch.bfloat16), rn(2, N, K, dt=torch.bfloat16), rn(3, M, N, dt=torch.bfloat16)
    v = blocks.gdn_linear_fwd(x, w, None, act, save=True)[1]
    dx, _, db = blocks.gdn_linear_bwd(x, w, dy, act, v, need=(True, False, True))
    total = torch.zeros(N, device="cuda", dtype=torch.float64)
    for m in range(0, M, 1 << 20):
        s = slice(m, m + (1 << 20))
        vs = None if v is None else v[s].contiguous()
        a, _, _ = blocks.gdn_linear_bwd(x[s], w, dy[s], act, vs, need=(True, False, False))
        assert torch.equal(a, dx[s])
        sig = None if v is None else torch.sigmoid(v[s].double())
        total += (dy[s].double() * (1 if v is None else sig + v[s] * sig * (1 - sig))).sum(0)
    # of terms whose magnitudes add up to at most 1.1 sum |dy|: 90 roundings each, as fp32 sums hold 64 rows
    within(db, total, 1.1 * dy.double().abs().sum(0), 90)
    with pytest.raises(GDNError, match="too large"):
        blocks.gdn_linear_bwd(x, w, dy, act, v)


def test_bias_gradient_of_very_wide_rows():
    """2^28 outputs and more, past one dimension of the joining launch: sums of a few whole numbers."""
    N = (1 << 28) + 45
    x, w = torch.ones(3, 1, device="cuda", dtype=torch.bfloat16), torch.zeros(N, 1, device="cuda", dtype=torch.bfloat16)
    dy = torch.randint(-9, 10, (3, N), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    _, dw, db = blocks.gdn_linear_bwd(x, w, dy, need=(False, True, True))
    want = (dy[0] + dy[1]) + dy[2]
    assert torch.equal(db, want) and torch.equal(dw[:, 0], want)


# ------------------------------------------------------------------ tiles
def kernels(f):
    """f's result and how often each kernel was launched for it."""
    binding.gdn_profile_reset()
    binding.gdn_profile_enable(True)
    try:
        out = f()
        torch.cuda.synchronize()
    finally:
        binding.gdn_profile_enable(False)
    return out, {n: c for n, (_, c) in binding.gdn_profile_read().items()}


def rms_within(name, got, want, n, more=0.0):
    """rms of the error over that of the result.  Of a sum of n products of random signs: a partial sum
    of j of them is sqrt(j) sigma, each rounding off by at most u32 of it, u32 / sqrt(3) in rms, so all n
    by u32 sigma sqrt(n^2 / 6) at most, against a result of sqrt(n) sigma.  Half as much again for
    what is not random, and the stored type's own rounding (2^-8 / sqrt(3) at most in bf16)."""
    off = float((got.double() - want).norm() / want.norm())
    most = 1.5 * U32 * math.sqrt(n / 6) + U[got.dtype] / math.sqrt(3) + more
    print(f"    {name}: rms {off:.2e} of {most:.2e}", flush=True)
    assert off <= most, name


def act_of(v, act):
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    return v, 1.0


@pytest.mark.parametrize("M,K,N,dt,act,tile", [
    (16301, 2041, 6131, "bf16", "silu", 256), (16304, 2040, 6136, "bf16", None, 256), (16301, 2041, 6131, "f32", "gelu", 256),
    (16304, 2040, 6136, "f32", None, 256), (3001, 522, 2100, "bf16", "gelu", 128), (2305, 513, 1153, "f32", "silu", 128)])
def test_every_output_of_many_ragged_tiles(M, K, N, dt, act, tile):
    """Each of the tiles' two sizes in all three products, more than eight tile rows and columns, the last
    ones cut; with the large ones the gradient copies x after the product of dx."""
    dt = DT[dt]
    x, w, b, r, dy = rn(1, M, K, dt=dt), rn(2, N, K, std=K ** -.5, dt=dt), rn(3, N, dt=dt), rn(4, M, N, dt=dt), rn(5, M, N, dt=dt)
    leaves = [t.requires_grad_(True) for t in (x, w, b)]
    (got, grads), names = kernels(lambda: (lambda y: (y.detach(), torch.autograd.grad(y, leaves, dy)))(gdn.linear(x, w, b, act, r)))
    assert {n: c for n, c in names.items() if n[:9] in ("linear_fw", "linear_dx", "linear_dw")} == {
        f"linear_{p}_{tile}": 1 for p in ("fwd", "dx", "dw")}, names
    odd = K * x.element_size() % 16 != 0        # (rows that are not whole 16 bytes are copied first: x, w)
    assert names["linear_pack"] == 2 * odd + (2 if tile == 256 else 1), names
    X, W, D = x.detach().double(), w.detach().double(), dy.double()
    v = X @ W.t() + b.detach().double()
    y, d = act_of(v, act)
    y += r.double()
    Sv = X.abs() @ W.abs().t() + b.detach().double().abs()
    # sums of K products: K roundings at most, a few more around them; |act'| < 1.13
    within(got, y, 1.13 * Sv + y.abs() + r.double().abs(), K + 24)
    rms_within("y", got, y, K)
    del y
    # bf16's dy act'(v) is rounded once more before its products (2^-8 of each term, in rms 2^-8 / sqrt(3) of
    # the sum); v's error moves act' by at most 0.5 of itself, in rms by that of v's own
    dv = D * d
    twice = U[dt] if act else 0.0
    dd = D.abs() * 0.5 * Sv * (K + 24) if act else torch.zeros_like(D)
    more = twice / math.sqrt(3) + (1.5 * U32 * math.sqrt(K / 6) if act else 0.0)
    del Sv
    want = dv @ W
    within(grads[0], want, (dv.abs() * (N + 24 + twice / U32) + dd) @ W.abs(), 1)
    rms_within("dx", grads[0], want, N, more)
    want = dv.t() @ X
    within(grads[1], want, (dv.abs() * (M + 24 + twice / U32) + dd).t() @ X.abs(), 1)
    rms_within("dw", grads[1], want, M, more)
    within(grads[2], dv.sum(0), (dv.abs() * 90 + dd).sum(0), 1)


@pytest.mark.parametrize("M,K,N,launches", [(32768, 1024, 1024, 1), (16384, 2048, 2048, 1), (6144, 8192, 4096, 2)])
def test_when_the_gradient_copies_x(M, K, N, launches):
    """With the other copies, or after the product of dx where the copies are large: the same gradients."""
    x, w, dy = rn(1, M, K, dt=torch.bfloat16), rn(2, N, K, dt=torch.bfloat16), rn(3, M, N, dt=torch.bfloat16)
    (dx, dw, _), names = kernels(lambda: blocks.gdn_linear_bwd(x, w, dy, need=(True, True, False)))
    assert names["linear_pack"] == launches
    assert torch.equal(dx, blocks.gdn_linear_bwd(x, w, dy, need=(True, False, False))[0])
    assert torch.equal(dw, blocks.gdn_linear_bwd(x, w, dy, need=(False, True, False))[1])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,tile", [(16301, 2041, 6131, 256), (16304, 2064, 6136, 256), (3001, 522, 2100, 128), (300, 8190, 300, 128)])
def test_every_8bit_output_of_many_ragged_tiles(M, K, N, tile, out):
    """fp32 results are those of sums in fp32: the 8-bit matrix instructions' 17 bits (1.3e-5) would show."""
    out = DT[out]
    q, s, X = rows8(rn(1, M, K))
    p, t, W = rows8(rn(2, N, K, std=K ** -.5))
    b, r = rn(3, N, dt=out), rn(4, M, N, dt=out)
    got, names = kernels(lambda: gdn.linear_8bit(q, s, p, t, b, "silu", r, out_dtype=out))
    assert names.get(f"linear_fwd_{tile}") == 1, names
    v = X @ W.t() + b.double()
    y = v * torch.sigmoid(v) + r.double()
    S = 1.13 * (X.abs() @ W.abs().t() + b.double().abs()) + y.abs() + r.double().abs()
    within(got, y, S, K + 24 + (256 if out == torch.bfloat16 else 0))
    rms_within("y", got, y, K, 2e-5 if out == torch.bfloat16 else 0.0)
    few, names = kernels(lambda: gdn.linear_8bit(q[:33], s[:33], p, t, b, "silu", r[:33], out_dtype=out))
    assert names == {"linear_few": 1}
    rms_within("few", few, y[:33], K, 2e-5 if out == torch.bfloat16 else 0.0)
