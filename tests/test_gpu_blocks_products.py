"""Projections where their sums, scales, sizes and tiles could go wrong, against plain forms
in 64 bits.  Tolerances are worst cases by arithmetic, as in the tests of the operators
themselves: half a step of the stored type, and (roundings in a row) u32 times the sum of
the magnitudes of the terms before it, u32 = 2^-24."""
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
from gated_deltanet_chunked_delta_amd import GDNError, blocks  # noqa: E402


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
