"""The layer operators' precision on the GPU, at lengths and sums where a lost
bit shows: outputs against the nearest value of their type to the 64-bit result,
and fp32 results of thousands of tokens against a chunked 64-bit form.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import torch.nn.functional as F  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def scan64(x, dt, A, B, C, D, bias, softplus, h0, lens, Q=64, keep=None):
    """The scan in 64 bits by chunks of Q tokens, differentiable; x [T, H, P], B, C [T, G, N],
    states [n, H, N, P].  Returns y and the final states; keep receives the steps and the log
    decays."""
    H, G = x.shape[1], B.shape[1]
    rep = H // G
    d = dt + bias if bias is not None else dt
    d = torch.logaddexp(d, torch.zeros_like(d)) if softplus else d
    a = d * A
    if keep is not None:
        keep.update(d=d, a=a)
    tri = torch.tril(torch.ones(Q, Q, dtype=torch.bool, device=x.device))
    ys, hs, at = [], [], 0
    for n, L in enumerate(lens):
        nc = (L + Q - 1) // Q

        def cut(a):  # [L, heads, k] -> [nc, heads, Q, k], zero rows behind the end
            a = torch.cat([a[at:at + L], a.new_zeros(nc * Q - L, *a.shape[1:])], 0)
            return a.reshape(nc, Q, *a.shape[1:]).transpose(1, 2)

        h = h0[n] if h0 is not None else x.new_zeros(H, B.shape[2], x.shape[2])
        X, K, O, dd = cut(x), cut(B).repeat_interleave(rep, 1), cut(C).repeat_interleave(rep, 1), cut(d[..., None])
        cum = cut(a[..., None]).cumsum(2)
        Lm = torch.exp(torch.where(tri, cum - cum.transpose(2, 3), torch.full_like(cum[:1, :1, :1, :1], -torch.inf)))
        V = dd * X
        inner = ((O @ K.transpose(2, 3)) * Lm) @ V
        tot = cum[:, :, -1:]
        add = K.transpose(2, 3) @ (torch.exp(tot - cum) * V)
        rows = []
        for c in range(nc):
            rows.append(inner[c] + torch.exp(cum[c]) * (O[c] @ h))
            h = torch.exp(tot[c]) * h + add[c]
        if L:
            y = torch.stack(rows).transpose(1, 2).reshape(nc * Q, H, -1)[:L]
            ys.append(y if D is None else y + D[:, None] * x[at:at + L])
        hs.append(h)
        at += L
    return (torch.cat(ys) if ys else torch.zeros_like(x)), torch.stack(hs)


def inputs(seed, T, H, G, Dk, Dv, n, dt=BF, dev="cuda:0"):
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    return dict(x=F.silu(rn(1, T, H, Dv)).to(dt), dt=rn(1, T, H).to(dt), A=-(1 + 15 * torch.rand(H, generator=g, device=dev)),
                B=F.silu(rn(1, T, G, Dk)).to(dt), C=F.silu(rn(1, T, G, Dk)).to(dt), D=rn(H), bias=rn(H) - 4,
                h0=0.3 * rn(n, H, Dk, Dv)), rn(1, T, H, Dv).to(dt), 0.3 * rn(n, H, Dk, Dv)


ORDER = ["x", "dt", "A", "B", "C", "D", "bias", "h0"]


def both(seed, lens, H, G, Dk, Dv, dt=BF, **opts):
    """{name: (got, 64-bit)} of the outputs and gradients of one packed batch; under "sums" the
    64-bit gradients of the steps and log decays, the steps and dt + bias."""
    from gated_deltanet_chunked_delta_amd import selective_scan
    T, n = sum(lens), len(lens)
    s, dy, dhT = inputs(seed, T, H, G, Dk, Dv, n, dt)
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    kw = dict(cu_seqlens=cu.to(dy.device), cu_seqlens_host=cu) if n > 1 else {}
    leaves = [s[k].requires_grad_(True) for k in ORDER]
    y, hT = selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], dt_bias=s["bias"], dt_softplus=True,
                           initial_state=s["h0"], output_final_state=True, **opts, **kw)
    grads = torch.autograd.grad([y, hT], leaves, [dy, dhT])
    torch.cuda.synchronize()
    r = {k: s[k].detach().double() for k in ORDER}
    r = {k: (v[0] if k in ("x", "dt", "B", "C") else v).requires_grad_(True) for k, v in r.items()}
    keep = {}
    ry, rh = scan64(*(r[k] for k in ORDER[:7]), True, r["h0"], lens, keep=keep)
    *rg, gd, ga = torch.autograd.grad([ry, rh], [r[k] for k in ORDER] + [keep["d"], keep["a"]],
                                      [dy[0].double(), dhT.double()])
    out = dict(y=(y[0], ry), hT=(hT, rh))
    for k, a, b in zip(ORDER, grads, rg):
        out["d" + k] = (a[0] if k in ("x", "dt", "B", "C") else a, b)
    out = {k: (a.detach(), b.detach()) for k, (a, b) in out.items()}
    out["sums"] = (gd, ga, keep["d"].detach(), (r["dt"] + r["bias"]).detach())
    return out


def rms(t):
    return t.double().square().mean().sqrt().item()


ROUNDED = [  # lens, H, G, Dk, Dv, seg_mode
    ([4096], 2, 1, 128, 128, 0),
    ([1000, 3, 900], 4, 2, 64, 64, 2),
    ([777], 3, 1, 128, 64, -1),
    ([500, 140], 1, 1, 64, 192, 1),
]


@pytest.mark.parametrize("lens,H,G,Dk,Dv,seg", ROUNDED)
def test_scan_outputs_are_rounded_once(dev, lens, H, G, Dk, Dv, seg):
    """With round_once bf16 outputs and gradients are the 64-bit result rounded once, but for what precedes the
    rounding: factors of the products off by 2^-18 each, two a product, so 2^-16 of the rms
    scale with room for their sums.  A pre-rounding error e turns the rounding over with
    probability 2 e / step, by one step, step <= 2^-7 of the value: rms
    sqrt(2 e step) = sqrt(2 2^-16 2^-7) = 2^-11 of the rms."""
    r = both(3, lens, H, G, Dk, Dv, seg_mode=seg, round_once=True)
    del r["sums"]
    for k, (got, want) in r.items():
        if got.dtype != BF:
            continue
        e = rms(got.double() - want.to(BF).double()) / rms(want)
        print(f"    {k} {e:.2e}", flush=True)
        assert e <= 2.0 ** -11, k



@pytest.mark.parametrize("lens,H,G,Dk,Dv,seg", ROUNDED)
def test_scan_outputs_by_default(dev, lens, H, G, Dk, Dv, seg):
    """Without round_once y and dx pass two more bf16 roundings, of a chunk's matrix and of the
    state, which enter through sums: each adds at most an error like the output's own, sqrt(3) of
    it in all.  dB, dC and ddt are rounded once as with round_once."""
    r = both(3, lens, H, G, Dk, Dv, seg_mode=seg)
    del r["sums"]
    for k, (got, want) in r.items():
        if got.dtype != BF:
            continue
        own = rms(want.to(BF).double() - want)
        e = rms(got.double() - want)
        print(f"    {k} {e / rms(want):.3e} (rounding alone {own / rms(want):.3e})", flush=True)
        if k in ("y", "dx"):
            assert e <= 3 ** 0.5 * own, k
        else:
            assert rms(got.double() - want.to(BF).double()) <= 2.0 ** -11 * rms(want), k


def chunk_scale(t, lens):
    """sqrt of the sum over chunks of 64 tokens of (the chunk's sum)^2, by head: what an error
    that goes with a chunk's terms, of either sign from chunk to chunk, adds up to."""
    at, tot = 0, 0.0
    for n in lens:
        for c in range(at, at + n, 64):
            tot = tot + t[c:min(c + 64, at + n)].sum(0).square()
        at += n
    return tot.sqrt()


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("lens,H,G,Dk,Dv", [([8192], 2, 1, 128, 128), ([5000, 3192], 4, 2, 64, 64)])
def test_scan_fp32_results_of_long_sequences(dev, lens, H, G, Dk, Dv, seed):
    """fp32 results of bf16 inputs over thousands of tokens.  An entry of a state is a sum of 64
    products a chunk: off by sqrt(64) = 8 fp32 roundings of its size (one standard deviation),
    and the decay forgets within a few chunks: 1e-6 of the largest entry, 17 roundings, has room.
    da_t is a product of two such states, so off by 8 sqrt(2) roundings of its size; as d da
    added up over the chunks that is the standard deviation of dA = sum d da (which may
    cancel far below its terms), and the same of the two parts of ddt = A da + (dh B) x that of the
    bias's gradient.  Four of them, 4 8 sqrt(2) = 45 roundings, hold for the 12 heads here
    (operands cut to 16 bits, short by 128 on average, would add up as the plain sum, sqrt(128
    chunks) = 11 times as fast)."""
    r = both(seed, lens, H, G, Dk, Dv)
    gd, ga, d, v = r.pop("sums")
    for k in ("hT", "dh0"):
        got, want = r[k]
        e = ((got.double() - want).abs().max() / want.abs().max()).item()
        print(f"    {k} {e:.2e}", flush=True)
        assert e <= 1e-6, k
    A = inputs(seed, sum(lens), H, G, Dk, Dv, len(lens))[0]["A"].double()
    u = 2.0 ** -24
    terms = dict(dA=(d * ga).abs(), dbias=((A * ga).abs() + (gd - A * ga).abs()) * torch.sigmoid(v))
    for k, t in terms.items():
        got, want = r[k]
        tol = 45 * u * chunk_scale(t, lens) + u * want.abs()
        e = ((got.double() - want).abs() / tol).max().item()
        print(f"    {k} {e:.3f} of the bound ({((got.double() - want).abs().max() / want.abs().max()).item():.2e} of the largest)", flush=True)
        assert e <= 1, k


def test_decay_gradient_does_not_drift(dev):
    """The matrix cores' sums come out low whatever their sign, and the scan keeps its states with
    alternating sign so that this cancels.  In the units of the test above the 48 heads' errors of
    dA have a mean of 0 with a standard deviation of 8 sqrt(2) / sqrt(48) = 1.6 roundings; three of
    them bound it (0.5 measured; 12 below zero with every state of one sign)."""
    mean = []
    for seed in (1, 2, 3):
        r = both(seed, [16384], 16, 1, 128, 128)
        gd, ga, d, v = r.pop("sums")
        got, want = r["dA"]
        mean.append(((got.double() - want) / chunk_scale((d * ga).abs(), [16384])).mean().item() * 2 ** 24)
        print(f"    seed {seed}: {mean[-1]:.1f} roundings", flush=True)
        del r
    assert abs(sum(mean) / 3) <= 3 * 8 * 2 ** 0.5 / 48 ** 0.5


def plain_dA(x, d, A, B, C, h0, dy, dhT, lens, Q=64):
    """dA by chunks in elementary fp32 operations, its decays and long sums in 64 bits."""
    H, rep = x.shape[1], x.shape[1] // B.shape[1]
    strict = torch.tril(torch.ones(Q, Q, device=x.device), -1)
    dA, at = 0.0, 0
    for n, L in enumerate(lens):
        nc = (L + Q - 1) // Q

        def cut(a):
            a = torch.cat([a[at:at + L].float(), a.new_zeros(nc * Q - L, *a.shape[1:], dtype=torch.float32)], 0)
            return a.reshape(nc, Q, *a.shape[1:]).transpose(1, 2).contiguous()

        X, Y, s = cut(x), cut(dy), cut(d[..., None])
        K, O = cut(B).repeat_interleave(rep, 1), cut(C).repeat_interleave(rep, 1)
        T = lambda a: a.transpose(2, 3).contiguous()
        cum = (s.double() * A.double()[:, None, None]).cumsum(2)
        tot = cum[:, :, -1:]
        w = torch.exp((cum - cum.transpose(2, 3)).clamp(max=0)).float() * strict
        e_in, e_out, e_tot = torch.exp(cum).float(), torch.exp(tot - cum).float(), torch.exp(tot).float()
        add, back = T(K) @ (e_out * s * X), T(O) @ (e_in * Y)
        hs, gs = [h0[n]], [dhT[n]]
        for c in range(nc):
            hs.append(e_tot[c] * hs[-1] + add[c])
            gs.append(e_tot[nc - 1 - c] * gs[-1] + back[nc - 1 - c])
        hs, gs = torch.stack(hs), torch.stack(gs[:-1][::-1])
        pair = (Y @ T(X)) * w * (O @ T(K)) * s.transpose(2, 3)
        sum64 = lambda a, dim: a.sum(dim, dtype=torch.float64)
        v = (sum64(pair, 3) + sum64(e_in * (Y @ T(hs[:-1])) * O, 3)) - (sum64(pair, 2) + sum64(s * e_out * X * (K @ gs), 3))
        da = sum64(gs * hs[1:], (2, 3))[..., None] + v.flip(2).cumsum(2).flip(2)
        dA = dA + (da * s[..., 0].double()).sum((0, 2))
        at += L
    return dA


@pytest.mark.parametrize("lens,H,G,Dk,Dv,dt", [([300, 1, 1027, 64, 2000], 4, 4, 64, 64, torch.float32),
                                               ([1024], 4, 4, 64, 64, BF), ([128], 4, 2, 128, 64, torch.float32)])
def test_decay_gradient_is_as_exact_as_a_plain_one(dev, lens, H, G, Dk, Dv, dt):
    """Rms error of dA over 24 inputs, in the units above, against that of plain fp32 operations.
    The kernels' terms pass about three times as many fp32 roundings (a decay is a product of three
    factors, a bf16 product is a sum of three parts' products): sqrt(3) times the plain error.  With
    the pairs of a chunk taken from two sweeps the ratio was 2.0, 2.4 and 2.2."""
    mine, plain = 0.0, 0.0
    for seed in range(24):
        r = both(seed, lens, H, G, Dk, Dv, dt)
        gd, ga, d, v = r.pop("sums")
        Qs = chunk_scale((d * ga).abs(), lens)
        s, dy, dhT = inputs(seed, sum(lens), H, G, Dk, Dv, len(lens), dt)
        step = F.softplus(s["dt"][0].float() + s["bias"])
        p = plain_dA(s["x"][0], step, s["A"], s["B"][0], s["C"][0], s["h0"], dy[0], dhT, lens)
        got, want = r["dA"]
        mine += ((got.double() - want) / Qs).square().mean().item()
        plain += ((p - want) / Qs).square().mean().item()
    mine, plain = ((t / 24) ** 0.5 * 2 ** 24 for t in (mine, plain))
    print(f"    {mine:.1f} roundings, plain {plain:.1f}", flush=True)
    assert mine <= 3 ** 0.5 * plain


MANY = {"65": [(3 * i) % 7 for i in range(64)] + [130], "1100": [(5 * i) % 4 for i in range(1099)] + [70]}
SHAPES = [("65", 2, 1, 64, 64), ("1100", 1, 1, 64, 64), ([200], 64, 1, 128, 64), ([70, 60], 128, 1, 128, 64)]


@pytest.mark.parametrize("lens,H,G,Dk,Dv", SHAPES)
@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_scan_of_many_sequences_and_heads(dev, lens, H, G, Dk, Dv, dt):
    """More sequences than one wave and than one workgroup plans, and many heads on one B and C.
    Tolerances as for the other shapes: bf16 outputs rounded once, fp32 results 2e-6 of the
    largest entry, the sums over all tokens 2e-5."""
    r = both(4, MANY.get(str(lens), lens), H, G, Dk, Dv, dt, round_once=True)
    del r["sums"]
    for k, (got, want) in r.items():
        if got.dtype == BF:
            e, tol = rms(got.double() - want.to(BF).double()) / rms(want), 2.0 ** -11
        else:
            e = ((got.double() - want).abs().max() / want.abs().max()).item()
            tol = {"dA": 2e-5, "dbias": 2e-5, "ddt": 1e-5, "dD": 4e-6}.get(k, 2e-6)
        print(f"    {k} {e:.2e} (<= {tol:.1e})", flush=True)
        assert e <= tol, k


def test_gates_of_fp32_tensors(dev):
    """silu(x) of fp32 tensors over the exponential's range, relative to every value: the
    exponential and the reciprocal off by 2^-23 each, and three roundings: 7 fp32 roundings,
    and one more for the norm's product.  Its derivative s + x (s - s s) likewise, relative to
    the size of its terms (s one rounding finer than 1 where x is large)."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, layers, short_conv
    x = torch.linspace(-80, 80, 64 * 1024, device=dev).view(1, -1, 64)
    x = torch.cat([x, x / 16], 1).contiguous()
    w = torch.zeros(64, 2, device=dev)
    w[:, 1] = 1                                                  # u = x
    want = x.double() * torch.sigmoid(x.double())
    live = x.abs() > 1e-3
    def worst(name, got, ref, size):
        e = ((got.double() - ref).abs() / size)[live].max().item() * 2 ** 24
        print(f"    {name} {e:.1f} roundings", flush=True)
        return e
    n = torch.ones_like(x)
    w1 = torch.ones(64, device=dev)
    conv = short_conv(x, w)
    step = layers.gdn_conv_step(x[0].contiguous(), torch.zeros(x.shape[1], 1, 64, device=dev), w)
    norm = gated_group_norm(n, w1, x, eps=1e-30)                 # n / sqrt(1) = 1
    long = gated_group_norm(torch.ones(23, 1, 5501, device=dev), torch.ones(5501, device=dev),
                            x.flatten()[:23 * 5501].view(23, 1, 5501), eps=1e-30)
    assert worst("convolution", conv, want, want.abs()) <= 8
    assert torch.equal(step[None], conv)
    assert worst("norm", norm, want, want.abs()) <= 8
    lw = want.flatten()[:23 * 5501].view(23, 1, 5501)
    assert ((long.double() - lw).abs() <= 8 * 2.0 ** -24 * lw.abs() + 1e-30).all()
    leaf = x.clone().requires_grad_(True)
    (dx,) = torch.autograd.grad(short_conv(leaf, w), leaf, torch.ones_like(x))
    s = torch.sigmoid(x.double())
    size = s + x.double().abs() * s * torch.clamp(1 - s, min=2.0 ** -24)
    assert worst("derivative", dx, s + x.double() * s * (1 - s), size) <= 24
    inf = float("inf")
    e = short_conv(torch.tensor([inf, 200.0, -200.0, float("nan")], device=dev).view(1, 1, 4), w[:4])
    assert e[0, 0, 0] == inf and e[0, 0, 1] == 200 and e[0, 0, 2] == 0 and e[0, 0, 3].isnan()


@pytest.mark.parametrize("rows,G,D", [(1 << 20, 1, 8), (300_000, 2, 24), (40_000, 1, 5501), (1 << 25, 1, 3)])
@pytest.mark.parametrize("shared", [False, True])
def test_weight_gradients_over_many_rows(dev, rows, G, D, shared):
    """Sums of many like terms, where an fp32 sum of n terms is off by up to n / 2 roundings: a
    thread's has at most 64 terms, a workgroup's 32 of those, the rest is summed in 64 bits."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm
    x = torch.full((rows, G, D), 1.5, device=dev)
    x[..., 1::2] = -0.75
    ws = (D,) if shared else (G, D)
    w, b = torch.ones(*ws, device=dev, requires_grad=True), torch.zeros(*ws, device=dev, requires_grad=True)
    dy = torch.full((rows, G, D), 0.1, device=dev)
    dw, db = torch.autograd.grad(gated_group_norm(x, w, bias=b), [w, b], dy)
    n = rows * (G if shared else 1)
    v = x[0, 0].double()
    want = 0.1 * n * v / torch.sqrt((v * v).mean() + 1e-5)
    for name, got, ref in (("dw", dw, want), ("db", db, torch.full_like(v, n * 0.1))):
        e = ((got.double() - ref) / ref).abs().max().item() * 2 ** 24
        print(f"    {name} {e:.1f} roundings", flush=True)
        assert e <= 32 + 16 + 8, name         # and a row's statistics, 0.1 and the result


def test_convolution_weight_gradients_over_many_tokens(dev):
    """The same: a thread's sum has at most 128 terms."""
    from gated_deltanet_chunked_delta_amd import short_conv
    T, D = 1 << 20, 8
    x = torch.full((1, T, D), 1.5, device=dev)
    w, b = torch.zeros(D, 4, device=dev, requires_grad=True), torch.zeros(D, device=dev, requires_grad=True)
    dy = torch.full_like(x, 0.1)
    dw, db = torch.autograd.grad(short_conv(x, w, b, silu=False), [w, b], dy)
    lag = torch.tensor([3.0, 2.0, 1.0, 0.0], device=dev, dtype=torch.float64)
    for name, got, ref in (("dw", dw, (0.15 * (T - lag)).expand(D, 4)), ("db", db, torch.full_like(db, 0.1 * T).double())):
        e = ((got.double() - ref) / ref).abs().max().item() * 2 ** 24
        print(f"    {name} {e:.1f} roundings", flush=True)
        assert e <= 64 + 4, name
