"""Calls of the layer operators that their documentation allows, on the GPU."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def scan_leaves(seed, T, H, G, Dk, Dv, dt=BF, B=1):
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda:0")
    return [t.requires_grad_(True) for t in (
        rn(B, T, H, Dv).to(dt), rn(B, T, H) * 0.1, -(1 + torch.rand(H, generator=g, device="cuda:0")),
        rn(B, T, G, Dk).to(dt), rn(B, T, G, Dk).to(dt))]


@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_gradients_that_start_anywhere(dev, dt):
    """Behind three other entries of a concatenation y's gradient starts off 16 bytes: the same
    gradients as from an aligned one.  Bit for bit from the scan, which gets a copy; the other
    two read it element by element and sum a row's 48 entries and the rows in another order:
    each side within (16 + 2 sqrt(48)) fp32 roundings of the exact sums."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, selective_scan, short_conv
    leaves = scan_leaves(1, 150, 2, 1, 64, 64, dt)
    x, w = torch.randn(1, 33, 40, device=dev).to(dt), torch.randn(40, 4, device=dev).to(dt)
    n, nw = torch.randn(9, 2, 48, device=dev).to(dt), torch.randn(48, device=dev).to(dt)
    calls = [(lambda: selective_scan(*leaves, dt_softplus=True), leaves),
             (lambda: short_conv(x, w), [x.requires_grad_(True), w.requires_grad_(True)]),
             (lambda: gated_group_norm(n, nw), [n.requires_grad_(True), nw.requires_grad_(True)])]
    for f, into in calls:
        y = f()
        dy = torch.randn(y.shape, device=dev).to(dt)
        want = torch.autograd.grad(y, into, dy)
        y = f()
        both = torch.cat([torch.zeros(3, dtype=dt, device=dev), y.flatten()])
        got = torch.autograd.grad(both, into, torch.cat([torch.zeros(3, dtype=dt, device=dev), dy.flatten()]))
        for a, b in zip(got, want):
            if into is leaves:
                assert torch.equal(a, b)
            else:
                e = (a.double() - b.double()).abs().max() / b.double().abs().max()
                assert e <= 2 * ((16 + 2 * 48 ** 0.5) * 2.0 ** -24 + (2.0 ** -8 if dt == BF else 0.0))


def test_chunk_rule_gradients_that_start_anywhere(dev):
    from gated_deltanet_chunked_delta_amd import chunk_gated_delta_rule
    g = torch.Generator(device=dev).manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    into = [t.requires_grad_(True) for t in (
        rn(1, 130, 2, 64).to(BF), rn(1, 130, 2, 64).to(BF), rn(1, 130, 2, 64).to(BF), -rn(1, 130, 2).abs(), rn(1, 130, 2).to(BF))]
    f = lambda: chunk_gated_delta_rule(*into, qk_norm=True)
    dy = rn(1, 130, 2, 64).to(BF)
    want = torch.autograd.grad(f(), into, dy)
    z = torch.zeros(3, dtype=BF, device=dev)
    got = torch.autograd.grad(torch.cat([z, f().flatten()]), into, torch.cat([z, dy.flatten()]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("lens", [None, [70, 0, 129]])
def test_captured_autograd_training(dev, lens):
    """The three operators with autograd, forward and backward captured together; every replay,
    with eager work between, gives what an eager pass of other leaves gives."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, selective_scan, short_conv
    H, Dk, Dv, T = 2, 64, 64, 199
    kw = {}
    if lens:
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        kw = dict(cu_seqlens=cu.to(dev), cu_seqlens_host=cu)
    g = torch.Generator(device=dev).manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    values = [rn(1, T, H * Dv).to(BF), rn(H * Dv, 4).to(BF), rn(1, T, H).to(BF), -1 - rn(H).abs(), rn(1, T, 1, Dk).to(BF),
              rn(1, T, 1, Dk).to(BF), rn(H), rn(Dv).to(BF), rn(1, T, H, Dv).to(BF)]
    dy = rn(1, T, H, Dv).to(BF)

    def train(leaves):
        x, w, dt, A, B, C, bias, nw, z = leaves
        c = short_conv(x, w, **kw).view(1, T, H, Dv)
        y = gated_group_norm(selective_scan(c, dt, A, B, C, dt_bias=bias, dt_softplus=True, seg_mode=1, **kw), nw, z)
        return [y.detach(), *torch.autograd.grad(y, leaves, dy)]

    fresh = lambda: [v.clone().requires_grad_(True) for v in values]
    side = torch.cuda.Stream()
    static = fresh()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        train(static)                       # (its eager graph is gone when the capture begins)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = train(static)
    torch.cuda.synchronize()
    for k in range(3):
        values[0] = rn(1, T, H * Dv).to(BF)
        with torch.no_grad():
            static[0].copy_(values[0])
        graph.replay()
        torch.cuda.synchronize()
        want = train(fresh())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_are_not_lost(dev, bad):
    """A value that is not finite makes its sequence not finite from its chunk of 64 tokens on,
    leaves the chunks before it as they are, and shows in every gradient summed over tokens."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, selective_scan, short_conv
    lens, at = [30, 200, 10], 30 + 70
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    kw = dict(cu_seqlens=cu.to(dev), cu_seqlens_host=cu)
    out = []
    for poison in (False, True):
        g = torch.Generator(device=dev).manual_seed(6)
        rn = lambda *s: torch.randn(*s, generator=g, device=dev)
        x, B, C, u = rn(1, 240, 2, 64).to(BF), rn(1, 240, 1, 64).to(BF), rn(1, 240, 1, 64).to(BF), rn(1, 240, 48).to(BF)
        dt, A, D, bias, w = rn(1, 240, 2) - 2, -1 - rn(2).abs(), rn(2), rn(2), rn(48, 4).to(BF)
        nw, cb = rn(64).to(BF), rn(48).to(BF)
        if poison:
            for t in (x, u):
                t[0, at] = bad
        leaves = [t.requires_grad_(True) for t in (A, D, bias)]
        y, hT = selective_scan(x, dt, A, B, C, D=D, dt_bias=bias, dt_softplus=True, output_final_state=True, **kw)
        sums = list(torch.autograd.grad(y, leaves, torch.ones_like(y)))
        c = short_conv(u, w.requires_grad_(True), cb.requires_grad_(True), **kw)
        sums += torch.autograd.grad(c, [w, cb], torch.ones_like(c))
        n = gated_group_norm(x, nw.requires_grad_(True))
        sums += torch.autograd.grad(n, [nw], torch.ones_like(n))
        out.append(([t.detach() for t in (y, hT, c, n)], sums))
    (y0, h0, c0, n0), clean = out[0]
    (y1, h1, c1, n1), dirty = out[1]
    assert all(t.isfinite().all() for t in out[0][0] + clean)
    assert torch.equal(y1[:, :94], y0[:, :94]) and torch.equal(y1[:, 230:], y0[:, 230:])
    assert not y1[:, 94:230].isfinite().any()
    assert not h1[1].isfinite().any() and torch.equal(h1[[0, 2]], h0[[0, 2]])
    assert not c1[:, at:at + 4].isfinite().any() and torch.equal(c1[:, :at], c0[:, :at]) and torch.equal(c1[:, at + 4:], c0[:, at + 4:])
    assert not n1[:, at].isfinite().any() and torch.equal(n1[:, at + 1:], n0[:, at + 1:])
    for k, t in enumerate(dirty):
        assert not t.isfinite().any(), k


@pytest.mark.parametrize("name", ["conv", "scan", "norm", "conv_step", "scan_step", "library"])
def test_inside_a_compiled_function(dev, name):
    """A function compiled by torch.compile leaves its graph for the calls: results and gradients
    are those of the function itself, bit for bit, in its first call and in later ones of
    another length."""
    from gated_deltanet_chunked_delta_amd import (gated_group_norm, gdn_conv_fwd, gdn_conv_step, gdn_norm_fwd,
                                                  gdn_scan_fwd, gdn_scan_step, selective_scan, short_conv)
    g = torch.Generator(device=dev).manual_seed(8)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    A = -1 - rn(2).abs()
    scan = lambda T: (rn(1, T, 2, 64), rn(1, T, 2), A, rn(1, T, 1, 64), rn(1, T, 1, 64))

    def library(x, dt, A, B, C):
        y, hT = gdn_scan_fwd(2 * x, dt, A, B, C, dt_softplus=True)
        z, fin = gdn_conv_fwd(y.flatten(2), torch.ones(128, 4, device=dev))
        return gdn_norm_fwd(z.view(x.shape), torch.ones(64, device=dev)), hT, fin

    f, inputs = {
        "conv": (lambda x, w: short_conv(2 * x, w, output_final_state=True), lambda T: (rn(1, T, 48), rn(48, 4))),
        "scan": (lambda *a: selective_scan(2 * a[0], *a[1:], dt_softplus=True, output_final_state=True), scan),
        "norm": (lambda x, w: (gated_group_norm(2 * x, w),), lambda T: (rn(T, 2, 64), rn(64))),
        "conv_step": (lambda x, w, state: (gdn_conv_step(2 * x, state, w), state), lambda T: (rn(T, 48), rn(48, 4), rn(T, 3, 48))),
        "scan_step": (lambda x, dt, A, B, C, state: (gdn_scan_step(2 * x, dt, A, B, C, state, dt_softplus=True), state),
                      lambda T: (rn(T, 2, 64), rn(T, 2), A, rn(T, 1, 64), rn(T, 1, 64), rn(T, 2, 64, 64))),
        "library": (library, scan),
    }[name]
    torch._dynamo.reset()
    compiled = torch.compile(f, backend="eager")
    trained = name in ("conv", "scan", "norm")
    for T in (70, 70, 5, 133):
        at, results = inputs(T), []
        for call in (f, compiled):
            leaves = [t.clone().requires_grad_(trained) for t in at]
            out = list(call(*leaves))
            results.append(out + (list(torch.autograd.grad(out, leaves, [torch.ones_like(t) for t in out])) if trained else []))
        assert all(torch.equal(a, b) for a, b in zip(*results))


def test_chunk_rule_inside_a_compiled_function(dev):
    from gated_deltanet_chunked_delta_amd import chunk_gated_delta_rule, gdn_decode_step
    g = torch.Generator(device=dev).manual_seed(9)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)

    def f(q, k, v, g, beta):
        with torch.no_grad():
            state = torch.zeros(1, 2, 64, 64, device=dev)
            step = gdn_decode_step(*(t[:, 0].contiguous() for t in (q, k, v, g, beta)), 0.125, state)
        return chunk_gated_delta_rule(q, 2 * k, v, g, beta, qk_norm=True, output_final_state=True) + (step, state)

    torch._dynamo.reset()
    compiled = torch.compile(f, backend="eager")
    for T in (70, 70, 5, 133):
        inputs = (rn(1, T, 2, 64).to(BF), rn(1, T, 2, 64).to(BF), rn(1, T, 2, 64).to(BF), -rn(1, T, 2).abs(), rn(1, T, 2).to(BF))
        results = []
        for call in (f, compiled):
            leaves = [t.clone().requires_grad_(True) for t in inputs]
            out = list(call(*leaves))
            results.append(out + list(torch.autograd.grad(out[:2], leaves, [torch.ones_like(t) for t in out[:2]])))
        assert all(torch.equal(a, b) for a, b in zip(*results))
