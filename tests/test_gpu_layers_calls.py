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
