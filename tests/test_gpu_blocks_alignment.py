"""Inputs, states and scales that start anywhere an element may, against the same call on
copies of their own: the same bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


import gated_deltanet_chunked_delta_amd as gdn  # noqa: E402
from gated_deltanet_chunked_delta_amd import blocks  # noqa: E402


def rn(seed, *s, std=1.0, dt=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda", dtype=torch.float64) * std).to(dt)


def off(t, n=1):
    """t's values, contiguous, n elements behind an allocation's start."""
    wide = torch.zeros(t.numel() + n, device=t.device, dtype=torch.uint8 if t.element_size() == 1 else t.dtype)
    wide[n:] = t.reshape(-1).view(wide.dtype)
    out = wide[n:].view(t.dtype).view(t.shape)
    assert out.data_ptr() % 16 != 0
    return out


def rows(t, n=1):
    """t's values as a slice of wider rows, n elements in."""
    raw = t.view(torch.uint8) if t.element_size() == 1 else t
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 5, device=t.device, dtype=raw.dtype)
    wide[..., n:n + t.shape[-1]] = raw
    return wide.view(t.dtype)[..., n:n + t.shape[-1]]


def same(a, b):
    a, b = ([t for t in (o if isinstance(o, tuple) else (o,)) if t is not None] for o in (a, b))
    assert len(a) == len(b)
    for p, q in zip(a, b):
        assert p.shape == q.shape and torch.equal(p.view(torch.uint8) if p.element_size() == 1 else p, q.view(torch.uint8) if q.element_size() == 1 else q)


@pytest.mark.parametrize("n", [1, 2, 3])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(5, 64, 80), (70, 64, 80), (300, 136, 260), (300, 67, 129)])
def test_projections(M, K, N, dt, n):
    dt = DT[dt]
    x, w, b, r, dy = rn(1, M, K, dt=dt), rn(2, N, K, std=.2, dt=dt), rn(3, N, dt=dt), rn(4, M, N, dt=dt), rn(5, M, N, dt=dt)
    same(blocks.gdn_linear_fwd(rows(x, n), off(w, n), off(b, n), "silu", rows(r, n), save=True), blocks.gdn_linear_fwd(x, w, b, "silu", r, save=True))
    v = blocks.gdn_linear_fwd(x, w, b, "silu", r, save=True)[1]
    same(blocks.gdn_linear_bwd(rows(x, n), off(w, n), off(dy, n), "silu", off(v, n)), blocks.gdn_linear_bwd(x, w, dy, "silu", v))
    same(blocks.gdn_linear_bwd(x, w, off(dy, n)), blocks.gdn_linear_bwd(x, w, dy))
    (q, s), (p, t) = gdn.quantize_rows(x), gdn.quantize_rows(w)
    for out in DT.values():
        b, r = b.to(out), r.to(out)
        same(gdn.linear_8bit(rows(q, n), off(s, n), off(p, n), off(t, n), off(b, n), "gelu", rows(r, n), out_dtype=out),
             gdn.linear_8bit(q, s, p, t, b, "gelu", r, out_dtype=out))


@pytest.mark.parametrize("dt,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("R,D", [(5, 40), (1100, 129), (300, 2304), (9, 20001)])
def test_norms_and_8_bits(R, D, dt, res):
    dt, res = DT[dt], DT[res]
    x, w, r, dy, ds = rn(1, R, D, dt=dt), rn(2, D, dt=dt), rn(3, R, D, dt=res), rn(4, R, D, dt=dt), rn(5, R, D, dt=res)
    same(gdn.add_rms_norm(rows(x), off(w), rows(r)), gdn.add_rms_norm(x, w, r))
    same(gdn.add_rms_norm_8bit(rows(x), off(w), rows(r)), gdn.add_rms_norm_8bit(x, w, r))
    same(gdn.quantize_rows(rows(x)), gdn.quantize_rows(x))
    same(blocks.gdn_addnorm_bwd(rows(r), off(w), off(dy), off(ds)), blocks.gdn_addnorm_bwd(r, w, dy, ds))


@pytest.mark.parametrize("dt,g32", [("bf16", 0), ("bf16", 1), ("f32", 0)])
@pytest.mark.parametrize("D", [1, 2, 63, 130])
def test_recurrences(D, dt, g32):
    dt = DT[dt]
    gt = torch.float32 if g32 else dt
    cu = torch.tensor([0, 3, 3, 150, 400], dtype=torch.int32, device="cuda")
    x, g, i, sc, h0 = rn(1, 1, 400, D, dt=dt), rn(2, 1, 400, D, dt=gt), rn(3, 1, 400, D, dt=dt), rn(4, D).abs() * .2, rn(5, 4, D)
    dy, dh = rn(6, 1, 400, D, dt=dt), rn(7, 4, D)
    kw, odd = dict(cu_seqlens=cu, cu_seqlens_host=cu.cpu()), dict(cu_seqlens=off(cu), cu_seqlens_host=cu.cpu())
    same(blocks.gdn_rec_fwd(rows(x), rows(g, 2), rows(i, 3), off(sc), off(h0), **odd), blocks.gdn_rec_fwd(x, g, i, sc, h0, **kw))
    st = blocks.gdn_rec_fwd(x, g, i, sc, h0, save_states=True, **kw)[2]
    same(blocks.gdn_rec_bwd(rows(x), rows(g, 2), off(dy), rows(i, 3), off(sc), off(h0), off(dh), states=off(st), **odd),
         blocks.gdn_rec_bwd(x, g, dy, i, sc, h0, dh, states=st, **kw))
    n, slots = 7, torch.tensor([5, 0, 11, 2, 9, -1, 3], dtype=torch.int32, device="cuda")
    a, b = rn(8, 12, D), off(rn(8, 12, D))
    ya, yb = torch.zeros(n, D, device="cuda", dtype=dt), off(torch.zeros(n, D, device="cuda", dtype=dt))
    gdn.gdn_rec_step(x[0, :n], g[0, :n], a, i[0, :n], sc, slots, ya)
    gdn.gdn_rec_step(rows(x)[0, :n], rows(g, 2)[0, :n], b, rows(i, 3)[0, :n], off(sc), off(slots), yb)
    same((a, ya), (b, yb))
