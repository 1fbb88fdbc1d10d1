"""The operators around the recurrence on the GPU, element by element against
plain forms in 64 bits on the same rounded inputs.

Tolerances.  A stored result is off by at most half a step of its type, u
relative to its value (bf16 2^-8 as a bound, fp32 2^-24); what is computed in
fp32 before that is off by a few fp32 roundings of the largest terms summed, far
below bf16's step.  So per element |got - want| <= u |want| + c u32 S with S the
root mean square scale of the terms' sum, for direct formulas.  The scan's bf16
outputs also round a chunk matrix and the state to bf16 once each inside: two
more relative errors of u on quantities of the output's own scale, which per
element can reach a few u times the tensor's rms; the bound is 8 u on
max|got - want| / max|want| (each error is below u max-term and they add in
quadrature over 64 terms).  States and fp32 gradients carry fp32 precision:
64 tokens a chunk, 24-bit operands: 2e-6 of the largest entry.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import torch.nn.functional as F  # noqa: E402

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rn(g, *s, std=1.0, dt=torch.float32, dev="cuda:0"):
    return (torch.randn(*s, generator=g, dtype=torch.float64) * std).to(dt).to(dev)


def d64(t):
    return None if t is None else t.detach().double().cpu()


def err(got, want):
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, (got.shape, want.shape)
    if want.numel() == 0:
        return 0.0
    s = want.abs().max().item()
    e = (got - want).abs().max().item()
    assert math.isfinite(e)
    return e / s if s > 0 else e


def close(name, got, want, tol):
    e = err(got, want)
    print(f"    {name} {e:.2e} (<= {tol:.1e})", flush=True)
    assert e <= tol, name


# ------------------------------------------------------------------ 64-bit plain forms
def ref_conv(x, w, b, init, bounds, silu):
    """x [B, T, D] in 64 bits, differentiable; final states [N, W-1, D]."""
    W = w.shape[1]
    y = torch.zeros_like(x)
    rows, fins = [], []
    for n, (row, lo, hi) in enumerate(bounds):
        head = init[n] if init is not None else x.new_zeros(W - 1, x.shape[2])
        full = torch.cat([head, x[row, lo:hi]], 0)
        u = sum(w[:, k] * full[k:k + hi - lo] for k in range(W))
        if b is not None:
            u = u + b
        rows.append((row, lo, hi, u * torch.sigmoid(u) if silu else u))
        fins.append(full[hi - lo:])
    for row, lo, hi, v in rows:
        y = y.index_put((torch.tensor(row).expand(hi - lo), torch.arange(lo, hi)), v)
    return y, torch.stack(fins)


def ref_scan(x, dt, A, B, C, D, bias, softplus, h0, bounds):
    """Token by token in 64 bits, differentiable."""
    H, G = x.shape[2], B.shape[2]
    head = torch.arange(H) // (H // G)
    d = dt + bias if bias is not None else dt
    d = torch.logaddexp(d, torch.zeros_like(d)) if softplus else d
    y = torch.zeros_like(x)
    hT = []
    for n, (row, lo, hi) in enumerate(bounds):
        h = h0[n] if h0 is not None else x.new_zeros(H, B.shape[3], x.shape[3])
        out = []
        for t in range(lo, hi):
            dd = d[row, t][:, None, None]
            h = torch.exp(dd * A[:, None, None]) * h + dd * B[row, t, head][:, :, None] * x[row, t][:, None, :]
            o = (h * C[row, t, head][:, :, None]).sum(1)
            out.append(o if D is None else o + D[:, None] * x[row, t])
        if hi > lo:
            y = y.index_put((torch.tensor(row).expand(hi - lo), torch.arange(lo, hi)), torch.stack(out))
        hT.append(h)
    return y, torch.stack(hT)


def ref_norm(x, w, z, b, eps, center, gate_first):
    act = None if z is None else z * torch.sigmoid(z)
    v = x * act if gate_first else x
    if center:
        v = v - v.mean(-1, keepdim=True)
    o = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w
    if b is not None:
        o = o + b
    return o * act if z is not None and not gate_first else o


def bounds_of(B, T, lens):
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return [(0, at[i], at[i + 1]) for i in range(len(lens))]


def cu_of(lens, dev):
    if lens is None:
        return {}
    host = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    return dict(cu_seqlens=host.to(dev), cu_seqlens_host=host)


def ref_grads(outs, gouts, leaves):
    pairs = [(o, g) for o, g in zip(outs, gouts) if g is not None and o.requires_grad]
    return torch.autograd.grad([o for o, _ in pairs], leaves, [g for _, g in pairs], allow_unused=True)


# ------------------------------------------------------------------ convolution
CONV = [  # B, T, lens, D, W, bias, silu, init, dtype
    (1, 1, None, 8, 4, True, True, True, "bf16"),
    (2, 5, None, 64, 3, False, True, False, "bf16"),
    (3, 67, None, 136, 4, True, False, True, "bf16"),
    (1, 300, None, 2048, 4, False, True, True, "bf16"),
    (1, 0, [1, 2, 3, 0, 130, 64, 17, 1], 200, 4, True, True, True, "bf16"),
    (1, 0, [0, 0, 5, 33, 0], 77, 2, True, True, True, "bf16"),      # odd width: element accesses
    (1, 0, [257, 3], 1001, 4, False, True, False, "bf16"),
    (2, 100, None, 60, 3, True, True, True, "f32"),
    (1, 0, [2, 40, 0, 9], 33, 4, True, False, True, "f32"),
]


@pytest.mark.parametrize("B,T,lens,D,W,bias,silu,init,dtype", CONV)
def test_conv_forward_and_gradients(dev, B, T, lens, D, W, bias, silu, init, dtype):
    from gated_deltanet_chunked_delta_amd import short_conv
    print(f"[conv] B={B} T={T} lens={lens} D={D} W={W} {dtype}", flush=True)
    g, dt = gen(D + W), DT[dtype]
    T = sum(lens) if lens else T
    n = len(lens) if lens else B
    x, w = rn(g, B, T, D, dt=dt), rn(g, D, W, std=0.5, dt=dt)
    b = rn(g, D, std=0.3, dt=dt) if bias else None
    st = rn(g, n, W - 1, D, dt=dt) if init else None
    dy, dfin = rn(g, B, T, D, dt=dt), rn(g, n, W - 1, D, dt=dt)
    leaves = [t.requires_grad_(True) for t in (x, w, b, st) if t is not None]
    y, fin = short_conv(x, w, b, silu=silu, initial_state=st, output_final_state=True, **cu_of(lens, dev))
    grads = torch.autograd.grad([y, fin], leaves, [dy, dfin])
    torch.cuda.synchronize()
    rl = [d64(t).requires_grad_(True) for t in (x, w, b, st) if t is not None]
    it = iter(rl)
    rx, rw = next(it), next(it)
    rb = next(it) if bias else None
    rs = next(it) if init else None
    ry, rf = ref_conv(rx, rw, rb, rs, bounds_of(B, T, lens), silu)
    rg = ref_grads([ry, rf], [d64(dy), d64(dfin)], rl)
    # W + 1 products and a sigmoid in fp32, then one rounding: u and 16 fp32 roundings;
    # the weights' gradients sum up to T terms in fp32
    tol = U[dt] + 16 * U[torch.float32]
    close("y", y, ry, tol)
    assert torch.equal(fin.cpu(), rf.to(dt))                       # copied inputs
    for name, got, want in zip("x w b init".split() if bias else ["x", "w", "init"], grads, rg):
        close("d" + name, got, want, U[dt] + (16 + 2 * math.sqrt(max(T, 1))) * U[torch.float32])


def test_conv_strided_rows_and_tail(dev):
    """x a slice of a wider projection; rows behind the last sequence stay as they were."""
    from gated_deltanet_chunked_delta_amd import layers
    g = gen(5)
    wide = rn(g, 1, 50, 400, dt=torch.bfloat16)
    w = rn(g, 160, 4, dt=torch.bfloat16)
    for off in (8, 3):                                             # 16-byte aligned, and not
        x = wide[:, :, off:off + 160]
        y, fin = layers.gdn_conv_fwd(x, w)
        y2, fin2 = layers.gdn_conv_fwd(x.contiguous(), w)
        assert torch.equal(y, y2) and torch.equal(fin, fin2)
    cu = torch.tensor([0, 20, 41], dtype=torch.int32, device=dev)
    y, _ = layers.gdn_conv_fwd(wide[:, :, :160], w, cu_seqlens=cu)
    assert torch.equal(y[:, 41:], torch.zeros_like(y[:, 41:]))
    full, _ = layers.gdn_conv_fwd(wide[:, 20:41, :160].contiguous(), w)
    assert torch.equal(y[:, 20:41], full)


@pytest.mark.parametrize("N,D,W,dtype", [(1, 64, 4, "bf16"), (5, 72, 2, "bf16"), (7, 1001, 3, "bf16"), (3, 20, 4, "f32")])
def test_conv_steps_continue_a_prompt(dev, N, D, W, dtype):
    """A prompt's final state continued token by token equals one longer prompt."""
    from gated_deltanet_chunked_delta_amd import layers
    g, dt, T, more = gen(N + D), DT[dtype], 6, 5
    x, w, b = rn(g, N, T + more, D, dt=dt), rn(g, D, W, dt=dt), rn(g, D, dt=dt)
    want, wfin = layers.gdn_conv_fwd(x, w, b)
    _, fin = layers.gdn_conv_fwd(x[:, :T].contiguous(), w, b)
    state = torch.full((N + 3, W - 1, D), 7.0, dtype=dt, device=dev)
    idx = torch.tensor([(3 * i + 1) % (N + 3) for i in range(N)] if N != 1 else [2], dtype=torch.int32, device=dev)
    if len(set(idx.tolist())) < N:
        idx = torch.arange(N, dtype=torch.int32, device=dev)
    state[idx.long()] = fin
    keep = [s for s in range(N + 3) if s not in idx.tolist()]
    for t in range(T, T + more):
        y = layers.gdn_conv_step(x[:, t], state, w, b, state_idx=idx)   # a strided slice
        assert torch.equal(y, want[:, t])
    assert torch.equal(state[idx.long()], wfin)
    assert bool((state[keep] == 7.0).all())
    # padding entries: skipped, their y as it was
    y0 = torch.full((N, D), 3.0, dtype=dt, device=dev)
    before = state.clone()
    layers.gdn_conv_step(x[:, 0], state, w, b, state_idx=torch.full_like(idx, -1), y=y0)
    layers.gdn_conv_step(x[:, 0], state, w, b, state_idx=torch.full_like(idx, N + 3), y=y0)
    assert bool((y0 == 3.0).all()) and torch.equal(state, before)


# ------------------------------------------------------------------ scan
def scan_inputs(g, lead, H, G, Dk, Dv, dt, raw, n, h0, dev):
    s = dict(x=F.silu(rn(g, *lead, H, Dv)).to(dt), B=F.silu(rn(g, *lead, G, Dk)).to(dt), C=F.silu(rn(g, *lead, G, Dk)).to(dt))
    s["A"] = -(1 + 15 * torch.rand(H, generator=g)).to(dev)
    s["D"] = rn(g, H)
    s["bias"] = rn(g, H) - 4 if raw else None
    s["dt"] = rn(g, *lead, H).to(dt) if raw else F.softplus(rn(g, *lead, H) - 4)
    s["h0"] = rn(g, n, H, Dk, Dv, std=0.3) if h0 else None
    return s


SCAN = [  # B, T, lens, H, G, Dk, Dv, raw, h0, seg_mode, dtype
    (1, 1, None, 1, 1, 64, 64, True, False, 0, "bf16"),
    (2, 63, None, 2, 2, 64, 64, True, True, 0, "bf16"),
    (1, 64, None, 3, 1, 128, 64, False, True, 0, "bf16"),
    (1, 65, None, 5, 1, 64, 128, True, True, 1, "bf16"),
    (2, 200, None, 4, 2, 128, 128, True, True, 1, "bf16"),
    (1, 333, None, 6, 1, 128, 64, True, False, 2, "bf16"),
    (1, 150, None, 1, 1, 64, 256, False, True, 1, "bf16"),
    (1, 100, None, 2, 1, 128, 192, True, True, -1, "bf16"),
    (1, 0, [1, 0, 64, 130, 0, 65, 2], 4, 1, 128, 128, True, True, 1, "bf16"),
    (1, 0, [300, 7], 2, 1, 64, 64, False, True, 3, "bf16"),
    (1, 0, [0, 0], 2, 1, 64, 64, True, True, 0, "bf16"),
    (2, 130, None, 3, 3, 64, 64, True, True, 1, "f32"),
    (1, 0, [70, 1, 129], 4, 2, 128, 128, False, True, 1, "f32"),
    (1, 90, None, 5, 1, 128, 64, True, False, -1, "f32"),
]


@pytest.mark.parametrize("B,T,lens,H,G,Dk,Dv,raw,h0,seg,dtype", SCAN)
def test_scan_forward_and_gradients(dev, B, T, lens, H, G, Dk, Dv, raw, h0, seg, dtype):
    from gated_deltanet_chunked_delta_amd import selective_scan
    print(f"[scan] B={B} T={T} lens={lens} H={H} G={G} Dk={Dk} Dv={Dv} raw={raw} seg={seg} {dtype}", flush=True)
    g, dt = gen(H * 1000 + Dk + Dv + T), DT[dtype]
    T = sum(lens) if lens is not None else T
    n = len(lens) if lens is not None else B
    s = scan_inputs(g, (B, T), H, G, Dk, Dv, dt, raw, n, h0, dev)
    dy, dhT = rn(g, B, T, H, Dv, dt=dt), rn(g, n, H, Dk, Dv, std=0.3)
    order = ["x", "dt", "A", "B", "C", "D", "bias", "h0"]
    leaves = [s[k].requires_grad_(True) for k in order if s[k] is not None]
    y, hT = selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], dt_bias=s["bias"], dt_softplus=raw,
                           initial_state=s["h0"], output_final_state=True, seg_mode=seg, **cu_of(lens, dev))
    grads = torch.autograd.grad([y, hT], leaves, [dy, dhT])
    torch.cuda.synchronize()
    r = {k: d64(s[k]).requires_grad_(True) if s[k] is not None else None for k in order}
    ry, rh = ref_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["D"], r["bias"], raw, r["h0"], bounds_of(B, T, lens))
    rl = [r[k] for k in order if r[k] is not None]
    rg = ref_grads([ry, rh], [d64(dy), d64(dhT)], rl)
    lo = 8 * U[dt] if dt == torch.bfloat16 else 2e-6
    close("y", y, ry, lo)
    close("hT", hT, rh, 2e-6)
    for k, got, want in zip([k for k in order if s[k] is not None], grads, rg):
        want = torch.zeros_like(got, device="cpu").double() if want is None else want
        # dA and dbias are sums with cancellation over all tokens: a few more bits
        tol = {"h0": 2e-6, "A": 2e-5, "D": 4e-6, "bias": 2e-5}.get(k)
        if tol is None:
            tol = lo if not (k == "dt" and got.dtype == torch.float32) else 1e-5
        close("d" + k, got, want, tol)


def test_scan_segments_agree_and_states_are_reused(dev):
    """Cut or not, with the forward's states or its own, the results are the same to fp32
    rounding, and a repeated call is the same bit for bit."""
    from gated_deltanet_chunked_delta_amd import layers
    g = gen(9)
    s = scan_inputs(g, (2, 500), 4, 1, 128, 64, torch.bfloat16, True, 2, True, dev)
    kw = dict(D=s["D"], dt_bias=s["bias"], dt_softplus=True, h0=s["h0"])
    a = [s[k] for k in ("x", "dt", "A", "B", "C")]
    dy = rn(g, 2, 500, 4, 64, dt=torch.bfloat16)
    y0, h0 = layers.gdn_scan_fwd(*a, seg_mode=-1, **kw)
    for seg in (1, 2, 3, 0):
        y, hT, st = layers.gdn_scan_fwd(*a, seg_mode=seg, save_states=True, **kw)
        close(f"hT seg {seg}", hT, d64(h0), 2e-6)
        close(f"y seg {seg}", y, d64(y0), 8 * U[torch.bfloat16])
        g1 = layers.gdn_scan_bwd(*a, dy, seg_mode=seg, states=st, **kw)
        g2 = layers.gdn_scan_bwd(*a, dy, seg_mode=seg, **kw)
        g3 = layers.gdn_scan_bwd(*a, dy, seg_mode=seg, **kw)
        for p, q, r in zip(g1, g2, g3):
            assert torch.equal(p, q) and torch.equal(q, r)


def test_scan_slices_of_one_projection(dev):
    """x, B, C and dt as slices of wider rows give what contiguous copies give."""
    from gated_deltanet_chunked_delta_amd import layers
    g = gen(10)
    H, G, Dk, Dv, T = 4, 2, 64, 64, 150
    wide = rn(g, 1, T, H * Dv + 2 * G * Dk + 8, dt=torch.bfloat16, std=0.5)
    x = wide[..., :H * Dv].view(1, T, H, Dv)
    B = wide[..., H * Dv:H * Dv + G * Dk].view(1, T, G, Dk)
    C = wide[..., H * Dv + G * Dk:H * Dv + 2 * G * Dk].view(1, T, G, Dk)
    dt = wide[..., -8:-8 + H]
    A, bias = -torch.rand(H, generator=g).to(dev) - 0.5, rn(g, H)
    dy = rn(g, 1, T, H, Dv, dt=torch.bfloat16)
    kw = dict(dt_bias=bias, dt_softplus=True)
    c = [t.contiguous() for t in (x, dt, B, C)]
    assert all(torch.equal(p, q) for p, q in zip(layers.gdn_scan_fwd(x, dt, A, B, C, **kw),
                                                 layers.gdn_scan_fwd(c[0], c[1], A, c[2], c[3], **kw)))
    got = layers.gdn_scan_bwd(x, dt, A, B, C, dy, **kw)
    want = layers.gdn_scan_bwd(c[0], c[1], A, c[2], c[3], dy, **kw)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("scale", [0.0, 1e-6, 30.0, 1e4])
def test_scan_extreme_decays(dev, scale):
    """Steps of zero (a padded token leaves the state as it is), tiny ones, and decays whose
    products underflow; nothing overflows and the gradients stay finite and right."""
    from gated_deltanet_chunked_delta_amd import selective_scan
    g = gen(11)
    s = scan_inputs(g, (1, 140), 2, 1, 64, 64, torch.bfloat16, False, 1, True, dev)
    s["dt"] = (s["dt"] / s["dt"].mean() * scale / 8).contiguous()
    dy, dhT = rn(g, 1, 140, 2, 64, dt=torch.bfloat16), rn(g, 1, 2, 64, 64)
    order = ["x", "dt", "A", "B", "C", "D", "h0"]
    leaves = [s[k].requires_grad_(True) for k in order]
    y, hT = selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], initial_state=s["h0"],
                           output_final_state=True, seg_mode=1)
    grads = torch.autograd.grad([y, hT], leaves, [dy, dhT])
    r = {k: d64(s[k]).requires_grad_(True) for k in order}
    ry, rh = ref_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["D"], None, False, r["h0"], bounds_of(1, 140, None))
    rg = ref_grads([ry, rh], [d64(dy), d64(dhT)], [r[k] for k in order])
    close("y", y, ry, 8 * U[torch.bfloat16])
    close("hT", hT, rh, 2e-6)
    if scale == 0.0:
        assert torch.equal(hT, s["h0"])
    for k, got, want in zip(order, grads, rg):
        # under decays of e^-30 a token and more, dA is what is left of terms e^30 times its size
        if k == "A" and scale >= 30:
            assert bool(torch.isfinite(got).all())
            continue
        close("d" + k, got, want, 8 * U[torch.bfloat16] if got.dtype == torch.bfloat16 else 2e-5)


@pytest.mark.parametrize("N,H,G,Dk,Dv,dtype", [(1, 1, 1, 64, 64, "bf16"), (5, 6, 2, 128, 64, "bf16"),
                                               (3, 4, 1, 64, 128, "f32"), (9, 2, 2, 128, 128, "bf16"),
                                               (2, 3, 1, 64, 192, "bf16"), (2, 2, 1, 128, 256, "f32")])
def test_scan_steps_continue_a_prompt(dev, N, H, G, Dk, Dv, dtype):
    from gated_deltanet_chunked_delta_amd import layers
    g, dt, T, more = gen(N + Dk), DT[dtype], 70, 3
    s = scan_inputs(g, (N, T + more), H, G, Dk, Dv, dt, True, N, True, dev)
    kw = dict(D=s["D"], dt_bias=s["bias"], dt_softplus=True)
    cut = {k: s[k][:, :T].contiguous() for k in ("x", "dt", "B", "C")}
    _, hT = layers.gdn_scan_fwd(cut["x"], cut["dt"], s["A"], cut["B"], cut["C"], h0=s["h0"], **kw)
    state = torch.full((N + 2, H, Dk, Dv), 5.0, device=dev)
    idx = torch.tensor([(i + 2) % (N + 2) for i in range(N)], dtype=torch.int32, device=dev)
    state[idx.long()] = hT
    ry, rh = ref_scan(*(d64(s[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias")), True, d64(s["h0"]),
                      bounds_of(N, T + more, None))
    for t in range(T, T + more):
        y = layers.gdn_scan_step(s["x"][:, t], s["dt"][:, t], s["A"], s["B"][:, t], s["C"][:, t], state, state_idx=idx, **kw)
        close("y", y, ry[:, t], U[dt] + 2e-6)
    close("state", state[idx.long()], rh, 2e-6)
    assert bool((state[:2] == 5.0).all())
    y0, before = torch.full((N, H, Dv), 3.0, dtype=dt, device=dev), state.clone()
    layers.gdn_scan_step(s["x"][:, 0], s["dt"][:, 0], s["A"], s["B"][:, 0], s["C"][:, 0], state,
                         state_idx=torch.full_like(idx, -5), y=y0, **kw)
    assert bool((y0 == 3.0).all()) and torch.equal(state, before)


def test_scan_device_lengths_that_disagree(dev):
    """A device cu_seqlens that disagrees with the host copy in its start, its end or its number
    of chunks (5 against 4 here): nothing is written."""
    import ctypes
    from gated_deltanet_chunked_delta_amd import layers
    g = gen(13)
    s = scan_inputs(g, (1, 200), 2, 1, 64, 64, torch.bfloat16, False, 2, False, dev)
    host = torch.tensor([0, 100, 200], dtype=torch.int32)
    y, hT = torch.full((1, 200, 2, 64), 9.0, dtype=torch.bfloat16, device=dev), torch.full((2, 2, 64, 64), 9.0, device=dev)
    for lens in ([0, 65, 200], [1, 100, 200], [0, 100, 199]):
        cu = torch.tensor(lens, dtype=torch.int32, device=dev)
        a, keep = layers._scan_args(s["x"], s["dt"], s["A"], s["B"], s["C"], None, None, False, None,
                                    cu, host, 1)
        f = layers.ScanFwdArgs()
        f.a, f.y, f.hT = a, y.data_ptr(), hT.data_ptr()
        ws = torch.empty(layers.lib().gdn_scan_fwd_workspace_size(ctypes.byref(f)), dtype=torch.uint8, device=dev)
        f.a.workspace, f.a.workspace_bytes = ws.data_ptr(), ws.numel()
        layers._call(layers.lib().gdn_scan_fwd, f, dev)
        torch.cuda.synchronize()
        assert bool((y == 9.0).all()) and bool((hT == 9.0).all())
        del keep


def test_scan_without_optional_inputs(dev):
    from gated_deltanet_chunked_delta_amd import selective_scan
    g = gen(12)
    s = scan_inputs(g, (1, 80), 2, 1, 64, 64, torch.float32, False, 1, False, dev)
    y = selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"])
    ry, _ = ref_scan(*(d64(s[k]) for k in ("x", "dt", "A", "B", "C")), None, None, False, None, bounds_of(1, 80, None))
    close("y", y, ry, 2e-6)


# ------------------------------------------------------------------ gated group norm
NORM = [  # lead, G, D, shared, center, gate, bias, dtype
    ((1,), 1, 1, False, False, None, False, "f32"),
    ((3, 5), 4, 64, True, False, "after", False, "bf16"),
    ((2, 33), 16, 128, True, False, "after", True, "bf16"),
    ((70,), 2, 256, False, True, "before", True, "bf16"),
    ((9,), 3, 77, False, True, "after", True, "bf16"),
    ((130,), 1, 1000, False, False, "before", False, "bf16"),
    ((40,), 1, 2000, False, True, "after", False, "bf16"),
    ((17,), 2, 4096, True, False, None, True, "bf16"),
    ((5,), 1, 8200, False, True, "before", True, "bf16"),      # a row past the registers
    ((6,), 2, 1031, False, False, "after", True, "f32"),
    ((21,), 3, 96, False, True, "before", False, "f32"),
    ((0,), 2, 64, False, False, "after", True, "bf16"),
]


@pytest.mark.parametrize("lead,G,D,shared,center,gate,bias,dtype", NORM)
def test_norm_forward_and_gradients(dev, lead, G, D, shared, center, gate, bias, dtype):
    from gated_deltanet_chunked_delta_amd import gated_group_norm
    print(f"[norm] lead={lead} G={G} D={D} shared={shared} center={center} gate={gate} {dtype}", flush=True)
    g, dt = gen(G * D), DT[dtype]
    x = (rn(g, *lead, G, D) + (0.7 if center else 0.0)).to(dt)
    z = rn(g, *lead, G, D, dt=dt) if gate else None
    ws = (D,) if shared else (G, D)
    w, b = (1 + rn(g, *ws, std=0.2)).to(dt), rn(g, *ws, std=0.2, dt=dt) if bias else None
    dy = rn(g, *lead, G, D, dt=dt)
    leaves = [t.requires_grad_(True) for t in (x, w, z, b) if t is not None]
    y = gated_group_norm(x, w, z=z, bias=b, eps=1e-5, center=center, gate_first=gate == "before")
    grads = torch.autograd.grad(y, leaves, dy)
    torch.cuda.synchronize()
    r = [d64(t).requires_grad_(True) if t is not None else None for t in (x, w, z, b)]
    ry = ref_norm(*r[:3], r[3], 1e-5, center, gate == "before")
    rg = torch.autograd.grad(ry, [t for t in r if t is not None], d64(dy))
    rows = max(1, int(np.prod(lead)) * (G if shared else 1))
    # sums of D (statistics) and of the rows (weights) in fp32
    tol = U[dt] + (16 + 2 * math.sqrt(D)) * U[torch.float32]
    close("y", y, ry, tol)
    for name, got, want in zip([k for k, t in zip("xwzb", (x, w, z, b)) if t is not None], grads, rg):
        if D == 1 and name == "x":
            continue  # a single channel: the exact gradient is eps-sized, a difference of equal numbers
        close("d" + name, got, want, 2 * tol + 2 * math.sqrt(rows) * U[torch.float32])


def test_norm_strided_gate(dev):
    from gated_deltanet_chunked_delta_amd import layers
    g = gen(3)
    wide = rn(g, 30, 4 * 64 + 12, dt=torch.bfloat16)
    x, w = rn(g, 30, 4, 64, dt=torch.bfloat16), rn(g, 64, dt=torch.bfloat16)
    for off in (8, 5):
        z = wide[:, off:off + 256].view(30, 4, 64)
        assert torch.equal(layers.gdn_norm_fwd(x, w, z), layers.gdn_norm_fwd(x, w, z.contiguous()))
        assert torch.equal(layers.gdn_norm_fwd(z, w, x), layers.gdn_norm_fwd(z.contiguous(), w, x))


# ------------------------------------------------------------------ together
def layer_weights(g, dev, dim, H, Dk, Dv, dt):
    W = 4
    return dict(proj=rn(g, dim, 2 * H * Dk + 2 * H * Dv + 2 * H, std=dim ** -0.5, dt=dt),
                conv=rn(g, 2 * H * Dk + H * Dv, W, std=0.5, dt=dt), norm=(1 + rn(g, Dv, std=0.1)).to(dt),
                out=rn(g, H * Dv, dim, std=(H * Dv) ** -0.5, dt=dt), A=-torch.rand(H, generator=g).to(dev) * 4 - 1,
                bias=rn(g, H) - 3, D=rn(g, H))


def run_layer(p, u, H, Dk, Dv, kind, state=None, cu=None, cu_host=None):
    """projection -> short convolution -> recurrence -> gated norm -> projection."""
    from gated_deltanet_chunked_delta_amd import chunk_gated_delta_rule, gated_group_norm, selective_scan, short_conv
    B, T, _ = u.shape
    r = u @ p["proj"]
    n1 = 2 * H * Dk + H * Dv
    conv_in, z = r[..., :n1], r[..., n1:n1 + H * Dv].view(B, T, H, Dv)
    c = short_conv(conv_in, p["conv"], silu=True, cu_seqlens=cu, cu_seqlens_host=cu_host)
    q, k, v = c[..., :H * Dk].view(B, T, H, Dk), c[..., H * Dk:2 * H * Dk].view(B, T, H, Dk), c[..., 2 * H * Dk:].view(B, T, H, Dv)
    if kind == "delta":
        o = chunk_gated_delta_rule(q.contiguous(), k.contiguous(), v.contiguous(), r[..., -2 * H:-H].float().contiguous(),
                                   r[..., -H:].contiguous(), cu_seqlens=cu, cu_seqlens_host=cu_host, qk_norm=True, gate_act=True)
    else:
        o = selective_scan(v, r[..., -H:], p["A"], k, q, D=p["D"], dt_bias=p["bias"], dt_softplus=True, cu_seqlens=cu,
                           cu_seqlens_host=cu_host)
    return gated_group_norm(o, p["norm"], z=z).reshape(B, T, H * Dv) @ p["out"]


def plain_layer(p, u, H, Dk, Dv, kind, bounds):
    """run_layer's formulas in 64 bits."""
    B, T, _ = u.shape
    r = u @ p["proj"]
    n1 = 2 * H * Dk + H * Dv
    c, _ = ref_conv(r[..., :n1], p["conv"], None, None, bounds, True)
    q, k, v = c[..., :H * Dk].reshape(B, T, H, Dk), c[..., H * Dk:2 * H * Dk].reshape(B, T, H, Dk), c[..., 2 * H * Dk:].reshape(B, T, H, Dv)
    if kind == "delta":
        unit = lambda a: a / torch.sqrt((a * a).sum(-1, keepdim=True) + 1e-6)
        q, k = unit(q), unit(k)
        gate, beta = -F.softplus(r[..., -2 * H:-H]), torch.sigmoid(r[..., -H:])
        rows = []
        for row, lo, hi in bounds:
            S = u.new_zeros(H, Dk, Dv)
            for t in range(lo, hi):
                S = torch.exp(gate[row, t])[:, None, None] * S
                e = v[row, t] - (S * k[row, t][:, :, None]).sum(1)
                S = S + beta[row, t][:, None, None] * k[row, t][:, :, None] * e[:, None, :]
                rows.append((row, t, Dk ** -0.5 * (S * q[row, t][:, :, None]).sum(1)))
        o = torch.stack([x for _, _, x in rows]).view(len(rows), H, Dv)
        o = u.new_zeros(B, T, H, Dv).index_put((torch.tensor([a for a, _, _ in rows]), torch.tensor([b for _, b, _ in rows])), o)
    else:
        o, _ = ref_scan(v, r[..., -H:], p["A"], k, q, p["D"], p["bias"], True, None, bounds)
    z = r[..., n1:n1 + H * Dv].reshape(B, T, H, Dv)
    return ref_norm(o, p["norm"], z, None, 1e-5, False, False).reshape(B, T, H * Dv) @ p["out"]


@pytest.mark.parametrize("kind", ["delta", "scan"])
@pytest.mark.parametrize("lens", [None, [70, 1, 59]])
def test_layer_in_one_run(dev, kind, lens):
    """The operators one after the other as a layer uses them, with gradients through all of
    them.  Six bf16 stages follow each other, each with a rounding of u relative to
    its values and sums of them: 16 u of the largest entry (32 u for gradients, which pass all stages twice)."""
    g, dim, H, Dk, Dv = gen(77), 96, 2, 64, 64
    B, T = (2, 65) if lens is None else (1, sum(lens))
    p = layer_weights(g, dev, dim, H, Dk, Dv, torch.bfloat16)
    u = rn(g, B, T, dim, dt=torch.bfloat16)
    names = [k for k in p if kind == "scan" or k not in ("A", "bias", "D")]
    for k in names:
        p[k].requires_grad_(True)
    cu = cu_of(lens, dev)
    y = run_layer(p, u.requires_grad_(True), H, Dk, Dv, kind, cu=cu.get("cu_seqlens"), cu_host=cu.get("cu_seqlens_host"))
    dy = rn(g, B, T, dim, dt=torch.bfloat16)
    grads = torch.autograd.grad(y, [u] + [p[k] for k in names], dy)
    torch.cuda.synchronize()
    r = {k: d64(v).requires_grad_(True) for k, v in p.items()}
    ru = d64(u).requires_grad_(True)
    ry = plain_layer(r, ru, H, Dk, Dv, kind, bounds_of(B, T, lens))
    rg = torch.autograd.grad(ry, [ru] + [r[k] for k in names], d64(dy))
    u8 = U[torch.bfloat16]
    close("y", y, ry, 16 * u8)
    for k, got, want in zip(["u"] + names, grads, rg):
        close("d" + k, got, want, 32 * u8)


# ------------------------------------------------------------------ streams, graphs, gradients by differences
def test_other_stream_and_captured_replays(dev):
    """The operators on a side stream, then a captured step (convolution, scan, norm, in place
    states) replayed with eager work between: every replay equals its eager twin."""
    from gated_deltanet_chunked_delta_amd import layers
    g = gen(21)
    N, H, Dk, Dv, W = 6, 4, 64, 64, 4
    D = H * Dv
    w, nw = rn(g, D, W, dt=torch.bfloat16), rn(g, Dv, dt=torch.bfloat16)
    A, bias = -torch.rand(H, generator=g).to(dev) - 1, rn(g, H)
    xs = [rn(g, N, D, dt=torch.bfloat16) for _ in range(4)]
    Bs, Cs = rn(g, N, 1, Dk, dt=torch.bfloat16), rn(g, N, 1, Dk, dt=torch.bfloat16)
    dts, zs = rn(g, N, H, dt=torch.bfloat16), rn(g, N, H, Dv, dt=torch.bfloat16)
    px = rn(g, 1, 300, H, Dv, dt=torch.bfloat16)
    pB, pC, pdt = rn(g, 1, 300, 1, Dk, dt=torch.bfloat16), rn(g, 1, 300, 1, Dk, dt=torch.bfloat16), rn(g, 1, 300, H, dt=torch.bfloat16)

    def step(x, cs, ss):
        c = layers.gdn_conv_step(x, cs, w)
        y = layers.gdn_scan_step(c.view(N, H, Dv), dts, A, Bs, Cs, ss, dt_bias=bias, dt_softplus=True)
        p, _ = layers.gdn_scan_fwd(px, pdt, A, pB, pC, dt_bias=bias, dt_softplus=True, seg_mode=1)
        return layers.gdn_norm_fwd(y, nw, zs), p

    def states():
        return (torch.zeros(N, W - 1, D, dtype=torch.bfloat16, device=dev), torch.zeros(N, H, Dk, Dv, device=dev))

    cs, ss = states()
    want = [step(x, cs, ss) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cs2, ss2 = states()
        got = [step(x, cs2, ss2) for x in xs]
    side.synchronize()
    assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q)) and torch.equal(ss, ss2)
    cs3, ss3 = states()
    xin = xs[0].clone()
    with torch.cuda.stream(side):
        step(xin, *states())
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = step(xin, cs3, ss3)
    torch.cuda.synchronize()
    for x, (wy, wp) in zip(xs, want):
        xin.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], wy) and torch.equal(out[1], wp)
        step(x, *states())                                        # eager work between the replays
        torch.cuda.synchronize()
    assert torch.equal(ss3, ss) and torch.equal(cs3, cs)


def test_captured_training_step(dev):
    """Forward and backward of the three operators captured together and replayed."""
    from gated_deltanet_chunked_delta_amd import layers
    g = gen(22)
    H, Dk, Dv, T = 2, 64, 64, 130
    D = H * Dv
    x, w, nw = rn(g, 1, T, D, dt=torch.bfloat16), rn(g, D, 4, dt=torch.bfloat16), rn(g, Dv, dt=torch.bfloat16)
    A, bias = -torch.rand(H, generator=g).to(dev) - 1, rn(g, H)
    B, C = rn(g, 1, T, 1, Dk, dt=torch.bfloat16), rn(g, 1, T, 1, Dk, dt=torch.bfloat16)
    dt, dy = rn(g, 1, T, H, dt=torch.bfloat16), rn(g, 1, T, H, Dv, dt=torch.bfloat16)

    def train():
        c, _ = layers.gdn_conv_fwd(x, w)
        cv = c.view(1, T, H, Dv)
        y, _, st = layers.gdn_scan_fwd(cv, dt, A, B, C, dt_bias=bias, dt_softplus=True, save_states=True, seg_mode=1)
        o = layers.gdn_norm_fwd(y, nw)
        gy, gw, _, _ = layers.gdn_norm_bwd(y, nw, dy)
        gs = layers.gdn_scan_bwd(cv, dt, A, B, C, gy, dt_bias=bias, dt_softplus=True, states=st, seg_mode=1)
        gx, gcw, _, _ = layers.gdn_conv_bwd(x, w, gs[0].view(1, T, D))
        return [o, gw, gx, gcw] + [t for t in gs if t is not None]

    want = [t.clone() for t in train()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        train()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = train()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        train()
        torch.cuda.synchronize()


def test_gradients_by_differences(dev):
    """Central differences of the fp32 operators along random directions."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, selective_scan, short_conv
    g = gen(31)
    T, H, Dk, Dv = 40, 2, 64, 64
    leaves = dict(x=rn(g, 1, T, H * Dv, std=0.5), w=rn(g, H * Dv, 3, std=0.5), B=rn(g, 1, T, 1, Dk, std=0.3),
                  C=rn(g, 1, T, 1, Dk, std=0.3), dt=rn(g, 1, T, H) - 2, A=-torch.rand(H, generator=g).to(dev) - 1,
                  nw=1 + rn(g, Dv, std=0.1), z=rn(g, 1, T, H, Dv))
    m = rn(g, 1, T, H, Dv)

    def f(p):
        c = short_conv(p["x"], p["w"]).view(1, T, H, Dv)
        y = selective_scan(c, p["dt"], p["A"], p["B"], p["C"], dt_softplus=True)
        return (gated_group_norm(y, p["nw"], z=p["z"], eps=1e-2).double() * m.double()).sum()

    q = {k: v.clone().requires_grad_(True) for k, v in leaves.items()}
    grads = dict(zip(q, torch.autograd.grad(f(q), list(q.values()))))
    for k in leaves:
        v = rn(g, *leaves[k].shape)
        v = v / v.norm() * leaves[k].norm()
        h = 2.0 ** -7
        with torch.no_grad():
            hi = f({**leaves, k: leaves[k] + h * v}).item()
            lo = f({**leaves, k: leaves[k] - h * v}).item()
        fd, an = (hi - lo) / (2 * h), (grads[k].double() * v.double()).sum().item()
        # third-order term h^2 and fp32 noise of f (about 1e-6 |f| / h)
        scale = max(abs(an), abs(fd), grads[k].double().norm().item() * v.norm().item() * 0.05)
        print(f"    {k} {fd:.6f} {an:.6f}", flush=True)
        assert abs(fd - an) <= 5e-3 * scale, k


def test_ragged_packed_batch(dev):
    """One long sequence among many short ones, the empty ones included: the right values, and
    a workspace that goes as the tokens and not as sequences times the longest one."""
    import ctypes
    from gated_deltanet_chunked_delta_amd import layers, selective_scan
    g, H = gen(31), 2
    lens = [3, 0, 700] + [1, 70, 2] * 20
    T, n = sum(lens), len(lens)
    s = scan_inputs(g, (1, T), H, 1, 64, 64, torch.bfloat16, True, n, True, dev)
    order = ["x", "dt", "A", "B", "C", "D", "bias", "h0"]
    r = {k: d64(s[k]).requires_grad_(True) for k in order}
    dy = rn(g, 1, T, H, 64, dt=torch.bfloat16)
    ry, rh = ref_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], r["D"], r["bias"], True, r["h0"], bounds_of(1, T, lens))
    rg = ref_grads([ry], [d64(dy)], [r[k] for k in order])
    chunks = sum((n_ + 63) // 64 for n_ in lens)
    for seg in (0, -1, 2 ** 31 - 1):
        leaves = [s[k].detach().requires_grad_(True) for k in order]
        y, hT = selective_scan(*leaves[:7], dt_softplus=True, initial_state=leaves[7], output_final_state=True,
                               seg_mode=seg, **cu_of(lens, dev))
        grads = torch.autograd.grad(y, leaves, dy)
        close("y", y, ry, 8 * U[torch.bfloat16])
        close("hT", hT, rh, 2e-6)
        for k, got, want in zip(order, grads, rg):
            tol = {"h0": 2e-6, "A": 2e-5, "D": 4e-6, "bias": 2e-5}.get(k, 8 * U[torch.bfloat16])
            close("d" + k, got, want, tol)
        f = layers.ScanBwdArgs()
        f.a, keep = layers._scan_args(*(s[k] for k in ("x", "dt", "A", "B", "C", "D", "bias")), True, s["h0"],
                                      cu_of(lens, dev)["cu_seqlens"], cu_of(lens, dev)["cu_seqlens_host"], seg)
        size = layers.lib().gdn_scan_bwd_workspace_size(ctypes.byref(f))
        # a state a chunk, three a segment and sequence, and what goes with the tokens
        assert size < 4 * H * 64 * 64 * (chunks + 3 * (chunks + n)) + 64 * T * H * 64 + (1 << 16), (seg, size)
        del keep


def test_lengths_reused_between_forward_and_backward(dev):
    """A loader that writes the next batch's lengths into the same host buffer before the
    backward pass does not change it."""
    from gated_deltanet_chunked_delta_amd import selective_scan, short_conv
    g, lens = gen(32), [70, 130, 20]
    s = scan_inputs(g, (1, 220), 2, 1, 64, 64, torch.float32, False, 1, False, dev)
    w, x = rn(g, 96, 4), rn(g, 1, 220, 96)
    dy, dx = rn(g, 1, 220, 2, 64), rn(g, 1, 220, 96)
    leaves = [s[k].requires_grad_(True) for k in ("x", "dt", "A", "B", "C")]
    cl = [x.requires_grad_(True), w.requires_grad_(True)]
    got = []
    for reuse in (False, True):
        kw = cu_of(lens, dev)
        y, u = selective_scan(*leaves, **kw), short_conv(*cl, **kw)
        if reuse:
            kw["cu_seqlens_host"].copy_(torch.tensor([0, 5, 6, 7], dtype=torch.int32))
        got.append(torch.autograd.grad(y, leaves, dy) + torch.autograd.grad(u, cl, dx))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_states_of_another_forward_are_refused(dev):
    from gated_deltanet_chunked_delta_amd import GDNError, layers
    g = gen(33)
    s = scan_inputs(g, (1, 300), 2, 1, 64, 64, torch.bfloat16, False, 1, False, dev)
    a, dy = [s[k] for k in ("x", "dt", "A", "B", "C")], rn(g, 1, 300, 2, 64, dt=torch.bfloat16)
    _, _, st = layers.gdn_scan_fwd(*a, seg_mode=1, save_states=True)
    layers.gdn_scan_bwd(*a, dy, seg_mode=1, states=st)
    for seg in (2, -1):
        with pytest.raises(GDNError, match="states"):
            layers.gdn_scan_bwd(*a, dy, seg_mode=seg, states=st)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_sequence(dev, bad):
    """A NaN or infinity anywhere in one packed sequence reaches no other one, nor their
    states and gradients; what is summed over tokens becomes NaN."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, selective_scan, short_conv
    g, lens = gen(34), [65, 90, 40]
    lo, hi = lens[0], lens[0] + lens[1]
    kw = cu_of(lens, dev)
    out = []
    for where in (None, lo, hi - 1, lo + 70):
        g = gen(34)
        s = scan_inputs(g, (1, sum(lens)), 2, 1, 64, 64, torch.bfloat16, True, 3, True, dev)
        x, w = rn(g, 1, sum(lens), 96, dt=torch.bfloat16), rn(g, 96, 4, dt=torch.bfloat16)
        dy, dx = rn(g, *s["x"].shape, dt=torch.bfloat16), rn(g, *x.shape, dt=torch.bfloat16)
        if where is not None:
            for t in (s["x"], s["B"], s["C"], x):
                t[0, where] = bad
        leaves = [s[k].requires_grad_(True) for k in ("x", "dt", "B", "C", "h0")]
        y, hT = selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], dt_bias=s["bias"], dt_softplus=True,
                               initial_state=s["h0"], output_final_state=True, seg_mode=1, **kw)
        u, fin = short_conv(x.requires_grad_(True), w, output_final_state=True, **kw)
        v = gated_group_norm(s["x"], torch.ones(64, dtype=torch.bfloat16, device=dev))
        grads = torch.autograd.grad(y, leaves, dy) + torch.autograd.grad(u, x, dx)
        rows = [t[0] for t in (y, u, v, *grads[:4], grads[5])]
        out.append([torch.cat([t[:lo], t[hi:]]).detach() for t in rows] +
                   [t[[0, 2]].detach() for t in (hT, fin, grads[4])])
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


def test_norm_of_more_rows_than_one_grid_row(dev):
    """70 million short rows: more threads than one launch dimension takes."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm
    R = 70_000_000
    x = torch.randint(-3, 4, (R, 1, 3), device=dev, dtype=torch.int8).to(torch.bfloat16)
    w = torch.tensor([1.0, 2.0, -0.5], device=dev, dtype=torch.bfloat16)
    y = gated_group_norm(x, w, eps=1.0)
    for lo in range(0, R, 10_000_000):
        v = x[lo:lo + 10_000_000].double()
        want = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1.0) * w.double()
        e = (y[lo:lo + 10_000_000].double() - want).abs().max().item()
        assert e <= want.abs().max().item() * (U[torch.bfloat16] + 1e-6), (lo, e)


def test_gradients_of_one_output_only(dev):
    """Only the final states are used, or only y: the other output's gradient is zero."""
    from gated_deltanet_chunked_delta_amd import selective_scan, short_conv
    g = gen(35)
    s = scan_inputs(g, (1, 150), 2, 1, 64, 64, torch.float32, False, 1, True, dev)
    order = ["x", "dt", "A", "B", "C", "h0"]
    leaves = [s[k].requires_grad_(True) for k in order]
    x, w, init = (rn(g, 2, 9, 40).requires_grad_(True), rn(g, 40, 3).requires_grad_(True),
                  rn(g, 2, 2, 40).requires_grad_(True))
    dh, df = rn(g, 1, 2, 64, 64), rn(g, 2, 2, 40)
    _, hT = selective_scan(*leaves[:5], initial_state=leaves[5], output_final_state=True, seg_mode=1)
    got = torch.autograd.grad(hT, leaves, dh)
    _, fin = short_conv(x, w, initial_state=init, output_final_state=True)
    cgot = torch.autograd.grad(fin, [x, w, init], df)
    r = {k: d64(s[k]).requires_grad_(True) for k in order}
    _, rh = ref_scan(r["x"], r["dt"], r["A"], r["B"], r["C"], None, None, False, r["h0"], bounds_of(1, 150, None))
    rg = ref_grads([rh], [d64(dh)], [r[k] for k in order])
    for k, a, b in zip(order, got, rg):
        if b is None:  # (hT does not depend on C)
            assert not bool(a.any())
        else:
            close("d" + k, a, b, {"A": 2e-5, "dt": 1e-5}.get(k, 2e-6))
    # the final state copies the last inputs: nothing else has a gradient
    want = torch.zeros_like(x)
    want[:, -2:] = df
    assert torch.equal(cgot[0], want) and not bool(cgot[1].any()) and not bool(cgot[2].any())


def test_empty_calls(dev):
    """No tokens, no rows, no sequences: empty outputs, zero gradients of the weights."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, layers, selective_scan, short_conv
    bf = torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device=dev)
    x, w, b = z(0, 3, 64).requires_grad_(True), (z(3, 64) + 1).requires_grad_(True), z(3, 64).requires_grad_(True)
    y = gated_group_norm(x, w, z(0, 3, 64), b)
    assert y.shape == (0, 3, 64)
    dx, dw, db = torch.autograd.grad(y, [x, w, b], torch.zeros_like(y))
    assert dx.shape == x.shape and not bool(dw.any()) and not bool(db.any())
    x, w, init = z(2, 0, 48).requires_grad_(True), (z(48, 4) + 1).requires_grad_(True), (z(2, 3, 48) + 2).requires_grad_(True)
    y, fin = short_conv(x, w, initial_state=init, output_final_state=True)
    assert y.shape == (2, 0, 48) and torch.equal(fin, init)
    dx, dw, di = torch.autograd.grad(fin, [x, w, init], torch.full_like(fin, 3.0))
    assert dx.shape == x.shape and not bool(dw.any()) and bool((di == 3.0).all())
    h0 = torch.randn(2, 2, 64, 64, device=dev).requires_grad_(True)
    A = -torch.ones(2, device=dev).requires_grad_(True)
    y, hT = selective_scan(z(2, 0, 2, 64), z(2, 0, 2), A, z(2, 0, 1, 64), z(2, 0, 1, 64), initial_state=h0,
                           output_final_state=True)
    assert y.shape == (2, 0, 2, 64) and torch.equal(hT, h0)
    dA, dh0 = torch.autograd.grad(hT, [A, h0], torch.full_like(hT, 3.0))
    assert not bool(dA.any()) and bool((dh0 == 3.0).all())
    st = z(4, 3, 48)
    assert layers.gdn_conv_step(z(0, 48), st, z(48, 4)).shape == (0, 48) and not bool(st.any())
    hs = torch.ones(4, 2, 64, 64, device=dev)
    y = layers.gdn_scan_step(z(0, 2, 64), z(0, 2), A.detach(), z(0, 1, 64), z(0, 1, 64), hs)
    assert y.shape == (0, 2, 64) and bool((hs == 1).all())


def test_two_streams_at_once(dev):
    """The same operators on two streams side by side give what they give alone."""
    from gated_deltanet_chunked_delta_amd import selective_scan, short_conv
    g = gen(36)
    s = scan_inputs(g, (2, 700), 4, 1, 64, 64, torch.bfloat16, True, 2, True, dev)
    x, w = rn(g, 2, 700, 160, dt=torch.bfloat16), rn(g, 160, 4, dt=torch.bfloat16)
    dy = rn(g, 2, 700, 4, 64, dt=torch.bfloat16)

    def run():
        leaves = [s[k].detach().requires_grad_(True) for k in ("x", "dt", "A", "B", "C")]
        y = selective_scan(*leaves, dt_bias=s["bias"], dt_softplus=True, initial_state=s["h0"])
        return [y, short_conv(x, w)] + list(torch.autograd.grad(y, leaves, dy))

    want = run()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(run())
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_offsets_past_32_bits(dev):
    """A short sequence packed behind more than 2^31 elements, and slots that far into a cache,
    give bit for bit what they give alone."""
    from gated_deltanet_chunked_delta_amd import gated_group_norm, layers, selective_scan, short_conv
    bf, H, Dv, tail = torch.bfloat16, 64, 128, 150
    T = (1 << 31) // (H * Dv) + 1000
    x = torch.randn(1, T, H, Dv, device=dev, dtype=bf)
    dt = torch.rand(1, T, H, device=dev) * 0.1
    B, C = torch.randn(1, T, 1, 64, device=dev, dtype=bf), torch.randn(1, T, 1, 64, device=dev, dtype=bf)
    A = -torch.rand(H, device=dev)
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32)
    alone = [t[:, -tail:].contiguous() for t in (x, dt, B, C)]

    def scan(x, dt, B, C, **kw):
        leaves = [t.detach().requires_grad_(True) for t in (x, dt, B, C)]
        y, hT = selective_scan(leaves[0], leaves[1], A, leaves[2], leaves[3], seg_mode=-1, output_final_state=True, **kw)
        grads = torch.autograd.grad(y, leaves, y.detach())
        return [t[:, -tail:].detach().clone() for t in (y, *grads)] + [hT[-1:].detach().clone()]

    print("[offsets] scan", flush=True)
    got = scan(x, dt, B, C, cu_seqlens=cu.to(dev), cu_seqlens_host=cu)
    assert all(torch.equal(a, b) for a, b in zip(got, scan(*alone)))
    del got, dt, B, C
    x, xa = x.view(1, T, H * Dv), alone[0].view(1, tail, H * Dv)
    w = torch.randn(H * Dv, 4, device=dev, dtype=bf)

    def conv(x, **kw):
        leaf = x.detach().requires_grad_(True)
        u, fin = short_conv(leaf, w, output_final_state=True, **kw)
        (dx,) = torch.autograd.grad(u, leaf, u.detach())
        return [u[:, -tail:].detach().clone(), dx[:, -tail:].clone(), fin[-1:].detach().clone()]

    print("[offsets] convolution", flush=True)
    got = conv(x, cu_seqlens=cu.to(dev), cu_seqlens_host=cu)
    assert all(torch.equal(a, b) for a, b in zip(got, conv(xa)))

    def norm(x):
        leaf = x.detach().view(1, -1, H, Dv).requires_grad_(True)
        y = gated_group_norm(leaf, w[:Dv, 0].contiguous(), x.view(leaf.shape))
        (dx,) = torch.autograd.grad(y, leaf, y.detach())
        return [y[:, -tail:].detach().clone(), dx[:, -tail:].clone()]

    print("[offsets] norm", flush=True)
    assert all(torch.equal(a, b) for a, b in zip(norm(x), norm(xa)))
    del x, got
    print("[offsets] steps", flush=True)
    slots = (1 << 31) // (H * 64 * Dv) + 9
    state = torch.zeros(slots, H, 64, Dv, device=dev)
    xs, dts, Bs, Cs = (t[0, :3].contiguous() for t in alone)
    idx = torch.tensor([slots - 1, 5, slots - 3], dtype=torch.int32, device=dev)
    y = layers.gdn_scan_step(xs, dts, A, Bs, Cs, state, state_idx=idx)
    small = torch.zeros(3, H, 64, Dv, device=dev)
    assert torch.equal(y, layers.gdn_scan_step(xs, dts, A, Bs, Cs, small))
    assert torch.equal(state[idx.long()], small) and bool(small.any())
    del state
    slots = (1 << 31) // (3 * H * Dv) + 9
    state = torch.zeros(slots, 3, H * Dv, device=dev, dtype=bf)
    idx = torch.tensor([slots - 1, 5, slots - 3], dtype=torch.int32, device=dev)
    u = layers.gdn_conv_step(xs.view(3, H * Dv), state, w, state_idx=idx)
    small = torch.zeros(3, 3, H * Dv, device=dev, dtype=bf)
    assert torch.equal(u, layers.gdn_conv_step(xs.view(3, H * Dv), small, w))
    assert torch.equal(state[idx.long()], small) and bool(small.any())
