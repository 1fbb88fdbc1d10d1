"""Argument checks of the operators around the recurrence: refusals of the C ABI
before a device is touched (no GPU), and of the Python entries."""
import ctypes

import numpy as np
import pytest
import torch

from gated_deltanet_chunked_delta_amd import GDNError, layers
from gated_deltanet_chunked_delta_amd import binding as B

FAKE = 1 << 20  # a 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def L():
    return layers.lib()


def fill(st, **kw):
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def conv(**kw):
    a = fill(layers.ConvArgs(), dtype=B.GDN_BF16, B=2, T=10, D=64, W=4, x=FAKE, x_stride=64, w=FAKE, num_seqs=2, silu=1)
    return fill(a, **kw)


def scan(**kw):
    a = fill(layers.ScanArgs(), dtype=B.GDN_BF16, dt_dtype=B.GDN_F32, B=1, T=128, H=4, G=2, Dk=64, Dv=64, x=FAKE,
             dt=FAKE, b=FAKE, c=FAKE, x_stride=256, dt_stride=4, b_stride=128, c_stride=128, A=FAKE, num_seqs=1,
             workspace=FAKE, workspace_bytes=1 << 40)
    return fill(a, **kw)


def norm(**kw):
    a = fill(layers.NormArgs(), dtype=B.GDN_BF16, R=5, G=2, D=64, x=FAKE, x_stride=128, w=FAKE, eps=1e-5)
    return fill(a, **kw)


BAD_CONV = [dict(dtype=7), dict(B=0), dict(T=-1), dict(D=0), dict(W=1), dict(W=5), dict(silu=2), dict(x=None),
            dict(w=None), dict(x_stride=63), dict(num_seqs=1), dict(cu_seqlens=FAKE), dict(x=FAKE + 1),
            dict(T=2 ** 31 - 1, D=2 ** 20, x_stride=2 ** 20), dict(B=1, cu_seqlens=FAKE, num_seqs=0)]
BAD_SCAN = [dict(dtype=9), dict(dt_dtype=3), dict(H=0), dict(G=3), dict(Dk=96), dict(Dv=32), dict(Dv=320),
            dict(dt_softplus=2), dict(x=None), dict(dt=None), dict(A=None), dict(x=FAKE + 8), dict(b=FAKE + 2),
            dict(x_stride=255), dict(x_stride=260), dict(b_stride=64), dict(dt_stride=3), dict(x_stride=1 << 22),
            dict(num_seqs=2), dict(seg_mode=-2), dict(cu_seqlens=FAKE), dict(h0=FAKE + 1)]
BAD_NORM = [dict(dtype=4), dict(R=-1), dict(G=0), dict(D=0), dict(eps=0.0), dict(eps=float("nan")), dict(x=None),
            dict(w=None), dict(x_stride=127), dict(gate_first=1), dict(center=2), dict(z=FAKE, z_stride=5),
            dict(R=2 ** 40)]


@pytest.mark.parametrize("kw", BAD_CONV)
def test_conv_refusals(L, kw):
    f = fill(layers.ConvFwdArgs(), a=conv(**kw), y=FAKE)
    assert L.gdn_conv_fwd(ctypes.byref(f), None) in (1, 2) and L.gdn_last_error()
    b = fill(layers.ConvBwdArgs(), a=conv(**kw), dy=FAKE, dx=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    assert L.gdn_conv_bwd(ctypes.byref(b), None) in (1, 2)
    assert L.gdn_conv_bwd_workspace_size(ctypes.byref(b)) == 0


def test_conv_refuses_missing_buffers(L):
    assert L.gdn_conv_fwd(ctypes.byref(fill(layers.ConvFwdArgs(), a=conv())), None) == 1
    assert L.gdn_conv_fwd(None, None) == 1
    ok = dict(dy=FAKE, dx=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    for missing, status in (("dy", 1), ("dx", 1), ("dw", 1), ("workspace", 3)):
        b = fill(layers.ConvBwdArgs(), a=conv(), **{**ok, missing: None})
        assert L.gdn_conv_bwd(ctypes.byref(b), None) == status, missing
    b = fill(layers.ConvBwdArgs(), a=conv(), **{**ok, "workspace_bytes": 16})
    assert L.gdn_conv_bwd(ctypes.byref(b), None) == 3


@pytest.mark.parametrize("kw,status", [(dict(W=7), 2), (dict(N=-1), 1), (dict(x=None), 1), (dict(state=None), 1),
                                       (dict(num_slots=3), 1), (dict(x_stride=10), 1), (dict(y=FAKE + 1), 1),
                                       (dict(N=0, x=None, state=None, y=None), 0)])
def test_conv_step_refusals(L, kw, status):
    a = fill(layers.ConvStepArgs(), dtype=B.GDN_BF16, N=4, D=64, W=4, x=FAKE, x_stride=64, state=FAKE, num_slots=4, w=FAKE, y=FAKE)
    assert L.gdn_conv_step(ctypes.byref(fill(a, **kw)), None) == status


@pytest.mark.parametrize("kw", BAD_SCAN)
def test_scan_refusals(L, kw):
    f = fill(layers.ScanFwdArgs(), a=scan(**kw), y=FAKE)
    assert L.gdn_scan_fwd(ctypes.byref(f), None) in (1, 2) and L.gdn_last_error()
    assert L.gdn_scan_fwd_workspace_size(ctypes.byref(f)) == 0
    b = fill(layers.ScanBwdArgs(), a=scan(**kw), dy=FAKE, dx=FAKE, ddt=FAKE, db=FAKE, dc=FAKE, dA=FAKE)
    assert L.gdn_scan_bwd(ctypes.byref(b), None) in (1, 2)
    assert L.gdn_scan_bwd_workspace_size(ctypes.byref(b)) == 0


def test_scan_refuses_missing_buffers_and_bad_sequences(L):
    assert L.gdn_scan_fwd(ctypes.byref(fill(layers.ScanFwdArgs(), a=scan())), None) == 1
    assert L.gdn_scan_fwd(ctypes.byref(fill(layers.ScanFwdArgs(), a=scan(), y=FAKE + 4)), None) == 1
    assert L.gdn_scan_fwd(ctypes.byref(fill(layers.ScanFwdArgs(), a=scan(workspace=None), y=FAKE)), None) == 3
    assert L.gdn_scan_fwd(ctypes.byref(fill(layers.ScanFwdArgs(), a=scan(workspace_bytes=8), y=FAKE)), None) == 3
    ok = dict(dy=FAKE, dx=FAKE, ddt=FAKE, db=FAKE, dc=FAKE, dA=FAKE)
    for missing in ok:
        b = fill(layers.ScanBwdArgs(), a=scan(), **{**ok, missing: None})
        assert L.gdn_scan_bwd(ctypes.byref(b), None) == 1, missing
    for cu in ([0, 50, 20, 128], [1, 128], [0, 100]):
        host = np.array(cu, dtype=np.int32)
        a = scan(cu_seqlens=FAKE, cu_seqlens_host=host.ctypes.data, num_seqs=len(cu) - 1)
        assert L.gdn_scan_fwd(ctypes.byref(fill(layers.ScanFwdArgs(), a=a, y=FAKE)), None) == 1, cu


def test_scan_sizes(L):
    f = fill(layers.ScanFwdArgs(), a=scan(T=4096, seg_mode=4))
    own = L.gdn_scan_fwd_workspace_size(ctypes.byref(f))
    states = L.gdn_scan_states_bytes(ctypes.byref(f.a))
    assert states == 16 * 4 * 64 * 64 * 4                      # 64 chunks in 16 segments
    f.h_save = FAKE
    assert own - L.gdn_scan_fwd_workspace_size(ctypes.byref(f)) >= states
    assert L.gdn_scan_states_bytes(ctypes.byref(scan(seg_mode=-1))) == 0
    b = fill(layers.ScanBwdArgs(), a=scan(T=4096, seg_mode=4))
    assert L.gdn_scan_bwd_workspace_size(ctypes.byref(b)) > own


@pytest.mark.parametrize("kw,status", [(dict(Dk=32), 2), (dict(Dv=320), 2), (dict(G=3), 1), (dict(b=None), 1),
                                       (dict(state=FAKE + 4), 1), (dict(x_stride=100), 1), (dict(num_slots=2), 1),
                                       (dict(N=0, x=None, state=None), 0)])
def test_scan_step_refusals(L, kw, status):
    a = fill(layers.ScanStepArgs(), dtype=B.GDN_BF16, dt_dtype=B.GDN_BF16, N=3, H=4, G=2, Dk=64, Dv=64, x=FAKE, dt=FAKE,
             b=FAKE, c=FAKE, x_stride=256, dt_stride=4, b_stride=128, c_stride=128, A=FAKE, state=FAKE, num_slots=3, y=FAKE)
    assert L.gdn_scan_step(ctypes.byref(fill(a, **kw)), None) == status


@pytest.mark.parametrize("kw", BAD_NORM)
def test_norm_refusals(L, kw):
    f = fill(layers.NormFwdArgs(), a=norm(**kw), y=FAKE)
    assert L.gdn_norm_fwd(ctypes.byref(f), None) in (1, 2) and L.gdn_last_error()
    b = fill(layers.NormBwdArgs(), a=norm(**kw), dy=FAKE, dx=FAKE, dz=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    assert L.gdn_norm_bwd(ctypes.byref(b), None) in (1, 2)
    assert L.gdn_norm_bwd_workspace_size(ctypes.byref(b)) == 0


def test_norm_refuses_missing_buffers(L):
    assert L.gdn_norm_fwd(ctypes.byref(fill(layers.NormFwdArgs(), a=norm())), None) == 1
    assert L.gdn_norm_fwd(ctypes.byref(fill(layers.NormFwdArgs(), a=norm(R=0, x=None))), None) == 0
    ok = dict(dy=FAKE, dx=FAKE, dz=FAKE, dw=FAKE, dbias=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    for missing, status in (("dy", 1), ("dx", 1), ("dz", 1), ("dw", 1), ("dbias", 1), ("workspace", 3)):
        b = fill(layers.NormBwdArgs(), a=norm(z=FAKE, z_stride=128, bias=FAKE), **{**ok, missing: None})
        assert L.gdn_norm_bwd(ctypes.byref(b), None) == status, missing


# ------------------------------------------------------------------ Python entries
def bad(fn, *a, match, **kw):
    with pytest.raises(GDNError, match=match):
        fn(*a, **kw)


def test_python_refusals():
    x, w = torch.zeros(2, 8, 64), torch.zeros(64, 4)
    bad(layers.short_conv, x[0], w, match=r"\[B, T, D\]")
    bad(layers.short_conv, x, w[:32], match="weight must be")
    bad(layers.short_conv, x, w.double(), match="torch.float32")
    bad(layers.short_conv, x.half(), w.half(), match="unsupported dtype")
    bad(layers.short_conv, x, w, torch.zeros(63), match="bias must be")
    bad(layers.short_conv, x, w, initial_state=torch.zeros(2, 4, 64), match="initial_state must be")
    bad(layers.short_conv, x, w, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32), match="batch size 1")
    bad(layers.short_conv, x[:1], w, cu_seqlens=torch.tensor([0, 8]), match="int32")
    bad(layers.short_conv, x[:1], w, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32),
        cu_seqlens_host=torch.tensor([0, 7]), match="rise from 0 to 8")
    bad(layers.short_conv, x.transpose(1, 2), torch.zeros(8, 4), match="contiguous")
    bad(layers.short_conv, x[:, ::2], w, match="evenly apart|on a GPU")
    bad(layers.short_conv, x, w, match="on a GPU")
    bad(layers.gdn_conv_step, x[0], torch.zeros(8, 2, 64), w, match="state must be")
    s = torch.zeros(1, 8, 4, 64)
    g = torch.zeros(1, 8, 2, 64)
    dt, A = torch.zeros(1, 8, 4), torch.zeros(4)
    bad(layers.selective_scan, s[0], dt, A, g, g, match=r"\[B, T, H, Dv\]")
    bad(layers.selective_scan, s, dt[:, :7], A, g, g, match="dt must be")
    bad(layers.selective_scan, s, dt.double(), A, g, g, match="dt must be")
    bad(layers.selective_scan, s, dt, A.double(), g, g, match="A must be")
    bad(layers.selective_scan, s, dt, A, g, g[:, :, :1], match="C must be")
    bad(layers.selective_scan, s, dt, A, g, g, initial_state=torch.zeros(1, 4, 64, 32), match="initial_state")
    bad(layers.selective_scan, s, dt, A, g, g, match="on a GPU")
    bad(layers.gdn_scan_step, s[0], dt[0], A, g[0], g[0], torch.zeros(8, 4, 64, 65), match="state must be")
    n = torch.zeros(3, 2, 64)
    bad(layers.gated_group_norm, n, torch.zeros(32), match="weight must be")
    bad(layers.gated_group_norm, n, torch.zeros(64), z=n[:2], match="z must be")
    bad(layers.gated_group_norm, n, torch.zeros(64), gate_first=True, match="gate_first needs z")
    bad(layers.gated_group_norm, n, torch.zeros(64), match="on a GPU")


def test_token_strides():
    t = torch.zeros(3, 5, 40)
    r = lambda x, shape, inner: layers._rows("t", x, shape, inner, torch.float32, x.device)
    assert r(t, (3, 5, 40), 1) == 40
    assert r(t[:, :, 4:20], (3, 5, 16), 1) == 40
    assert r(t[:, :1], (3, 1, 40), 1) == 200                   # one token a row: the row's distance
    assert r(t[:1, :1], (1, 1, 40), 1) == 40
    assert r(t[:, :, 8:24].view(3, 5, 2, 8), (3, 5, 2, 8), 2) == 40
    with pytest.raises(GDNError, match="evenly apart"):
        r(t[:, :4], (3, 4, 40), 1)
    with pytest.raises(GDNError, match="contiguous"):
        r(t[..., ::2], (3, 5, 20), 1)
