"""Sizes that a block's operators take and refuse (C ABI, no GPU: nothing here reaches a launch)."""
import ctypes

import pytest
import torch

from gated_deltanet_chunked_delta_amd import GDNError, blocks, layers
from gated_deltanet_chunked_delta_amd import binding as B

FAKE = 1 << 20  # a 16-byte aligned fake device address; never dereferenced
ref = ctypes.byref


@pytest.fixture(scope="module")
def L():
    return blocks.lib()


def lin(**kw):
    a = blocks.LinearArgs()
    for k, v in dict(dict(dtype=B.GDN_BF16, out_dtype=B.GDN_BF16, M=100, N=64, K=32, x_stride=kw.get("K", 32), x=FAKE, w=FAKE), **kw).items():
        setattr(a, k, v)
    return a


def fwd(L, a):
    f = blocks.LinearFwdArgs(a, FAKE)
    return L.gdn_linear_fwd(ref(f), None), L.gdn_linear_fwd_workspace_size(ref(f))


Q = dict(dtype=2, x_scale=FAKE, w_scale=FAKE)


@pytest.mark.parametrize("kw", [dict(), Q, dict(Q, out_dtype=B.GDN_F32), dict(dtype=B.GDN_F32, out_dtype=B.GDN_F32)])
@pytest.mark.parametrize("M,N", [(131077, 131103), (131072, 152064), (1 << 24, 8192), ((1 << 31) - 1, 64), (1000, 100_000_000)])
@pytest.mark.parametrize("K", [8, 2048])
def test_large_products_are_taken(L, kw, M, N, K):
    """Below 2^39 elements a tensor: such a call comes as far as its missing workspace."""
    if max(M, N) * K >= 1 << 39:
        pytest.skip("too large an input")
    status, need = fwd(L, lin(M=M, N=N, K=K, **kw))
    assert status == 3 and need > 0, L.gdn_last_error()


@pytest.mark.parametrize("M,N,K", [(1 << 20, 1 << 19, 8), (60, (1 << 31) - 1024, 8), (1 << 31, 8, 8), (1 << 30, 4, 512), (4, 1 << 30, 512)])
def test_products_of_larger_tensors_are_refused(L, M, N, K):
    status, need = fwd(L, lin(M=M, N=N, K=K))
    assert status == 1 and need == 0 and b"too large" in L.gdn_last_error()


def test_large_gradients_are_taken(L):
    for kw in (dict(M=131077, N=131103, K=8), dict(M=131077, N=8, K=131104), dict(M=100, N=131103, K=131104)):
        b = blocks.LinearBwdArgs(lin(**kw), None, FAKE, FAKE, FAKE, FAKE)
        assert L.gdn_linear_bwd(ref(b), None) == 3 and L.gdn_linear_bwd_workspace_size(ref(b)) > 0, kw


@pytest.mark.parametrize("kw,taken", [
    (dict(M=1 << 22, N=48, K=32), "xb"), (dict(M=(1 << 22) - 8, N=48, K=32), "xwb"), (dict(M=40, N=1 << 22, K=32), "wb"),
    (dict(M=1 << 22, N=1 << 16, K=8), "xb"), (dict(M=1 << 21, N=48, K=32, dtype=B.GDN_F32, out_dtype=B.GDN_F32), "xb"),
    (dict(M=8, N=1 << 30, K=8), "wb"), (dict(M=(1 << 31) - 1, N=8, K=8), "xb")])
def test_each_gradient_is_refused_for_its_own_sums(L, kw, taken):
    """dx sums along N, dw along M, the bias's gradient has no product."""
    for name, field in zip("xwb", ("dx", "dw", "dbias")):
        b = blocks.LinearBwdArgs(lin(**kw), None, FAKE, **{field: FAKE})
        status = L.gdn_linear_bwd(ref(b), None)
        assert status == (3 if name in taken else 1) and (L.gdn_linear_bwd_workspace_size(ref(b)) > 0) == (name in taken), name


@pytest.mark.parametrize("M,N", [(0, 1 << 22), (3, 1 << 22), (1 << 22, 2)])
def test_training_calls_are_refused_by_their_forward_pass(monkeypatch, M, N):
    """Whatever the rows, none among them: not later, by the gradient."""
    monkeypatch.setattr(layers, "_on_gpu", lambda name, t: t.device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    x, w = torch.zeros(M, 1, dtype=torch.bfloat16), torch.zeros(N, 1, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(GDNError, match="too large"):
        blocks.linear(x, w)


def rec(B_, T, D, N=None, **kw):
    a = blocks.RecArgs()
    d = dict(dtype=B.GDN_BF16, g_dtype=B.GDN_BF16, B=B_, T=T, D=D, x=FAKE, x_stride=D, g=FAKE, g_stride=D, num_seqs=N or B_)
    for k, v in dict(d, **kw).items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("T,D", [((1 << 31) - 1025, 1), (600_000_007, 3), (1 << 20, 1 << 17), (1 << 10, 1 << 23)])
@pytest.mark.parametrize("dt", [B.GDN_BF16, B.GDN_F32])
def test_long_recurrences_are_taken(L, T, D, dt):
    """Below 2^31 - 1024 tokens and 2^40 entries: such a call comes as far as its missing workspace."""
    a = rec(1, T, D, dtype=dt, g_dtype=dt, cu_seqlens=FAKE)
    assert L.gdn_rec_fwd(ref(blocks.RecFwdArgs(a, FAKE, FAKE)), None) == 3, L.gdn_last_error()
    b = blocks.RecBwdArgs(a, None, FAKE, None, FAKE, FAKE)
    assert L.gdn_rec_bwd(ref(b), None) == 3 and L.gdn_rec_bwd_workspace_size(ref(b)) > 0


def test_longer_recurrences_are_refused(L):
    for a in (rec(1, (1 << 31) - 1024, 1), rec(1, 1 << 23, 1 << 17), rec(1, 8, 1 << 20, N=1 << 17, cu_seqlens=FAKE)):
        f = blocks.RecFwdArgs(a, FAKE, FAKE)
        assert L.gdn_rec_fwd(ref(f), None) == 1 and b"too large" in L.gdn_last_error() and L.gdn_rec_fwd_workspace_size(ref(f)) == 0
