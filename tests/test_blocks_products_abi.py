"""Sizes that the projections take and refuse (C ABI, no GPU: nothing here reaches a launch)."""
import ctypes

import pytest

from gated_deltanet_chunked_delta_amd import binding as B
from gated_deltanet_chunked_delta_amd import blocks

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
