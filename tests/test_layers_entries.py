"""The layer operators' entries without a GPU: refusals that need no device, and
what the Python entries hand on."""
import ctypes

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


def scan(**kw):
    a = fill(layers.ScanArgs(), dtype=B.GDN_BF16, dt_dtype=B.GDN_F32, B=1, T=128, H=4, G=2, Dk=64, Dv=64, x=FAKE,
             dt=FAKE, b=FAKE, c=FAKE, x_stride=256, dt_stride=4, b_stride=128, c_stride=128, A=FAKE, num_seqs=1,
             workspace=FAKE, workspace_bytes=1 << 40)
    return fill(a, **kw)


def test_round_once_field(L):
    """The choice lies where the struct had padding: no other field has moved."""
    f = layers.ScanArgs
    assert f.round_once.offset == f.dt_softplus.offset + 4 and f.h0.offset == f.dt_softplus.offset + 8
    for v in (2, -1):
        a = fill(layers.ScanFwdArgs(), a=scan(round_once=v), y=FAKE)
        assert L.gdn_scan_fwd(ctypes.byref(a), None) == 1 and b"round_once" in L.gdn_last_error()
        assert L.gdn_scan_fwd_workspace_size(ctypes.byref(a)) == 0
