"""The layer operators' entries without a GPU: refusals that need no device, and
what the Python entries hand on."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fw

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


def test_sizes_past_32_bits_are_refused():
    """A size of 2^32 + 5 is not taken for 5."""
    m = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="meta")
    n = 2 ** 32 + 5
    for f in (lambda: layers.short_conv(m(1, n, 1), m(1, 4)), lambda: layers.gdn_conv_fwd(m(1, 8, 1), m(1, n)),
              lambda: layers.gdn_conv_bwd(m(1, n, 1), m(1, 4), m(1, n, 1)),
              lambda: layers.gdn_conv_step(m(1, n), m(1, 3, n), m(n, 4)),
              lambda: layers.gdn_conv_step(m(5, 1), m(n, 3, 1), m(1, 4)),
              lambda: layers.selective_scan(m(1, n, 1, 64), m(1, n, 1), m(1, dt=torch.float32), m(1, n, 1, 64), m(1, n, 1, 64)),
              lambda: layers.gated_group_norm(m(3, 2, n), m(n)), lambda: layers.gated_group_norm(m(3, n, 1), m(1))):
        with pytest.raises(GDNError, match="too large"):
            f()


def test_launches_of_2_32_threads_are_refused(L):
    """Before anything is enqueued: many sequences' states, many channels' weight gradients."""
    conv = dict(dtype=B.GDN_BF16, B=1, T=1 << 21, D=1001, W=4, x=FAKE, x_stride=1001, w=FAKE, cu_seqlens=FAKE,
                num_seqs=1 << 21, silu=1)
    f = fill(layers.ConvFwdArgs(), a=fill(layers.ConvArgs(), **conv), y=FAKE, final_state=FAKE)
    assert L.gdn_conv_fwd(ctypes.byref(f), None) == 1 and b"too large" in L.gdn_last_error()
    grad = dict(dy=FAKE, dx=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 60)
    b = fill(layers.ConvBwdArgs(), a=fill(layers.ConvArgs(), **conv), dinit=FAKE, **grad)
    assert L.gdn_conv_bwd(ctypes.byref(b), None) == 1 and b"too large" in L.gdn_last_error()
    wide = dict(conv, T=2, D=1 << 27, x_stride=1 << 27, cu_seqlens=None, num_seqs=1)
    b = fill(layers.ConvBwdArgs(), a=fill(layers.ConvArgs(), **wide), **grad)
    assert L.gdn_conv_bwd(ctypes.byref(b), None) == 1 and b"too large" in L.gdn_last_error()
    n = fill(layers.NormArgs(), dtype=B.GDN_BF16, R=2, G=1, D=1 << 28, x=FAKE, x_stride=1 << 28, w=FAKE, eps=1e-5)
    b = fill(layers.NormBwdArgs(), a=n, dy=FAKE, dx=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 60)
    assert L.gdn_norm_bwd(ctypes.byref(b), None) == 1 and b"too large" in L.gdn_last_error()


# ------------------------------------------------------------------ derivatives
@pytest.fixture
def stub(monkeypatch):
    """The entries on CPU tensors, the library's calls replaced by a record of their names."""
    class Calls(list):
        args = None
    calls = Calls()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size") or name.endswith("_bytes"):
                return lambda args: 256

            def call(args, stream):
                calls.append(name)
                calls.args = args._obj
            return call
    monkeypatch.setattr(layers, "lib", Lib)
    monkeypatch.setattr(layers, "_on_gpu", lambda name, t: t.device)
    monkeypatch.setattr(layers, "_raw_stream", lambda index: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    return calls


def operators():
    """{name: (function of its first input, that input)}"""
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)
    A, w, nw, dt, k = -torch.ones(2), r(8, 4), r(8), r(1, 6, 2), r(1, 6, 1, 64)
    st, hs = torch.zeros(3, 3, 8), torch.zeros(3, 2, 64, 64)
    return dict(short_conv=(lambda x: layers.short_conv(x, w), r(1, 5, 8)),
                selective_scan=(lambda x: layers.selective_scan(x, dt, A, k, k), r(1, 6, 2, 64)),
                gated_group_norm=(lambda x: layers.gated_group_norm(x, nw), r(4, 2, 8)),
                gdn_conv_step=(lambda x: layers.gdn_conv_step(x, st, w), r(3, 8)),
                gdn_scan_step=(lambda x: layers.gdn_scan_step(x, dt[0, :3], A, k[0, :3], k[0, :3], hs), r(3, 2, 64)))


NAMES = ["short_conv", "selective_scan", "gated_group_norm", "gdn_conv_step", "gdn_scan_step"]


@pytest.mark.parametrize("name", NAMES)
def test_forward_mode_is_refused(stub, name):
    """No result without its tangent, in grad mode and outside it."""
    f, x = operators()[name]
    f(x)
    assert len(stub) == 1
    for grad in (True, False):
        with fw.dual_level(), torch.set_grad_enabled(grad), pytest.raises((NotImplementedError, GDNError)):
            f(fw.make_dual(x, torch.ones_like(x)))
    with fw.dual_level():                       # a level without a tangent changes nothing
        assert torch.is_tensor(f(x))


@pytest.mark.parametrize("name", ["gdn_conv_step", "gdn_scan_step"])
def test_steps_refuse_a_gradient(stub, name):
    """A step has no gradient; it does not return a detached result without saying so."""
    f, x = operators()[name]
    with pytest.raises(GDNError, match="no_grad"):
        f(x.requires_grad_(True))
    assert not stub
    with torch.no_grad():
        f(x)
    assert len(stub) == 1


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead", [1, 3, 8])
def test_gradients_that_start_anywhere(stub, dt, lead):
    """The gradient of y behind `lead` other entries of a concatenation is contiguous and starts
    off 16 bytes; the library gets an aligned one with its values."""
    x = torch.randn(1, 6, 2, 64).to(dt).requires_grad_(True)
    A, d, k = -torch.ones(2), torch.randn(1, 6, 2), torch.randn(1, 6, 1, 64).to(dt)
    seen = []

    class Watch(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y):
            return y.view_as(y)

        @staticmethod
        def backward(ctx, g):
            seen.append(g)
            return g

    y = Watch.apply(layers.selective_scan(x, d, A, k, k))
    both = torch.cat([torch.zeros(lead, dtype=dt), y.flatten()])
    both.backward(torch.arange(both.numel()).to(dt))
    g = seen[0]
    assert g.is_contiguous() and g.data_ptr() % 16 == lead * dt.itemsize % 16
    at = stub.args.dy
    assert stub[-1] == "gdn_scan_bwd" and at % 16 == 0 and (at == g.data_ptr()) == (lead * dt.itemsize % 16 == 0)
    assert torch.equal(layers._gradient(g), g)


def test_chunk_rule_gradients_that_start_anywhere(monkeypatch):
    """The same for the delta rule's own gradient."""
    import gated_deltanet_chunked_delta_amd as pkg
    seen = []

    def fwd(q, k, v, *a, **kw):
        return torch.zeros_like(v), torch.zeros(1), torch.zeros(1), torch.zeros(1)

    def bwd(q, k, v, g, beta, scale, do, **kw):
        seen.append(do)
        return tuple(torch.zeros_like(t) for t in (q, k, v, g, beta)) + (None,)
    monkeypatch.setattr(pkg, "gdn_chunk_fwd", fwd)
    monkeypatch.setattr(pkg, "gdn_chunk_bwd", bwd)
    q = torch.randn(1, 6, 2, 64).bfloat16().requires_grad_(True)
    o = pkg.chunk_gated_delta_rule(q, q, q, torch.zeros(1, 6, 2), torch.zeros(1, 6, 2).bfloat16())
    both = torch.cat([torch.zeros(3).bfloat16(), o.flatten()])
    w = torch.arange(both.numel()).bfloat16()
    both.backward(w)
    assert seen[0].data_ptr() % 16 == 0 and torch.equal(seen[0].flatten(), w[3:])


# ------------------------------------------------------------------ tracers
@pytest.mark.parametrize("name", NAMES)
def test_traces_hold_the_call_or_are_refused(stub, name):
    f, x = operators()[name]
    if name.startswith("gdn_"):
        with pytest.raises(GDNError, match="traced"):
            torch.jit.trace(f, (x,), check_trace=False)
    else:
        t = torch.jit.trace(f, (x,), check_trace=False)
        for n in (1, 2):
            del stub[:]
            t(x)
            assert len(stub) == 1               # the replay calls the library
    from torch._subclasses.fake_tensor import FakeTensorMode
    from torch.fx.experimental.proxy_tensor import make_fx
    del stub[:]
    with pytest.raises(GDNError, match="traced"):
        make_fx(f)(x)
    with pytest.raises((GDNError, RuntimeError)), FakeTensorMode(allow_non_fake_inputs=True) as m:
        f(m.from_tensor(x))
    assert not stub


def test_traces_of_direct_calls_are_refused(stub):
    x, w = torch.randn(1, 5, 8), torch.randn(8, 4)
    with pytest.raises(GDNError, match="traced"):
        torch.jit.trace(lambda a: layers.gdn_conv_fwd(a, w), (x,), check_trace=False)
    assert not stub


def test_modes_that_only_watch_are_no_tracers(stub):
    from torch.utils.flop_counter import FlopCounterMode
    f, x = operators()["short_conv"]
    with FlopCounterMode(display=False):
        f(x)
    assert stub == ["gdn_conv_fwd"]


@pytest.mark.parametrize("final", [False, True])
@pytest.mark.parametrize("grad", [False, True])
def test_compiled_functions_leave_their_graph_for_a_call(stub, final, grad):
    """torch.compile cannot follow what fills a C structure in; the library gets it whole:
    outputs of the right shapes, and the fields that are written after nesting."""
    f = {"short_conv": lambda x: layers.short_conv(x, torch.ones(8, 4), output_final_state=final),
         "selective_scan": lambda x: layers.selective_scan(
             x, torch.ones(1, 6, 2), -torch.ones(2), torch.ones(1, 6, 1, 64), torch.ones(1, 6, 1, 64),
             output_final_state=final, round_once=True)}
    for name, call in f.items():
        torch._dynamo.reset()
        for T in (6, 6, 9) if name == "short_conv" else (6, 6):
            x = torch.zeros(1, T, 8) if name == "short_conv" else torch.zeros(1, T, 2, 64)
            out = torch.compile(lambda x: call(x.requires_grad_(grad)), backend="eager")(x)
            y, state = out if final else (out, None)
            a = stub.args.a
            assert y.shape == x.shape and y.requires_grad == grad and stub.args.y
            assert (a.B, a.T, a.num_seqs) == (1, T, 1) and a.x == x.data_ptr()
            if name == "short_conv":
                assert not final or (state.shape == (1, 3, 8) and stub.args.final_state)
            else:
                assert a.workspace and a.workspace_bytes == 256 and a.round_once == 1
                assert not final or (state.shape == (1, 2, 64, 64) and stub.args.hT)
