"""Argument checks of a block's operators: refusals of the C ABI before a device is
touched (no GPU), and what the Python entries refuse or hand on."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fw

from gated_deltanet_chunked_delta_amd import GDNError, blocks, layers
from gated_deltanet_chunked_delta_amd import binding as B

FAKE = 1 << 20  # a 16-byte aligned fake device address; never dereferenced
BIG = 1 << 60


@pytest.fixture(scope="module")
def L():
    return blocks.lib()


def fill(st, **kw):
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def norm(**kw):
    a = fill(blocks.AddNormFwdArgs(), dtype=B.GDN_BF16, res_dtype=B.GDN_F32, R=5, D=64, eps=1e-5, x=FAKE, x_stride=64, r=FAKE,
             r_stride=64, w=FAKE, s=FAKE, y=FAKE)
    return fill(a, **kw)


def norm_bwd(**kw):
    a = fill(blocks.AddNormBwdArgs(), dtype=B.GDN_BF16, res_dtype=B.GDN_F32, R=5, D=64, eps=1e-5, s=FAKE, s_stride=64, w=FAKE,
             dy=FAKE, ds=FAKE, dx=FAKE, dr=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=BIG)
    return fill(a, **kw)


def quant(**kw):
    return fill(fill(blocks.QuantArgs(), dtype=B.GDN_BF16, R=5, D=64, x=FAKE, x_stride=64, q=FAKE, q_scale=FAKE), **kw)


def lin(**kw):
    a = fill(blocks.LinearArgs(), dtype=B.GDN_BF16, out_dtype=B.GDN_BF16, M=100, N=64, K=32, x=FAKE, x_stride=32, w=FAKE,
             workspace=FAKE, workspace_bytes=BIG)
    return fill(a, **kw)


def rec(**kw):
    a = fill(blocks.RecArgs(), dtype=B.GDN_BF16, g_dtype=B.GDN_BF16, B=2, T=100, D=64, x=FAKE, x_stride=64, g=FAKE, g_stride=64,
             i=FAKE, i_stride=64, scale=FAKE, num_seqs=2, workspace=FAKE, workspace_bytes=BIG)
    return fill(a, **kw)


ref = ctypes.byref


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 2), (dict(dtype=7), 2), (dict(res_dtype=7), 2), (dict(dtype=B.GDN_F32, res_dtype=B.GDN_BF16), 2),
    (dict(r=None), 2), (dict(R=-1), 1), (dict(D=0), 1), (dict(R=1 << 31), 1), (dict(D=1 << 24, x_stride=1 << 24), 1), (dict(eps=0.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(s=None), 1), (dict(y=None), 1),
    (dict(q=FAKE), 1), (dict(y=None, q=FAKE), 1), (dict(x_stride=63), 1), (dict(r_stride=63), 1), (dict(x=FAKE + 1), 1),
    (dict(s=FAKE + 2), 1), (dict(y=FAKE + 1), 1), (dict(R=0, x=None, y=None, s=None), 0)])
def test_norm_refusals(L, kw, status):
    assert L.gdn_addnorm_fwd(ref(norm(**kw)), None) == status
    assert status == 0 or L.gdn_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), 2), (dict(dtype=B.GDN_F32, res_dtype=B.GDN_BF16), 2), (dict(D=-3), 1), (dict(eps=-1.0), 1), (dict(s=None), 1),
    (dict(dy=None), 1), (dict(w=None), 1), (dict(dx=None, dr=None, dw=None), 1), (dict(s_stride=10), 1), (dict(dr=FAKE + 2), 1),
    (dict(workspace=None), 3), (dict(workspace_bytes=64), 3), (dict(workspace=FAKE + 8), 1)])
def test_norm_gradient_refusals(L, kw, status):
    a = norm_bwd(**kw)
    assert L.gdn_addnorm_bwd(ref(a), None) == status and L.gdn_last_error()
    if status == 2 or "D" in kw or "eps" in kw:
        assert L.gdn_addnorm_bwd_workspace_size(ref(a)) == 0


@pytest.mark.parametrize("kw,status", [(dict(dtype=2), 2), (dict(R=-2), 1), (dict(x=None), 1), (dict(q=None), 1), (dict(q_scale=None), 1),
                                       (dict(x_stride=1), 1), (dict(q_scale=FAKE + 2), 1), (dict(R=0, x=None), 0)])
def test_quant_refusals(L, kw, status):
    assert L.gdn_quant_rows(ref(quant(**kw)), None) == status


Q = dict(dtype=2, x_scale=FAKE, w_scale=FAKE)
BAD_LINEAR = [(dict(dtype=3), 2), (dict(out_dtype=B.GDN_F32), 2), (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(act=3), 2),
              (dict(act=-1), 2), (dict(x=None), 1), (dict(w=None), 1), (dict(x_stride=31), 1), (dict(x=FAKE + 1), 1), (dict(w=FAKE + 1), 1),
              (dict(K=1 << 22, x_stride=1 << 22), 1), (dict(M=1 << 31), 1), (dict(x_scale=FAKE), 1)]


@pytest.mark.parametrize("kw,status", BAD_LINEAR + [(dict(Q, x_scale=None), 1), (dict(Q, out_dtype=2), 2), (dict(r=FAKE, r_stride=63), 1),
                                                    (dict(bias=FAKE + 1), 1), (dict(workspace=None), 3), (dict(M=0, x=None), 0),
                                                    (dict(M=1 << 30, N=1 << 30, K=8, x_stride=8), 1)])
def test_linear_refusals(L, kw, status):
    f = fill(blocks.LinearFwdArgs(), a=lin(**kw), y=FAKE)
    assert L.gdn_linear_fwd(ref(f), None) == status
    if status in (1, 2):
        assert L.gdn_linear_fwd_workspace_size(ref(f)) == 0


@pytest.mark.parametrize("kw,status", BAD_LINEAR + [(Q, 2), (dict(M=1 << 22), 1), (dict(N=1 << 22), 1),
                                                    (dict(M=1 << 20, K=1 << 19, x_stride=1 << 19), 1), (dict(N=1 << 20, K=1 << 19, x_stride=1 << 19), 1)])
def test_linear_gradient_refusals(L, kw, status):
    b = fill(blocks.LinearBwdArgs(), a=lin(**kw), dy=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE)
    assert L.gdn_linear_bwd(ref(b), None) == status
    assert L.gdn_linear_bwd_workspace_size(ref(b)) == 0


def test_linear_missing_buffers(L):
    assert L.gdn_linear_fwd(ref(fill(blocks.LinearFwdArgs(), a=lin())), None) == 1
    ok = dict(dy=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE)
    for kw, act in ((dict(ok, dy=None), 0), (dict(dy=FAKE), 0), (ok, 1), (dict(ok, dw=FAKE + 1), 0)):
        assert L.gdn_linear_bwd(ref(fill(blocks.LinearBwdArgs(), a=lin(act=act), **kw)), None) == 1
    small = fill(blocks.LinearBwdArgs(), a=lin(workspace_bytes=1000), **ok)
    assert L.gdn_linear_bwd(ref(small), None) == 3
    need = L.gdn_linear_bwd_workspace_size(ref(small))
    assert need > L.gdn_linear_bwd_workspace_size(ref(fill(blocks.LinearBwdArgs(), a=lin(), dy=FAKE, dx=FAKE)))
    assert need >= 2 * (64 * 104 + 32 * 104 + 32 * 64)        # turned copies of dy, x and w


BAD_REC = [(dict(dtype=2), 2), (dict(dtype=B.GDN_F32), 2), (dict(g_dtype=4), 2), (dict(B=0), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(x=None), 1),
           (dict(g=None), 1), (dict(x_stride=63), 1), (dict(g_stride=2), 1), (dict(i_stride=63), 1), (dict(num_seqs=1), 1),
           (dict(cu_seqlens=FAKE), 1), (dict(B=1, cu_seqlens=FAKE, num_seqs=0), 1), (dict(B=1, num_seqs=3, cu_seqlens=FAKE + 2), 1),
           (dict(scale=FAKE + 2), 1), (dict(h0=FAKE + 1), 1), (dict(x=FAKE + 1), 1), (dict(B=1 << 15, num_seqs=1 << 15, T=1 << 16), 1),
           (dict(B=1, T=1 << 30, num_seqs=1, D=1 << 12, x_stride=1 << 12, g_stride=1 << 12, i_stride=1 << 12), 1)]


@pytest.mark.parametrize("kw,status", BAD_REC)
def test_recurrence_refusals(L, kw, status):
    f = fill(blocks.RecFwdArgs(), a=rec(**kw), y=FAKE)
    assert L.gdn_rec_fwd(ref(f), None) == status and L.gdn_rec_fwd_workspace_size(ref(f)) == 0
    assert L.gdn_rec_states_bytes(ref(f.a)) == 0
    b = fill(blocks.RecBwdArgs(), a=rec(**kw), dy=FAKE, dx=FAKE, dg=FAKE, di=FAKE, dscale=FAKE)
    assert L.gdn_rec_bwd(ref(b), None) == status and L.gdn_rec_bwd_workspace_size(ref(b)) == 0


def test_recurrence_missing_buffers_and_sizes(L):
    assert L.gdn_rec_fwd(ref(fill(blocks.RecFwdArgs(), a=rec())), None) == 1
    assert L.gdn_rec_fwd(ref(fill(blocks.RecFwdArgs(), a=rec(workspace_bytes=100), y=FAKE)), None) == 3
    ok = dict(dy=FAKE, dx=FAKE, dg=FAKE, di=FAKE, dscale=FAKE)
    for k in ok:
        assert L.gdn_rec_bwd(ref(fill(blocks.RecBwdArgs(), a=rec(), **{**ok, k: None})), None) == 1, k
    assert L.gdn_rec_bwd(ref(fill(blocks.RecBwdArgs(), a=rec(workspace_bytes=100), **ok)), None) == 3
    assert L.gdn_rec_states_bytes(ref(rec())) == 4 * 4 * 64          # 200 tokens: four states of 64 channels
    own = L.gdn_rec_bwd_workspace_size(ref(fill(blocks.RecBwdArgs(), a=rec(), **ok)))
    kept = L.gdn_rec_bwd_workspace_size(ref(fill(blocks.RecBwdArgs(), a=rec(), h_saved=FAKE, **ok)))
    assert own - kept == 4 * 4 * 64
    # more sequences' final states than one launch has threads
    many = rec(B=1, T=8, D=1 << 20, x_stride=1 << 20, g_stride=1 << 20, i_stride=1 << 20, cu_seqlens=FAKE, num_seqs=1 << 17)
    assert L.gdn_rec_fwd(ref(fill(blocks.RecFwdArgs(), a=many, y=FAKE, hT=FAKE)), None) == 1 and b"too large" in L.gdn_last_error()


@pytest.mark.parametrize("kw,status", [(dict(dtype=2), 2), (dict(g_dtype=9), 2), (dict(N=-1), 1), (dict(D=0), 1), (dict(x=None), 1),
                                       (dict(state=None), 1), (dict(y=None), 1), (dict(x_stride=3), 1), (dict(i=FAKE, i_stride=3), 1),
                                       (dict(num_slots=3), 1), (dict(state=FAKE + 2), 1), (dict(N=1 << 30), 1), (dict(N=0, x=None), 0)])
def test_recurrence_step_refusals(L, kw, status):
    a = fill(blocks.RecStepArgs(), dtype=B.GDN_BF16, g_dtype=B.GDN_BF16, N=4, D=64, x=FAKE, x_stride=64, g=FAKE, g_stride=64, state=FAKE,
             num_slots=4, y=FAKE)
    assert L.gdn_rec_step(ref(fill(a, **kw)), None) == status


def test_null_arguments(L):
    for name, _ in blocks._SIGNATURES:
        assert getattr(L, name)(None, None) == 1, name
    for name, _ in blocks._SIZES:
        assert getattr(L, name)(None) == 0, name


# ------------------------------------------------------------------ the Python entries
@pytest.fixture
def stub(monkeypatch):
    """The entries on CPU tensors, the library's calls replaced by a record of their names."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size") or name.endswith("_bytes"):
                return lambda args: 4 * 64

            def call(args, stream):
                calls.append(name)
            return call
    monkeypatch.setattr(blocks, "lib", Lib)
    monkeypatch.setattr(layers, "_on_gpu", lambda name, t: t.device)
    monkeypatch.setattr(layers, "_raw_stream", lambda index: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    return calls


def entries():
    """{name: (function of its first input, that input)}"""
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)
    w, W, gg, st = r(8), r(5, 8), r(2, 6, 8), torch.zeros(3, 8)
    return dict(add_rms_norm=(lambda x: blocks.add_rms_norm(x, w), r(4, 8)), add_rms_norm_8bit=(lambda x: blocks.add_rms_norm_8bit(x, w), r(4, 8)),
                quantize_rows=(lambda x: blocks.quantize_rows(x), r(4, 8)), linear=(lambda x: blocks.linear(x, W, None, "silu"), r(4, 8)),
                gated_recurrence=(lambda x: blocks.gated_recurrence(x, gg), r(2, 6, 8)),
                gdn_rec_step=(lambda x: blocks.gdn_rec_step(x, gg[0, :3].contiguous(), st), r(3, 8)))


DIFFERENTIABLE = ("add_rms_norm", "linear", "gated_recurrence")


@pytest.mark.parametrize("name", list(entries()))
def test_derivatives_are_taken_or_refused(stub, name):
    f, x = entries()[name]
    f(x)
    assert len(stub) == 1
    if name in DIFFERENTIABLE:
        y = f(x.clone().requires_grad_(True))
        assert (y[0] if isinstance(y, tuple) else y).requires_grad
    else:
        with pytest.raises(GDNError, match="no gradient"):
            f(x.clone().requires_grad_(True))
    n = len(stub)
    for grad in (True, False):
        with torch.set_grad_enabled(grad), fw.dual_level():
            with pytest.raises((RuntimeError, NotImplementedError)):   # (GDNError is a RuntimeError)
                f(fw.make_dual(x, torch.ones_like(x)))
    assert name in DIFFERENTIABLE or len(stub) == n


@pytest.mark.parametrize("name", list(entries()))
def test_tracers(stub, name):
    """One operation of a trace, or refused: never a trace without the kernels."""
    from torch.fx.experimental.proxy_tensor import make_fx
    f, x = entries()[name]
    with pytest.raises(GDNError, match="traced"):
        make_fx(f)(x)
    if name not in DIFFERENTIABLE:
        with pytest.raises(Exception, match="traced"):
            torch.jit.trace(f, (x,), check_trace=False)


@pytest.mark.parametrize("name", DIFFERENTIABLE)
def test_one_operation_of_a_jit_trace(stub, name):
    """A trace holds the operator as one operation, whose replay calls the library."""
    f, x = entries()[name]
    with torch.no_grad():
        t = torch.jit.trace(f, (x,), check_trace=False)
        n = len(stub)
        assert n >= 1
        t(x)
    assert len(stub) == n + 1


@pytest.mark.parametrize("name", list(entries()))
def test_compiled_functions_leave_their_graph(stub, name):
    f, x = entries()[name]
    torch._dynamo.reset()
    g = torch.compile(lambda t: f(t * 1.0), backend="eager")
    with torch.no_grad():
        g(x)
        g(x)
    assert len(stub) == 2


def test_sizes_past_32_bits_are_refused():
    m = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="meta")
    n = 2 ** 32 + 5
    for f in (lambda: blocks.add_rms_norm(m(3, n), m(n)), lambda: blocks.add_rms_norm(m(n, 1), m(1)), lambda: blocks.quantize_rows(m(3, n)),
              lambda: blocks.linear(m(3, n), m(4, n)), lambda: blocks.linear(m(3, 4), m(n, 4)), lambda: blocks.linear(m(n, 4), m(3, 4)),
              lambda: blocks.gated_recurrence(m(1, n, 1), m(1, n, 1)), lambda: blocks.gdn_rec_step(m(n, 1), m(n, 1), m(3, 1, dt=torch.float32))):
        with pytest.raises(GDNError, match="too large"):
            f()


def test_python_checks(stub):
    r = torch.randn
    f8 = lambda *s: torch.zeros(*s).to(torch.float8_e4m3fn)
    one = torch.ones
    bad = [(lambda: blocks.add_rms_norm(r(8), r(8)), "x must be"), (lambda: blocks.add_rms_norm(r(2, 8), r(7)), "weight"),
           (lambda: blocks.add_rms_norm(r(2, 8), r(8), r(2, 7)), "residual"), (lambda: blocks.add_rms_norm(r(2, 8), r(8), r(2, 8).bfloat16()), "residual"),
           (lambda: blocks.add_rms_norm(r(2, 8).half(), r(8).half()), "dtype"), (lambda: blocks.linear(r(2, 8), r(5, 7)), "weight"),
           (lambda: blocks.linear(r(2, 8), r(5, 8), None, "relu"), "activation"), (lambda: blocks.linear(r(2, 8), r(5, 8), r(4)), "bias"),
           (lambda: blocks.linear(r(2, 8), r(5, 8), None, None, r(2, 4)), "residual"), (lambda: blocks.linear(f8(2, 8), f8(5, 8)), "dtype"),
           (lambda: blocks.linear_8bit(r(2, 8), one(2), f8(5, 8), one(5)), "float8"), (lambda: blocks.linear_8bit(f8(2, 8), one(3), f8(5, 8), one(5)), "x_scale"),
           (lambda: blocks.linear_8bit(f8(2, 8), one(2), f8(5, 8), one(4)), "weight_scale"),
           (lambda: blocks.linear_8bit(f8(2, 8), one(2), f8(5, 8), one(5), one(5)), "bias"),
           (lambda: blocks.gdn_linear_bwd(r(2, 8), r(5, 8), r(2, 5), "silu"), "v is missing"),
           (lambda: blocks.gated_recurrence(r(2, 8), r(2, 8)), "x must be"), (lambda: blocks.gated_recurrence(r(1, 2, 8), r(1, 2, 7)), "g must be"),
           (lambda: blocks.gated_recurrence(r(1, 2, 8).bfloat16(), r(1, 2, 8).half()), "g must be"),
           (lambda: blocks.gated_recurrence(r(1, 2, 8), r(1, 2, 8), scale=r(7)), "scale"),
           (lambda: blocks.gated_recurrence(r(1, 2, 8), r(1, 2, 8), initial_state=r(2, 8)), "initial_state"),
           (lambda: blocks.gated_recurrence(r(1, 5, 8), r(1, 5, 8), cu_seqlens=torch.tensor([0, 3], dtype=torch.int32),
                                            cu_seqlens_host=torch.tensor([0, 3])), "rise from 0 to 5"),
           (lambda: blocks.gdn_rec_bwd(r(1, 5, 8), r(1, 5, 8), r(1, 5, 8), states=r(3)), "states are not"),
           (lambda: blocks.gdn_rec_step(r(2, 8), r(2, 8), r(3, 7)), "state must be")]
    for f, text in bad:
        with pytest.raises(GDNError, match=text):
            f()
    assert not stub


@pytest.mark.parametrize("M,N,K,dt", [(1 << 22, 3, 1, torch.bfloat16), (1 << 21, 2, 1, torch.float32)])
@pytest.mark.parametrize("activation", (None, "silu"))
def test_training_calls_whose_gradient_would_be_refused_are_refused_at_once(stub, monkeypatch, M, N, K, dt, activation):
    """Rows along which the weight's gradient sums are below 2^23 bytes: a call that asks for one
    is refused by its forward pass, not later; one without a gradient runs, as do fewer rows."""
    L, recorded = B.lib(), blocks.lib()

    class Sizes:   # the library's sizes, launches recorded
        def __getattr__(self, name):
            if not name.endswith("_size"):
                return getattr(recorded, name)
            fn = getattr(L, name)
            fn.argtypes, fn.restype = [ctypes.POINTER(dict(blocks._SIZES)[name])], ctypes.c_size_t
            return fn
    monkeypatch.setattr(blocks, "lib", Sizes)
    x, w = torch.zeros(M, K, dtype=dt), torch.zeros(N, K, dtype=dt)
    for leaf in ("x", "w"):
        with pytest.raises(GDNError, match="too large"):
            blocks.linear(x.clone().requires_grad_(leaf == "x"), w.clone().requires_grad_(leaf == "w"), None, activation)
    assert stub == []
    blocks.linear(x, w, None, activation)
    blocks.linear(x[:M - 8].clone().requires_grad_(True), w, None, activation)
    assert stub == ["gdn_linear_fwd"] * 2
