"""Workloads of the operators of a block around its mixer: the residual norm
(also with an output in 8 bits), rows in 8 bits with scales, projections with
their epilogue, and the gated linear recurrence.

``run`` takes a prepared state through one pass: in plain torch operations where
``own`` is false, through this package's entry points where it is true.

Shapes follow the workloads of this repository (a width of 16 heads of 128,
projections to 3 x 16 x 128 channels, 8,192 to 65,536 tokens, 4 x 4,096 tokens in
training, a decode batch of 16 or 64, packed sequences of 1 to 16,384 tokens) and
smaller, odd and ragged ones.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_TOP = 448.0            # e4m3's largest value
_LEAST = 2.0 ** -100    # a row's largest magnitude counts as this at least


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the residual norm in front of a decode step's 8-bit projection: launch latency
        dict(name="norm8_step_64", op="norm8", dtype="bf16", R=64, D=2048, res="bf16"),
        # the same for a 32k prompt
        dict(name="norm8_prefill_32k", op="norm8", dtype="bf16", R=32768, D=2048, res="bf16"),
        # a training batch of an odd number of rows on an fp32 residual stream, forward and backward
        dict(name="norm_train_f32_stream", op="norm_train", dtype="bf16", R=12345, D=2304, res="f32"),
        # a projection's weight laid out in 8 bits once a model is loaded
        dict(name="quant_weight", op="quant", dtype="bf16", R=6144, D=2048),
        # odd rows of fp32
        dict(name="quant_odd_f32", op="quant", dtype="f32", R=1000, D=1001),
        # the q, k, v projection of a decode batch: the weight streams through
        dict(name="linear_step_16", op="linear", dtype="bf16", M=16, K=2048, N=6144, bias=True, act="silu", res=False),
        # the same projection of a 32k prompt in 8 bits
        dict(name="linear8_prefill_32k", op="linear8", dtype="bf16", M=32768, K=2048, N=6144, bias=True, act="",
             res=False),
        # an output projection added to the residual stream, 8,192 tokens, forward and backward
        dict(name="linear_train_out_8k", op="linear_train", dtype="bf16", M=8192, K=2048, N=2048, bias=False, act="",
             res=True),
        # a training step's input projection, 4 x 4,096 tokens, forward and backward
        dict(name="linear_train_4x4k", op="linear_train", dtype="bf16", M=16384, K=2048, N=6144, bias=True, act="silu",
             res=False),
        # one token each for a decode batch
        dict(name="rec_step_64", op="rec_step", dtype="bf16", N=64, slots=80, D=2048, scaled=True, inp=True, g32=False),
        # one long prompt, gates as logits
        dict(name="rec_prefill_64k", op="rec", dtype="bf16", B=1, T=65536, lens="", D=2048, scaled=True, inp=True,
             g32=False, init=True),
        # a packed training batch of ragged sequences, forward and backward
        dict(name="rec_train_packed", op="rec_train", dtype="bf16", B=1, T=0, lens="5121 777 3000 6384 513 1 0 588",
             D=2304, scaled=True, inp=True, g32=False, init=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _lens(rng, total):
    """Ragged sequence lengths, some of them tiny, adding up to `total` tokens."""
    out, left = [], total
    while left > 0 and len(out) < 11:
        n = min(left, _log_int(rng, 1, max(2, total)))
        out.append(n)
        left -= n
    return " ".join(map(str, out + ([left] if left else [])))


def draw(rng):
    op = rng.choice(["norm8", "norm_train", "quant", "linear", "linear8", "linear_train", "linear_train", "rec_step",
                     "rec", "rec_train", "rec_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm8", "norm_train", "quant"):
        D = rng.choice([1024, 2048, 4096, _log_int(rng, 33, 8192), _log_int(rng, 33, 8192)])
        R = _log_int(rng, 1, min(65536, (24 << 20) // D))
        c = dict(op=op, dtype=dtype, R=R, D=D)
        if op != "quant":
            c["res"] = rng.choice(["", dtype, dtype, "f32"])
        return c
    if op.startswith("linear"):
        K, N = (rng.choice([1024, 2048, 4096, _log_int(rng, 33, 6144)]) for _ in range(2))
        most = (1 << 37) // (1 if dtype == "bf16" or op == "linear8" else 8)   # multiply-adds
        M = _log_int(rng, 1, max(2, min(32768, most // (K * N))))
        if op == "linear" and rng.random() < .5:
            M = rng.randint(1, 64)
        return dict(op=op, dtype=dtype, M=M, K=K, N=N, bias=rng.random() < .5, act=rng.choice(["", "silu", "gelu"]),
                    res=rng.random() < .5)
    D = rng.choice([1024, 2048, 2304, _log_int(rng, 33, 6144)])
    gates = dict(D=D, scaled=rng.random() < .6, inp=rng.random() < .6, g32=rng.random() < .3)
    if op == "rec_step":
        n = _log_int(rng, 1, 256)
        return dict(op=op, dtype=dtype, N=n, slots=n + rng.randint(0, 9), **gates)
    total = _log_int(rng, 1, min(65536, (32 << 20) // D))
    packed = rng.random() < .5
    b = 1 if packed else rng.choice([1, 1, 2, 4])
    return dict(op=op, dtype=dtype, B=b, T=0 if packed else max(1, total // b), lens=_lens(rng, total) if packed else "",
                init=rng.random() < .5, **gates)


def _lengths(case):
    """Lengths of a packed batch's sequences; empty for sequences of one length."""
    return [int(n) for n in case.get("lens", "").split()]


def _tokens(case):
    return sum(_lengths(case)) or case["B"] * case["T"]


def _nseq(case):
    return len(_lengths(case)) or case["B"]


def work(case):
    es, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op in ("norm8", "norm_train", "quant"):
        n, r = case["R"] * case["D"], case["R"]
        if op == "quant":
            return dict(bytes=n * (es + 1) + 4 * r, flops=3 * n)
        rs = {"": 0, "bf16": 2, "f32": 4}[case["res"]]
        if op == "norm8":  # x, residual in; residual out, 8 bits, scales
            return dict(bytes=n * (es + 2 * rs + 1) + es * case["D"] + 4 * r, flops=8 * n)
        # forward x, residual -> sum, y; backward dy, the sum's gradient, the sum -> one or two gradients
        back = es + es + (3 * rs if rs else es)
        return dict(bytes=n * (2 * es + 2 * rs + back) + 3 * es * case["D"], flops=18 * n)
    if op.startswith("linear"):
        m, k, n = case["M"], case["K"], case["N"]
        mac = m * k * n
        if op == "linear8":
            return dict(bytes=m * k + n * k + 4 * (m + n) + es * (m * n * (1 + case["res"]) + n * case["bias"]),
                        flops=2 * mac)
        by = es * (m * k + n * k + n * case["bias"] + m * n * (1 + case["res"]))
        if op == "linear":
            return dict(bytes=by, flops=2 * mac)
        return dict(bytes=by + es * (m * n + m * k + n * k + n * case["bias"]), flops=6 * mac)
    gs = 4 if case["g32"] else es
    if op == "rec_step":
        n = case["N"] * case["D"]
        return dict(bytes=n * (es * (2 + case["inp"]) + gs + 8) + 4 * case["D"] * case["scaled"], flops=20 * n)
    n, st = _tokens(case) * case["D"], 4 * _nseq(case) * case["D"]
    by = n * (es * (2 + case["inp"]) + gs) + st * (1 + case["init"]) + 4 * case["D"] * case["scaled"]
    if op == "rec":
        return dict(bytes=by, flops=20 * n)
    by += n * (es * (2 + case["inp"]) + gs) + 2 * st * case["init"] + 4 * case["D"] * case["scaled"]
    return dict(bytes=by, flops=60 * n)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)
    dt, op = _DT[case["dtype"]], case["op"]

    def rn(*s, std=1.0):
        return torch.randn(*s, generator=gen, device=DEV) * std

    s = dict(case=case)
    if op in ("norm8", "norm_train", "quant"):
        R, D = case["R"], case["D"]
        # a few channels far larger than the rest, as in a residual stream
        wide = 1.0 + 9.0 * (torch.rand(D, generator=gen, device=DEV) < 0.01)
        s["x"] = (rn(R, D) * wide).to(dt)
        if op != "quant":
            s["w"] = (1.0 + rn(D, std=0.1)).to(dt)
            s["r"] = (rn(R, D) * wide * 2.0).to(_DT[case["res"]]) if case["res"] else None
            if op == "norm_train":
                s["dy"] = rn(R, D).to(dt)
                s["ds"] = rn(R, D).to(s["r"].dtype) if case["res"] else None
                leaves = ("x", "w", "r")
    elif op.startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        x, w = rn(M, K), rn(N, K, std=K ** -0.5)
        if op == "linear8":  # 8 bits with a scale for each token and each output channel
            s["xs"], s["ws"] = (t.abs().amax(1) / _TOP for t in (x, w))
            s["x"], s["w"] = (x / s["xs"][:, None]).to(_F8), (w / s["ws"][:, None]).to(_F8)
        else:
            s["x"], s["w"] = x.to(dt), w.to(dt)
        s["b"] = rn(N, std=0.3).to(dt) if case["bias"] else None
        s["r"] = rn(M, N).to(dt) if case["res"] else None
        if op == "linear_train":
            s["dy"] = rn(M, N).to(dt)
            leaves = ("x", "w", "b", "r")
    else:
        D, lens = case["D"], _lengths(case)
        if lens:
            host = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
            s["cu_host"], s["cu"] = host, host.to(DEV)
        lead = (case["N"],) if op == "rec_step" else (1, sum(lens)) if lens else (case["B"], case["T"])
        gdt = torch.float32 if case["g32"] else dt
        s["x"] = rn(*lead, D).to(dt)
        s["i"] = rn(*lead, D).to(dt) if case["inp"] else None
        if case["scaled"]:  # logits; a token that keeps its gate open decays by 0.9 to 0.995
            s["g"] = rn(*lead, D).to(gdt)
            s["l"] = -torch.log(0.9 + 0.095 * torch.rand(D, generator=gen, device=DEV))
        else:               # log decays, as the delta rule's
            s["g"] = (-0.1 * torch.log1p(torch.exp(rn(*lead, D)))).to(gdt)
            s["l"] = None
        if op == "rec_step":
            s["state"] = rn(case["slots"], D, std=2.0)
            s["idx"] = torch.randperm(case["slots"], generator=gen, device=DEV)[:case["N"]].to(torch.int32)
        else:
            s["h0"] = rn(_nseq(case), D, std=2.0) if case["init"] else None
            if op == "rec_train":
                s["dy"] = rn(*lead, D).to(dt)
                s["dh"] = rn(_nseq(case), D) if case["init"] else None
                leaves = ("x", "g", "i", "l", "h0")
    if op.endswith("train"):
        s["leaves"] = [s[k].requires_grad_(True) for k in leaves if s[k] is not None]
    return s


def run(state):
    if own:
        return _run_own(state)
    with torch.no_grad():
        return _run_plain(state)


def _values(q, scale, dt):
    """What 8-bit rows stand for."""
    return (q.float() * scale[:, None]).to(dt)


# ------------------------------------------------------------------ this package's calls
def _grads(s, outs, gouts):
    pairs = [(o, g) for o, g in zip(outs, gouts) if g is not None]
    return list(torch.autograd.grad([o for o, _ in pairs], s["leaves"], [g for _, g in pairs]))


def _run_own(s):
    import gated_deltanet_chunked_delta_amd as gdn
    case, op = s["case"], s["case"]["op"]
    act = case.get("act") or None
    if op == "norm8":
        q, scale, total = gdn.add_rms_norm_8bit(s["x"], s["w"], s["r"], eps=1e-6)
        return [_values(q, scale, torch.bfloat16), scale] + ([total] if case["res"] else [])
    if op == "quant":
        q, scale = gdn.quantize_rows(s["x"])
        return [_values(q, scale, torch.bfloat16), scale]
    if op == "norm_train":
        y, total = gdn.add_rms_norm(s["x"], s["w"], s["r"], eps=1e-6)
        outs, gouts = ([y, total], [s["dy"], s["ds"]]) if case["res"] else ([y], [s["dy"]])
        return [o.detach() for o in outs] + _grads(s, outs, gouts)
    if op == "linear8":
        return [gdn.linear_8bit(s["x"], s["xs"], s["w"], s["ws"], s["b"], act, s["r"], out_dtype=_DT[case["dtype"]])]
    if op == "linear":
        with torch.no_grad():
            return [gdn.linear(s["x"], s["w"], s["b"], act, s["r"])]
    if op == "linear_train":
        y = gdn.linear(s["x"], s["w"], s["b"], act, s["r"])
        return [y.detach()] + _grads(s, [y], [s["dy"]])
    if op == "rec_step":
        y = gdn.gdn_rec_step(s["x"], s["g"], s["state"], i=s["i"], scale=s["l"], state_idx=s["idx"])
        return [y, s["state"]]
    seqs = dict(cu_seqlens=s.get("cu"), cu_seqlens_host=s.get("cu_host"))
    with torch.set_grad_enabled(op == "rec_train"):
        y, hT = gdn.gated_recurrence(s["x"], s["g"], i=s["i"], scale=s["l"], initial_state=s["h0"],
                                     output_final_state=True, **seqs)
    if op == "rec":
        return [y, hT]
    return [y.detach(), hT.detach()] + _grads(s, [y, hT], [s["dy"], s["dh"]])


# ------------------------------------------------------------------ the plain forms (fp32)
def _run_plain(s):
    op = s["case"]["op"]
    if op in ("norm8", "quant"):
        return _plain_rows8(s, op == "norm8")
    if op == "norm_train":
        return _plain_norm(s)
    if op.startswith("linear"):
        return _plain_linear(s, op)
    if op == "rec_step":
        return _plain_rec_step(s)
    return _plain_rec(s, op == "rec_train")


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _plain_sum(s):
    """x plus the residual, as the stream holds it: the norm reads what it stores."""
    return s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["r"].dtype)


def _plain_rows8(s, norm):
    case = s["case"]
    v = s["x"].float()
    if norm:
        total = _plain_sum(s)
        v = total.float()
        v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * s["w"].float()
    top = torch.clamp(v.abs().amax(1), min=_LEAST)
    scale = top / _TOP
    # 448 v / top: a quotient halfway between two 8-bit values comes out exactly (v / scale would round it to a side)
    q = (0.875 * v / top[:, None] * 512.0).to(_F8)
    return [_values(q, scale, torch.bfloat16), scale] + ([total] if norm and case["res"] else [])


def _plain_norm(s):
    x, w, dy = s["x"], s["w"].float(), s["dy"].float()
    total = _plain_sum(s)
    v = total.float()
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    n = v * rstd
    dn = dy * w
    dv = (dn - n * (dn * n).mean(1, keepdim=True)) * rstd
    dw = (dy * n).sum(0, dtype=torch.float64)
    y = (n * w).to(x.dtype)
    if s["r"] is None:
        return [y, dv.to(x.dtype), dw.to(x.dtype)]
    dv = dv + s["ds"].float()
    return [y, total, dv.to(x.dtype), dw.to(x.dtype), dv.to(total.dtype)]


def _act(v, act):
    """act(v) and its derivative."""
    if act == "silu":
        sg = _sigmoid(v)
        return v * sg, sg * (1.0 + v * (1.0 - sg))
    if act == "gelu":  # v sigmoid(2 u), u = sqrt(2 / pi) (v + 0.044715 v^3)
        c = math.sqrt(8.0 / math.pi)
        sg = _sigmoid(c * (v + 0.044715 * v * v * v))
        return v * sg, sg + v * sg * (1.0 - sg) * c * (1.0 + 3.0 * 0.044715 * v * v)
    return v, None


def _plain_linear(s, op):
    case = s["case"]
    x, w = s["x"].float(), s["w"].float()
    if op == "linear8":
        x, w = x * s["xs"][:, None], w * s["ws"][:, None]
    v = torch.mm(x, w.t())
    if s["b"] is not None:
        v = v + s["b"].float()
    y, d = _act(v, case["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    dt = _DT[case["dtype"]]
    if op != "linear_train":
        return [y.to(dt)]
    dv = s["dy"].float() if d is None else s["dy"].float() * d
    out = [y.to(dt), torch.mm(dv, w).to(dt), torch.mm(dv.t(), x).to(dt)]
    if s["b"] is not None:
        out.append(dv.sum(0, dtype=torch.float64).to(dt))
    return out + ([s["dy"]] if s["r"] is not None else [])


def _gates(s):
    """Decay, factor of the input from the decay (None: 1), sigmoids of g and i."""
    g = s["g"].float()
    si = None if s["i"] is None else _sigmoid(s["i"].float())
    if s["l"] is None:
        return torch.exp(g), None, None, si
    sg = _sigmoid(g)
    lg = -s["l"] * sg
    return torch.exp(lg), torch.sqrt(-torch.expm1(2.0 * lg)), sg, si


def _inputs(s, m, si):
    u = s["x"].float()
    u = u if m is None else u * m
    return u if si is None else u * si


def _plain_rec_step(s):
    a, m, _, si = _gates(s)
    idx = s["idx"].long()
    h = a * s["state"][idx] + _inputs(s, m, si)
    s["state"][idx] = h
    return [h.to(s["x"].dtype), s["state"]]


def _firsts(s):
    """(sequences that have tokens, the flat index of each one's first and last token)."""
    case = s["case"]
    lens = _lengths(case) or [case["T"]] * case["B"]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    live = [n for n in range(len(lens)) if lens[n]]
    ix = lambda v: torch.tensor(v, device=DEV, dtype=torch.long)  # noqa: E731
    return ix(live), ix([starts[n] for n in live]), ix([starts[n + 1] - 1 for n in live]), max(lens, default=0)


def _doubling(a, u, longest):
    """h_t = a_t h_{t-1} + u_t over [tokens, D] by doubling; a is 0 where a sequence starts."""
    a, u, k = a.clone(), u.clone(), 1
    while k < longest:
        u[k:] = u[k:] + a[k:] * u[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return u


def _plain_rec(s, train):
    case, x, D = s["case"], s["x"], s["case"]["D"]
    live, first, last, longest = _firsts(s)
    a, m, sg, si = _gates(s)
    u = _inputs(s, m, si).reshape(-1, D)
    a = a.reshape(-1, D)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(_nseq(case), D, device=DEV)
    cut, start = a.clone(), u.clone()
    cut[first] = 0.0
    start[first] = start[first] + a[first] * h0[live]
    h = _doubling(cut, start, longest)
    hT = h0.clone()
    hT[live] = h[last]
    y = h.to(x.dtype).reshape(x.shape)
    if not train:
        return [y, hT]
    # dh_t = dy_t + a_{t+1} dh_{t+1}, the scan turned round in time
    dh = s["dy"].float().reshape(-1, D).clone()
    dlast = s["dh"] if s["dh"] is not None else torch.zeros_like(h0)
    dh[last] = dh[last] + dlast[live]
    nxt = torch.zeros_like(a)
    nxt[:-1] = cut[1:]
    dh = _doubling(nxt.flip(0), dh.flip(0), longest).flip(0)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[first] = h0[live]
    xf = x.float().reshape(-1, D)
    one = torch.ones_like(xf)
    si = one if si is None else si.reshape(-1, D)
    mm = one if m is None else m.reshape(-1, D)
    out = [y, hT, (dh * mm * si).to(x.dtype).reshape(x.shape)]
    dlog = a * dh * prev                                   # gradient of the log decay
    if m is None:
        out.append(dlog.to(s["g"].dtype).reshape(x.shape))
    else:
        sg = sg.reshape(-1, D)
        dlog = dlog - torch.where(mm > 0, dh * si * xf * a * a / mm, torch.zeros_like(mm))
        out.append((-dlog * s["l"] * sg * (1.0 - sg)).to(s["g"].dtype).reshape(x.shape))
    if s["i"] is not None:
        out.append((dh * mm * xf * si * (1.0 - si)).to(x.dtype).reshape(x.shape))
    if m is not None:
        out.append((-dlog * sg).sum(0, dtype=torch.float64).float())
    if s["h0"] is not None:
        dh0 = dlast.clone()
        dh0[live] = a[first] * dh[first]
        out.append(dh0)
    return out


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        op = case["op"]
        if op in ("norm8", "norm_train", "quant"):
            return _exact_rows(s, op)
        if op.startswith("linear"):
            return _exact_linear(s, op)
        if op == "rec_step":
            return _exact_rec_step(s)
        return _exact_rec(s, op == "rec_train")


def _nearest8(v):
    """v rounded to e4m3: four significant bits, steps of 2^-9 at least, ties to even."""
    e = torch.clamp(torch.frexp(v).exponent - 1, min=-6)
    step = torch.ldexp(torch.ones_like(v), (e - 3).to(torch.int32))
    return torch.clamp(torch.round(v / step) * step, -_TOP, _TOP)


def _exact_rows(s, op):
    v = s["x"].double()
    total = None
    if op != "quant":
        if s["r"] is not None:
            total = (v + s["r"].double()).to(s["r"].dtype)
            v = total.double()
        rms = torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + 1e-6)
        n = v / rms
        v = n * s["w"].double()
    if op == "norm_train":
        dn = s["dy"].double() * s["w"].double()
        dv = (dn - n * (dn * n).sum(1, keepdim=True) / n.shape[1]) / rms
        dw = torch.einsum("rd,rd->d", s["dy"].double(), n)
        if total is None:
            return [v, dv, dw]
        dv = dv + s["ds"].double()
        return [v, total, dv, dw, dv]
    top = torch.clamp(v.abs().amax(1), min=_LEAST)
    scale = top / _TOP
    out = [_nearest8(v * _TOP / top[:, None]) * scale[:, None], scale]
    return out if total is None else out + [total]


def _exact_linear(s, op):
    act = s["case"]["act"]
    x, w = s["x"].double(), s["w"].double()
    if op == "linear8":
        x, w = x * s["xs"].double()[:, None], w * s["ws"].double()[:, None]
    v = x @ w.t() + (0.0 if s["b"] is None else s["b"].double())
    r = 0.0 if s["r"] is None else s["r"].double()
    c = math.sqrt(2.0 / math.pi)
    if act == "gelu":
        th = torch.tanh(c * (v + 0.044715 * v ** 3))
        y, d = 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * c * (1 + 0.134145 * v * v)
    elif act == "silu":
        sg = torch.sigmoid(v)
        y, d = v * sg, sg + v * sg * (1 - sg)
    else:
        y, d = v, torch.ones_like(v)
    if op != "linear_train":
        return [y + r]
    dv = s["dy"].double() * d
    out = [y + r, dv @ w, dv.t() @ x]
    if s["b"] is not None:
        out.append(dv.sum(0))
    return out + ([s["dy"]] if s["r"] is not None else [])


def _exact_gates(s):
    g = s["g"].double()
    si = torch.ones_like(g) if s["i"] is None else torch.sigmoid(s["i"].double())
    if s["l"] is None:
        return g, torch.ones_like(g), si, None
    sg = torch.sigmoid(g)
    lg = -s["l"].double() * sg
    return lg, torch.sqrt(-torch.expm1(2 * lg)), si, sg


def _exact_rec_step(s):
    lg, m, si, _ = _exact_gates(s)
    idx = s["idx"].long()
    state = s["state"].double()
    state[idx] = lg.exp() * state[idx] + m * si * s["x"].double()
    return [state[idx], state]


def _blocked(a, u):
    """h_t = a_t h_{t-1} + u_t over [tokens, D], token by token inside blocks and then block by block."""
    T, D = a.shape
    C = 128
    nb = (T + C - 1) // C
    pad = lambda t: torch.cat([t, t.new_zeros(nb * C - T, D)]).reshape(nb, C, D)  # noqa: E731
    a, h = pad(a), pad(u)
    for t in range(1, C):
        h[:, t] += a[:, t] * h[:, t - 1]
        a[:, t] *= a[:, t - 1]
    for b in range(1, nb):
        h[b] += a[b] * h[b - 1, -1]
    return h.reshape(-1, D)[:T]


def _exact_rec(s, train):
    case, D = s["case"], s["case"]["D"]
    live, first, last, _ = _firsts(s)
    shape = s["x"].shape
    lg, m, si, sg = (None if t is None else t.reshape(-1, D) for t in _exact_gates(s))
    x = s["x"].double().reshape(-1, D)
    h0 = s["h0"].double() if s["h0"] is not None else torch.zeros(_nseq(case), D, device=DEV, dtype=torch.float64)
    a = lg.exp()
    entering = torch.zeros_like(x)
    entering[first] = h0[live]
    inside = a.clone()
    inside[first] = 0
    h = _blocked(inside, m * si * x + a * entering)
    hT = h0.clone()
    hT[live] = h[last]
    if not train:
        return [h.reshape(shape), hT]
    before = entering + torch.roll(h, 1, 0) * (inside != 0)
    before[first] = h0[live]
    dhT = s["dh"].double() if s["dh"] is not None else torch.zeros_like(h0)
    gy = s["dy"].double().reshape(-1, D)
    gy[last] += dhT[live]
    dh = _blocked(torch.roll(inside, -1, 0).flip(0), gy.flip(0)).flip(0)
    out = [h.reshape(shape), hT, (dh * m * si).reshape(shape)]
    dl = a * dh * before
    if sg is not None:
        dl = dl - torch.where(m > 0, dh * si * x * a.square() / m, torch.zeros_like(m))
        out.append((-dl * s["l"].double() * sg * (1 - sg)).reshape(shape))
    else:
        out.append(dl.reshape(shape))
    if s["i"] is not None:
        out.append((dh * m * x * si * (1 - si)).reshape(shape))
    if sg is not None:
        out.append((-dl * sg).sum(0))
    if s["h0"] is not None:
        d0 = dhT.clone()
        d0[live] = a[first] * dh[first]
        out.append(d0)
    return out
