"""Timed cases of the training block's operators: the gated feed-forward (forward and backward),
the norms before and after a block with its gate and residual scale (forward and backward), and the
8-bit activation checkpoints that both backward passes can read.

`run` computes a case with elementary torch operations in fp32, or, with `own` set, through the
calls of block_sliding_window_gb300 that a training or serving program makes.  `exact` is the
definition in 64 bits, written apart from both.

A checkpoint of a [rows, cols] tensor is int8 codes [rows, cols] and uint8 exponents
[rows, cols / 32]: code c of a group with exponent E stands for c 2^(E - 127).
"""
import math
import random

import torch

own = False

GROUP = 32
EPS = 1e-5


# ------------------------------------------------------------------------------------- the cases --

def listed():
    ffn = dict(kind="ffn")
    norm = dict(kind="norm", alpha=1.0)
    back = dict(kind="norm_bwd", alpha=1.0)
    return [
        # One new token through the feed-forward of the 13B-class width: the weights' bytes.
        dict(ffn, name="ffn_1_token", tokens=1, hidden=5120, ffn=13824, act="silu", resid=False),
        # The new tokens of a batch of answers, added to the residual stream.
        dict(ffn, name="ffn_24_tokens", tokens=24, hidden=5120, ffn=13824, act="gelu", resid=True),
        # The training sequence of the 175B-class width.
        dict(ffn, name="ffn_2048_175b", tokens=2048, hidden=12288, ffn=32768, act="silu", resid=False),
        # The backward pass from bf16 activations, the 13B-class training sequence.
        dict(kind="ffn_bwd", name="ffn_bwd_2048", tokens=2048, hidden=5120, ffn=13824, act="silu", bits=16),
        # The same from 8-bit checkpoints of gate, up and x, 64-wide remainders of ffn.
        dict(kind="ffn_bwd", name="ffn_bwd_8bit", tokens=1555, hidden=5120, ffn=13632, act="gelu", bits=8),
        # A whole training step that keeps 8 bits: forward, checkpoint of x, backward.
        dict(kind="ffn_step", name="ffn_step_8bit", tokens=777, hidden=2048, ffn=5440, act="silu"),
        # One new token between two blocks: latency.
        dict(norm, name="norm_1_row", seqs=1, rows=1, hidden=5120, rms=True, post=True, gate="none", pre=True),
        # A training batch, norms with a bias, a learned gate for each channel.
        dict(norm, name="norm_8192", seqs=4, rows=2048, hidden=5120, rms=False, post=True, gate="channel", pre=True),
        # Backward at the 175B-class width, a gate of its own for each sequence.
        dict(back, name="norm_bwd_175b", seqs=4, rows=1000, hidden=12288, rms=False, post=True, gate="sequence",
             pre=True, bits=16),
        # Backward of rms norms with a scaled residual, the block's output kept in 8 bits.
        dict(back, name="norm_bwd_8bit", seqs=1, rows=8190, hidden=5120, rms=True, post=True, gate="channel",
             pre=True, bits=8, alpha=0.8125),
        # The output of a block on one short sequence, kept and read back: latency.
        dict(kind="checkpoint", name="checkpoint_333", rows=333, cols=5120),
        # Gate and up of a 13B-class layer written as a checkpoint and read back.
        dict(kind="checkpoint", name="checkpoint_2048", rows=2048, cols=27648),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    kind = rng.choice(["ffn", "ffn", "ffn_bwd", "ffn_step", "norm", "norm_bwd", "norm_bwd", "checkpoint"])
    if kind.startswith("ffn"):
        hidden = 64 * int(_log(rng, 4, 160))
        ffn = 64 * max(4, round(hidden * rng.uniform(1.5, 4.0) / 64))
        most = 4.0e11 if kind == "ffn" else 1.4e11  # tokens x hidden x ffn
        tokens = max(1, int(_log(rng, 1, min(4096, most / (hidden * ffn)) + 1)))
        c = dict(kind=kind, tokens=tokens, hidden=hidden, ffn=ffn, act=rng.choice(["silu", "gelu"]))
        if kind == "ffn":
            c["resid"] = rng.random() < 0.5
        elif kind == "ffn_bwd":
            c["bits"] = rng.choice([8, 16])
        return c
    if kind == "checkpoint":
        cols = 32 * int(_log(rng, 2, 1024))
        return dict(kind=kind, rows=int(_log(rng, 1, min(1 << 16, 5.0e7 / cols))), cols=cols)
    hidden = 32 * int(_log(rng, 4, 640))
    seqs = rng.choice([1, 1, 2, 3, 8])
    rows = max(1, int(_log(rng, 1, 4.0e7 / (hidden * seqs))))
    post = rng.random() < 0.8
    c = dict(kind=kind, seqs=seqs, rows=rows, hidden=hidden, rms=rng.random() < 0.5, post=post,
             gate=rng.choice(["none", "channel", "sequence"]), pre=rng.random() < 0.8 or not post,
             alpha=rng.choice([1.0, 0.5, 1.25]))
    if kind == "norm_bwd":
        c["bits"] = rng.choice([8, 16])
    return c


# ------------------------------------------------------------------------------------- the inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(torch.bfloat16)


def _stream_like(g, rows, hidden):
    """Rows of a residual stream: a mean of their own, and some channels far larger than the others."""
    loud = 1 + 15 * (torch.rand(hidden, generator=g, device="cuda") < 0.005)
    x = torch.randn(rows, hidden, generator=g, device="cuda") * loud
    return (x + torch.randn(rows, 1, generator=g, device="cuda") * 0.3).to(torch.bfloat16)


def _weights(g, c):
    h, f = c["hidden"], c["ffn"]
    return dict(w_gate=_normal(g, f, h, std=1.2 / math.sqrt(h)), w_up=_normal(g, f, h, std=1.2 / math.sqrt(h)),
                w_down=_normal(g, h, f, std=1 / math.sqrt(f)))


def _power(e):
    """2^e in fp32 for whole numbers e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x):
    """(codes, exponents) of a checkpoint of x [rows, cols]."""
    rows, cols = x.shape
    v = x.float().view(rows, cols // GROUP, GROUP)
    most = v.abs().amax(2)
    f, e = torch.frexp(most)  # most = f 2^e, f in [0.5, 1)
    e = torch.where(f >= 127.5 / 128, e + 1, e) - 7
    e = torch.where(most == 0, torch.full_like(e, -126), e).clamp(min=-126)
    codes = torch.round(v * _power(-e.unsqueeze(2)))
    return codes.to(torch.int8).view(rows, cols), (e + 127).to(torch.uint8)


def _values(codes, exps):
    rows, cols = codes.shape
    v = codes.float().view(rows, cols // GROUP, GROUP)
    return (v * _power(exps.int() - 127).unsqueeze(2)).view(rows, cols)


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=c)
    if c["kind"].startswith("ffn"):
        t, h, f = c["tokens"], c["hidden"], c["ffn"]
        s.update(_weights(g, c))
        s["x"] = _normal(g, t, h)
        s["resid"] = _normal(g, t, h, std=2.0) if c.get("resid") else None
        if c["kind"] != "ffn":
            s["dy"] = _normal(g, t, h, std=0.02)
        if c["kind"] == "ffn_bwd":
            # What the forward pass kept: gate and up as the weights above distribute them.
            s["saved"] = _normal(g, t, 2 * f, std=1.2)
            if c["bits"] == 8:
                s["saved"] = _quantised(s["saved"])
                s["x"] = _quantised(s["x"])
        return s
    if c["kind"] == "checkpoint":
        s["x"] = _stream_like(g, c["rows"], c["cols"])
        return s
    n, h = c["seqs"] * c["rows"], c["hidden"]
    s["post_gamma"] = s["post_beta"] = s["pre_gamma"] = s["pre_beta"] = s["gate"] = None
    if c["post"]:
        s["post_gamma"] = _normal(g, h, std=0.2, mean=1.0)
        s["post_beta"] = None if c["rms"] else _normal(g, h, std=0.1)
    if c["pre"]:
        s["pre_gamma"] = _normal(g, h, std=0.2, mean=1.0)
        s["pre_beta"] = None if c["rms"] else _normal(g, h, std=0.1)
    if c["gate"] != "none":
        s["gate"] = _normal(g, 1 if c["gate"] == "channel" else c["seqs"], h, std=0.2, mean=0.5)
    s["o"] = _normal(g, n, h, std=0.7)
    if c["kind"] == "norm":
        s["x"] = _stream_like(g, n, h)
        return s
    s["y"] = _stream_like(g, n, h)
    s["dy"] = _normal(g, n, h, std=0.01)
    s["dh"] = _normal(g, n, h, std=0.02) if c["pre"] else None
    if c["bits"] == 8:
        s["o"] = _quantised(s["o"])
    # The statistics that the forward pass kept for each row.
    s["stats"] = torch.zeros(n, 4, device="cuda")
    if c["post"]:
        s["stats"][:, 0:2] = _row_stats(_values(*s["o"]) if c["bits"] == 8 else s["o"], c["rms"])
    if c["pre"]:
        s["stats"][:, 2:4] = _row_stats(s["y"], c["rms"])
    return s


def _row_stats(v, rms):
    out = torch.empty(v.shape[0], 2, dtype=torch.float64, device=v.device)
    for lo in range(0, v.shape[0], 1024):
        d = v[lo:lo + 1024].double()
        mean = d.new_zeros(d.shape[0]) if rms else d.mean(1)
        out[lo:lo + 1024, 0] = mean
        out[lo:lo + 1024, 1] = ((d - mean.unsqueeze(1)).square().mean(1) + EPS).rsqrt()
    return out.float()


# ---------------------------------------------------------------------------------- the plain form --

def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))


def _act_grad(z, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * z * z)


def _plain_ffn(s, x):
    g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    y = (_act(g, s["case"]["act"]) * u) @ s["w_down"].float().t()
    return g, u, (y if s["resid"] is None else y + s["resid"].float()).to(torch.bfloat16)


def _plain_ffn_bwd(s, x, g, u):
    act, dy = s["case"]["act"], s["dy"].float()
    da = dy @ s["w_down"].float()
    av = _act(g, act)
    dw_down = (dy.t() @ (av * u)).to(torch.bfloat16)
    du = da * av
    dg = da * u * _act_grad(g, act)
    dx = (dg @ s["w_gate"].float() + du @ s["w_up"].float()).to(torch.bfloat16)
    return dict(dx=dx, dw_gate=(dg.t() @ x).to(torch.bfloat16), dw_up=(du.t() @ x).to(torch.bfloat16), dw_down=dw_down)


def _normalised(v, rms):
    mean = 0.0 if rms else v.mean(1, keepdim=True)
    d = v - mean
    r = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    return d * r, r


def _norm_bwd(dv, vh, r, rms):
    """Gradient through the normalisation for the gradient dv of its result vh."""
    m2 = (dv * vh).mean(1, keepdim=True)
    m1 = 0.0 if rms else dv.mean(1, keepdim=True)
    return r * (dv - m1 - vh * m2)


def _gate_rows(s, n):
    g = s["gate"].float()
    return g if g.shape[0] == 1 else g.repeat_interleave(n // g.shape[0], 0)


def _plain_norm(s):
    c, p = s["case"], s["o"].float()
    if c["post"]:
        p = _normalised(p, c["rms"])[0] * s["post_gamma"].float()
        if s["post_beta"] is not None:
            p = p + s["post_beta"].float()
    if s["gate"] is not None:
        p = p * _gate_rows(s, p.shape[0])
    y = (c["alpha"] * s["x"].float() + p).to(torch.bfloat16)
    if not c["pre"]:
        return dict(y=y)
    h = _normalised(y.float(), c["rms"])[0] * s["pre_gamma"].float()
    if s["pre_beta"] is not None:
        h = h + s["pre_beta"].float()
    return dict(y=y, h=h.to(torch.bfloat16))


def _plain_norm_bwd(s):
    c = s["case"]
    o = _values(*s["o"]) if c["bits"] == 8 else s["o"].float()
    out, d = {}, s["dy"].float()
    if c["pre"]:
        yh, r = _normalised(s["y"].float(), c["rms"])
        dh = s["dh"].float()
        d = d + _norm_bwd(dh * s["pre_gamma"].float(), yh, r, c["rms"])
        out["dpre_gamma"] = (dh * yh).sum(0)
        if s["pre_beta"] is not None:
            out["dpre_beta"] = dh.sum(0)
    out["dx"] = (c["alpha"] * d).to(torch.bfloat16)
    oh, r = _normalised(o, c["rms"]) if c["post"] else (o, None)
    p = oh * s["post_gamma"].float() if c["post"] else oh
    if s["post_beta"] is not None:
        p = p + s["post_beta"].float()
    dp = d
    if s["gate"] is not None:
        k = s["gate"].shape[0]
        out["dgate"] = (d * p).view(k, -1, c["hidden"]).sum(1)
        dp = d * _gate_rows(s, d.shape[0])
    if c["post"]:
        out["dpost_gamma"] = (dp * oh).sum(0)
        if s["post_beta"] is not None:
            out["dpost_beta"] = dp.sum(0)
        dp = _norm_bwd(dp * s["post_gamma"].float(), oh, r, c["rms"])
    out["do"] = dp.to(torch.bfloat16)
    return out


def _plain(s):
    c = s["case"]
    if c["kind"] == "ffn":
        return _plain_ffn(s, s["x"].float())[2]
    if c["kind"] == "ffn_bwd":
        f = c["ffn"]
        kept = _values(*s["saved"]) if c["bits"] == 8 else s["saved"].float()
        x = _values(*s["x"]) if c["bits"] == 8 else s["x"].float()
        return _plain_ffn_bwd(s, x, kept[:, :f], kept[:, f:])
    if c["kind"] == "ffn_step":
        g, u, y = _plain_ffn(s, s["x"].float())
        g, u, x = (_values(*_quantised(v)) for v in (g, u, s["x"]))
        return dict(_plain_ffn_bwd(s, x, g, u), y=y)
    if c["kind"] == "checkpoint":
        return _values(*_quantised(s["x"])).to(torch.bfloat16)
    return _plain_norm(s) if c["kind"] == "norm" else _plain_norm_bwd(s)


# ----------------------------------------------------------------------------- the framework's calls --

def _own(s):
    import block_sliding_window_gb300 as bsw
    c = s["case"]
    if c["kind"].startswith("ffn"):
        w = s["w_gate"], s["w_up"], s["w_down"]
    if c["kind"] == "ffn":
        return bsw.gated_ffn(s["x"], *w, activation=c["act"], residual=s["resid"])
    if c["kind"] == "ffn_bwd":
        return bsw.gated_ffn_backward(s["dy"], s["x"], *w, s["saved"], activation=c["act"])
    if c["kind"] == "ffn_step":
        y, saved = bsw.gated_ffn_train(s["x"], *w, activation=c["act"], bits=8)
        kept = bsw.checkpoint_pack(s["x"])
        return dict(bsw.gated_ffn_backward(s["dy"], kept, *w, saved, activation=c["act"]), y=y)
    if c["kind"] == "checkpoint":
        return bsw.checkpoint_unpack(*bsw.checkpoint_pack(s["x"]))
    how = dict(post_gamma=s["post_gamma"], post_beta=s["post_beta"], gate=s["gate"], pre_gamma=s["pre_gamma"],
               pre_beta=s["pre_beta"], alpha=c["alpha"], rms=c["rms"], eps=EPS)
    if c["kind"] == "norm":
        y, h = bsw.norm_residual(s["x"], s["o"], **how)
        return dict(y=y, h=h) if c["pre"] else dict(y=y)
    how.pop("eps")
    return bsw.norm_residual_backward(s["dy"], s["dh"], s["y"], s["o"], s["stats"], **how)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- the work --

def work(case):
    c = case
    if c["kind"].startswith("ffn"):
        t, h, f = c["tokens"], c["hidden"], c["ffn"]
        unit, w = 2 * t * h * f, 2 * 3 * h * f
        kept = 1 + 1 / GROUP  # bytes of a value in 8 bits
        if c["kind"] == "ffn":
            return dict(bytes=w + 2 * t * h * (3 if c["resid"] else 2), flops=3 * unit)
        if c["kind"] == "ffn_bwd":
            each = 2 if c["bits"] == 16 else kept
            return dict(bytes=2 * w + 2 * t * h * 2 + each * (2 * t * f + t * h), flops=6 * unit)
        return dict(bytes=2 * w + 2 * t * h * 4, flops=9 * unit)
    if c["kind"] == "checkpoint":
        return dict(bytes=c["rows"] * c["cols"] * (4 + 2 * (1 + 1 / GROUP)), flops=0)
    n = c["seqs"] * c["rows"] * c["hidden"]
    if c["kind"] == "norm":
        return dict(bytes=2 * n * (4 if c["pre"] else 3), flops=0)
    o = 2 if c["bits"] == 16 else 1 + 1 / GROUP
    return dict(bytes=n * (2 * (5 if c["pre"] else 3) + (o if c["post"] or c["gate"] != "none" else 0)), flops=0)


# ---------------------------------------------------------------------------------- in 64 bits --

def _d(t):
    return None if t is None else t.double()


def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _from8(codes, exps):
    scale = _two_to(exps.long() - 127)
    return codes.double() * scale.repeat_interleave(GROUP, 1)


def _to8(v):
    """The values that a checkpoint of v (64 bits) holds."""
    r, n = v.shape
    w = v.reshape(r, n // GROUP, GROUP)
    m = w.abs().max(2, keepdim=True).values
    e = torch.floor(torch.log2(m.clamp(min=1e-300)))
    e = e - (_two_to(e) > m).double() + (_two_to(e + 1) <= m).double()  # log2 near a power of two
    e = e - 6
    e = e + (m >= 127.5 * _two_to(e)).double()
    step = _two_to(e.clamp(min=-126))
    return ((w / step).round() * step).reshape(r, n)


def _exact_gate(z, act):
    """act(z) and its derivative."""
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t ** 2) * k * (1 + 3 * 0.044715 * z ** 2)


def _exact_ffn_bwd(s, act, x, g, u):
    v, slope = _exact_gate(g, act)
    dy = _d(s["dy"])
    out = dict(dw_down=torch.einsum("th,tf->hf", dy, v * u))
    da = torch.einsum("th,hf->tf", dy, _d(s["w_down"]))
    dg, du = da * u * slope, da * v
    out["dw_gate"] = torch.einsum("tf,th->fh", dg, x)
    out["dw_up"] = torch.einsum("tf,th->fh", du, x)
    out["dx"] = torch.einsum("tf,fh->th", dg, _d(s["w_gate"])) + torch.einsum("tf,fh->th", du, _d(s["w_up"]))
    return out


def _exact_rows(v, rms):
    m = torch.zeros_like(v[:, :1]) if rms else v.sum(1, keepdim=True) / v.shape[1]
    dev = ((v - m) ** 2).sum(1, keepdim=True) / v.shape[1]
    sd = torch.sqrt(dev + EPS)
    return (v - m) / sd, sd


def _through_norm(w, vh, sd, rms):
    """J^T w of v -> vh = (v - mean) / sd."""
    n = vh.shape[1]
    inner = w - vh * ((w * vh).sum(1, keepdim=True) / n)
    return (inner if rms else inner - w.sum(1, keepdim=True) / n) / sd


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"].startswith("ffn"):
        if 6 * c["tokens"] * c["hidden"] * c["ffn"] * (1 if c["kind"] == "ffn" else 3) > 1e13:
            return None
        f = c["ffn"]
        if c["kind"] == "ffn_bwd":
            both = _from8(*s["saved"]) if c["bits"] == 8 else _d(s["saved"])
            x = _from8(*s["x"]) if c["bits"] == 8 else _d(s["x"])
            return _exact_ffn_bwd(s, c["act"], x, both[:, :f], both[:, f:])
        x = _d(s["x"])
        g = torch.einsum("th,fh->tf", x, _d(s["w_gate"]))
        u = torch.einsum("th,fh->tf", x, _d(s["w_up"]))
        y = torch.einsum("tf,hf->th", _exact_gate(g, c["act"])[0] * u, _d(s["w_down"]))
        if c["kind"] == "ffn":
            return y if s["resid"] is None else y + _d(s["resid"])
        return dict(_exact_ffn_bwd(s, c["act"], _to8(x), _to8(g), _to8(u)), y=y)
    if c["kind"] == "checkpoint":
        return _to8(_d(s["x"]))
    k = 1 if s["gate"] is None else s["gate"].shape[0]
    n, h = c["seqs"] * c["rows"], c["hidden"]
    gate = torch.ones(1, h, dtype=torch.float64, device="cuda") if s["gate"] is None else _d(s["gate"])
    wide = lambda v: v.view(k, n // k, h)  # noqa: E731
    o = _from8(*s["o"]) if c.get("bits") == 8 else _d(s["o"])
    p = oh = o
    if c["post"]:
        oh, sd_o = _exact_rows(o, c["rms"])
        p = oh * _d(s["post_gamma"]) + (0 if s["post_beta"] is None else _d(s["post_beta"]))
    if c["kind"] == "norm":
        y = c["alpha"] * _d(s["x"]) + (wide(p) * gate.unsqueeze(1)).view(n, h)
        if not c["pre"]:
            return dict(y=y)
        # h is the norm of y as it is stored.
        yh, _ = _exact_rows(y.to(torch.bfloat16).double(), c["rms"])
        return dict(y=y, h=yh * _d(s["pre_gamma"]) + (0 if s["pre_beta"] is None else _d(s["pre_beta"])))
    out, d = {}, _d(s["dy"])
    if c["pre"]:
        yh, sd_y = _exact_rows(_d(s["y"]), c["rms"])
        dh = _d(s["dh"])
        out["dpre_gamma"] = torch.einsum("th,th->h", dh, yh)
        if s["pre_beta"] is not None:
            out["dpre_beta"] = dh.sum(0)
        d = d + _through_norm(dh * _d(s["pre_gamma"]), yh, sd_y, c["rms"])
    out["dx"] = d * c["alpha"]
    dp = (wide(d) * gate.unsqueeze(1)).view(n, h)
    if s["gate"] is not None:
        out["dgate"] = torch.einsum("kth,kth->kh", wide(d), wide(p))
    if c["post"]:
        out["dpost_gamma"] = torch.einsum("th,th->h", dp, oh)
        if s["post_beta"] is not None:
            out["dpost_beta"] = dp.sum(0)
        dp = _through_norm(dp * _d(s["post_gamma"]), oh, sd_o, c["rms"])
    out["do"] = dp
    return out
