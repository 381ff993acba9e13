"""64-bit model of the gated feed-forward, the norms around a block and the 8-bit checkpoints, with
bounds on what a kernel may be off by.

U16 is half a step of bf16 relative to the value, U32 that of fp32.  A contraction of K terms in
fp32 is held to K 2^-23 of the sum of magnitudes: every addition of K may be off by one step (the
tensor cores need not round to nearest), each product is exact.  F is what a handful of fp32
operations and CUDA's fast exponential and division lose, relative to the terms."""
import math

import torch

U16 = 2.0 ** -8
U32 = 2.0 ** -24
F = 2.0 ** -18
GROUP = 32


def d(t):
    return None if t is None else t.detach().double().cpu()


# ------------------------------------------------------------------ checkpoints --

def pack(x):
    """(codes, exps) of x [rows, cols] in 64 bits, as integers."""
    rows, cols = x.shape
    v = x.reshape(rows, cols // GROUP, GROUP)
    m = v.abs().amax(2)
    bad = ~torch.isfinite(v).all(2) | (m >= 255.0 * 2.0 ** 120)
    safe = torch.where(bad | (m == 0), torch.ones_like(m), m)
    f, e = torch.frexp(safe)                      # safe = f 2^e, 1/2 <= f < 1
    e = e.long() - 7 + (f >= 127.5 / 128).long()  # smallest e with safe < 127.5 2^e
    e = torch.where(m == 0, torch.full_like(e, -126), e.clamp(min=-126))
    step = torch.ldexp(torch.ones_like(m), e).unsqueeze(2)
    codes = torch.where(bad.unsqueeze(2), torch.zeros_like(v), torch.where(torch.isfinite(v), v, torch.zeros_like(v)) / step).round()
    exps = torch.where(bad, torch.full_like(e, 255), e + 127)
    return codes.reshape(rows, cols).to(torch.int8), exps.to(torch.uint8)


def unpack(codes, exps):
    scale = torch.ldexp(torch.ones(exps.shape, dtype=torch.float64), exps.long() - 127)
    scale = torch.where(exps == 255, torch.full_like(scale, math.nan), scale)
    return codes.double() * scale.repeat_interleave(GROUP, 1)


def values(t):
    """The 64-bit values of a bf16 tensor or of a checkpoint."""
    if isinstance(t, tuple):
        return unpack(t[0].cpu(), t[1].cpu())
    return d(t)


def kept_bound(exact, err, kept):
    """What rounding `exact` (itself known to `err`) to kept may be off by; checks the exponents."""
    if not isinstance(kept, tuple):
        return U16 * exact.abs() + err
    exps = kept[1].cpu().long() - 127
    step = torch.ldexp(torch.ones(exps.shape, dtype=torch.float64), exps)
    rows, cols = exact.shape
    m = (exact.abs() + err).reshape(rows, -1, GROUP).amax(2)
    least = (exact.abs() - err).clamp(min=0).reshape(rows, -1, GROUP).amax(2)
    assert (least < 127.5 * step).all(), "a scale is too small"
    assert ((m >= 127.5 * step / 2) | (exps == -126)).all(), "a scale is larger than it has to be"
    return step.repeat_interleave(GROUP, 1) / 2 + err


# ------------------------------------------------------------ gated feed-forward --

def act(z, name):
    """act(z), act'(z)"""
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


SLOPE = 1.2  # |act'| stays below


def contraction(a, b):
    """a b^T and its error bound in fp32."""
    return a @ b.t(), a.shape[1] * 2 * U32 * (a.abs() @ b.abs().t())


def ffn(x, wg, wu, wd, name, resid=None):
    """(g, e_g, u, e_u, y, e_y)"""
    g, eg = contraction(x, wg)
    u, eu = contraction(x, wu)
    v, _ = act(g, name)
    a = v * u
    ea = SLOPE * eg * (u.abs() + eu) + v.abs() * eu + (U16 + F) * a.abs() + F * g.abs() * u.abs()
    y, ey = contraction(a, wd)
    ey = ey + ea @ wd.abs().t()
    if resid is not None:
        y = y + resid
        ey = ey + U32 * resid.abs()
    return g, eg, u, eu, y, ey + U16 * y.abs()


def ffn_backward(dy, x, wg, wu, wd, g, u, name, grad_rounding):
    """{name: (value, bound)} from kept g and u; grad_rounding: U16 or U32 for the weight gradients."""
    v, s = act(g, name)
    a = v * u
    ea = (U16 + F) * a.abs() + F * g.abs() * u.abs()
    da, eda = contraction(dy, wd.t())
    dg, du = da * u * s, da * v
    edg = eda * (u * s).abs() + (U16 + F) * dg.abs() + F * (1 + g.abs()) * (da * u).abs()
    edu = eda * v.abs() + (U16 + F) * du.abs() + F * (da * g).abs()

    def product(p, ep, q, rounding):
        r, e = contraction(p, q)
        return r, e + ep @ q.abs().t() + rounding * r.abs()

    x1, e1 = contraction(dg, wg.t())
    x2, e2 = contraction(du, wu.t())
    dx = x1 + x2
    edx = e1 + e2 + edg @ wg.abs() + edu @ wu.abs() + U16 * dx.abs()
    out = dict(dx=(dx, edx), dw_gate=product(dg.t(), edg.t(), x.t(), grad_rounding),
               dw_up=product(du.t(), edu.t(), x.t(), grad_rounding))
    w, ew = contraction(a.t(), dy.t())
    out["dw_down"] = (w.t(), (ew + ea.t() @ dy.abs()).t() + grad_rounding * w.t().abs())
    return out


# --------------------------------------------------------------------- the norms --

def normal(v, rms, eps):
    """(v - mean) / sd, mean, 1 / sd"""
    mean = torch.zeros_like(v[:, :1]) if rms else v.mean(1, keepdim=True)
    r = ((v - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    return (v - mean) * r, mean, r


def gate_rows(gate, rows):
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64)
    gate = gate.reshape(-1, gate.shape[-1])
    return gate.repeat_interleave(rows // gate.shape[0], 0)


def norm_error(v, vh, r):
    """Error bound of an fp32 (v - mean) / sd: the statistics' sums and the operations on each value."""
    return F * (vh.abs() + v.abs().mean(1, keepdim=True) * r + v.abs() * r)


def norm_residual(x, o, pg, pb, gate, alpha, ng, nb, rms, eps, y_stored=None):
    """(y, e_y, h, e_h, stats); h from y_stored, the y that was rounded."""
    p, st, ep = o, [torch.zeros(o.shape[0], 1).double()] * 4, torch.zeros_like(o)
    if pg is not None:
        oh, m, r = normal(o, rms, eps)
        st[0], st[1] = m, r
        p = oh * pg + (0 if pb is None else pb)
        ep = norm_error(o, oh, r) * pg.abs() + F * p.abs()
    g = gate_rows(gate, o.shape[0])
    y = alpha * x + g * p
    ey = U16 * y.abs() + g.abs() * ep + F * (abs(alpha) * x.abs() + (g * p).abs())
    if ng is None:
        return y, ey, None, None, torch.cat(st, 1)
    ys = y if y_stored is None else y_stored
    yh, m, r = normal(ys, rms, eps)
    st[2], st[3] = m, r
    h = yh * ng + (0 if nb is None else nb)
    return y, ey, h, U16 * h.abs() + norm_error(ys, yh, r) * ng.abs() + F * h.abs(), torch.cat(st, 1)


def norm_backward(dy, dh, y, o, pg, pb, gate, alpha, ng, rms, eps):
    """{name: (value, bound)}"""
    rows, n = o.shape
    out = {}
    dd = torch.zeros_like(o) if dy is None else dy
    ed = F * dd.abs()
    more = rows * 2 * U32  # the additions of a sum over rows

    def through(w, ew, v, vh, r):
        m1 = 0 if rms else w.mean(1, keepdim=True)
        m2 = (w * vh).mean(1, keepdim=True)
        t = r * (w - m1 - vh * m2)
        eh = norm_error(v, vh, r)
        size = w.abs() + w.abs().mean(1, keepdim=True) + vh.abs() * (w * vh).abs().mean(1, keepdim=True)
        e = ew + ew.mean(1, keepdim=True) + vh.abs() * (ew * vh.abs()).mean(1, keepdim=True)
        e = e + eh * m2.abs() + vh.abs() * (w.abs() * eh).mean(1, keepdim=True)
        return t, r * (e + F * size)

    if ng is not None:
        yh, _, r = normal(y, rms, eps)
        eh = norm_error(y, yh, r)
        out["dpre_gamma"] = ((dh * yh).sum(0), (dh.abs() * eh).sum(0) + more * (dh * yh).abs().sum(0))
        out["dpre_beta"] = (dh.sum(0), more * dh.abs().sum(0))
        t, e = through(dh * ng, F * (dh * ng).abs(), y, yh, r)
        dd, ed = dd + t, ed + e
    out["dx"] = (alpha * dd, abs(alpha) * ed + (U16 + F) * (alpha * dd).abs())
    oh, eo = o, torch.zeros_like(o)
    if pg is not None:
        oh, _, r = normal(o, rms, eps)
        eo = norm_error(o, oh, r)
    p, epp = oh, eo
    if pg is not None:
        p = oh * pg + (0 if pb is None else pb)
        epp = eo * pg.abs() + F * p.abs()
    g = gate_rows(gate, rows)
    if gate is not None:
        k = gate.reshape(-1, n).shape[0]
        fold = lambda v: v.reshape(k, rows // k, n).sum(1)  # noqa: E731
        # S1 and S0 are summed on their own: their terms count, not their sum's
        terms = (dd * oh).abs() * (1 if pg is None else pg.abs()) + (0 if pb is None else (dd * pb).abs())
        out["dgate"] = (fold(dd * p), fold(ed * p.abs() + dd.abs() * epp + (more + F) * terms))
    w, ew = g * dd, g.abs() * ed + F * (g * dd).abs()
    if pg is not None:
        out["dpost_gamma"] = ((w * oh).sum(0), (ew * oh.abs() + w.abs() * eo + more * (w * oh).abs()).sum(0))
        out["dpost_beta"] = (w.sum(0), (ew + more * w.abs()).sum(0))
        w, ew = through(w * pg, ew * pg.abs() + F * (w * pg).abs(), o, oh, r)
    out["do"] = (w, ew + U16 * w.abs())
    return out


def held_to(name, got, want, bound):
    got = d(got).reshape(want.shape)
    assert torch.isfinite(got).all(), f"{name} is not finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), (f"{name}: {int((over > 0).sum())} of {over.numel()} values beyond the bound, by up to "
                               f"{over.max():.3e}")
