"""Plain 64-bit forms of the operators of the block around the experts (the
product with bias, activation and residual, the norms before and after a block,
their gradients, the layer for a few tokens), each with an element-wise bound on what
a kernel that works in fp32 and rounds once may be off. U = 2^-24 is half a step of fp32.

Activations. e^-|v| is v_exp_f32 (1 ulp = 2 U) of the rounded product of |v| and a rounded log2 e, which is off by 1.25 |v| U
more; with 1 + e one rounding and the reciprocal 1 ulp a sigmoid is within (5 + 1.25 |v|) U of its value and a curve within
(7 + 1.25 |z|) U, which is below 8 U (1 + z^2). Where the sigmoid's (or erfc's) argument is itself formed with
roundings, its relative error grows by as many times the argument's size, which costs as much again.
So a curve is allowed 16 U (1 + z^2) |value|, its derivative, a sum of terms of size 1 + |z|
that may cancel, 32 U (1 + z^2). Curves change by at most 1.2 times what their argument does.

Norms. A mean of d squares is within (d + 32) U, its root within half of that and 4 U (square root, reciprocal).
"""
import math

import torch

from grouped_reference import F8, U, d, stored, sums, within  # noqa: F401

GATED = {"swiglu": "silu", "geglu": "gelu_tanh"}


def curve(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))


def slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    v = c * (z + 0.044715 * z ** 3)
    return torch.sigmoid(v) + z * torch.sigmoid(v) * torch.sigmoid(-v) * c * (1.0 + 3.0 * 0.044715 * z ** 2)


def curve_slack(name, z, value):
    return torch.zeros_like(z) if name in ("none", "relu") else 16 * U * (1 + z * z) * value.abs() + 1e-36 * (1 + z.abs())


def slope_slack(name, z):
    return torch.zeros_like(z) if name in ("none", "relu") else 32 * U * (1 + z * z)


def linear(x, W, bias, act, residual):
    """(y, slack of y before it is stored, z, slack of z)."""
    x, W = d(x), d(W)
    z = x @ W.T
    mag = x.abs() @ W.abs().T
    if bias is not None:
        z, mag = z + d(bias), mag + d(bias).abs()
    zs = sums(x.shape[1] + 1, mag)
    if act in GATED:
        h = z.shape[1] // 2
        g, u, gs, us = z[:, :h], z[:, h:], zs[:, :h], zs[:, h:]
        v = curve(GATED[act], g)
        vs = 1.2 * gs + curve_slack(GATED[act], g, v)
        y, ys = v * u, vs * (u.abs() + us) + v.abs() * us
    else:
        y = curve(act, z)
        ys = 1.2 * zs + curve_slack(act, z, y)
    if residual is not None:
        y = y + d(residual)
    return y, ys + 2 * U * y.abs(), z, zs


def act_grad(dy, pre, act, dtype):
    """(dz, slack of dz in fp32, slack of dz rounded to dtype)."""
    dy = d(dy)
    if act == "none":
        return dy, torch.zeros_like(dy), torch.zeros_like(dy)
    z = d(pre)
    if act in GATED:
        h, name = z.shape[1] // 2, GATED[act]
        g, u = z[:, :h], z[:, h:]
        v, s = curve(name, g), slope(name, g)
        dz = torch.cat([dy * u * s, dy * v], 1)
        slack = torch.cat([(dy * u).abs() * slope_slack(name, g), dy.abs() * curve_slack(name, g, v)], 1)
    else:
        dz = dy * slope(act, z)
        slack = dy.abs() * slope_slack(act, z)
    slack = slack + 3 * U * dz.abs()
    return dz, slack, stored(dz, slack, dtype)


def linear_grad(dy, x, W, pre, act, dtype):
    """((dx, slack), (dW, slack), (db, slack))."""
    dz, s32, s16 = act_grad(dy, pre, act, dtype)
    x, W = d(x), d(W)
    T, N = dz.shape
    return ((dz @ W, s16 @ W.abs() + sums(N, dz.abs() @ W.abs())), (dz.T @ x, s16.T @ x.abs() + sums(T, dz.abs().T @ x.abs())),
            (dz.sum(0), s32.sum(0) + sums(T, dz.abs().sum(0))))


def _root(v, eps):
    return (v * v).mean(1, keepdim=True).add(eps).rsqrt()


def _spread(gate, T):
    g = d(gate)
    g = g[None] if g.dim() == 1 else g
    return g.repeat_interleave(T // g.shape[0], 0)


def norm(o, x, w_o, gate, scale, w_n, eps):
    """((y, slack), (n, slack) or None)."""
    T, width = (o if o is not None else x).shape
    rr = (width + 32) * U / 2 + 4 * U
    y = torch.zeros((T, width), dtype=F8)
    ys = torch.zeros_like(y)
    if o is not None:
        p = d(o)
        if w_o is not None:
            p = p * _root(p, eps) * d(w_o)
        if gate is not None:
            p = p * _spread(gate, T)
        y, ys = p, p.abs() * (rr + 5 * U)
    if x is not None:
        part = scale * d(x)
        y, ys = y + part, ys + 3 * U * part.abs()
    ys = ys + U * y.abs()
    if w_n is None:
        return (y, ys), None
    r, w = _root(y, eps), d(w_n)
    n = y * r * w
    moved = (y.abs() * ys).mean(1, keepdim=True) * r * r
    return (y, ys), (n, ys * r * w.abs() + n.abs() * (moved + rr + 4 * U))


def _back(g, gs, v, w, eps):
    """Gradient of v root(v) w from g (known within gs): value and slack, and g vh with its own."""
    width = v.shape[1]
    rr = (width + 32) * U / 2 + 4 * U
    r = _root(v, eps)
    hat = v * r
    wg = w * g
    m = (wg * hat).mean(1, keepdim=True)
    mag = (wg * hat).abs().mean(1, keepdim=True)
    ms = mag * (rr + 4 * U + (width + 32) * U) + ((w * hat).abs() * gs).mean(1, keepdim=True)
    out = r * (wg - hat * m)
    slack = r * (w.abs() * gs + 2 * U * wg.abs() + hat.abs() * ms + (hat * m).abs() * (rr + 3 * U)) * (1 + rr) + out.abs() * (rr + 3 * U)
    return (out, slack), (g * hat, gs * hat.abs() + (g * hat).abs() * (rr + 2 * U))


def norm_grad(dy, dn, o, y, w_o, gate, scale, w_n, eps):
    """Dict of (value, slack): dx, and where they exist d_o, dw_o, dgate, dw_n."""
    some = next(t for t in (dy, dn) if t is not None)
    T, width = some.shape
    rr = (width + 32) * U / 2 + 4 * U
    gy = torch.zeros((T, width), dtype=F8) if dy is None else d(dy)
    gs = torch.zeros_like(gy)
    out = {}

    def column_sums(pair, per):
        v, s = pair
        shape = (-1, per, width)
        return v.reshape(shape).sum(1), s.reshape(shape).sum(1) + sums(per, v.abs().reshape(shape).sum(1))
    if dn is not None:
        (b, bs), pair = _back(d(dn), torch.zeros_like(gy), d(y), d(w_n), eps)
        gy, gs = gy + b, gs + bs
        v, s = column_sums(pair, T)
        out["dw_n"] = (v[0], s[0])
    gs = gs + U * gy.abs()
    out["dx"] = (scale * gy, abs(scale) * gs + 2 * U * (scale * gy).abs())
    if o is not None:
        of = d(o)
        dp, dps = gy, gs
        if gate is not None:
            p = of if w_o is None else of * _root(of, eps) * d(w_o)
            per = T // (1 if gate.dim() == 1 else gate.shape[0])
            v, s = column_sums((gy * p, gs * p.abs() + (gy * p).abs() * (rr + 4 * U)), per)
            out["dgate"] = (v.reshape(gate.shape), s.reshape(gate.shape))
            g = _spread(gate, T)
            dp, dps = g * gy, g.abs() * gs + U * (g * gy).abs()
        if w_o is not None:
            (b, bs), pair = _back(dp, dps, of, d(w_o), eps)
            v, s = column_sums(pair, T)
            out["dw_o"] = (v[0], s[0])
            dp, dps = b, bs
        out["d_o"] = (dp, dps)
    return out


def layer(x, logits, gu, dn, k, sh_gu, sh_dn, add):
    """(y, slack of y before it is stored, ids, gates)."""
    x, lg = d(x), d(logits)
    T, width = x.shape
    ranked = torch.sort(lg, dim=1, descending=True, stable=True)
    ids = ranked.indices[:, :k]
    gates = torch.softmax(ranked.values[:, :k], 1)
    y = torch.zeros((T, dn.shape[1] if dn is not None else width), dtype=F8) if add is None else d(add).clone()
    mag, ys = y.abs(), torch.zeros_like(y)

    def block(v, g, w):
        g, w = d(g), d(w)
        h = g.shape[0] // 2
        z, zs = v @ g.T, sums(v.shape[1], v.abs() @ g.abs().T)
        c = curve("silu", z[:, :h])
        cs = 1.2 * zs[:, :h] + curve_slack("silu", z[:, :h], c)
        a = c * z[:, h:]
        s = cs * (z[:, h:].abs() + zs[:, h:]) + c.abs() * zs[:, h:] + U * a.abs()
        return a @ w.T, s @ w.abs().T + sums(3 * h, a.abs() @ w.abs().T), a.abs() @ w.abs().T
    for j in range(k):
        for e in ids[:, j].unique().tolist():
            at = (ids[:, j] == e).nonzero()[:, 0]
            v, s, m = block(x[at], gu[e], dn[e])
            w = gates[at, j, None]
            y[at] += w * v
            # a gate: exponentials of rounded differences (the logits' magnitude is below 16 in the tests) and their sum
            ys[at] += w * (s + v.abs() * 64 * U)
            mag[at] += w * v.abs()
    if sh_gu is not None:
        v, s, m = block(x, sh_gu, sh_dn)
        y, ys, mag = y + v, ys + s, mag + v.abs()
    return y, ys + sums(k + 2, mag), ids, gates
