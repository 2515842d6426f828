"""The activation checkpoints' operators in 64 bits, elementary torch operations
on the CPU, with bounds on what fp32 arithmetic may add to one rounding.

A bound is `u * |x| + tiny + e`: u is half a step of the stored type relative to
the value (finfo.eps / 2), tiny half its smallest subnormal, and e what the fp32
operations before that rounding may have added, written beside each formula in
units of F = 2^-24."""
import math

import torch

F = 2.0 ** -24
BLOCK = 128


def dec(t):
    return None if t is None else t.detach().cpu().double()


def check(got, want, err, name=""):
    """got, in its own type, is want rounded once, `err` apart."""
    t = got.dtype
    got, f = dec(got), torch.finfo(t)
    bound = f.eps / 2 * want.abs() + f.smallest_normal * f.eps / 2 + err
    off = (got - want).abs()
    both = (got == want) | (got.isnan() & want.isnan())
    bad = ~(both | (off <= bound))
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist(),
                           (bound.expand_as(off))[bad][:4].tolist())


def blocks(x):
    rows, cols = x.shape
    y = x.new_zeros(rows, -(-cols // BLOCK) * BLOCK)
    y[:, :cols] = x
    return y.view(rows, -(-cols // BLOCK), BLOCK)


def grid(y):
    """The e4m3 value next to y, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def encode(x):
    """Values of the codes [rows, cols] and scales [rows, blocks] of x (double)."""
    y = blocks(x)
    top = torch.where(y.isfinite(), y.abs(), 0.0).amax(2) if y.numel() else y.new_zeros(y.shape[:2])
    scale = torch.exp2(torch.ceil(torch.log2((top / 448).clamp_min(2.0 ** -126))))
    v = y / scale[:, :, None]
    v = torch.where(v.isfinite(), grid(torch.where(v.isfinite(), v, 0.0)), math.nan)
    return v.flatten(1)[:, :x.shape[1]], scale


def value(code, scale=None):
    v = code.detach().cpu().float().double()
    if scale is None:
        return v
    return v * dec(scale)[:, torch.arange(v.shape[1]) // BLOCK]


# --------------------------------------------------------------------------- feed-forward activations

def act(name, a):
    """f(a), f'(a), and the size that their fp32 errors are relative to, in units of F."""
    if name == "gelu":
        q = 0.5 * torch.erfc(-a / math.sqrt(2))
        f, slope = a * q, q + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        # erfc is within 16 units; rounding its argument x = a / sqrt 2 twice moves it by 2 * 2 x^2 units
        return f, slope, 24 + 2 * a * a, q + a.abs() * torch.exp(-a * a / 2)
    u = a if name == "silu" else 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
    du = torch.ones_like(a) if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * a * a)
    q = 1 / (1 + torch.exp(-u))
    # the exponent is rounded at a few units of |u|; exp, 1 + and the reciprocal add four more
    return a * q, q + a * q * (1 - q) * du, 24 + 6 * u.abs(), q + (a * q * du).abs()


def glu(name, a, b):
    """out and its fp32 error."""
    f, _, k, _ = act(name, a)
    o = f if b is None else f * b
    return o, (k + 2) * F * o.abs()


def glu_back(name, d, a, b):
    """da, db (None), out, and their fp32 errors."""
    f, slope, k, size = act(name, a)
    v = 1.0 if b is None else b
    ref = (d * v * slope, None if b is None else d * f, f * v)
    err = ((k + 4) * F * (d * v).abs() * size, None if b is None else (k + 4) * F * (d * f).abs(), (k + 4) * F * (f * v).abs())
    return ref, err


# --------------------------------------------------------------------------- block norms

SUMS = 48    # additions one after the other in a row's sum: 16 on a lane, 6 in a wave, 16 waves, and the last steps


def norm(z, ez, kind, eps):
    """Normalised values, r, and the errors of both; ez: the error of z."""
    m = z.mean(1, keepdim=True) if kind == "layer" else torch.zeros(z.shape[0], 1, dtype=z.dtype)
    em = (ez + SUMS * F * z.abs()).mean(1, keepdim=True) if kind == "layer" else m
    c, ec = z - m, ez + em + F * (z - m).abs()
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    # the mean square is off by 2 mean(c ec) and its own additions; its root halves that
    er = r ** 3 * (c.abs() * ec).mean(1, keepdim=True) + (SUMS / 2 + 6) * F * r
    return c * r, r[:, 0], c.abs() * er + ec * r + F * (c * r).abs(), er[:, 0]


def by_row(v, seg, rows):
    if v is None:
        return 1.0
    return v[None].expand(rows, -1) if v.dim() == 1 else v[seg]


def segments(starts, rows):
    """The segment of each row, -1 for none."""
    if starts is None:
        return torch.zeros(rows, dtype=torch.long)
    seg = torch.full((rows,), -1)
    for b in range(len(starts) - 1):
        seg[starts[b]:starts[b + 1]] = b
    return seg


def forward(c, x, y):
    """The forward pass over the rows of x that are in a segment: a dict of outputs and their fp32 errors.
    c: a dict of the norm's settings, vectors in double."""
    rows, seg = x.shape[0], c["seg"]
    out, h, eh = {}, x, torch.zeros_like(x)
    if y is not None:
        v, ev = y, torch.zeros_like(y)
        if c["post"] != "none":
            v, r, ev, er = norm(y, ev, c["post"], c["post_eps"])
            out.update(y_hat=(v, ev), y_rstd=(r, er))
        k = by_row(c["w1"], seg, rows) * by_row(c["gate"], seg, rows) * c["beta"]
        h = c["alpha"] * x + k * v
        eh = (k * ev).abs() if torch.is_tensor(k) else abs(k) * ev
        eh = eh + F * (4 * (k * v).abs() + 2 * (c["alpha"] * x).abs() + h.abs())
        out["h"] = (h, eh)
    hat, r, e, er = norm(h, eh, c["pre"], c["pre_eps"])
    out.update(h_hat=(hat, e), h_rstd=(r, er))
    m = by_row(c["mul"], seg, rows) + (1.0 if c["plus_one"] else 0.0)
    n = hat * m
    en = (e * m).abs() if torch.is_tensor(m) else e * abs(m)
    en = en + 3 * F * n.abs()
    if c["add"] is not None:
        n = n + by_row(c["add"], seg, rows)
        en = en + F * n.abs()
    out["n"] = (n, en)
    return out


def back(g, eg, z, r, kind):
    """The gradient through a norm, and its error; z, r exact."""
    r = r[:, None]
    gz, egz = (g * z).mean(1, keepdim=True), ((eg + SUMS * F * g.abs()) * z.abs()).mean(1, keepdim=True)
    m, em = 0.0, 0.0
    if kind == "layer":
        m, em = g.mean(1, keepdim=True), (eg + SUMS * F * g.abs()).mean(1, keepdim=True)
    d = g - z * gz - m
    return r * d, r * (eg + z.abs() * egz + em + 3 * F * (g.abs() + (z * gz).abs() + abs(m)))


def backward(c, dn, dh, xh, r, yh, ry):
    """The backward pass over the rows in a segment: outputs and errors. yh: the saved branch values (None without
    a gate or post norm), ry: their r; dy is made if c["branch"]."""
    rows, seg = dn.shape[0], c["seg"]
    out = {}

    def total(name, like, t, e):
        """Sums over the rows (like: [cols]) or each segment's."""
        adds = rows + 24
        if like.dim() == 1:
            out[name] = (t.sum(0), (e + adds * F * t.abs()).sum(0))
        else:
            z = torch.zeros_like(like)
            out[name] = (z.index_add(0, seg, t), z.index_add(0, seg, e + adds * F * t.abs()))
    m = by_row(c["mul"], seg, rows) + (1.0 if c["plus_one"] else 0.0)
    if c["mul"] is not None:
        total("d_mul", c["mul"], dn * xh, F * (dn * xh).abs())
    if c["add"] is not None:
        total("d_add", c["add"], dn, torch.zeros_like(dn))
    a = dn * m
    g, eg = back(a, 2 * F * a.abs(), xh, r, c["pre"])
    if dh is not None:
        g = g + dh
        eg = eg + F * g.abs()
    if not c["branch"]:
        out["dx"] = (c["alpha"] * g, abs(c["alpha"]) * (eg + 2 * F * g.abs()))
        return out
    out["dx"] = (c["alpha"] * g, abs(c["alpha"]) * (eg + 2 * F * g.abs()))
    p, ep = c["beta"] * g, abs(c["beta"]) * (eg + 2 * F * g.abs())
    w, gate = by_row(c["w1"], seg, rows), by_row(c["gate"], seg, rows)
    if c["gate"] is not None:
        total("d_gate", c["gate"], p * yh * w, (ep * yh * w).abs() + 4 * F * (p * yh * w).abs())
    if c["w1"] is not None:
        total("d_post_weight", c["w1"], p * gate * yh, (ep * gate * yh).abs() + 4 * F * (p * gate * yh).abs())
    q = p * gate * w
    k = gate * w
    eq = (ep * k).abs() if torch.is_tensor(k) else ep * abs(k)
    eq = eq + 3 * F * q.abs()
    if c["post"] != "none":
        q, eq = back(q, eq, yh, ry, c["post"])
    out["dy"] = (q, eq)
    return out


# --------------------------------------------------------------------------- weight gradients

def wgrad(dy, z, mul, add):
    """dw, db and their fp32 errors. Products of two 16-bit values are exact; a sum takes one step for 16 tokens, at
    most 16 inside one, and the joins of splits and strips; a step of the matrix cores may cut instead of round."""
    t = dy.shape[0]
    k = 2 * F * (t / 16 + 16 + 80)
    dw, e = dy.t() @ z, k * (dy.abs().t() @ z.abs())
    db, eb = dy.sum(0), (t / 8 + 80) * F * dy.abs().sum(0)
    if mul is not None:
        dw, e = dw * mul, e * mul.abs() + 2 * F * (dw * mul).abs()
    if add is not None:
        e = e + add.abs() * eb[:, None] + 2 * F * (add * db[:, None]).abs()
        dw = dw + add * db[:, None]
        e = e + F * dw.abs()
    return dw, e, db, eb
