"""More measured operators: activation checkpoints in 8 bits (e4m3) and what a
training step does with them. The codec of saved activations; the norms before
and after a transformer block, fused with its gate, its residual scale and the
residual sum, with the normalised values saved in 8 bits, and their backward
pass from those; the activation of a feed-forward layer, gated or not, with its
inputs saved in 8 bits, and its backward pass; the weight gradient of a linear
layer whose input was saved in 8 bits.

`own = False` computes them in elementary torch operations, `own = True` through
precision_state_amd.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
E4M3 = torch.float8_e4m3fn
BLOCK = 128             # columns of a row that share a scale
EPS_POST, EPS_PRE = 1e-5, 1e-6
MOST_VALUES = 100_000_000       # rows * cols of the largest drawn case but weight gradients
MOST_PRODUCTS = 800_000_000_000  # tokens * outputs * inputs of the largest drawn weight gradient

# op: encode, decode (saved activations of any layer), norm_fwd, norm_bwd, glu_fwd, glu_bwd, wgrad
# type: of activations and their gradients; vec: of norm weights, gates and modulations
# pad: columns between the end of one row and the next
# norms: pre, post: rms, layer (post also none); branch: a block's output joins the residual stream; gate: it is
#   gated, mod: weight (one vector for all rows) or ada (scale and shift, like the gate a vector for each sequence);
#   segs: packed sequences (0: gate and weight serve all rows), tail: rows behind the last sequence
# glu: act: silu, gelu, gelu_tanh; gated: times a second input; again: the backward pass gives the output once more
# wgrad: tokens x out gradients, tokens x inp saved inputs; saved: block (a scale for each 128 columns) or norm
#   (normalised values and the norm's weight); bias: the bias gradient too; grad: the type of the gradient
NORM = dict(type="bf16", vec="bf16", pre="rms", post="none", branch=True, gate=False, mod="weight", segs=0, tail=0,
            alpha=1.0, beta=1.0)


def listed():
    return [
        # saving the input of a wide feed-forward layer's last product
        dict(name="encode_wide", op="encode", type="bf16", rows=16384, cols=12288, pad=0),
        # reading back half-precision activations of odd width, rows with a stride
        dict(name="decode_odd", op="decode", type="f16", rows=4097, cols=2731, pad=13),
        # a block's exit and the next one's entry in a language model: norms before and after, scaled branch
        dict(NORM, name="norm_fwd_sandwich", op="norm_fwd", rows=16384, cols=4096, post="rms", beta=0.5),
        # the short sequences of an adapter run on a small model
        dict(NORM, name="norm_fwd_short", op="norm_fwd", rows=77, cols=1024, vec="f32"),
        # a diffusion transformer: images of different sizes in one batch, each with its own gate, scale and shift
        dict(NORM, name="norm_bwd_modulated", op="norm_bwd", rows=9216, cols=5120, pre="layer", gate=True, mod="ada",
             segs=6, tail=100),
        dict(NORM, name="norm_bwd_sandwich", op="norm_bwd", rows=16384, cols=4096, post="rms", beta=0.5),
        # odd width in 32 bits
        dict(NORM, name="norm_bwd_odd", op="norm_bwd", type="f32", vec="f32", rows=1537, cols=1001, pre="layer",
             post="layer", gate=True, segs=0),
        # gated feed-forward layer of a language model
        dict(name="glu_fwd_wide", op="glu_fwd", type="bf16", act="silu", gated=True, rows=8192, cols=11008, again=False),
        dict(name="glu_bwd_wide", op="glu_bwd", type="bf16", act="silu", gated=True, rows=8192, cols=11008, again=True),
        # the ungated layer of a text encoder, odd width
        dict(name="gelu_bwd_odd", op="glu_bwd", type="f16", act="gelu_tanh", gated=False, rows=1537, cols=2731,
             again=False),
        # the first product of a feed-forward layer: its input was saved by the norm before it
        dict(name="wgrad_wide", op="wgrad", type="bf16", tokens=16384, out=11008, inp=4096, saved="norm", bias=False,
             grad="f32"),
        # a low-rank adapter's gradient: few outputs, many tokens
        dict(name="wgrad_adapter", op="wgrad", type="bf16", tokens=4096, out=16, inp=2048, saved="block", bias=True,
             grad="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["encode", "decode", "norm_fwd", "norm_bwd", "norm_fwd", "norm_bwd", "glu_fwd", "glu_bwd", "wgrad",
                     "wgrad"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    while True:
        rows, cols = _log(rng, 1, 16384), _log(rng, 8, 12288 if op in ("encode", "decode", "glu_fwd", "glu_bwd") else 8192)
        if rng.random() < 0.5:
            cols = -(-cols // 64) * 64
        if rows * cols <= MOST_VALUES * (1 if kind != "f32" else 0.5):
            break
    if op in ("encode", "decode"):
        return dict(op=op, type=kind, rows=rows, cols=cols, pad=rng.choice([0, 0, 1, 8, 64]))
    if op in ("glu_fwd", "glu_bwd"):
        return dict(op=op, type=kind, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]), gated=rng.random() < 0.7,
                    rows=rows, cols=cols, again=op == "glu_bwd" and rng.random() < 0.5)
    if op == "wgrad":
        while True:
            c = dict(op=op, type=rng.choice(["bf16", "bf16", "f16"]), tokens=_log(rng, 16, 16384),
                     out=_log(rng, 8, 12288), inp=_log(rng, 8, 12288), saved=rng.choice(["block", "norm"]),
                     bias=rng.random() < 0.5, grad=rng.choice(["f32", "bf16", "f16"]))
            if rng.random() < 0.5:
                c["out"], c["inp"] = -(-c["out"] // 64) * 64, -(-c["inp"] // 64) * 64
            if c["tokens"] * c["out"] * c["inp"] <= MOST_PRODUCTS:
                return c
    c = dict(NORM, op=op, type=kind, vec=rng.choice([kind, "f32"]), rows=rows, cols=cols, pre=rng.choice(["rms", "layer"]))
    if rng.random() < 0.8:
        c.update(post=rng.choice(["none", "none", "rms", "layer"]), gate=rng.random() < 0.5,
                 alpha=rng.choice([1.0, 1.0, 1.5]), beta=rng.choice([1.0, 0.5]))
    else:
        c["branch"] = False
    if rng.random() < 0.5:
        c.update(segs=rng.randint(1, 12), mod=rng.choice(["weight", "ada"]), tail=rng.choice([0, 0, rows // 10]))
    return c


def work(case):
    if case["op"] == "wgrad":
        t, n, k = case["tokens"], case["out"], case["inp"]
        scales = 4 * t * -(-k // BLOCK) if case["saved"] == "block" else 4 * k
        return {"bytes": t * n * SIZE[case["type"]] + t * k + scales + n * k * SIZE[case["grad"]]
                + (4 * n if case["bias"] else 0), "flops": 2 * t * n * k}
    rows, cols, e = case["rows"], case["cols"], SIZE[case["type"]]
    n, coded = rows * cols, rows * cols + 4 * rows * -(-cols // BLOCK)
    if case["op"] in ("encode", "decode"):
        return {"bytes": e * n + coded, "flops": 2 * n}
    if case["op"] == "glu_fwd":
        k = 2 if case["gated"] else 1
        return {"bytes": (k + 1) * e * n + k * coded, "flops": 10 * n}
    if case["op"] == "glu_bwd":
        k = 2 if case["gated"] else 1
        return {"bytes": (k + 1 + case["again"]) * e * n + k * coded, "flops": 15 * n}
    n -= case["tail"] * cols
    rows -= case["tail"]
    groups, v = max(1, case["segs"]), SIZE[case["vec"]]
    saved = n + 4 * rows
    if case["branch"]:
        saved += (n + 4 * rows if case["post"] != "none" else n + 4 * rows * -(-cols // BLOCK) if case["gate"] else 0)
    mods = cols * (2 * groups if case["mod"] == "ada" else 1)
    vectors = mods + (cols if case["post"] != "none" else 0) + (cols * groups if case["gate"] else 0)
    streams = (4 if case["branch"] else 2) if case["op"] == "norm_fwd" else (4 if case["branch"] else 3)
    grads = 0 if case["op"] == "norm_fwd" else 4 * vectors
    return {"bytes": streams * e * n + saved + v * vectors + grads, "flops": (12 if case["op"] == "norm_fwd" else 25) * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _activations(rand, rows, cols):
    """Activations of a layer: some channels much larger than the others, rows of different size."""
    level = torch.exp(0.5 * rand(rows, 1))
    wide = torch.exp(0.4 * rand(1, cols))
    wide[rand(1, cols) > 2.6] *= 20
    return rand(rows, cols).mul_(level).mul_(wide)


def _padded(x, dtype, pad):
    """x as `dtype`, rows `pad` columns apart."""
    y = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=dtype, device=DEV)
    y[:, :x.shape[1]] = x
    return y[:, :x.shape[1]]


def _empty_code(rows, cols):
    return torch.zeros(rows, cols, dtype=E4M3, device=DEV), torch.zeros(rows, -(-cols // BLOCK), device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    s = dict(case=case)
    if own:
        import precision_state_amd as ps
        s["ps"] = ps
    op = case["op"]
    if op == "wgrad":
        return _prepare_wgrad(s, case, rand)
    dtype, rows, cols = DT[case["type"]], case["rows"], case["cols"]
    if op in ("encode", "decode"):
        s["x"] = _padded(_activations(rand, rows, cols), dtype, case["pad"])
        s["code"], s["scale"] = _empty_code(rows, cols)
        if op == "decode":
            s["code"], s["scale"] = _encode(s["x"])
            s["x"].zero_()
        return s
    if op in ("glu_fwd", "glu_bwd"):
        k = 2 if case["gated"] else 1
        x = torch.zeros(rows, k * cols, dtype=dtype, device=DEV)   # both inputs come from one product
        for i in range(k):
            x[:, i * cols:(i + 1) * cols] = _activations(rand, rows, cols)
        s["x"] = [x[:, i * cols:(i + 1) * cols] for i in range(k)]
        if op == "glu_fwd":
            s["out"] = torch.zeros(rows, cols, dtype=dtype, device=DEV)
            s["codes"] = [_empty_code(rows, cols) for _ in s["x"]]
        else:
            s["codes"] = [_encode(v) for v in s["x"]]
            x.zero_()                                               # takes the gradients
            s["dout"] = rand(rows, cols).mul_(1e-2).to(dtype)
            s["out"] = torch.zeros(rows, cols, dtype=dtype, device=DEV) if case["again"] else None
        if own:
            s["act"] = {"silu": ps.ACT_SILU, "gelu": ps.ACT_GELU, "gelu_tanh": ps.ACT_GELU_TANH}[case["act"]]
        return s
    return _prepare_norm(s, case, rand, seed)


def _prepare_norm(s, case, rand, seed):
    dtype, vec, rows, cols = DT[case["type"]], DT[case["vec"]], case["rows"], case["cols"]
    used = rows - case["tail"]
    starts, groups = None, 1
    if case["segs"]:
        cpu = torch.Generator().manual_seed(seed)
        cuts = torch.randint(0, used + 1, (case["segs"] - 1,), generator=cpu).sort().values
        starts = torch.cat([torch.tensor([0]), cuts, torch.tensor([used])]).to(torch.int32).to(DEV)
        groups = case["segs"]
    s.update(used=used, starts=starts, groups=groups)
    if starts is not None:
        s["seg"] = torch.searchsorted(starts[1:].contiguous(), torch.arange(used, dtype=torch.int32, device=DEV),
                                      right=True).clamp_max(groups - 1)
    per = (groups, cols) if starts is not None else (cols,)
    s["post_weight"] = (1 + 0.2 * rand(cols)).to(vec) if case["post"] != "none" else None
    s["gate"] = (0.5 + 0.3 * rand(*per)).to(vec) if case["gate"] else None
    if case["mod"] == "ada":
        s["mul"], s["add"] = (0.2 * rand(*per)).to(vec), (0.3 * rand(*per)).to(vec)
    else:
        s["mul"], s["add"] = (1 + 0.2 * rand(cols)).to(vec), None
    zeros = lambda *z: torch.zeros(*z, dtype=dtype, device=DEV)  # noqa: E731
    x = _activations(rand, rows, cols).to(dtype)
    y = _activations(rand, rows, cols).to(dtype) if case["branch"] else None
    saves_y = case["branch"] and (case["post"] != "none" or case["gate"])
    s["h_code"], s["h_rstd"] = torch.zeros(rows, cols, dtype=E4M3, device=DEV), torch.zeros(rows, device=DEV)
    s.update(y_code=None, y_scale=None, y_rstd=None)
    if saves_y:
        s["y_code"], s["y_scale"] = _empty_code(rows, cols)
        if case["post"] != "none":
            s["y_scale"], s["y_rstd"] = None, torch.zeros(rows, device=DEV)
    if case["op"] == "norm_fwd":
        s.update(x=x, y=y, h=zeros(rows, cols) if case["branch"] else None, n=zeros(rows, cols))
    else:
        if case["branch"]:
            v = y
            if case["post"] != "none":
                v, s["y_rstd"] = _norm(y.float(), case["post"], EPS_POST)
                s["y_code"] = v.to(E4M3)
            elif saves_y:
                s["y_code"], s["y_scale"] = _encode(y)
            x = x.float() + v.float()
        hat, s["h_rstd"] = _norm(x.float(), case["pre"], EPS_PRE)
        s["h_code"] = hat.to(E4M3)
        s["dn"] = rand(rows, cols).mul_(1e-2).to(dtype)
        s["dh"] = rand(rows, cols).mul_(1e-2).to(dtype)
        s["dx"], s["dy"] = zeros(rows, cols), zeros(rows, cols) if case["branch"] else None
        for k in ("post_weight", "gate", "mul", "add"):
            s["d_" + k] = None if s[k] is None else torch.zeros(s[k].shape, device=DEV)
    if own:
        ps = s["ps"]
        kind = {"none": ps.NORM_NONE, "rms": ps.NORM_RMS, "layer": ps.NORM_LAYER}
        s["norm"] = ps.BlockNorm(pre_norm=kind[case["pre"]], pre_eps=EPS_PRE, post_norm=kind[case["post"]],
                                 post_eps=EPS_POST, residual_scale=case["alpha"], branch_scale=case["beta"],
                                 post_weight=s["post_weight"], gate=s["gate"], mul=s["mul"], add=s["add"],
                                 mul_plus_one=case["mod"] == "ada", segments=s["starts"])
        if case["op"] == "norm_bwd":
            size = ps.block_norm_workspace_size(s["norm"], rows, cols)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


def _prepare_wgrad(s, case, rand):
    t, n, k = case["tokens"], case["out"], case["inp"]
    s["dy"] = rand(t, n).mul_(torch.exp(0.5 * rand(t, 1))).mul_(1e-2).to(DT[case["type"]])
    x = _activations(rand, t, k)
    s.update(mul=None, add=None, scale=None)
    if case["saved"] == "norm":
        s["code"] = _norm(x, "rms", EPS_PRE)[0].to(E4M3)
        s["mul"] = 1 + 0.2 * rand(k)
    else:
        s["code"], s["scale"] = _encode(x)
    s["dw"] = torch.zeros(n, k, dtype=DT[case["grad"]], device=DEV)
    s["db"] = torch.zeros(n, device=DEV) if case["bias"] else None
    if own:
        ps = s["ps"]
        s["workspace"] = torch.empty(ps.linear_wgrad_workspace_size(t, n, k), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"encode": _run_encode, "decode": _run_decode, "norm_fwd": _run_norm_fwd, "norm_bwd": _run_norm_bwd,
            "glu_fwd": _run_glu_fwd, "glu_bwd": _run_glu_bwd, "wgrad": _run_wgrad}[s["case"]["op"]](s)


def _run_encode(s):
    if own:
        s["ps"].encode_act(s["x"], s["code"], s["scale"])
    else:
        code, scale = _encode(s["x"])
        s["code"].copy_(code)
        s["scale"].copy_(scale)
    return s["code"], s["scale"]


def _run_decode(s):
    if own:
        s["ps"].decode_act(s["code"], s["scale"], s["x"])
    else:
        s["x"].copy_(_decode(s["code"], s["scale"]))
    return s["x"]


def _run_glu_fwd(s):
    (a, *b), ((a_code, a_scale), *b_saved) = s["x"], s["codes"]
    b = b[0] if b else None
    b_code, b_scale = b_saved[0] if b_saved else (None, None)
    if own:
        s["ps"].glu_forward(a, s["out"], s["act"], a_code=a_code, a_scale=a_scale, b=b, b_code=b_code, b_scale=b_scale)
    else:
        f, _ = _act(s["case"]["act"], a.float())
        s["out"].copy_(f if b is None else f * b.float())
        for x, code, scale in [(a, a_code, a_scale), (b, b_code, b_scale)][:len(s["x"])]:
            c, sc = _encode(x)
            code.copy_(c)
            scale.copy_(sc)
    return s["out"], s["codes"]


def _run_glu_bwd(s):
    (da, *db), ((a_code, a_scale), *b_saved) = s["x"], s["codes"]
    db = db[0] if db else None
    b_code, b_scale = b_saved[0] if b_saved else (None, None)
    if own:
        s["ps"].glu_backward(s["dout"], s["act"], a_code, a_scale, da, b_code=b_code, b_scale=b_scale, db=db,
                             out=s["out"])
    else:
        g = s["dout"].float()
        f, slope = _act(s["case"]["act"], _decode(a_code, a_scale))
        if db is not None:
            b = _decode(b_code, b_scale)
            db.copy_(g * f)
            g, f = g * b, f * b
        da.copy_(g * slope)
        if s["out"] is not None:
            s["out"].copy_(f)
    return {"dx": s["x"], "out": s["out"]}


def _run_wgrad(s):
    if own:
        s["ps"].linear_wgrad(s["dy"], s["code"], s["dw"], scale=s["scale"], db=s["db"], mul=s["mul"],
                             workspace=s["workspace"])
    else:
        g = s["dy"].float()
        x = s["code"].float() if s["scale"] is None else _decode(s["code"], s["scale"])
        if s["mul"] is not None:
            x = x * s["mul"]
        s["dw"].copy_(g.t() @ x)
        if s["db"] is not None:
            s["db"].copy_(g.sum(0))
    return {"dw": s["dw"], "db": s["db"]}


def _run_norm_fwd(s):
    if own:
        s["ps"].block_norm_forward(s["norm"], s["x"], s["n"], y=s["y"], h=s["h"], h_code=s["h_code"],
                                   h_rstd=s["h_rstd"], y_code=s["y_code"], y_scale=s["y_scale"], y_rstd=s["y_rstd"])
    else:
        _norm_forward(s)
    return {k: s[k] for k in ("h", "n", "h_code", "h_rstd", "y_code", "y_scale", "y_rstd")}


def _run_norm_bwd(s):
    if own:
        s["ps"].block_norm_backward(s["norm"], s["dn"], s["h_code"], s["h_rstd"], s["dx"], dh=s["dh"], dy=s["dy"],
                                    y_code=s["y_code"], y_scale=s["y_scale"], y_rstd=s["y_rstd"],
                                    d_post_weight=s["d_post_weight"], d_gate=s["d_gate"], d_mul=s["d_mul"],
                                    d_add=s["d_add"], workspace=s["workspace"])
    else:
        _norm_backward(s)
    return {k: s[k] for k in ("dx", "dy", "d_post_weight", "d_gate", "d_mul", "d_add")}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _blocks(x):
    """x [rows, cols] as [rows, blocks, 128], the last block filled up with zeros."""
    rows, cols = x.shape
    y = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=x.dtype, device=x.device)
    y[:, :cols] = x
    return y.view(rows, -1, BLOCK)


def _encode(x):
    """Codes, and for each block the smallest power of two s with max |x| <= 448 s (and s >= 2^-126)."""
    y = _blocks(x.float())
    top = y.abs().amax(2)
    e = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp_min(1)
    code = (y * ((254 - e) << 23).view(torch.float32)[:, :, None]).to(E4M3)
    return code.view(x.shape[0], -1)[:, :x.shape[1]].contiguous(), (e << 23).view(torch.float32)


def _decode(code, scale):
    return code.float() * scale.repeat_interleave(BLOCK, 1)[:, :code.shape[1]]


def _act(name, a):
    """The activation and its slope."""
    if name == "silu":
        r = 1 / (1 + torch.exp(-a))
        return a * r, r * (1 + a * (1 - r))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * p, p + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * (c * (1 + 3 * 0.044715 * a * a))


def _norm(x, kind, eps):
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(x.square().mean(1) + eps)
    return x * r[:, None], r


def _norm_back(g, hat, r, kind):
    """Gradient of a norm's input from that of its normalised values."""
    d = g - hat * (g * hat).mean(1, keepdim=True)
    return r[:, None] * (d - g.mean(1, keepdim=True) if kind == "layer" else d)


def _by_row(s, v, dtype=torch.float32):
    """A vector, or a sequence's vector for each of its rows."""
    return v.to(dtype) if v.dim() == 1 else v.to(dtype)[s["seg"]]


def _sums(s, like, x):
    """Sums over the rows, or over each sequence's."""
    if like.dim() == 1:
        return x.sum(0)
    own_rows = torch.arange(s["groups"], device=DEV)[:, None] == s["seg"]
    return own_rows.to(x.dtype) @ x


def _norm_forward(s):
    case, u = s["case"], s["used"]
    h = s["x"][:u].float()
    if case["branch"]:
        v = s["y"][:u].float()
        if case["post"] != "none":
            v, r = _norm(v, case["post"], EPS_POST)
            s["y_code"][:u] = v.to(E4M3)
            s["y_rstd"][:u] = r
            v = v * s["post_weight"].float()
        elif case["gate"]:
            code, scale = _encode(s["y"][:u])
            s["y_code"][:u] = code
            s["y_scale"][:u] = scale
        if case["gate"]:
            v = v * _by_row(s, s["gate"])
        h = case["alpha"] * h + case["beta"] * v
        s["h"][:u] = h
    hat, r = _norm(h, case["pre"], EPS_PRE)
    s["h_code"][:u] = hat.to(E4M3)
    s["h_rstd"][:u] = r
    mul = _by_row(s, s["mul"])
    n = hat * (1 + mul if case["mod"] == "ada" else mul)
    s["n"][:u] = n + _by_row(s, s["add"]) if s["add"] is not None else n


def _norm_backward(s):
    case, u = s["case"], s["used"]
    dn, hat = s["dn"][:u].float(), s["h_code"][:u].float()
    mul = _by_row(s, s["mul"])
    s["d_mul"].copy_(_sums(s, s["mul"], dn * hat))
    if s["add"] is not None:
        s["d_add"].copy_(_sums(s, s["add"], dn))
    g = dn * (1 + mul if case["mod"] == "ada" else mul)
    g = s["dh"][:u].float() + _norm_back(g, hat, s["h_rstd"][:u], case["pre"])
    if not case["branch"]:
        s["dx"][:u] = g
        return
    s["dx"][:u] = case["alpha"] * g
    g = case["beta"] * g
    gate = _by_row(s, s["gate"]) if case["gate"] else 1.0
    if case["post"] == "none":
        if case["gate"]:
            s["d_gate"].copy_(_sums(s, s["gate"], g * _decode(s["y_code"][:u], s["y_scale"][:u])))
        s["dy"][:u] = g * gate
        return
    hat, w = s["y_code"][:u].float(), s["post_weight"].float()
    if case["gate"]:
        s["d_gate"].copy_(_sums(s, s["gate"], g * (hat * w)))
    s["d_post_weight"].copy_((g * gate * hat).sum(0))
    s["dy"][:u] = _norm_back(g * gate * w, hat, s["y_rstd"][:u], case["post"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _grid64(y):
    """y rounded to the values of e4m3: to the nearest, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _encode64(x):
    y = _blocks(x.double())
    scale = torch.exp2(torch.ceil(torch.log2((y.abs().amax(2) / 448).clamp_min(2.0 ** -126))))
    return _grid64(y / scale[:, :, None]).view(x.shape[0], -1)[:, :x.shape[1]], scale


def _value64(code, scale):
    column = torch.arange(code.shape[1], device=DEV) // BLOCK
    return code.double() if scale is None else code.double() * scale.double()[:, column]


def _act64(name, a):
    if name == "silu":
        return a / (1 + torch.exp(-a)), (1 + torch.exp(-a) + a * torch.exp(-a)) / (1 + torch.exp(-a)) ** 2
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-a / 2 ** 0.5)
        return a * cdf, cdf + a * torch.exp(-a * a / 2) / (2 * math.pi) ** 0.5
    u = (2 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3)
    p = 1 / (1 + torch.exp(-2 * u))         # (1 + tanh u) / 2
    return a * p, p + 2 * a * p * (1 - p) * (2 / math.pi) ** 0.5 * (1 + 0.134145 * a ** 2)


def _norm64(x, kind, eps):
    if kind == "layer":
        return (x - x.mean(1, keepdim=True)) / (x.var(1, keepdim=True, correction=0) + eps).sqrt(), \
            (x.var(1, correction=0) + eps) ** -0.5
    return x / ((x * x).mean(1, keepdim=True) + eps).sqrt(), ((x * x).mean(1) + eps) ** -0.5


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode":
        return _encode64(s["x"])
    if op == "decode":
        return _value64(s["code"], s["scale"])
    if op == "glu_fwd":
        f = _act64(case["act"], s["x"][0].double())[0]
        return f * s["x"][1].double() if case["gated"] else f, [_encode64(x) for x in s["x"]]
    if op == "glu_bwd":
        g = s["dout"].double()
        f, slope = _act64(case["act"], _value64(*s["codes"][0]))
        b = _value64(*s["codes"][1]) if case["gated"] else 1.0
        return {"dx": [g * slope * b] + ([g * f] if case["gated"] else []), "out": f * b if case["again"] else None}
    if op == "wgrad":
        g = s["dy"].double()
        dw = g.t() @ _value64(s["code"], s["scale"])
        return {"dw": dw if s["mul"] is None else dw * s["mul"].double(), "db": g.sum(0) if case["bias"] else None}
    return _norm_forward64(s) if op == "norm_fwd" else _norm_backward64(s)


def _whole(s, x):
    """x with zeros for the rows behind the last sequence."""
    return None if x is None else torch.cat([x, x.new_zeros(s["case"]["rows"] - x.shape[0], *x.shape[1:])])


def _norm_forward64(s):
    case, u = s["case"], s["used"]
    vec = lambda k: 1.0 if s[k] is None else _by_row(s, s[k], torch.float64)  # noqa: E731
    h, out = s["x"][:u].double(), dict.fromkeys(("h", "y_code", "y_scale", "y_rstd"))
    if case["branch"]:
        y = s["y"][:u].double()
        if case["post"] != "none":
            y, out["y_rstd"] = _norm64(y, case["post"], EPS_POST)
            out["y_code"] = _grid64(y)
        elif case["gate"]:
            out["y_code"], out["y_scale"] = _encode64(s["y"][:u])
        h = out["h"] = case["alpha"] * h + case["beta"] * vec("gate") * vec("post_weight") * y
    hat, out["h_rstd"] = _norm64(h, case["pre"], EPS_PRE)
    out["h_code"] = _grid64(hat)
    n = hat * (vec("mul") + (case["mod"] == "ada"))
    out["n"] = n if s["add"] is None else n + vec("add")
    return {k: _whole(s, v) for k, v in out.items()}


def _norm_backward64(s):
    case, u = s["case"], s["used"]
    vec = lambda k: 1.0 if s[k] is None else _by_row(s, s[k], torch.float64)  # noqa: E731
    out = dict.fromkeys(("dx", "dy", "d_post_weight", "d_gate", "d_mul", "d_add"))

    def sums(k, x):
        if s[k].dim() == 1:
            return x.sum(0)
        return torch.zeros(s["groups"], x.shape[1], dtype=x.dtype, device=DEV).index_add_(0, s["seg"], x)

    def back(g, hat, r, kind):
        c = case["cols"]
        total = (g * hat).sum(1, keepdim=True) * hat + (g.sum(1, keepdim=True) if kind == "layer" else 0)
        return (g - total / c) * r.double()[:, None]
    dn, hat = s["dn"][:u].double(), s["h_code"][:u].double()
    out["d_mul"] = sums("mul", dn * hat)
    if s["add"] is not None:
        out["d_add"] = sums("add", dn)
    g = back(dn * (vec("mul") + (case["mod"] == "ada")), hat, s["h_rstd"][:u], case["pre"]) + s["dh"][:u].double()
    dx, dy = g, None
    if case["branch"]:
        dx, dv = case["alpha"] * g, case["beta"] * g
        dy = dv * vec("gate") * vec("post_weight")
        if s["y_code"] is not None:
            hat = _value64(s["y_code"][:u], None if s["y_scale"] is None else s["y_scale"][:u])
            if case["gate"]:
                out["d_gate"] = sums("gate", dv * hat * vec("post_weight"))
            if case["post"] != "none":
                out["d_post_weight"] = (dv * hat * vec("gate")).sum(0)
                dy = back(dy, hat, s["y_rstd"][:u], case["post"])
    out["dx"], out["dy"] = _whole(s, dx), _whole(s, dy)
    return out
