"""The measured operators: one AdamW step over many tensors with 32-bit or with
8-bit (e4m3) moments, the global gradient norm that clips it, and the codec of
the 8-bit moments.

A case of the step holds the parameters of a small language model (embedding,
attention and feed-forward matrices, norm vectors) or of low-rank adapters. All
tensors of one kind of state lie in one array, each tensor at a multiple of 256
elements, so a moment block of 256 elements never crosses a tensor and the plain
form works on [blocks, 256] views. Matrices are in hyperparameter group 0 (weight
decay), vectors in group 1 (none).

`own = False` computes the operators in elementary torch operations, `own = True`
through precision_state_amd.
"""
import math

import torch

own = False

BLOCK = 256
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "": 0}
LR, BETA1, BETA2, EPS, DECAY, PSI, MAX_NORM = 2e-4, 0.9, 0.999, 1e-8, 0.1, 4e-3, 1.0
GOLDEN = 0x9E3779B97F4A7C15
MOST_PARAMS = 520_000_000

# op: step (m, v in 32 bits: state f32; in 8 bits: state e4m3), norm, encode, decode
# param: f32 (a master weight, with a 16-bit copy if `copy` names its type), bf16 with a 16-bit residual
#   (split trunc), or bf16 alone, rounded stochastically (split stochastic)
# round: how the second moment's e4m3 code is rounded
# clip: the gradient norm first, its clip factor in the step
STEP = dict(op="step", state="f32", param="f32", grad="bf16", copy="", split="trunc", algo="adam", round="nearest",
            clip=False, kind="model", layers=1, d=64, f=128, vocab=0, rank=0, step=100)


def listed():
    return [
        # fine-tuning low-rank adapters: 64 small fp32 tensors, the step is one short launch
        dict(STEP, name="step32_adapters", kind="adapter", layers=8, d=512, rank=8, grad="f32"),
        # one large transformer layer with fp32 master weights and the bf16 copy that the model runs on
        dict(STEP, name="step32_layer", d=4096, f=11008, copy="bf16"),
        # odd widths: rows and tensor ends that no vector width divides; fp16 gradients and copy
        dict(STEP, name="step32_odd", layers=3, d=1001, f=2731, vocab=5003, grad="f16", copy="f16"),
        # a whole small model with its embedding, clipped, as one training step ends
        dict(STEP, name="step32_model_clipped", layers=8, d=2048, f=5632, vocab=50304, copy="bf16", clip=True),
        # adapters again, bf16 weights with residuals and 8-bit moments
        dict(STEP, name="step8_adapters", state="e4m3", kind="adapter", layers=8, d=512, rank=8, param="bf16"),
        # odd widths, Nesterov momentum, no residual: weights and second moment rounded stochastically
        dict(STEP, name="step8_odd", state="e4m3", layers=3, d=1001, f=2731, vocab=5003, param="bf16",
             split="stochastic", algo="nadam", round="stochastic"),
        # one layer, fp32 master weights and bf16 copy, clipped
        dict(STEP, name="step8_layer_clipped", state="e4m3", d=4096, f=11008, copy="bf16", round="stochastic",
             clip=True),
        # the whole small model in the framework's own weight format
        dict(STEP, name="step8_model", state="e4m3", layers=8, d=2048, f=5632, vocab=50304, param="bf16"),
        # the norm alone: one odd small model, and the whole small model's fp32 gradients
        dict(STEP, name="norm_odd", op="norm", layers=3, d=1001, f=2731, vocab=5003, clip=True),
        dict(STEP, name="norm_model", op="norm", layers=8, d=2048, f=5632, vocab=50304, grad="f32", clip=True),
        # moving a run's moments into 8 bits and back: a large second moment, a small first moment
        dict(op="encode", name="encode_large", signed=False, n=150_000_001),
        dict(op="decode", name="decode_small", signed=True, n=1_000_003),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "step", "step", "step", "norm", "encode", "decode"])
    if op in ("encode", "decode"):
        return dict(op=op, signed=rng.random() < 0.5, n=_log(rng, 1, 150_000_000))
    while True:
        c = dict(STEP, op=op, layers=rng.randint(1, 8), d=_log(rng, 16, 4096), step=_log(rng, 1, 20000))
        c["f"] = int(c["d"] * rng.uniform(1.5, 4.0))
        if rng.random() < 0.3:
            c.update(kind="adapter", rank=rng.randint(1, 64), vocab=0)
        elif rng.random() < 0.5:
            c["vocab"] = _log(rng, 100, 60000)
        if sum(_sizes(c)[0]) <= MOST_PARAMS:
            break
    c["grad"] = rng.choice(["bf16", "f16", "f32"])
    c["clip"] = op == "norm" or rng.random() < 0.4
    if op == "step":
        c["state"] = rng.choice(["f32", "e4m3"])
        c["algo"] = rng.choice(["adam", "adam", "nadam"])
        c["param"] = rng.choice(["f32", "bf16"])
        if c["param"] == "f32":
            c["copy"] = rng.choice(["", "bf16", "f16"])
        else:
            c["split"] = rng.choice(["trunc", "stochastic"])
        if c["state"] == "e4m3":
            c["round"] = rng.choice(["nearest", "stochastic"])
    return c


def _sizes(c):
    """Element counts of the case's tensors, and the group of each."""
    d, f = c["d"], c["f"]
    if c["kind"] == "adapter":
        layer = [(c["rank"] * d, 0)] * 8
    else:
        layer = [(d * d, 0)] * 4 + [(d * f, 0)] * 3 + [(d, 1)] * 2
    t = ([(c["vocab"] * d, 0)] if c["vocab"] else []) + layer * c["layers"] + ([(d, 1)] if c["kind"] == "model" else [])
    return [n for n, _ in t], [g for _, g in t]


def work(case):
    if case["op"] in ("encode", "decode"):
        n = case["n"]
        return {"bytes": 5 * n + 4 * (-(-n // BLOCK)), "flops": 4 * n}
    sizes = _sizes(case)[0]
    n, nb = sum(sizes), sum(-(-k // BLOCK) for k in sizes)
    g = SIZE[case["grad"]] * n
    if case["op"] == "norm":
        return {"bytes": g + 8, "flops": 2 * n}
    w = 4 if case["param"] == "f32" or case["split"] == "trunc" else 2
    moments = 16 * n if case["state"] == "f32" else 4 * n + 16 * nb
    return {"bytes": g + 2 * w * n + SIZE[case["copy"]] * n + moments + (8 if case["clip"] else 0),
            "flops": (20 if case["state"] == "f32" else 30) * n + (2 * n if case["clip"] else 0)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _e4m3(x):
    """Some 8-bit moments of x [blocks, 256] to start from: codes, and a power of two for each block."""
    top = x.abs().amax(1, keepdim=True).clamp_min(1e-30)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn), scale.flatten()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    s = dict(case=case, seed=seed)
    if case["op"] in ("encode", "decode"):
        n = case["n"]
        nb = -(-n // BLOCK)
        x = torch.randn(nb, BLOCK, device=DEV, generator=gen).mul_(torch.exp(3 * rand(nb, 1))).mul_(1e-3)
        x = x if case["signed"] else x.square_()
        if case["op"] == "encode":
            s.update(x=x.flatten()[:n], code=torch.zeros(n, dtype=torch.float8_e4m3fn, device=DEV),
                     scale=torch.zeros(nb, device=DEV))
        else:
            code, scale = _e4m3(x if case["signed"] else x.sqrt_())
            s.update(code=code.flatten()[:n], scale=scale, x=torch.zeros(n, device=DEV))
        if own:
            import precision_state_amd as ps
            s.update(ps=ps, kind=ps.MOMENT_SIGNED if case["signed"] else ps.MOMENT_UNSIGNED)
        return s

    sizes, groups = _sizes(case)
    blocks = torch.tensor([-(-n // BLOCK) for n in sizes], device=DEV)
    nb = int(blocks.sum())
    first = torch.cumsum(blocks, 0) - blocks
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), blocks)   # of each block
    index = torch.arange(nb, device=DEV) - first[tensor]                             # of the block in its tensor
    left = torch.tensor(sizes, device=DEV)[tensor] - index * BLOCK
    inside = torch.arange(BLOCK, device=DEV) < left[:, None]
    group = torch.tensor(groups, device=DEV)[tensor]

    level = torch.exp(rand(nb, 1))                   # gradients differ in size from row to row
    level[rand(nb, 1) > 2.3] = 0.0                   # rows of tokens that the batch does not hold
    mask = lambda x: x.mul_(inside)                  # noqa: E731
    grad = mask(rand(nb, BLOCK).mul_(level).mul_(1e-3)).to(DT[case["grad"]])
    s.update(grad=grad, tensor=tensor, index=index, group=group, n_tensors=len(sizes))
    if case["op"] == "step":
        w = mask(rand(nb, BLOCK).mul_(0.02))
        if case["param"] == "f32":
            s["w"] = w
            s["copy"] = torch.zeros(nb, BLOCK, dtype=DT[case["copy"]], device=DEV) if case["copy"] else None
        else:
            bits = w.view(torch.int32)
            s["hi"] = (bits >> 16).to(torch.int16).view(torch.bfloat16)
            s["lo"] = (bits & 0xFFFF).to(torch.int16) if case["split"] == "trunc" else None
        m = mask(rand(nb, BLOCK).mul_(level).mul_(3e-4))
        v = mask(rand(nb, BLOCK).square_().add_(0.5).mul_(level.square()).mul_(1e-6))
        if case["state"] == "f32":
            s.update(m=m, v=v, ms=None, vs=None)
        else:
            s["m"], s["ms"] = _e4m3(m)
            s["v"], s["vs"] = _e4m3(v.sqrt_())
    if own:
        import precision_state_amd as ps
        starts = (first * BLOCK).tolist()
        flat = {k: s[k].view(-1) for k in ("w", "hi", "lo", "copy", "grad", "m", "v") if s.get(k) is not None}
        cut = lambda k, o, n: flat[k][o:o + n] if k in flat else None  # noqa: E731
        scales = lambda k, o, n: s[k][o // BLOCK:(o + n + BLOCK - 1) // BLOCK] if s.get(k) is not None else None  # noqa: E731
        if case["op"] == "norm":
            tensors = [ps.AdamWTensor(None, cut("grad", o, n)) for o, n in zip(starts, sizes)]
        else:
            tensors = [ps.AdamWTensor(cut("w", o, n) if "w" in flat else cut("hi", o, n), cut("grad", o, n),
                                      cut("m", o, n), cut("v", o, n), scales("ms", o, n), scales("vs", o, n),
                                      residual=cut("lo", o, n), copy=cut("copy", o, n), group=g)
                       for o, n, g in zip(starts, sizes, groups)]
        s["plan"] = ps.AdamWPlan(tensors)
        s["groups"] = [ps.HParams(algo=ps.ALGO_ADAM if case["algo"] == "adam" else ps.ALGO_NADAM,
                                  split_mode=ps.SPLIT_TRUNC if case["split"] == "trunc" else ps.SPLIT_STOCHASTIC,
                                  lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=wd, momentum_decay=PSI,
                                  seed=seed) for wd in (DECAY, 0.0)]
        s["rounding"] = ps.ROUND_NEAREST if case["round"] == "nearest" else ps.ROUND_STOCHASTIC
    return s


def run(s):
    case = s["case"]
    if case["op"] == "encode":
        if own:
            s["ps"].encode_fp8(s["x"], s["code"], s["scale"], s["kind"])
            return s["code"], s["scale"]
        return _encode(s)
    if case["op"] == "decode":
        if own:
            s["ps"].decode_fp8(s["code"], s["scale"], s["x"], s["kind"])
            return s["x"]
        return _decode(s)
    if own:
        plan = s["plan"]
        if case["clip"]:
            plan.grad_norm(max_norm=MAX_NORM)
        if case["op"] == "norm":
            return plan.norm, plan.grad_mul
        plan.step(s["groups"], case["step"], clipped=case["clip"], rounding=s["rounding"])
        return _state(s, plan.norm if case["clip"] else None)
    norm, mul = _norm(s["grad"]) if case["clip"] else (None, None)
    if case["op"] == "norm":
        return norm, mul
    _step(s, mul)
    return _state(s, norm)


def _state(s, norm):
    return {k: v for k, v in dict(w=s.get("w"), hi=s.get("hi"), lo=s.get("lo"), copy=s.get("copy"), m=s["m"], v=s["v"],
                                  ms=s["ms"], vs=s["vs"], norm=norm).items() if v is not None}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _norm(grad):
    """The 2-norm of all gradients and the factor that brings it down to MAX_NORM."""
    norm = grad.double().square().sum().sqrt()
    return norm.float(), (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()


def _block_scale(top):
    """The smallest power of two s with top <= 448 s (and s >= 2^-126), from the bits of top; and 1 / s."""
    e = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp_min(1)
    return (e << 23).view(torch.float32), ((254 - e) << 23).view(torch.float32)


def _scalars(case, decay):
    """The update's scalars in double, [group] values for the weight decay."""
    t, b1, b2 = case["step"], BETA1, BETA2
    k = dict(b1=b1, c1=1 - b1, b2=b2, c2=1 - b2, a=LR / (1 - b1 ** t), rs2=1 / math.sqrt(1 - b2 ** t),
             cwd=[LR * x for x in decay])
    if case["algo"] == "nadam":
        mu = lambda i: b1 * (1 - 0.5 * 0.96 ** (i * PSI))  # noqa: E731
        p = math.prod(mu(i) for i in range(1, min(t, 2000) + 1))
        k.update(ag=LR * (1 - mu(t)) / (1 - p), am=LR * mu(t + 1) / (1 - p * mu(t + 1)))
    return k


def _mix(z):
    """SplitMix64's output function on int64 (multiplications wrap, shifts are logical)."""
    c1, c2 = 0xBF58476D1CE4E5B9 - (1 << 64), 0x94D049BB133111EB - (1 << 64)
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * c1
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * c2
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _bits16(s, high):
    """The random 16 bits of every element, [blocks, 256], in 0 .. 65535: element e of tensor i takes bits
    16 (e mod 4) .. of output e / 4 of the stream of (seed, step, i); `high`: the streams of i + 2^31."""
    i = torch.arange(s["n_tensors"], device=DEV) | (1 << 31 if high else 0)
    start = _mix(s["seed"] ^ _mix((s["case"]["step"] << 32) | i))
    at = s["index"][:, None] * (BLOCK // 4) + torch.arange(1, BLOCK // 4 + 1, device=DEV)
    z = _mix(start[s["tensor"]][:, None] + at * (GOLDEN - (1 << 64)))
    return ((z[:, :, None] >> torch.tensor([0, 16, 32, 48], device=DEV)) & 0xFFFF).view(-1, BLOCK)


def _second_code(r, inv, bits):
    """sqrt(v) times 1 / scale as e4m3; a value above zero stays above zero."""
    y = r * inv
    if bits is not None:      # random bits below the last kept place, then cut there
        small = y < 2 ** -6   # below the smallest normal value the places stay those of 2^-6
        z = torch.where(small, y + 2 ** -6, y).view(torch.int32) + (bits << 4).to(torch.int32)
        z = (z & -0x100000).view(torch.float32)
        y = torch.where(small, z - 2 ** -6, z)
    return torch.where(r > 0, y.clamp_min(2 ** -9), y).to(torch.float8_e4m3fn)


def _step(s, mul):
    case = s["case"]
    k = _scalars(case, (DECAY, 0.0))
    g = s["grad"].float()
    if mul is not None:
        g = g * mul
    if case["param"] == "f32":
        w = s["w"]
    else:
        w = s["hi"].view(torch.int16).to(torch.int32) << 16
        w = (w if s["lo"] is None else w | (s["lo"].to(torch.int32) & 0xFFFF)).view(torch.float32)
    if case["state"] == "f32":
        m, v = s["m"], s["v"]
    else:
        m = s["m"].float() * s["ms"][:, None]
        v = (s["v"].float() * s["vs"][:, None]).square()
    m = m * k["b1"] + g * k["c1"]
    v = v * k["b2"] + (g * g) * k["c2"]
    r = v.sqrt()
    d = r * k["rs2"] + EPS
    u = (m / d) * k["a"] if case["algo"] == "adam" else (g * k["ag"] + m * k["am"]) / d
    u = u + w * torch.tensor(k["cwd"], device=DEV)[s["group"]][:, None]
    w = w - u
    if case["param"] == "f32":
        s["w"].copy_(w)
        if case["copy"]:
            s["copy"].copy_(w)
    else:
        b = w.view(torch.int32)
        if case["split"] == "trunc":
            s["lo"].copy_(b)
        else:
            b = b + _bits16(s, False).to(torch.int32)
        s["hi"].view(torch.int16).copy_(b >> 16)
    if case["state"] == "f32":
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        ms, inv_m = _block_scale(m.abs().amax(1))
        vs, inv_v = _block_scale(r.amax(1))
        s["m"].copy_((m * inv_m[:, None]).to(torch.float8_e4m3fn))
        s["v"].copy_(_second_code(r, inv_v[:, None], _bits16(s, True) if case["round"] == "stochastic" else None))
        s["ms"].copy_(ms)
        s["vs"].copy_(vs)


def _blocks(x):
    n = x.numel()
    y = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=x.dtype, device=x.device)
    y[:n] = x
    return y.view(-1, BLOCK)


def _encode(s):
    n, x = s["x"].numel(), _blocks(s["x"])
    x = x if s["case"]["signed"] else x.sqrt()
    scale, inv = _block_scale(x.abs().amax(1))
    code = (x * inv[:, None]).to(torch.float8_e4m3fn) if s["case"]["signed"] else _second_code(x, inv[:, None], None)
    s["code"].copy_(code.view(-1)[:n])
    s["scale"].copy_(scale)
    return s["code"], s["scale"]


def _decode(s):
    x = s["code"].float() * s["scale"].repeat_interleave(BLOCK)[:s["code"].numel()]
    s["x"].copy_(x if s["case"]["signed"] else x.square())
    return s["x"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _scale64(top):
    return torch.exp2(torch.ceil(torch.log2((top / 448).clamp_min(2.0 ** -126))))


def _grid64(y, bits=None):
    """y rounded to the values of e4m3: to the nearest, ties to even, or by the random 16 bits."""
    a = y.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    q = torch.round(a / step) if bits is None else torch.floor(a / step + bits.double() / 65536)
    return (q * step).copysign(y)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        n = case["n"]
        x = s["code"].double() * s["scale"].double()[torch.arange(n, device=DEV) // BLOCK]
        return x if case["signed"] else x * x
    if case["op"] == "encode":
        n = case["n"]
        x = _blocks(s["x"]).double()
        x = x if case["signed"] else x ** 0.5
        scale = _scale64(x.abs().amax(1))
        q = _grid64(x / scale[:, None])
        if not case["signed"]:
            q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
        return q.view(-1)[:n], scale
    g, norm = s["grad"].double(), None
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        g = g * min(1.0, MAX_NORM / (float(norm) + 1e-6))
        if case["op"] == "norm":
            return norm, torch.tensor(min(1.0, MAX_NORM / (float(norm) + 1e-6)), dtype=torch.float64)
    t, out = case["step"], {"norm": norm}
    if case["param"] == "f32":
        w = s["w"].double()
    else:
        w = s["hi"].double()
        if s["lo"] is not None:   # the residual's places: 2^-16 of the bf16 value's last place
            _, e = torch.frexp(w)
            place = torch.exp2((e - 8).clamp_min(-133).double()) * 2.0 ** -16
            w = (w.abs() + (s["lo"].to(torch.int64) & 0xFFFF).double() * place).copysign(w)
    if case["state"] == "f32":
        m, v = s["m"].double(), s["v"].double()
    else:
        m, v = s["m"].double() * s["ms"].double()[:, None], (s["v"].double() * s["vs"].double()[:, None]) ** 2
    m.mul_(BETA1).add_(g, alpha=1 - BETA1)
    v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    d = (v / (1 - BETA2 ** t)).sqrt_().add_(EPS)
    if case["algo"] == "adam":
        u = m / (1 - BETA1 ** t) / d
    else:
        mu = [BETA1 * (1 - 0.5 * 0.96 ** (i * PSI)) for i in range(1, t + 2)]
        p = math.prod(mu[:t])
        u = (m * (mu[t] / (1 - p * mu[t])) + g * ((1 - mu[t - 1]) / (1 - p))) / d
    del d, g
    u.add_(w * torch.tensor([DECAY, 0.0], dtype=torch.float64, device=DEV)[s["group"]][:, None])
    w = w.sub_(u, alpha=LR)
    del u
    if case["param"] == "f32":
        out.update(w=w, copy=w if case["copy"] else None)
    else:
        b = w.float().view(torch.int32)
        if case["split"] == "stochastic":
            b = b + _bits16(s, False).to(torch.int32)
        out.update(hi=(b & -0x10000).view(torch.float32).double(), lo=None)
    if case["state"] == "f32":
        out.update(m=m, v=v)
    else:
        r = v.sqrt_()
        ms, vs = _scale64(m.abs().amax(1)), _scale64(r.amax(1))
        y = _grid64(r / vs[:, None], _bits16(s, True) if case["round"] == "stochastic" else None)
        out.update(m=_grid64(m / ms[:, None]), v=torch.where(r > 0, y.clamp_min(2.0 ** -9), y), ms=ms, vs=vs)
    return out
