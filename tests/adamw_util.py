"""Device tensors of an AdamW plan with guard bytes around every array, and the
numpy state that steps along with them."""
import numpy as np

import adamw_ref as ref
import oracle

GUARD, FILL = 64, 0xA5


def torch():
    import torch as t
    return t


class Guarded:
    """A device array between guard bytes, from a numpy array."""

    def __init__(self, a, dtype):
        T = torch()
        raw = np.ascontiguousarray(a).view(np.uint8).reshape(-1)
        buf = np.full(raw.size + 2 * GUARD + (-raw.size) % 16, FILL, np.uint8)
        buf[GUARD:GUARD + raw.size] = raw
        self.buf, self.n = T.from_numpy(buf).cuda(), raw.size
        self.np_dtype = np.asarray(a).dtype
        self.t = self.buf[GUARD:GUARD + raw.size].view(dtype)

    def host(self):
        return self.buf.cpu().numpy()[GUARD:GUARD + self.n].view(self.np_dtype)

    def guards_intact(self):
        b = self.buf.cpu().numpy()
        return bool(np.all(b[:GUARD] == FILL) and np.all(b[GUARD + self.n:] == FILL))


def grad_bits(x, kind):
    """x as gradient array of the kind, and the float32 values it holds."""
    if kind == "f32":
        return x, x
    if kind == "f16":
        h = x.astype(np.float16)
        return h, h.astype(np.float32)
    b = ref.bf16_round(x)
    return b, ref.bf16_to_f32(b)


class Param:
    """One tensor: n, param "f32"/"bf16", grad "f32"/"bf16"/"f16", state "f32"/"e4m3", copy ""/"bf16"/"f16"."""

    def __init__(self, n, rng, param="f32", grad="bf16", state="f32", copy="", residual=True, group=0, index=0,
                 zero_state=False):
        T = torch()
        self.n, self.param, self.grad, self.state, self.copy, self.group, self.index = n, param, grad, state, copy, group, index
        w = rng.normal(0, 0.02, n).astype(np.float32)
        if param == "f32":
            self.w, self.lo = w, None
        else:
            u = w.view(np.uint32)
            self.w, self.lo = (u >> 16).astype(np.uint16), (u & 0xFFFF).astype(np.uint16) if residual else None
        m = np.zeros(n, np.float32) if zero_state else rng.normal(0, 3e-4, n).astype(np.float32)
        v = np.zeros(n, np.float32) if zero_state else (rng.normal(0, 1e-3, n) ** 2).astype(np.float32)
        if state == "f32":
            self.m, self.v, self.ms, self.vs = m, v, None, None
        elif zero_state:
            self.m, self.v = np.zeros(n, np.uint8), np.zeros(n, np.uint8)
            self.ms, self.vs = np.zeros(ref.blocks_of(n), np.float32), np.zeros(ref.blocks_of(n), np.float32)
        else:
            self.m, self.ms = ref.encode(m, True)
            self.v, self.vs = ref.encode(v, False)
        self.c = np.zeros(n, np.uint16) if copy else None
        self.set_grad(rng.normal(0, 1e-3, n).astype(np.float32))
        b16 = {"f32": T.float32, "bf16": T.bfloat16, "f16": T.float16}
        dev = lambda a, dt: None if a is None else Guarded(a, dt)  # noqa: E731
        self.d = dict(w=dev(self.w, b16[param]), lo=dev(self.lo, T.int16), c=dev(self.c, b16[copy or "bf16"]),
                      g=dev(self.gbits, b16[grad]), m=dev(self.m, T.float32 if state == "f32" else T.uint8),
                      v=dev(self.v, T.float32 if state == "f32" else T.uint8), ms=dev(self.ms, T.float32),
                      vs=dev(self.vs, T.float32))

    def set_grad(self, x):
        self.gbits, self.g = grad_bits(x, self.grad)

    def new_grad(self, x):
        """Another gradient into the device array."""
        T = torch()
        self.set_grad(x)
        raw = np.ascontiguousarray(self.gbits).view(np.uint8)
        d = self.d["g"]
        d.buf[GUARD:GUARD + d.n].copy_(T.from_numpy(raw.copy()))

    def tensor(self, ps):
        t = {k: (None if a is None else a.t) for k, a in self.d.items()}
        return ps.AdamWTensor(t["w"], t["g"], t["m"], t["v"], t["ms"], t["vs"], residual=t["lo"], copy=t["c"],
                              group=self.group)

    def weights(self, split):
        if self.param == "f32":
            return self.w
        if split == 2:
            return ref.bf16_to_f32(self.w)
        return oracle.join(self.w, self.lo, split)

    def moments(self):
        if self.state == "f32":
            return self.m, self.v
        return ref.decode(self.m, self.ms, True), ref.decode(self.v, self.vs, False)

    def random(self, seed, step, high):
        return oracle.sr_rand16(seed, step, self.index + ((1 << 31) if high else 0), 0, self.n)

    def step(self, hp, step, mul=1.0, rounding=0, coeffs=None):
        """The fp32 reference's step, bit-exact. hp: oracle.HParams of the group."""
        c = coeffs or oracle.coeffs(hp, step)
        m0, v0 = self.moments()
        w, m, v, r = ref.update(self.weights(hp.split_mode), self.g, m0, v0, c, mul, hp.algo == 1, np.float32)
        if self.param == "f32":
            self.w = w
            if self.copy:
                self.c = ref.bf16_round(w) if self.copy == "bf16" else w.astype(np.float16).view(np.uint16)
        elif hp.split_mode == 2:
            self.w = ((w.view(np.uint32) + self.random(hp.seed, step, False).astype(np.uint32)) >> 16).astype(np.uint16)
        else:
            self.w, self.lo = oracle.split(w, hp.split_mode)
        if self.state == "f32":
            self.m, self.v = m, v
        else:
            self.ms, self.vs = ref.block_scale(ref.per_block_max(m)), ref.block_scale(ref.per_block_max(r))
            self.m = ref.e4m3_code(m / ref.spread(self.ms, self.n))
            self.v = ref.second_code(r, ref.spread(self.vs, self.n), self.random(hp.seed, step, True) if rounding else None)

    def differences(self):
        """Arrays of the device that are not bit-equal to the numpy state, and broken guards."""
        host = dict(w=self.w, lo=self.lo, c=self.c, g=self.gbits, m=self.m, v=self.v, ms=self.ms, vs=self.vs)
        bad = []
        for k, d in self.d.items():
            if d is None:
                continue
            a, b = d.host().view(np.uint8), np.ascontiguousarray(host[k]).view(np.uint8)
            if not np.array_equal(a, b):
                at = np.flatnonzero(a != b)
                bad.append((k, self.n, f"{at.size} bytes, first at {at[0]}"))
            if not d.guards_intact():
                bad.append((k, self.n, "guard bytes"))
        return bad
