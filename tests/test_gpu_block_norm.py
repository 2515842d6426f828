"""GPU tests of the block norms against 64 bits (act_ref)."""
import dataclasses
import math

import pytest
import torch

import act_ref as ref
from act_util import DT, Padded, POISON, acts, codes, gen, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


KIND = {"none": 0, "rms": 1, "layer": 2}


class Case:
    """One norm with its inputs, outputs and reference."""

    def __init__(self, ps, rows, cols, dtype="bf16", vec=None, pre="rms", post="none", branch=True, gate=False, mul=True,
                 add=False, plus_one=False, starts=None, gate_seg=False, mod_seg=False, alpha=1.0, beta=1.0, pad=0,
                 offset=0.0, seed=0, weight=True):
        g = gen(seed + rows * 7 + cols)
        self.ps, self.rows, self.cols, self.dtype, self.pad = ps, rows, cols, dtype, pad
        vdt = DT[vec or dtype]
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        segs = len(starts) - 1 if starts is not None else 0
        row_seg = ref.segments(starts, rows)
        self.used = row_seg >= 0
        per = lambda by: (segs, cols) if by else (cols,)  # noqa: E731
        v = dict(w1=(1 + 0.2 * rand(cols)).to(vdt) if post != "none" and weight else None,
                 gate=(0.5 + 0.4 * rand(*per(gate_seg))).to(vdt) if gate else None,
                 mul=((0.0 if plus_one else 1.0) + 0.3 * rand(*per(mod_seg))).to(vdt) if mul else None,
                 add=(0.3 * rand(*per(mod_seg))).to(vdt) if add else None)
        self.c = dict(pre=pre, post=post, pre_eps=1e-6, post_eps=1e-5, alpha=alpha, beta=beta, plus_one=plus_one,
                      branch=branch, seg=row_seg[self.used], **{k: None if x is None else x.double() for k, x in v.items()})
        dev = {k: None if x is None else x.cuda() for k, x in v.items()}
        self.norm = ps.BlockNorm(pre_norm=KIND[pre], pre_eps=1e-6, post_norm=KIND[post], post_eps=1e-5, residual_scale=alpha,
                                 branch_scale=beta, post_weight=dev["w1"], gate=dev["gate"], mul=dev["mul"], add=dev["add"],
                                 mul_plus_one=plus_one,
                                 segments=None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda())
        self.v = v
        self.x = acts(g, rows, cols, dtype, 0.4) + offset
        self.y = acts(g, rows, cols, dtype, 0.4) + offset if branch else None
        self.x = self.x.to(DT[dtype])
        self.y = self.y.to(DT[dtype]) if branch else None
        self.dn, self.dh = acts(g, rows, cols, dtype, 0.3), acts(g, rows, cols, dtype, 0.3)
        self.saves_y = branch and (post != "none" or gate)

    def mat(self, fill=None, shift=0):
        return Padded(self.rows, self.cols, self.dtype, self.pad, shift, fill)

    def forward(self):
        rows, cols, post = self.rows, self.cols, self.c["post"] != "none"
        self.o = dict(n=self.mat(shift=1), h=self.mat() if self.y is not None else None)
        self.s = dict(h_code=codes(rows, cols), h_rstd=torch.full((rows,), POISON, device="cuda"))
        if self.saves_y:
            self.s["y_code"] = codes(rows, cols)
            if post:
                self.s["y_rstd"] = torch.full((rows,), POISON, device="cuda")
            else:
                self.s["y_scale"] = scales(rows, cols)
        x, y = self.mat(self.x), self.mat(self.y, 1) if self.y is not None else None
        self.ps.block_norm_forward(self.norm, x.m, self.o["n"].m, y=None if y is None else y.m,
                                   h=None if self.o["h"] is None else self.o["h"].m, **self.s)
        return self

    def check_forward(self):
        u = self.used
        want = ref.forward(self.c, self.x[u].double(), None if self.y is None else self.y[u].double())
        for name in ("n", "h"):
            if self.o[name] is not None:
                ref.check(self.o[name].m[u.cuda()], *want[name], name)
                assert self.o[name].outside_is_untouched()
                assert (self.o[name].m[~u.cuda()] == POISON).all()
        for name, hat in (("h", "h_hat"), ("y", "y_hat")):
            if f"{name}_rstd" in self.s:
                ref.check(self.s[f"{name}_rstd"][u.cuda()], *want[f"{name}_rstd"], name)
                assert (self.s[f"{name}_rstd"][~u.cuda()] == POISON).all()
                z, e = want[hat]
                got = ref.value(self.s[f"{name}_code"])[u]
                assert ((got - z).abs() <= torch.maximum(z.abs() * 2 ** -4, torch.tensor(2.0 ** -10)) + e).all(), name
        if "y_scale" in self.s:
            v, s = ref.encode(self.y[u].double())
            assert torch.equal(ref.value(self.s["y_code"])[u], v) and torch.equal(ref.dec(self.s["y_scale"])[u], s)
        for k in ("h_code", "y_code"):
            if k in self.s:
                assert (self.s[k].view(torch.uint8)[~u.cuda()] == 0x55).all()

    def grads(self, fill=POISON):
        return {f"d_{n}": torch.full(v.shape, fill, device="cuda")
                for n, v in (("post_weight", self.v["w1"]), ("gate", self.v["gate"]), ("mul", self.v["mul"]), ("add", self.v["add"]))
                if v is not None}

    def backward(self, with_dh=True, dx=None, dy=None, dh=None, dn=None, grads=None, **kw):
        self.dx, self.dy = dx or self.mat(), dy or (self.mat(shift=1) if self.y is not None else None)
        dn, dh = dn or self.mat(self.dn, 1), dh or (self.mat(self.dh) if with_dh else None)
        self.g = self.grads() if grads is None else grads
        self.ps.block_norm_backward(self.norm, dn.m, dx=self.dx.m, dh=None if dh is None else dh.m,
                                    dy=None if self.dy is None else self.dy.m, **self.s, **self.g, **kw)
        return self

    def want_backward(self, with_dh=True):
        u = self.used
        value = lambda k, sc=None: ref.value(self.s[k], self.s.get(sc))[u] if k in self.s else None  # noqa: E731
        return ref.backward(self.c, self.dn[u].double(), self.dh[u].double() if with_dh else None, value("h_code"),
                            ref.dec(self.s["h_rstd"])[u], value("y_code", "y_scale"),
                            ref.dec(self.s["y_rstd"])[u] if "y_rstd" in self.s else None)

    def check_backward(self, with_dh=True, base=0.0):
        u, want = self.used, self.want_backward(with_dh)
        for name, m in (("dx", self.dx), ("dy", self.dy)):
            if m is not None:
                ref.check(m.m[u.cuda()], *want[name], name)
                assert m.outside_is_untouched()
                assert (m.m[~u.cuda()] == POISON).all()
        for name, d in self.g.items():
            t, e = want[name]
            ref.check(d, t + base, e, name)


ADA = dict(pre="layer", gate=True, gate_seg=True, mod_seg=True, add=True, plus_one=True)
CASES = [
    dict(rows=1, cols=1), dict(rows=1, cols=8, branch=False), dict(rows=5, cols=512), dict(rows=9, cols=513, pad=3),
    dict(rows=3, cols=1024, branch=False, pre="layer", add=True), dict(rows=7, cols=1001, post="rms", beta=0.5, pad=1),
    dict(rows=11, cols=2048, post="layer", gate=True, alpha=1.5), dict(rows=4, cols=2049, gate=True),
    dict(rows=6, cols=4096, post="rms", vec="f32"), dict(rows=3, cols=5120, pre="layer", post="layer", mul=False),
    dict(rows=2, cols=8192, gate=True, beta=-0.25), dict(rows=3, cols=12289, post="rms", gate=True, pre="layer"),
    dict(rows=2, cols=16384, post="layer", pad=2), dict(rows=40, cols=136, post="rms", weight=False),
    dict(rows=37, cols=264, starts=[0, 10, 10, 31, 37], **ADA), dict(rows=50, cols=264, starts=[3, 4, 20, 45], **ADA),
    dict(rows=20, cols=130, starts=[0, 0, 0], **ADA), dict(rows=33, cols=520, starts=[0, 33], post="rms", **ADA),
    dict(rows=70, cols=72, starts=[0, 1, 2, 70], post="layer", gate=True, alpha=0.5),
    dict(rows=30, cols=640, starts=[0, 12, 29], gate=True, gate_seg=True, post="rms"),
    dict(rows=30, cols=640, starts=[0, 12, 30], gate=True, mod_seg=True, add=True),
    dict(rows=30, cols=640, starts=[5, 12, 30], branch=False, mod_seg=True, add=True, pre="layer", plus_one=True),
    dict(rows=25, cols=192, pre="layer", post="layer", offset=30.0), dict(rows=25, cols=192, offset=30.0, gate=True, post="rms"),
    dict(rows=2500, cols=72, post="rms", gate=True), dict(rows=3000, cols=40, starts=[0, 7, 1500, 1501, 2999], **ADA),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items())[:60])
def test_forward_and_backward(ps, case, dtype):
    t = Case(ps, dtype=dtype, **case)
    t.forward().check_forward()
    t.backward().check_backward()
    t.backward(with_dh=False).check_backward(with_dh=False)


@pytest.mark.parametrize("case", [CASES[7], CASES[14], CASES[18], CASES[24]], ids=str)
def test_accumulated_gradients(ps, case):
    t = Case(ps, dtype="f32", **case).forward().backward()
    first = {k: v.clone() for k, v in t.g.items()}
    t.backward(grads=t.grads(2.0), accumulate=True)
    for k, v in t.g.items():
        assert torch.equal(v, 2.0 + first[k]), k


def test_outputs_in_place_of_inputs(ps):
    """h in x, dx in dh or dn, dy in the other: the same results."""
    t = Case(ps, rows=19, cols=1001, post="rms", gate=True).forward()
    x, y, n = t.mat(t.x), t.mat(t.y), t.mat()
    ps.block_norm_forward(t.norm, x.m, n.m, y=y.m, h=x.m)
    assert torch.equal(x.m, t.o["h"].m) and torch.equal(n.m, t.o["n"].m)
    t.backward()
    want = t.dx.m.clone(), t.dy.m.clone(), {k: v.clone() for k, v in t.g.items()}
    for which in (0, 1):
        dn, dh = t.mat(t.dn), t.mat(t.dh)
        t.backward(dn=dn, dh=dh, dx=dh if which else dn, dy=dn if which else dh)
        assert torch.equal(t.dx.m, want[0]) and torch.equal(t.dy.m, want[1])
        assert all(torch.equal(t.g[k], v) for k, v in want[2].items())


def test_parts_of_a_call(ps):
    """Without saved values the forward pass gives the same; single gradients are those of the whole call."""
    t = Case(ps, rows=70, cols=264, starts=[0, 30, 66], post="rms", **ADA).forward()
    x, y, n, h = t.mat(t.x), t.mat(t.y), t.mat(), t.mat()
    ps.block_norm_forward(t.norm, x.m, n.m, y=y.m, h=h.m)
    assert torch.equal(n.m[:66], t.o["n"].m[:66]) and torch.equal(h.m[:66], t.o["h"].m[:66])
    t.backward()
    whole = {k: v.clone() for k, v in t.g.items()}
    dx, dy = t.dx.m.clone(), t.dy.m.clone()
    for k in whole:
        t.backward(grads={k: torch.full_like(whole[k], 5.0)})
        assert torch.equal(t.g[k], whole[k]), k
        assert torch.equal(t.dx.m, dx) and torch.equal(t.dy.m, dy)


@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_rows_of_equal_values(ps, pre):
    """A row of zeros has r = 1 / sqrt(eps); a constant one a variance of 0 under LAYER."""
    x = torch.zeros(3, 136, device="cuda")
    x[1], x[2] = 2.0, -3.5
    n, r, c = torch.empty_like(x), torch.empty(3, device="cuda"), codes(3, 136)
    ps.block_norm_forward(ps.BlockNorm(pre_norm=KIND[pre], pre_eps=1e-4), x, n, h_code=c, h_rstd=r)
    ref.check(r[:1], torch.tensor([100.0], dtype=torch.float64), torch.tensor(8 * ref.F * 100))
    assert (n[0] == 0).all() and (ref.value(c)[0] == 0).all()
    if pre == "layer":      # the mean of 136 equal values is within 16 roundings of them
        assert (n[1:].abs() <= 16 * ref.F * 3.5 * 100 + 1e-6).all()
    dx = torch.empty_like(x)
    ps.block_norm_backward(ps.BlockNorm(pre_norm=KIND[pre], pre_eps=1e-4), torch.ones_like(x), c, r, dx)
    assert dx.isfinite().all()


def test_non_finite_rows_stay_alone(ps):
    """A row with NaN or infinities becomes NaN where it depends on them; the other rows are what they were."""
    t = Case(ps, rows=12, cols=200, post="rms", gate=True).forward()
    good, saved = t.o["n"].m.clone(), {k: v.clone() for k, v in t.s.items()}
    t.x[3, 5], t.y[7, 100], t.y[9, 0] = math.nan, math.inf, math.nan
    t.forward()
    rest = [i for i in range(12) if i not in (3, 7, 9)]
    assert torch.equal(t.o["n"].m[rest], good[rest])
    for i in (3, 9):
        assert t.o["n"].m[i].isnan().all() and t.s["h_rstd"][i].isnan()
        assert t.s["h_code"][i].float().isnan().all()
    assert t.o["n"].m[7].isnan().any()
    assert torch.equal(t.s["h_code"].view(torch.uint8)[rest], saved["h_code"].view(torch.uint8)[rest])
    t.backward()
    assert t.dx.m[3].isnan().all() and t.dx.m[rest].isfinite().all()
    assert t.g["d_mul"].isnan().any()


def test_same_results_every_time(ps):
    t = Case(ps, rows=1500, cols=264, starts=[0, 400, 1400], post="rms", **ADA).forward().backward()
    want = [t.dx.m.clone(), t.dy.m.clone()] + [v.clone() for v in t.g.values()]
    for _ in range(3):
        t.backward(workspace=torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(want, [t.dx.m, t.dy.m] + list(t.g.values())))


def test_odd_segment_offsets_stay_inside(ps):
    """Offsets outside the rows, or out of order, read and write nothing that is not the call's."""
    t = Case(ps, rows=40, cols=136, starts=[0, 20, 40], post="rms", **ADA)
    for bad in ([-5, 20, 90], [30, 10, 40], [1 << 30, 5, 3], [40, 0, 0], [-1, -1, -1]):
        t.norm = dataclasses.replace(t.norm, segments=torch.tensor(bad, dtype=torch.int32).cuda())
        t.forward().backward()
        assert all(m.outside_is_untouched() for m in (t.o["n"], t.o["h"], t.dx, t.dy))


def test_no_rows(ps):
    """No rows: gradients of the vectors are zero."""
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    norm, r, c, d = ps.BlockNorm(mul=w), torch.empty(0, device="cuda"), codes(0, 64), torch.full((64,), 3.0, device="cuda")
    ps.block_norm_forward(norm, x, x.clone(), h_code=c, h_rstd=r)
    ps.block_norm_backward(norm, x, c, r, x.clone(), d_mul=d)
    assert (d == 0).all()


def test_rows_past_32_bit_offsets(ps):
    """Rows so far apart that offsets pass 2^31 elements."""
    rows, cols, ld = 9, 264, 300_000_000
    g = gen(3)
    base = torch.zeros((rows - 1) * ld + cols, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(base, (rows, cols), (ld, 1))
    v = acts(g, rows, cols, "bf16")
    x.copy_(v)
    n, want = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    c, r = codes(rows, cols), torch.empty(rows, device="cuda")
    ps.block_norm_forward(ps.BlockNorm(), x, n, h_code=c, h_rstd=r)
    ps.block_norm_forward(ps.BlockNorm(), v.cuda(), want)
    assert torch.equal(n, want)
    ps.block_norm_backward(ps.BlockNorm(), n, c, r, x)
    ps.block_norm_backward(ps.BlockNorm(), n, c, r, want)
    assert torch.equal(x, want)


def test_refusals_of_the_binding(ps):
    t = Case(ps, rows=8, cols=64, post="rms", gate=True).forward().backward()
    x = t.x.cuda()
    n = torch.empty_like(x)
    for change, says in ((dict(gate=torch.ones(3, 64).cuda().bfloat16()), "gate"), (dict(mul=torch.ones(64).cuda()), "mul"),
                         (dict(post_weight=torch.ones(65).cuda().bfloat16()), "post_weight"), (dict(mul=torch.ones(64).bfloat16()), "mul"),
                         (dict(segments=torch.zeros(2, dtype=torch.int64).cuda()), "segments")):
        norm = dataclasses.replace(t.norm, **change)
        with pytest.raises(ValueError, match=says):
            ps.block_norm_forward(norm, x, n, y=x.clone(), h=n.clone())
    with pytest.raises(ValueError, match="d_add"):
        t.backward(grads=dict(d_add=torch.ones(64).cuda()))
    with pytest.raises(ps.PSError, match="workspace"):
        t.backward(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
