"""GPU tests of the activation checkpoints used together: a feed-forward block's
training step with the AdamW plan at its end, captured calls, streams."""
import pytest
import torch

import act_ref as ref
from act_util import E4M3, codes, gen, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


class Block:
    """x -> norm -> gate and up products -> SiLU gated -> down product -> norm, gate, residual sum -> norm: a
    pre-and-post-norm feed-forward block with its input saved in 8 bits only, and its gradients."""

    def __init__(self, ps, tokens, width, hidden, seed):
        g = gen(seed)
        self.ps, self.t, self.c, self.f = ps, tokens, width, hidden
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        bf = lambda v: v.bfloat16().cuda()  # noqa: E731
        self.p = dict(w1=bf(1 + 0.2 * r(width)), wg=bf(r(hidden, width) / width ** 0.5), wu=bf(r(hidden, width) / width ** 0.5),
                      wd=bf(r(width, hidden) / hidden ** 0.5), post=bf(1 + 0.2 * r(width)), gate=bf(0.5 + 0.2 * r(width)),
                      w2=bf(1 + 0.2 * r(width)))
        self.x, self.dn, self.dh = bf(r(tokens, width)), bf(r(tokens, width) * 0.1), bf(r(tokens, width) * 0.1)
        self.before = ps.BlockNorm(mul=self.p["w1"])
        self.after = ps.BlockNorm(post_norm=ps.NORM_RMS, branch_scale=0.5, post_weight=self.p["post"], gate=self.p["gate"],
                                  mul=self.p["w2"])
        self.grads = {k: torch.empty(v.shape, device="cuda") for k, v in self.p.items()}

    def forward(self):
        ps, t, c, f = self.ps, self.t, self.c, self.f
        e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        st = lambda: torch.empty(t, device="cuda")  # noqa: E731
        n, out, h, n2 = e(t, c), e(t, f), e(t, c), e(t, c)
        s = self.saved = dict(x=(codes(t, c), st()), a=(codes(t, f), scales(t, f)), b=(codes(t, f), scales(t, f)),
                              y=(codes(t, c), st()), h=(codes(t, c), st()))
        ps.block_norm_forward(self.before, self.x, n, h_code=s["x"][0], h_rstd=s["x"][1])
        a, b = n @ self.p["wg"].t(), n @ self.p["wu"].t()
        ps.glu_forward(a, out, ps.ACT_SILU, *s["a"], b=b, b_code=s["b"][0], b_scale=s["b"][1])
        y = out @ self.p["wd"].t()
        ps.block_norm_forward(self.after, self.x, n2, y=y, h=h, h_code=s["h"][0], h_rstd=s["h"][1], y_code=s["y"][0],
                              y_rstd=s["y"][1])
        return h, n2

    def backward(self):
        ps, t, c, f, s, g = self.ps, self.t, self.c, self.f, self.saved, self.grads
        e = lambda *z: torch.empty(*z, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        dx, dy, dab, out, dx1 = e(t, c), e(t, c), e(t, 2 * f), e(t, f), e(t, c)
        ps.block_norm_backward(self.after, self.dn, s["h"][0], s["h"][1], dx, dh=self.dh, dy=dy, y_code=s["y"][0],
                               y_rstd=s["y"][1], d_post_weight=g["post"], d_gate=g["gate"], d_mul=g["w2"])
        do = dy @ self.p["wd"]
        ps.glu_backward(do, ps.ACT_SILU, *s["a"], dab[:, :f], b_code=s["b"][0], b_scale=s["b"][1], db=dab[:, f:], out=out)
        oc, os = codes(t, f), scales(t, f)
        ps.encode_act(out, oc, os)
        ps.linear_wgrad(dy, oc, g["wd"], scale=os)
        w1 = self.p["w1"].float()
        ps.linear_wgrad(dab[:, :f], s["x"][0], g["wg"], mul=w1)
        ps.linear_wgrad(dab[:, f:], s["x"][0], g["wu"], mul=w1)
        dn = (dab @ torch.cat([self.p["wg"], self.p["wu"]]))
        ps.block_norm_backward(self.before, dn, s["x"][0], s["x"][1], dx1, dh=dx, d_mul=g["w1"])
        return dx1


def _autograd(b):
    """The block's gradients in 64 bits, nothing saved in few bits."""
    p = {k: v.cpu().double().requires_grad_() for k, v in b.p.items()}
    x = b.x.cpu().double().requires_grad_()
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    n = rms(x) * p["w1"]
    y = (torch.nn.functional.silu(n @ p["wg"].t()) * (n @ p["wu"].t())) @ p["wd"].t()
    h = x + 0.5 * p["gate"] * (rms(y) * p["post"])
    n2 = rms(h) * p["w2"]
    ((n2 * b.dn.cpu().double()).sum() + (h * b.dh.cpu().double()).sum()).backward()
    return h.detach(), n2.detach(), x.grad, {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("tokens,width,hidden", [(200, 256, 640), (77, 136, 304), (1500, 512, 1024)])
def test_block_gradients_and_step(ps, tokens, width, hidden):
    """A saved value is off by at most 2^-4 of itself, 2^-4 / sqrt 3 in the mean square; a gradient here holds at most
    four of them, so its 2-norm is off by about 2 * 2^-4 / sqrt 3 = 0.072: 0.125 leaves a factor of 1.7. The forward pass
    saves nothing it then uses and is as exact as bf16 products: four roundings of 2^-8."""
    b = Block(ps, tokens, width, hidden, tokens)
    h, n2 = b.forward()
    dx = b.backward()
    want_h, want_n2, want_dx, want = _autograd(b)
    off = lambda got, w: float((got.cpu().double() - w).norm() / w.norm())  # noqa: E731
    assert off(h, want_h) < 4 * 2 ** -8 and off(n2, want_n2) < 4 * 2 ** -8
    assert off(dx, want_dx) < 0.125
    for k, w in want.items():
        assert off(b.grads[k], w) < 0.125, (k, off(b.grads[k], w))
    # the gradients go on as they are: one AdamW step over the block's weights, their norm first
    masters = {k: v.float() for k, v in b.p.items()}
    z = lambda v: torch.zeros_like(v)  # noqa: E731
    plan = ps.AdamWPlan([ps.AdamWTensor(m, b.grads[k], z(m), z(m), copy=b.p[k]) for k, m in masters.items()])
    before = {k: v.clone() for k, v in masters.items()}
    plan.grad_norm(max_norm=1.0)
    plan.step([ps.HParams(algo=ps.ALGO_ADAM, lr=1e-3)], step=1, clipped=True)
    total = torch.sqrt(sum((v.double() ** 2).sum() for v in b.grads.values()))
    assert abs(float(plan.norm) / float(total) - 1) < 1e-6
    for k, m in masters.items():
        # a first step moves by lr * g / (|g| + eps) of the clipped g, here up to the rounding of masters of up to 8
        # (2^-22); the copy that the block runs on follows
        g = b.grads[k] * plan.grad_mul
        assert torch.allclose(before[k] - m, 1e-3 * g / (g.abs() + 1e-8), rtol=1e-5, atol=2.0 ** -22), k
        assert torch.equal(b.p[k], m.bfloat16())
    assert all(torch.isfinite(v).all() for v in b.forward())


def test_a_gradient_that_overflowed_reaches_the_norm(ps):
    """An infinity in an activation becomes NaN in its code, then in the gradient, and the plan skips the step."""
    b = Block(ps, 64, 128, 256, 1)
    b.x[5, 7] = float("inf")
    b.forward()
    b.backward()
    m = b.p["wd"].float()
    plan = ps.AdamWPlan([ps.AdamWTensor(m, b.grads["wd"], torch.zeros_like(m), torch.zeros_like(m))])
    plan.grad_norm(max_norm=1.0)
    was = m.clone()
    plan.step([ps.HParams(algo=ps.ALGO_ADAM)], step=1, clipped=True)
    assert int(plan.skip) == 1 and torch.equal(m, was)


class Chain:
    """All operators one after the other on buffers of its own."""

    def __init__(self, ps, seed):
        self.ps = ps
        t, c, f = self.shape = 700, 264, 520
        e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.y, self.ab, self.dn, self.dy = e(t, c), e(t, c), e(t, 2 * f), e(t, c), e(t, f)
        self.starts = torch.tensor([0, 100, 350, t - 10], dtype=torch.int32).cuda()
        g = gen(seed)
        v = lambda *s: (0.3 * torch.randn(*s, generator=g)).cuda()  # noqa: E731
        self.norm = ps.BlockNorm(pre_norm=ps.NORM_LAYER, post_norm=ps.NORM_RMS, post_weight=v(c), gate=v(3, c), mul=v(3, c),
                                 add=v(3, c), mul_plus_one=True, segments=self.starts)
        self.n, self.h, self.hc, self.hr, self.yc, self.yr = e(t, c), e(t, c), codes(t, c), torch.zeros(t, device="cuda"), \
            codes(t, c), torch.zeros(t, device="cuda")
        self.out, self.ac, self.as_, self.bc, self.bs = e(t, f), codes(t, f), scales(t, f), codes(t, f), scales(t, f)
        self.dx, self.dyy, self.dab, self.back = e(t, c), e(t, c), e(t, 2 * f), e(t, f)
        self.vec = [torch.zeros(s, device="cuda") for s in ((c,), (3, c), (3, c), (3, c))]
        self.dw, self.db = torch.zeros(f, c, device="cuda"), torch.zeros(f, device="cuda")
        self.w1 = torch.empty(ps.block_norm_workspace_size(self.norm, t, c), dtype=torch.uint8, device="cuda")
        self.w2 = torch.empty(ps.linear_wgrad_workspace_size(t, f, c), dtype=torch.uint8, device="cuda")
        assert self.w2.numel() > 0       # split over the tokens and joined

    def fill(self, seed):
        g = gen(seed)
        for x in (self.x, self.y, self.ab, self.dn, self.dy):
            x.copy_(torch.randn(x.shape, generator=g))

    def run(self, stream=None):
        ps, f = self.ps, self.shape[2]
        ps.block_norm_forward(self.norm, self.x, self.n, y=self.y, h=self.h, h_code=self.hc, h_rstd=self.hr, y_code=self.yc,
                              y_rstd=self.yr, stream=stream)
        ps.glu_forward(self.ab[:, :f], self.out, ps.ACT_GELU, self.ac, self.as_, b=self.ab[:, f:], b_code=self.bc,
                       b_scale=self.bs, stream=stream)
        ps.glu_backward(self.dy, ps.ACT_GELU, self.ac, self.as_, self.dab[:, :f], b_code=self.bc, b_scale=self.bs,
                        db=self.dab[:, f:], out=self.back, stream=stream)
        ps.linear_wgrad(self.dab[:, :f], self.hc, self.dw, db=self.db, workspace=self.w2, stream=stream)
        ps.block_norm_backward(self.norm, self.dn, self.hc, self.hr, self.dx, dy=self.dyy, y_code=self.yc, y_rstd=self.yr,
                               d_post_weight=self.vec[0], d_gate=self.vec[1], d_mul=self.vec[2], d_add=self.vec[3],
                               workspace=self.w1, stream=stream)
        ps.encode_act(self.back, self.ac, self.as_, stream=stream)
        ps.decode_act(self.ac, self.as_, self.back, stream=stream)

    def results(self):
        u = int(self.starts[-1])
        return [x.clone() for x in (self.n[:u], self.h[:u], self.out, self.dab, self.back, self.dx[:u], self.dyy[:u], self.dw,
                                    self.db, *self.vec)] + [self.hc[:u].float(), self.ac.float(), self.as_.clone()]


def _expected(ps, seeds):
    c, out = Chain(ps, 1), []
    for s in seeds:
        c.fill(s)
        c.run()
        torch.cuda.synchronize()
        out.append(c.results())
    return out


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_calls_replay(ps):
    """Two graphs, each with workspaces of its own, replayed in turn with eager work between: every replay has the
    results of an eager run on its inputs."""
    seeds = [11, 12, 13, 14, 15, 16]
    want = _expected(ps, seeds)
    chains, graphs = [Chain(ps, 1), Chain(ps, 1)], []
    side = torch.cuda.Stream()
    for c in chains:
        c.fill(1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.run()
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                c.run()
        graphs.append(g)
    torch.cuda.synchronize()
    for i, s in enumerate(seeds):
        c, g = chains[i % 2], graphs[i % 2]
        c.fill(s)
        g.replay()
        other = Chain(ps, 1)
        other.fill(seeds[i - 1])
        other.run()                       # eager work beside the replay
        torch.cuda.synchronize()
        assert _equal(c.results(), want[i]), i
        assert _equal(other.results(), want[i - 1]), i


def test_streams(ps):
    """On a stream that is not the current one, as an object and as an integer, two at a time."""
    want = _expected(ps, [21, 22])
    a, b = Chain(ps, 1), Chain(ps, 1)
    a.fill(21)
    b.fill(22)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(stream=s)
        b.run(stream=t.cuda_stream)
    s.synchronize()
    t.synchronize()
    assert _equal(a.results(), want[0]) and _equal(b.results(), want[1])


def test_workspaces_of_the_call(ps):
    """Without a workspace the call takes one from the stream's allocator: the same results, on any stream."""
    t, n, k = 2000, 96, 640
    g = gen(4)
    dy = torch.randn(t, n, generator=g).bfloat16().cuda()
    code = torch.randn(t, k, generator=g).to(E4M3).cuda()
    want = torch.empty(n, k, device="cuda")
    size = ps.linear_wgrad_workspace_size(t, n, k)
    ps.linear_wgrad(dy, code, want, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        outs = [torch.empty(n, k, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        for o in outs:
            ps.linear_wgrad(dy, code, o, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_norms_share_no_state_between_threads(ps):
    """Two threads use one norm with different rows at a time."""
    import threading
    w = torch.ones(256, device="cuda")
    norm = ps.BlockNorm(mul=w)
    xs = [torch.randn(r, 256, generator=gen(r)).cuda() for r in (3, 700)]
    want = [torch.empty_like(x) for x in xs]
    for x, o in zip(xs, want):
        ps.block_norm_forward(norm, x, o)
    got = [torch.zeros_like(x) for x in xs]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(200):
            ps.block_norm_forward(norm, xs[i], got[i])
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in ts:
        th.start()
    for th in ts:
        th.join()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_reference_of_the_block_by_its_codes(ps):
    """The weight gradients are those of the saved values, to fp32: dw of the gate product from its own inputs."""
    b = Block(ps, 120, 128, 256, 9)
    b.forward()
    b.backward()
    x = ref.value(b.saved["x"][0])
    da = torch.empty(120, 512, dtype=torch.bfloat16, device="cuda")
    do = torch.randn(120, 256, generator=gen(2)).bfloat16().cuda()
    ps.glu_backward(do, ps.ACT_SILU, *b.saved["a"], da[:, :256], b_code=b.saved["b"][0], b_scale=b.saved["b"][1], db=da[:, 256:])
    w = torch.empty(256, 128, device="cuda")
    ps.linear_wgrad(da[:, :256], b.saved["x"][0], w, mul=b.p["w1"].float())
    want, e, _, _ = ref.wgrad(da[:, :256].cpu().double(), x, b.p["w1"].cpu().double(), None)
    ref.check(w, want, e)
