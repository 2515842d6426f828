"""GPU tests of the AdamW plan (step, gradient norm, device-counted steps) and
the e4m3 codec against plain references: bit for bit against the formulas in
float32, and within derived bounds of the formulas in 64 bits."""
import ctypes
import threading

import numpy as np
import pytest

import adamw_ref as ref
import oracle
from adamw_util import Param

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import precision_state_amd as ps  # noqa: E402

SIZES = [1, 2, 7, 8, 9, 255, 256, 257, 511, 512, 513, 1000, 2049, 30011]
HALF = 2.0 ** -24


def hps(algo=0, split=0, wd=(0.1, 0.0), **kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, seed=77)
    a.update(kw)
    return ([ps.HParams(algo=algo, split_mode=split, weight_decay=w, **a) for w in wd],
            [oracle.HParams(algo=algo, split_mode=split, weight_decay=w, **a) for w in wd])


def build(specs, seed=0, sizes=SIZES, **kw):
    rng = np.random.default_rng(seed)
    out = []
    for spec in specs:
        for n in sizes:
            out.append(Param(n, rng, group=len(out) % 2, index=len(out), **{**spec, **kw}))
    return out


def agree(params):
    torch.cuda.synchronize()
    bad = [(i, p.param, p.grad, p.state, p.copy, d) for i, p in enumerate(params) for d in p.differences()]
    assert not bad, bad[:6]


def run_steps(params, plan, dev, host, steps, rng, rounding=0, first=1):
    for t in range(first, first + steps):
        for p in params:
            p.new_grad(rng.normal(0, 1e-3, p.n).astype(np.float32))
        plan.step(dev, t, rounding=rounding)
        for p in params:
            p.step(host[p.group], t, rounding=rounding)
        agree(params)


# ---------------------------------------------------------------------------
# the step, bit for bit
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("state,rounding", [("f32", 0), ("e4m3", 0), ("e4m3", 1)])
@pytest.mark.parametrize("algo", [0, 1])
def test_step_all_fp32_weight_kinds(state, algo, rounding):
    """Every gradient and copy type and every ragged size in one plan, two groups."""
    params = build([dict(param="f32", grad=g, copy=c) for g in ("f32", "bf16", "f16") for c in ("", "bf16", "f16")],
                   state=state)
    dev, host = hps(algo)
    run_steps(params, ps.AdamWPlan([p.tensor(ps) for p in params]), dev, host, 3, np.random.default_rng(1), rounding)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("split", [0, 1, 2])
@pytest.mark.parametrize("algo", [0, 1])
def test_step_all_bf16_weight_kinds(state, split, algo):
    params = build([dict(param="bf16", grad=g, residual=r) for g in ("f32", "bf16", "f16")
                    for r in ((True, False) if split == 2 else (True,))], state=state)
    dev, host = hps(algo, split)
    run_steps(params, ps.AdamWPlan([p.tensor(ps) for p in params]), dev, host, 3, np.random.default_rng(2),
              rounding=split % 2, first=1000)


def test_step_mixes_kinds_and_starts_from_zero_state():
    params = build([dict(param="f32", state="f32", copy="bf16"), dict(param="bf16", state="e4m3"),
                    dict(param="f32", state="e4m3", grad="f32"), dict(param="bf16", state="f32", grad="f16")],
                   zero_state=True)
    dev, host = hps()
    run_steps(params, ps.AdamWPlan([p.tensor(ps) for p in params]), dev, host, 4, np.random.default_rng(3), rounding=1)


@pytest.mark.parametrize("level", [0.0, 1e-30, 1e-22, 1e-12, 1e-4, 1.0, 1e8, 1e17])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_step_over_gradient_magnitudes(level, state):
    """From gradients whose squares vanish to squares near the largest float; zero gradients in between, blocks of
    zeros, and one outlier a block."""
    rng = np.random.default_rng(4)
    params = build([dict(param="f32", grad="f32"), dict(param="bf16", grad="f32")], sizes=[700, 2048], state=state,
                   zero_state=True)
    dev, host = hps()
    plan = ps.AdamWPlan([p.tensor(ps) for p in params])
    for t in (1, 2, 3):
        for p in params:
            g = (rng.normal(0, 1, p.n) * level).astype(np.float32)
            g[rng.random(p.n) < 0.2] = 0.0
            g[256:512] = 0.0
            g[::300] *= 30
            p.new_grad(g)
        plan.step(dev, t)
        for p in params:
            with np.errstate(over="ignore"):
                p.step(host[p.group], t)
        agree(params)


@pytest.mark.parametrize("algo", [0, 1])
@pytest.mark.parametrize("kw", [dict(eps=1e-40), dict(eps=1e20), dict(beta1=0.0), dict(beta2=0.0), dict(lr=0.0),
                                dict(lr=50.0), dict(beta2=1 - 2.0 ** -50), dict(beta2=1 - 2.0 ** -53), dict(beta1=1e-30),
                                dict(eps=2.0 ** -61), dict(wd=(100.0, 0.0))])
def test_step_at_extreme_hyperparameters(algo, kw):
    """Where the scalars leave the ranges of the fast quotient, at their ends, and where terms vanish."""
    params = build([dict(param="f32", grad="f32", state=s) for s in ("f32", "e4m3")] +
                   [dict(param="bf16", state="e4m3")], sizes=[5, 700, 1024])
    dev, host = hps(algo, **kw)
    run_steps(params, ps.AdamWPlan([p.tensor(ps) for p in params]), dev, host, 2, np.random.default_rng(50), first=2)


def test_step_numbers_in_any_order():
    """The plan carries NAdam's product from call to call: ascending, repeated, earlier and far steps, other schedules in
    between, each as if it were the plan's first."""
    p = Param(300, np.random.default_rng(53), param="f32", grad="f32", state="f32")
    plan = ps.AdamWPlan([p.tensor(ps)])
    for t, kw in ((5, {}), (6, {}), (6, {}), (7, dict(lr=5e-4)), (3, {}), (2000, {}), (2001, {}), (8, dict(beta1=0.8)),
                  (9, dict(beta1=0.8)), (10, {}), (11, dict(beta1=0.999)), (12, dict(beta1=0.999)), (1, {})):
        dev, host = hps(1, wd=(0.1,), **kw)
        plan.step(dev, t)
        p.step(host[0], t)
        agree([p])


def test_first_moments_that_have_decayed_away():
    """First moments far below the fast quotient's range beside ordinary ones; second moments of zero and below 2^-96."""
    rng = np.random.default_rng(51)
    p = Param(4096, rng, param="f32", grad="f32", state="f32")
    p.m = (p.m * np.exp(rng.uniform(-90, 0, p.n))).astype(np.float32)
    p.v = np.where(rng.random(p.n) < 0.3, 0, p.v * np.exp(rng.uniform(-75, 0, p.n))).astype(np.float32)
    g = np.where(rng.random(p.n) < 0.5, 0, p.g).astype(np.float32)
    for k in ("m", "v"):
        p.d[k].t.copy_(torch.from_numpy(getattr(p, k)))
    p.new_grad(g)
    for algo in (0, 1):
        dev, host = hps(algo, wd=(0.1,))
        ps.AdamWPlan([p.tensor(ps)]).step(dev, 3)
        p.step(host[0], 3)
        agree([p])


@pytest.mark.parametrize("algo", [0, 1])
def test_step_against_64_bits(algo):
    """fp32 weights and moments against the formula in 64 bits with the same fp32 scalars. Roundings, each at most half
    a step: m: two products and a sum; v: three products and a sum; r: half of v's and its own; d: two more; the quotient, the factor
    (NADAM: two products and a sum over terms of one size before the quotient), the decay's product and sum, the
    difference."""
    rng = np.random.default_rng(5)
    p = Param(100_003, rng, param="f32", grad="f32", state="f32")
    dev, host = hps(algo, wd=(0.1,))
    c = oracle.coeffs(host[0], 9)
    w64, m64, v64, r64 = ref.update(p.w, p.g, p.m, p.v, c, 1.0, algo == 1, np.float64)
    m_terms = np.abs(float(c["B1"]) * p.m) + np.abs(float(c["C1"]) * p.g)
    g_terms = np.abs(float(c["AG"]) * p.g) if algo else 0.0
    a = float(c["AM"] if algo else c["A"])
    u_terms = (g_terms + a * m_terms) / (r64 * float(c["RS2"]) + float(c["EPS"]))
    ps.AdamWPlan([p.tensor(ps)]).step(dev, 9)
    torch.cuda.synchronize()
    got = {k: p.d[k].host().astype(np.float64) for k in ("w", "m", "v")}
    slack = 1 + 1e-5                                       # products of the roundings
    assert np.all(np.abs(got["m"] - m64) <= 2 * HALF * m_terms * slack + 2.0 ** -149)
    assert np.all(np.abs(got["v"] - v64) <= 3 * HALF * v64 * slack + 2.0 ** -148)
    # u: m 2, (NADAM: product and sum 2), r 3/2 + 1, d 2 (product, sum), quotient 1, factor 1, sum with decay 1
    bound = 10.5 * HALF * u_terms + 2 * HALF * np.abs(float(c["CWD"]) * p.w) + HALF * np.abs(w64)
    assert np.all(np.abs(got["w"] - w64) <= bound * slack)


def test_e4m3_moments_are_within_half_a_step():
    """Stored m and sqrt(v) against the values in 64 bits: half a step of e4m3 is 2^-4 of the value, or half of the
    smallest step 2^-9 times the block's scale; the fp32 arithmetic before it adds at most 4 half steps of fp32."""
    rng = np.random.default_rng(6)
    p = Param(50_001, rng, param="bf16", state="e4m3")
    dev, host = hps(wd=(0.0,))
    m0, v0 = p.moments()
    _, m64, v64, r64 = ref.update(p.weights(0), p.g, m0, v0, oracle.coeffs(host[0], 5), 1.0, False, np.float64)
    m_terms = 0.9 * np.abs(m0) + 0.1 * np.abs(p.g)
    ps.AdamWPlan([p.tensor(ps)]).step(dev, 5)
    torch.cuda.synchronize()
    ms, vs = p.d["ms"].host(), p.d["vs"].host()
    m = ref.e4m3_value(p.d["m"].host()).astype(np.float64) * ref.spread(ms, p.n)
    r = ref.e4m3_value(p.d["v"].host()).astype(np.float64) * ref.spread(vs, p.n)
    for got, want, s, slack in ((m, m64, ms, 4 * HALF * m_terms), (r, r64, vs, 4 * HALF * r64)):
        s = ref.spread(s, p.n)
        step = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s)
        floor = (got == 2.0 ** -9 * s) & (np.abs(want) < 2.0 ** -9 * s)    # above zero stays above zero
        assert np.all((np.abs(got - want) <= step * (1 + 1e-5) + slack) | (floor if got is r else False))
    assert np.all((r > 0) == (r64 > 0))


def test_stochastic_second_moment_decays_where_nearest_stays():
    """With zero gradients sqrt(v) falls by sqrt(0.999) a step: nearest codes of a block keep their values, stochastic
    ones fall on average. The largest element is kept up by its gradient, so the scale stays."""
    n, steps = 256 * 64, 60
    rng = np.random.default_rng(7)
    out = {}
    for rounding in (0, 1):
        p = Param(n, rng, param="f32", grad="f32", state="e4m3", zero_state=True)
        r = np.full(n, 1.0, np.float32)
        r[::256] = 1.5
        p.v, p.vs = ref.encode(r * r, False)
        p.d["v"].t.copy_(torch.from_numpy(p.v)), p.d["vs"].t.copy_(torch.from_numpy(p.vs))
        g = np.zeros(n, np.float32)
        g[::256] = 1.5
        p.new_grad(g)
        plan = ps.AdamWPlan([p.tensor(ps)])
        dev, _ = hps(wd=(0.0,))
        for t in range(1, steps + 1):
            plan.step(dev, t, rounding=rounding)
        x = torch.zeros(n, device="cuda")
        ps.decode_fp8(p.d["v"].t, p.d["vs"].t, x, ps.MOMENT_UNSIGNED)
        out[rounding] = np.sqrt(np.delete(x.cpu().numpy(), np.s_[::256]))
    assert np.all(out[0] == 1.0)
    # mean of n - n/256 elements that each moved down by 1/16 with probability p in all: sqrt(0.999)^60 = 0.9704,
    # a standard error of sqrt(p (1 - p) / n) / 16 with p about 0.5 is 2.5e-4; 6 of them, and the step doubles (1/8)
    # nowhere since values stay in [0.5, 1]
    assert abs(out[1].mean() - 0.999 ** (steps / 2)) < 1.5e-3


def test_large_tensors_pass_32_bit_offsets():
    """A bf16 weight with 8-bit moments of 2^31 + 777 elements: blocks at the start, beyond 2^31 and at the end."""
    n = (1 << 31) + 777
    nb = ref.blocks_of(n)
    dev = "cuda"
    w = torch.full((n,), 0.02, dtype=torch.bfloat16, device=dev)
    g = torch.full((n,), 1e-3, dtype=torch.bfloat16, device=dev)
    m, v = torch.zeros(n, dtype=torch.uint8, device=dev), torch.zeros(n, dtype=torch.uint8, device=dev)
    ms, vs = torch.zeros(nb, device=dev), torch.zeros(nb, device=dev)
    rng = np.random.default_rng(8)
    spans = [(0, 1024), ((1 << 31) - 512, 1024), ((1 << 31) + 512, 265)]
    for a, k in spans:
        g[a:a + k] = torch.from_numpy(rng.normal(0, 1e-3, k).astype(np.float32)).to(dev)
    plan = ps.AdamWPlan([ps.AdamWTensor(w, g, m, v, ms, vs)])
    hd, ho = hps(split=2, wd=(0.1,))
    plan.grad_norm()
    plan.step(hd, 3, rounding=1)
    torch.cuda.synchronize()
    exact = float(torch.linalg.vector_norm(g, dtype=torch.float64))
    assert abs(float(plan.norm) - exact) <= 2 * HALF * exact
    c = oracle.coeffs(ho[0], 3)
    for a, k in spans:
        gg = g[a:a + k].float().cpu().numpy()
        w0 = np.full(k, ref.bf16_to_f32(ref.bf16_round(np.full(1, 0.02, np.float32)))[0], np.float32)
        z = np.zeros(k, np.float32)
        w1, m1, _, r1 = ref.update(w0, gg, z, z, c, 1.0, False, np.float32)
        bits = [oracle.sr_rand16(77, 3, h, a, k) for h in (0, 1 << 31)]
        want = ((w1.view(np.uint32) + bits[0].astype(np.uint32)) >> 16).astype(np.uint16)
        assert np.array_equal(w[a:a + k].view(torch.int16).cpu().numpy().view(np.uint16), want)
        s = ref.spread(ref.block_scale(ref.per_block_max(m1)), k)
        t = ref.spread(ref.block_scale(ref.per_block_max(r1)), k)
        assert np.array_equal(m[a:a + k].cpu().numpy(), ref.e4m3_code(m1 / s))
        assert np.array_equal(v[a:a + k].cpu().numpy(), ref.second_code(r1, t, bits[1]))
        b0, b1 = a // 256, (a + k + 255) // 256
        assert np.array_equal(ms[b0:b1].cpu().numpy(), s[::256]) and np.array_equal(vs[b0:b1].cpu().numpy(), t[::256])


def test_large_fp32_tensors_pass_32_bit_offsets():
    """The other lane layout: fp32 weights and gradients with 8-bit moments and a copy, 2^30 + 777 elements (byte offsets
    beyond 2^32), and the codec over arrays of that size."""
    n = (1 << 30) + 777
    nb, k = ref.blocks_of(n), 777 + 256
    a = n - k                                               # the last blocks
    dev = "cuda"
    w, g = torch.full((n,), 0.02, device=dev), torch.full((n,), 1e-3, device=dev)
    copy = torch.zeros(n, dtype=torch.float16, device=dev)
    m, v = torch.zeros(n, dtype=torch.uint8, device=dev), torch.zeros(n, dtype=torch.uint8, device=dev)
    ms, vs = torch.zeros(nb, device=dev), torch.zeros(nb, device=dev)
    gg = np.random.default_rng(54).normal(0, 1e-3, k).astype(np.float32)
    g[a:] = torch.from_numpy(gg).to(dev)
    hd, ho = hps(wd=(0.1,))
    ps.AdamWPlan([ps.AdamWTensor(w, g, m, v, ms, vs, copy=copy)]).step(hd, 3)
    torch.cuda.synchronize()
    z = np.zeros(k, np.float32)
    w1, m1, v1, r1 = ref.update(np.full(k, 0.02, np.float32), gg, z, z, oracle.coeffs(ho[0], 3), 1.0, False, np.float32)
    s, t = ref.block_scale(ref.per_block_max(m1)), ref.block_scale(ref.per_block_max(r1))
    assert np.array_equal(w[a:].cpu().numpy(), w1)
    assert np.array_equal(copy[a:].cpu().numpy(), w1.astype(np.float16))
    assert np.array_equal(m[a:].cpu().numpy(), ref.e4m3_code(m1 / ref.spread(s, k)))
    assert np.array_equal(v[a:].cpu().numpy(), ref.second_code(r1, ref.spread(t, k)))
    assert np.array_equal(ms[a // 256:].cpu().numpy(), s) and np.array_equal(vs[a // 256:].cpu().numpy(), t)
    assert float(w[0]) == float(w[a - 1]) and int(m[0]) == int(m[a - 1])
    x = w
    x.fill_(1e-6)
    x[a:] = torch.from_numpy(v1).to(dev)
    ps.encode_fp8(x, m, ms, ps.MOMENT_UNSIGNED)
    c1, s1 = ref.encode(v1, False)
    assert np.array_equal(m[a:].cpu().numpy(), c1) and np.array_equal(ms[a // 256:].cpu().numpy(), s1)
    ps.decode_fp8(m, ms, g, ps.MOMENT_UNSIGNED)
    assert np.array_equal(g[a:].cpu().numpy(), ref.decode(c1, s1, False))
    assert float(g[0]) == float(g[a - 1]) == float(ref.decode(*ref.encode(np.full(256, 1e-6, np.float32), False), False)[0])


# ---------------------------------------------------------------------------
# gradient norm, clipping, skipped steps
# ---------------------------------------------------------------------------

def norm64(params):
    return np.sqrt(sum(float(np.sum(p.g.astype(np.float64) ** 2)) for p in params))


@pytest.mark.parametrize("grad", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", [[1], [8], SIZES, [8191, 8192, 8193], [3_000_001, 5, 2_000_000], [1] * 300])
def test_norm_and_clip_factor(grad, sizes):
    params = build([dict(param="f32", grad=grad)], sizes=sizes, seed=9)
    plan = ps.AdamWPlan([p.tensor(ps) for p in params])
    want = norm64(params)
    for max_norm, scale in ((float("inf"), 1.0), (want / 3, 1.0), (want * 3, 1.0), (0.5, 1 / 1024)):
        plan.grad_norm(max_norm, scale)
        n = want * scale
        mul = scale * min(1.0, max_norm / (n + 1e-6))
        # sums in double: 2^-53 for each of at most 5e6 terms, far below the final rounding to fp32
        assert abs(float(plan.norm) - n) <= n * (HALF + 1e-9)
        assert abs(float(plan.grad_mul) - mul) <= mul * (HALF + 1e-9)
        assert int(plan.skip) == 0 and int(plan.skipped) == 0


def test_norm_of_extreme_values_and_repeatability():
    rng = np.random.default_rng(10)
    for level in (1e-42, 1e-30, 1e19, 3e38):
        p = Param(40_000, rng, grad="f32")
        p.new_grad((np.clip(rng.normal(0, 0.3, p.n), -1, 1) * level).astype(np.float32))
        plan = ps.AdamWPlan([p.tensor(ps)])
        seen = set()
        for _ in range(5):
            plan.grad_norm(1.0)
            seen.add((plan.norm.cpu().numpy().tobytes(), plan.grad_mul.cpu().numpy().tobytes()))
        want = norm64([p])
        assert len(seen) == 1 and int(plan.skip) == 0
        if want < 3.4e38:
            assert abs(float(plan.norm) - want) <= max(HALF * want * 1.001, 2.0 ** -149)
        else:                                             # the norm is no fp32 value, the factor still is one
            assert np.isinf(float(plan.norm))
        assert abs(float(plan.grad_mul) - min(1.0, 1.0 / (want + 1e-6))) <= max(HALF * float(plan.grad_mul) * 1.001, 2.0 ** -149)


@pytest.mark.parametrize("sizes", [[700], [8192 * 40 + 5], [3_000_001, 5, 6_000_000], [4_000_000] * 5])
def test_norms_in_a_row_see_their_own_gradients(sizes):
    """Many calls with nothing between them but an exact doubling or halving of the gradients: every norm is the first one
    or its double, so no call reads a partial sum of the one before."""
    rng = np.random.default_rng(55)
    gs = [torch.from_numpy(rng.normal(0, 1e-3, n).astype(np.float32)).cuda() for n in sizes]
    plan = ps.AdamWPlan([ps.AdamWTensor(None, g) for g in gs])
    seen = torch.zeros(400, device="cuda")
    for i in range(400):
        plan.grad_norm(1.0)
        seen[i].copy_(plan.norm)
        for g in gs:
            g.mul_(0.5 if i % 2 else 2.0)
    seen = seen.cpu().numpy()
    assert np.all(seen[0::2] == seen[0]) and np.all(seen[1::2] == 2 * seen[0])


def test_norm_of_nothing():
    plan = ps.AdamWPlan([])
    plan.grad_norm(1.0)
    plan.step([ps.HParams(algo=ps.ALGO_ADAM)], 1, clipped=True)
    assert float(plan.norm) == 0.0 and float(plan.grad_mul) == 1.0 and int(plan.skip) == 0
    e = torch.empty(0, device="cuda")
    plan = ps.AdamWPlan([ps.AdamWTensor(e, e, e, e), ps.AdamWTensor(torch.ones(4, device="cuda"), None,
                                                                     torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"))])
    plan.grad_norm(1.0)
    assert float(plan.norm) == 0.0


@pytest.mark.parametrize("clip", [0.01, 100.0])
@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_clipped_steps_as_a_training_loop_ends(clip, state):
    """Norm, then step, several times, mixed types; the loss scale's inverse in the factor."""
    params = build([dict(param="f32", grad="f16", copy="f16"), dict(param="bf16", grad="bf16")], state=state)
    plan = ps.AdamWPlan([p.tensor(ps) for p in params])
    dev, host = hps()
    rng = np.random.default_rng(11)
    for t in (1, 2, 3, 4):
        for p in params:
            p.new_grad(rng.normal(0, 1e-2, p.n).astype(np.float32))
        plan.grad_norm(clip, 0.25)
        plan.step(dev, t, clipped=True)
        n = 0.25 * norm64(params)
        mul = np.float32(0.25 * min(1.0, clip / (n + 1e-6)))
        got = plan.grad_mul.cpu().numpy()
        assert abs(float(got) - float(mul)) <= 2 * HALF * float(mul)      # the double sums' order may tip the rounding
        for p in params:
            p.step(host[p.group], t, mul=got)
        agree(params)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_steps_with_infinite_gradients_change_nothing(bad):
    params = build([dict(param="f32", grad="f32"), dict(param="bf16", grad="f16", state="e4m3")], sizes=[700, 9000])
    plan = ps.AdamWPlan([p.tensor(ps) for p in params])
    dev, host = hps()
    for t in (1, 2, 3):
        rng = np.random.default_rng(20 + t)
        for i, p in enumerate(params):
            g = rng.normal(0, 1e-3, p.n).astype(np.float32)
            if t == 2 and i == 3:
                g[8999] = bad
            p.new_grad(g)
        plan.grad_norm(1e9)
        plan.step(dev, t, clipped=True)
        assert int(plan.skip) == (t == 2) and int(plan.skipped) == (t >= 2)
        if t != 2:
            for p in params:
                p.step(host[p.group], t)
        agree(params)


def test_bad_values_of_passed_by_tensors_do_not_count():
    params = build([dict(param="f32", grad="f32")], sizes=[300, 400, 500])
    params[1].new_grad(np.full(400, np.nan, np.float32))
    plan = ps.AdamWPlan([p.tensor(ps) for p in params])
    plan.set_grads([params[0].d["g"].t, None, params[2].d["g"].t])
    dev, host = hps()
    plan.grad_norm(1e9)
    plan.step(dev, 1, clipped=True)
    assert int(plan.skip) == 0
    for p in (params[0], params[2]):
        p.step(host[p.group], 1)
    agree(params)


# ---------------------------------------------------------------------------
# new gradients, streams, graphs, counted steps
# ---------------------------------------------------------------------------

def test_set_grads_over_many_tensors():
    """More tensors than one launch's pointers; gradients come, go and return."""
    params = build([dict(param="f32", grad="f32", state="e4m3")], sizes=[1 + 3 * (k % 40) for k in range(900)])
    tensors = [p.tensor(ps) for p in params]
    for t in tensors[::7]:
        t.grad = None
    plan = ps.AdamWPlan([ps.AdamWTensor(t.param, t.grad if t.grad is not None else None, t.m, t.v, t.m_scale, t.v_scale,
                                        group=t.group) for t in tensors])
    dev, host = hps()
    plan.step(dev, 1)
    for i, p in enumerate(params):
        if i % 7:
            p.step(host[p.group], 1)
    agree(params)
    fresh = [torch.randn(p.n, device="cuda") * 1e-3 if i % 5 else None for i, p in enumerate(params)]
    plan.set_grads(fresh)
    plan.grad_norm(1.0)
    plan.step(dev, 2)
    for p, g in zip(params, fresh):
        if g is not None:
            p.g = g.cpu().numpy()
            p.step(host[p.group], 2)
    want = np.sqrt(sum(float((g.double() ** 2).sum()) for g in fresh if g is not None))
    assert abs(float(plan.norm) - want) <= want * (HALF + 1e-9)
    for p in params:
        p.d["g"], p.gbits = None, None
    agree(params)


def test_gradients_that_come_later():
    """Tensors without a gradient at first, with the dtype the later one has."""
    p = Param(700, np.random.default_rng(52), param="f32", grad="bf16", copy="bf16")
    t = p.tensor(ps)
    g, t.grad = t.grad, None
    t.grad_dtype = torch.bfloat16
    plan = ps.AdamWPlan([t])
    dev, host = hps(wd=(0.1,))
    plan.step(dev, 1)
    agree([p])
    plan.set_grads([g])
    plan.step(dev, 1)
    p.step(host[0], 1)
    agree([p])
    with pytest.raises(ValueError):
        ps.AdamWPlan([ps.AdamWTensor(t.param, g, t.m, t.v, grad_dtype=torch.float16)])


def test_side_streams_and_two_plans_at_once():
    sets = [build([dict(param="f32", grad="bf16", copy="bf16", state="e4m3")], seed=30 + k, sizes=[100_003, 77]) for k in range(3)]
    dev, host = hps()
    errors = []
    torch.cuda.synchronize()

    def work(params):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                plan = ps.AdamWPlan([p.tensor(ps) for p in params])
                for t in range(1, 9):
                    plan.grad_norm(1e9)
                    plan.step(dev, t, clipped=True, rounding=1)
                s.synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(p,)) for p in sets]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for params in sets:
        for t in range(1, 9):
            for p in params:
                p.step(host[p.group], t, rounding=1)
        agree(params)


def test_explicit_stream_orders_with_its_own_work():
    p = Param(3_000_000, np.random.default_rng(31), grad="f32")
    s = torch.cuda.Stream()
    g = p.d["g"].t
    torch.cuda.synchronize()
    plan = ps.AdamWPlan([p.tensor(ps)])
    dev, host = hps(wd=(0.1,))
    with torch.cuda.stream(s):
        for _ in range(20):
            g.mul_(1.0)
        g.mul_(2.0)
    plan.grad_norm(stream=s)
    plan.step(dev, 4, clipped=True, stream=s)
    s.synchronize()
    p.set_grad(p.g * np.float32(2))
    p.step(host[0], 4)
    agree([p])


def device_coeffs(hp, t, lr_mul=1.0):
    c = dict(oracle.coeffs(hp, t))
    lr = hp.lr * float(np.float32(lr_mul))
    c["A"], c["CWD"] = np.float32(lr / (1.0 - hp.beta1 ** t)), np.float32(lr * hp.weight_decay)
    return c


def test_device_counted_steps_equal_numbered_ones():
    """The device's double pow may differ from the host's in its last place, which moves an fp32 scalar by at most one
    step, and only where the value lies at a border: the moments do not depend on it (bit-equal), weights by 3 half steps of the
    update beside their own rounding."""
    rng = np.random.default_rng(32)
    a, b = [Param(5000, np.random.default_rng(33), grad="f32", state="f32") for _ in range(2)]
    dev, _ = hps(wd=(0.1,))
    pa, pb = ps.AdamWPlan([a.tensor(ps)]), ps.AdamWPlan([b.tensor(ps)])
    for t in range(1, 31):
        g = rng.normal(0, 1e-3, 5000).astype(np.float32)
        a.new_grad(g), b.new_grad(g)
        pa.step(dev, t)
        pb.step(dev)
    torch.cuda.synchronize()
    assert int(pb.step_count) == 30
    for k in ("m", "v"):
        assert np.array_equal(a.d[k].host(), b.d[k].host())
    x, y = a.d["w"].host().astype(np.float64), b.d["w"].host().astype(np.float64)
    # 30 updates of at most lr * 10 (|m / sqrt(v)| <= 1 / sqrt(1 - beta2) * (1 - beta1) < 10, bias corrections < 3.2)
    assert np.all(np.abs(x - y) <= 30 * (4 * HALF * 1e-3 * 32 + 2 * HALF * np.abs(x)))


def test_counted_steps_skip_and_scale():
    p = Param(4000, np.random.default_rng(34), grad="f32", state="f32")
    plan = ps.AdamWPlan([p.tensor(ps)])
    dev, host = hps(wd=(0.1,))
    plan.step_count.fill_(41)
    plan.lr_mul.fill_(0.5)
    bad = p.g.copy()
    bad[7] = np.inf
    good = p.g.copy()
    for g, count in ((good, 42), (bad, 42), (good, 43)):
        p.new_grad(g)
        plan.grad_norm(1e9)
        plan.step(dev, clipped=True)
        assert int(plan.step_count) == count
        if np.isfinite(g).all():
            m0, v0 = p.moments()
            w, m, v, _ = ref.update(p.w, p.g, m0, v0, device_coeffs(host[0], count, 0.5), 1.0, False, np.float32)
            assert np.array_equal(p.d["m"].host(), m) and np.array_equal(p.d["v"].host(), v)
            got = p.d["w"].host()
            assert np.all(np.abs(got.astype(np.float64) - w) <= 4 * HALF * (np.abs(w) + 1e-2))
            p.w, p.m, p.v = got.copy(), m, v
    agree([p])


def test_captured_training_step_replays():
    """Norm and counted step in a graph, replayed with new gradients, eager work and synchronizations in between, the
    learning rate changed on the way; against the same calls made eagerly."""
    mk = lambda: build([dict(param="f32", grad="bf16", copy="bf16", state="e4m3"),   # noqa: E731
                        dict(param="bf16", grad="f16", state="f32")], sizes=[3, 700, 40_001], seed=35)
    a, b = mk(), mk()
    pa, pb = ps.AdamWPlan([p.tensor(ps) for p in a]), ps.AdamWPlan([p.tensor(ps) for p in b])
    dev, _ = hps()

    def once(plan):
        plan.grad_norm(0.02)
        plan.step(dev, clipped=True, rounding=1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        once(pb)
    rng = np.random.default_rng(36)
    for t in range(1, 8):
        for x, y in zip(a, b):
            g = rng.normal(0, 1e-3, x.n).astype(np.float32)
            if t == 4 and x.n == 700:
                g[3] = np.nan
            x.new_grad(g), y.new_grad(g)
        if t == 3:
            pa.lr_mul.fill_(0.25), pb.lr_mul.fill_(0.25)
        once(pa)
        graph.replay()
        torch.randn(1000, device="cuda").sum().item()
        for x, y in zip(a, b):
            for k, d in x.d.items():
                if d is not None:
                    assert np.array_equal(d.host().view(np.uint8), y.d[k].host().view(np.uint8)), (t, k, x.n)
    assert int(pa.step_count) == int(pb.step_count) == 6 and int(pb.skipped) == 1


def test_two_graphs_of_one_plan_replayed_in_turn():
    p, q = [Param(9000, np.random.default_rng(37), grad="f32", state="e4m3") for _ in range(2)]
    pp, pq = ps.AdamWPlan([p.tensor(ps)]), ps.AdamWPlan([q.tensor(ps)])
    dev, _ = hps(wd=(0.1,))
    graphs = []
    torch.cuda.synchronize()
    for clip in (1e-3, 1e9):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pq.grad_norm(clip)
            pq.step(dev, clipped=True)
        graphs.append(g)
    for t in range(6):
        pp.grad_norm((1e-3, 1e9)[t % 2])
        pp.step(dev, clipped=True)
        graphs[t % 2].replay()
        torch.cuda.synchronize()
        for k in ("w", "m", "v", "ms", "vs"):
            assert np.array_equal(p.d[k].host(), q.d[k].host()), (t, k)


# ---------------------------------------------------------------------------
# refusals that need a plan
# ---------------------------------------------------------------------------

def test_step_refusals():
    p = Param(300, np.random.default_rng(38), param="bf16", residual=False)
    f = Param(300, np.random.default_rng(39), group=1)
    plan = ps.AdamWPlan([p.tensor(ps), f.tensor(ps)])
    ok = [ps.HParams(algo=0, split_mode=2, lr=1e-3)] * 2

    def status(groups=ok, step=1, clipped=0, rounding=0):
        arr = (ps.CHParams * max(1, len(groups)))(*[g.c() for g in groups])
        return ps.lib().ps_adamw_step(plan._h, arr, len(groups), step, clipped, rounding, None)
    H = ps.HParams
    cases = [(dict(groups=[]), 1, "n_groups"), (dict(groups=ok[:1]), 1, "group 1"), (dict(groups=ok * 9), 1, "n_groups"),
             (dict(groups=[H(algo=0, split_mode=2), H(algo=1, split_mode=2)]), 1, "algo"),
             (dict(groups=[H(algo=0, split_mode=2), H(algo=0, split_mode=0)]), 1, "split_mode"),
             (dict(groups=[H(algo=0)] * 2), 1, "STOCHASTIC"), (dict(groups=[ok[0], H(algo=0, split_mode=2, lr=-1.0)]), 1, "lr"),
             (dict(step=-1), 1, "step"), (dict(clipped=2), 1, "clipped"), (dict(rounding=2), 1, "rounding"),
             (dict(groups=[H(algo=1, split_mode=2)] * 2, step=0), 4, "ADAM")]
    for kw, want, says in cases:
        assert status(**kw) == want and says in ps.last_error(), (kw, ps.last_error())
    L = ps.lib()
    for args in ((0.0, 1.0), (-1.0, 1.0), (float("nan"), 1.0), (1.0, 0.0), (1.0, float("inf")), (1.0, float("nan"))):
        assert L.ps_adamw_grad_norm(plan._h, *args, None) == 1
    ptrs = (ctypes.c_void_p * 2)(p.d["g"].t.data_ptr(), f.d["m"].t.data_ptr())
    assert L.ps_adamw_set_grads(plan._h, ptrs, 1, None) == 1
    assert L.ps_adamw_set_grads(plan._h, ptrs, 2, None) == 1 and "overlap" in ps.last_error()
    ptrs[1] = f.d["g"].t.data_ptr() + 2
    assert L.ps_adamw_set_grads(plan._h, ptrs, 2, None) == 2
    with pytest.raises(ValueError):
        plan.set_grads([p.d["g"].t])
    with pytest.raises(ValueError):
        plan.set_grads([p.d["g"].t, torch.zeros(300, device="cuda", dtype=torch.float64)])
    agree([p, f])                                           # nothing was touched
    plan.close()
    with pytest.raises(ValueError, match="closed"):
        plan.step(ok, 1)
    plan.close()


def test_plan_creation_is_refused_under_capture():
    t = Param(300, np.random.default_rng(40)).tensor(ps)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    rec = (ps.CAdamWTensor * 1)(ps._adamw_record(0, t))
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1.0)
        h = ctypes.c_void_p()
        st = ps.lib().ps_adamw_plan_create(rec, 1, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream,
                                           ctypes.byref(h))
        says = ps.last_error()
    assert st == 4 and "captured" in says
    g.replay()
    torch.cuda.synchronize()
    assert float(x[0]) == 1.0                               # the capture went on


# ---------------------------------------------------------------------------
# the e4m3 codec
# ---------------------------------------------------------------------------

def code_of(x, signed):
    d = torch.from_numpy(x).cuda()
    c = torch.full((x.size,), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.zeros(ref.blocks_of(x.size), device="cuda")
    ps.encode_fp8(d, c, s, ps.MOMENT_SIGNED if signed else ps.MOMENT_UNSIGNED)
    return c, s


@pytest.mark.parametrize("signed", [True, False])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 256, 257, 2047, 2048, 2049, 1_000_003])
def test_codec_equals_the_reference(signed, n):
    rng = np.random.default_rng(n)
    x = (rng.normal(0, 1, n) * np.exp(3 * rng.normal(0, 1, n))).astype(np.float32)
    x[rng.random(n) < 0.05] = 0.0
    if not signed:
        x = x * x
    c, s = code_of(x, signed)
    wc, ws = ref.encode(x, signed)
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().numpy(), ws)
    y = torch.full((n,), 7.0, device="cuda")
    ps.decode_fp8(c, s, y, ps.MOMENT_SIGNED if signed else ps.MOMENT_UNSIGNED)
    assert np.array_equal(y.cpu().numpy().view(np.uint32), ref.decode(wc, ws, signed).view(np.uint32))
    c2, s2 = code_of(y.cpu().numpy(), signed)               # decoded and encoded again: the same values
    z = torch.empty_like(y)
    ps.decode_fp8(c2, s2, z, ps.MOMENT_SIGNED if signed else ps.MOMENT_UNSIGNED)
    assert torch.equal(y, z)


def test_conversion_rounds_every_border():
    """All e4m3 borders and their neighbours, both signs, in blocks whose scale is 1 (largest value 448)."""
    mids = ref.MIDS.astype(np.float32)
    y = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(1000)),
                        ref.VALUES.astype(np.float32), np.float32(2.0) ** np.arange(-149, -8).astype(np.float32)])
    y = np.concatenate([y, -y])
    y = np.concatenate([y, np.zeros(-y.size % 255, np.float32)]).reshape(-1, 255)
    x = np.concatenate([np.full((y.shape[0], 1), 448, np.float32), y], 1).reshape(-1).astype(np.float32)
    c, s = code_of(x, True)
    assert np.all(s.cpu().numpy() == 1.0)
    assert np.array_equal(c.cpu().numpy(), ref.e4m3_code(x))
    k = torch.arange(256, dtype=torch.uint8, device="cuda")
    d = torch.empty(256, device="cuda")
    ps.decode_fp8(k, torch.ones(1, device="cuda"), d, ps.MOMENT_SIGNED)
    got, fine = d.cpu().numpy(), np.arange(256) % 128 != 127
    assert np.array_equal(got[fine], ref.e4m3_value(np.arange(256))[fine]) and np.all(np.isnan(got[~fine]))


@pytest.mark.parametrize("top", [0.0, 1e-45, 1e-40, 2.0 ** -126, 1e-36, 1e-20, 447.99, 448.0, 448.01, 1e20, 3e38])
def test_codec_at_extreme_levels(top):
    rng = np.random.default_rng(41)
    x = (rng.uniform(-1, 1, 600) * top).astype(np.float32)
    x[100] = top
    for signed in (True, False):
        v = x if signed else np.abs(x)
        c, s = code_of(v, signed)
        wc, ws = ref.encode(v, signed)
        assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(c.cpu().numpy(), wc)


def test_moments_move_between_32_and_8_bits():
    """A run with fp32 moments goes on with e4m3 ones: encode, step, decode, step."""
    rng = np.random.default_rng(42)
    p = Param(10_007, rng, grad="f32", state="f32")
    dev, host = hps(wd=(0.1,))
    plan = ps.AdamWPlan([p.tensor(ps)])
    plan.step(dev, 1)
    p.step(host[0], 1)
    t, nb = p.tensor(ps), ref.blocks_of(p.n)
    c = {k: torch.zeros(p.n, dtype=torch.float8_e4m3fn, device="cuda") for k in "mv"}
    s = {k: torch.zeros(nb, device="cuda") for k in "mv"}
    ps.encode_fp8(t.m, c["m"], s["m"], ps.MOMENT_SIGNED)
    ps.encode_fp8(t.v, c["v"], s["v"], ps.MOMENT_UNSIGNED)
    ps.AdamWPlan([ps.AdamWTensor(t.param, t.grad, c["m"], c["v"], s["m"], s["v"])]).step(dev, 2)
    ps.decode_fp8(c["m"], s["m"], t.m, ps.MOMENT_SIGNED)
    ps.decode_fp8(c["v"], s["v"], t.v, ps.MOMENT_UNSIGNED)
    plan.step(dev, 3)
    p.m, p.ms = ref.encode(p.m, True)
    p.v, p.vs = ref.encode(p.v, False)
    p.state = "e4m3"
    p.step(host[0], 2)
    p.m, p.v = p.moments()
    p.ms = p.vs = None
    p.state = "f32"
    p.step(host[0], 3)
    agree([p])
