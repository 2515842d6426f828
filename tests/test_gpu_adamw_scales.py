"""GPU tests of the AdamW step on 8-bit moments at the ends of their scales'
range and with scales that ps_encode_fp8 would not make, bit for bit against the
formulas in float32."""
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

# fp32 weights: a lane has 4 elements of each of two blocks; bf16 weights: 8 of one. Ragged ends in both.
KINDS = [dict(param="f32", grad="f32"), dict(param="f32", grad="f32", copy="bf16"), dict(param="bf16", grad="f32")]
SIZES = [1, 9, 255, 512, 700, 2049]
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, seed=77)


def build(rng, **kw):
    out = []
    for kind in KINDS:
        for n in SIZES:
            out.append(Param(n, rng, state="e4m3", index=len(out), **{**kind, **kw}))
    return out


def agree(params):
    torch.cuda.synchronize()
    bad = [(i, p.param, d) for i, p in enumerate(params) for d in p.differences()]
    assert not bad, bad[:6]


def put(p, **arrays):
    """Other moments into the device arrays and the numpy state."""
    for k, a in arrays.items():
        setattr(p, k, a)
        p.d[k].t.copy_(torch.from_numpy(a))


def steps(params, grads, algo, rounding, split=0):
    dev, host = ps.HParams(algo=algo, split_mode=split, **HP), oracle.HParams(algo=algo, split_mode=split, **HP)
    plan = ps.AdamWPlan([p.tensor(ps) for p in params])
    for t in (1, 2, 3):
        for p in params:
            p.new_grad(grads(p.n))
        plan.step([dev], t, rounding=rounding)
        for p in params:
            p.step(host, t, rounding=rounding)
        agree(params)


@pytest.mark.parametrize("level", [1e-35, 1e-36, 1e-38, 1e-42, 1e-45])
@pytest.mark.parametrize("algo,rounding", [(0, 0), (1, 1)])
def test_first_moments_at_the_scales_floor(level, algo, rounding):
    """Blocks whose largest first moment is below 448 * 2^-126, down to subnormal moments: the scale stays at 2^-126."""
    rng = np.random.default_rng(60)
    params = build(rng, zero_state=True)

    def grads(n):
        g = (rng.normal(0, 1, n) * level).astype(np.float32)
        g[rng.random(n) < 0.2] = 0.0
        return g
    steps(params, grads, algo, rounding)
    held = [(p.ms == np.float32(2.0 ** -126)) & (ref.per_block_max(p.m & 127) > 0) for p in params]
    assert np.any(np.concatenate(held)) == (level > 1e-39)  # below, every code is zero


@pytest.mark.parametrize("split", [0, 2])
@pytest.mark.parametrize("gradient", [0.0, 1e-37])
def test_stored_codes_at_the_scales_floor(gradient, split):
    """Every code from stored moments with the smallest scales, decaying."""
    rng = np.random.default_rng(61)
    params = build(rng)
    for p in params:
        nb = ref.blocks_of(p.n)
        code = rng.integers(0, 127, p.n).astype(np.uint8)
        put(p, m=code | (rng.integers(0, 2, p.n) << 7).astype(np.uint8), v=rng.permutation(code),
            ms=np.full(nb, 2.0 ** -126, np.float32), vs=(2.0 ** rng.integers(-90, -60, nb)).astype(np.float32))
    steps(params, lambda n: (rng.normal(0, 1, n) * gradient).astype(np.float32), 0, 1, split)


@pytest.mark.parametrize("algo,rounding,split", [(0, 0, 0), (1, 1, 0), (0, 1, 2), (1, 0, 2)])
def test_scales_that_are_no_powers_of_two(algo, rounding, split):
    """A moment is its code times its scale, the one that ps_decode_fp8 gives, whoever made the scale."""
    rng = np.random.default_rng(62)
    params = build(rng)
    for p in params:
        nb = ref.blocks_of(p.n)
        put(p, ms=(p.ms * rng.uniform(1, 2, nb)).astype(np.float32), vs=(p.vs * rng.uniform(1, 2, nb)).astype(np.float32))
        for code, scale, kind, want in ((p.m, "ms", ps.MOMENT_SIGNED, p.moments()[0]), (p.v, "vs", ps.MOMENT_UNSIGNED, p.moments()[1])):
            x = torch.empty(p.n, device="cuda")
            ps.decode_fp8(torch.from_numpy(code).cuda(), p.d[scale].t, x, kind)
            assert np.array_equal(x.cpu().numpy(), want)
    steps(params, lambda n: rng.normal(0, 1e-3, n).astype(np.float32), algo, rounding, split)


def test_scales_of_zero_and_extreme_size():
    """Zero scales (a fresh state's, with codes left in place), subnormal and the largest ones."""
    rng = np.random.default_rng(63)
    params = build(rng)
    for p in params:
        nb = ref.blocks_of(p.n)
        level = np.array([0.0, 1e-45, 1e-40, 2.0 ** -127, 3e-38, 1.0, 3e16, 2.0 ** 56], np.float32)
        put(p, ms=level[rng.integers(0, 8, nb)], vs=np.minimum(level, 3e4)[rng.integers(0, 8, nb)].astype(np.float32))
    steps(params, lambda n: rng.normal(0, 1e-3, n).astype(np.float32), 0, 0)
