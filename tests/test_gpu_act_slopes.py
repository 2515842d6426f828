"""GPU tests of the activations' slopes against 64 bits, to the places that fp32
arithmetic leaves them."""
import pytest
import torch

import act_ref as ref
from act_util import codes, gen, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


def slopes(ps, act, a, gen):
    """f' at about a, and where exactly: codes times scales with all their places."""
    c, s = codes(*a.shape), scales(*a.shape)
    ps.encode_act(a.cuda(), c, s)
    s *= torch.rand(s.shape, generator=gen).cuda() / 4 + 0.75
    kind = {"silu": ps.ACT_SILU, "gelu": ps.ACT_GELU, "gelu_tanh": ps.ACT_GELU_TANH}[act]
    da = torch.empty_like(a, device="cuda")
    ps.glu_backward(torch.ones_like(da), kind, c, s, da)
    x = (c.float() * s.repeat_interleave(128, 1)).cpu().double()     # a is this product in fp32
    return da.cpu().double(), ref.act(act, x)[1], x


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("size", [0.3, 2.0, 6.0])
def test_logistic_slopes_keep_their_places(ps, act, size):
    """f' = q + a q (1 - q) u' with q = 1 / (1 + e), e = exp(-u). Errors in units of F = 2^-24, each relative to its
    term: u is off by at most 6 (tanh's form: two constants, three products, a sum), which moves e by 6 |u|; the
    exponent's product and constant make that 8 |u|; exp2 and the reciprocal are within 2 (two more are left to
    exp2), 1 + e and a product within 1. So q is off by (8 |u| + 4)(1 - q) + 3 and 1 - q = e q by (8 |u| + 4) q + 6,
    since e's error moves q the other way, the whole term by both and 8 more (u' 6, two products), and the sum by one
    of the result. Nothing is relative to 1 where 1 - q is small. Where q is below 2^-126 it may be 0."""
    g = gen(int(10 * size))
    got, want, a = slopes(ps, act, torch.randn(256, 1024, generator=g) * size, g)
    u, du = a, torch.ones_like(a)
    if act == "gelu_tanh":
        c = (2 / torch.pi) ** 0.5
        u, du = 2 * c * (a + 0.044715 * a ** 3), 2 * c * (1 + 3 * 0.044715 * a * a)
    e = torch.exp(-u)
    q = 1 / (1 + e)
    p = e * q
    p = torch.where(p.isnan(), 1.0, p)
    k = 8 * u.abs() + 4
    eq, ep = k * p + 3, k * q + 6
    err = ref.F * (q * eq + (a * q * p * du).abs() * (eq + ep + 8) + want.abs()) + 2.0 ** -125 * (1 + (a * du).abs())
    off = (got - want).abs()
    assert (off <= err).all(), (float((off / err).max()), a[off > err][:4].tolist())


@pytest.mark.parametrize("size", [0.3, 2.0, 4.0])
def test_gelu_and_its_slope(ps, size):
    """w = Phi(-|a|) is e t P(t), e = exp(-a^2 / 2), t = 1 / (1 + 0.35 |a|), P of nine coefficients. In units of F: the
    exponent has two products and a constant, which move e by 1.5 a^2, and exp2 is within 2; t is off by 4 (a constant,
    a sum, the reciprocal within 2), which P takes with the factor sum i |c_i| t^i / P; each step of P adds one of its
    own size, at most 2 sum |c_i| t^i / P together; two more products, and one of the fit. q is w, or 1 - w with one
    rounding; f = a q has one more, and f' = q + a e / sqrt(2 pi) a product and a constant beside e's error, and its
    own. Below 2^-120 there may be nothing left."""
    g = gen(int(10 * size) + 1)
    got, want, a = slopes(ps, "gelu", torch.randn(256, 1024, generator=g) * size, g)
    out = torch.empty(256, 1024, device="cuda")
    ps.glu_forward(a.float().cuda(), out, ps.ACT_GELU)
    z = a.abs()
    t = 1 / (1 + 0.35 * z)
    c = [0.1396, 0.1399, 0.1198, 0.1056, 0.0232, 0.1593, 0.2558, 0.1440, 0.0292]       # sizes
    p = 0.5 * torch.special.erfcx(z / 2 ** 0.5) / t
    spread = sum(i * v * t ** i for i, v in enumerate(c)) / p
    size_p = sum(v * t ** i for i, v in enumerate(c)) / p
    ee = 1.5 * z * z + 2
    ew = ee + 4 + 4 * spread + 2 * size_p + 2 + 1
    w = 0.5 * torch.special.erfc(z / 2 ** 0.5)
    q = torch.where(a < 0, w, 1 - w)
    eq = ref.F * (ew * w + q)
    phi = torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    for name, g_, w_, err in (("f", out.cpu().double(), a * q, z * eq + ref.F * (a * q).abs()),
                              ("slope", got, want, eq + ref.F * (z * phi * (ee + 3) + want.abs()))):
        off = (g_ - w_).abs()
        assert (off <= err + 2.0 ** -120 * (1 + z)).all(), (name, float((off / err).max()))
