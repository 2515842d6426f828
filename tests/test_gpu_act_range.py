"""GPU tests of the activation checkpoints at the top of each type's range: a
finite value that was saved is finite when it is read.

The largest codes of a block are rounded up past the type's largest value: of
fp16 from 63488 on (to 2^16), of bf16 and fp32 from 1.9375 * 2^127 on (to 2^128;
the weight gradient leaves those infinite).
Infinities are compared as they are."""
import math

import pytest
import torch

import act_ref as ref
from act_util import DT, codes, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


def top(dtype):
    """Values on both sides of the border, all finite, and the border itself, in the middle of a block."""
    f = torch.finfo(DT[dtype])
    border = 63488.0 if dtype == "f16" else 1.9375 * 2.0 ** 127
    below = border * (1 - f.eps / 2)
    x = torch.zeros(2, 200, dtype=torch.float64)
    x[0, 40:48] = torch.tensor([below, border, f.max, -below, -border, -f.max, f.max / 2, 1.0], dtype=torch.float64)
    x[1, 199] = f.max
    x = x.to(DT[dtype])
    assert x.isfinite().all()
    return x


def want_of(code, scale, dtype):
    """What codes and scales stand for: their product, or the type's largest value where it is the power of two behind."""
    past, most = (2.0 ** 16, 65504.0) if dtype == "f16" else (2.0 ** 128, torch.finfo(DT[dtype]).max)
    v = ref.value(code, scale)
    return torch.where(v.abs() == past, v.sign() * most, v)


@pytest.mark.parametrize("dtype", list(DT))
def test_finite_values_decode_to_finite_ones(ps, dtype):
    x = top(dtype)
    c, s = codes(*x.shape), scales(*x.shape)
    ps.encode_act(x.cuda(), c, s)
    o = torch.empty_like(x, device="cuda")
    ps.decode_act(c, s, o)
    assert o.isfinite().all()
    want = want_of(c, s, dtype)
    assert torch.equal(o.cpu(), want.to(DT[dtype]))
    big = x.double().abs() > 1
    assert ((o.cpu().double() - x.double()).abs()[big] <= x.double().abs()[big] * 2.0 ** -4).all()    # half a step of a code


def test_what_was_not_finite_stays_so(ps):
    """NaN for NaN and infinities; values that fp16 has no room for are infinite in it, as in any conversion."""
    x = torch.zeros(1, 128)
    x[0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    for t in DT.values():
        c, s = codes(1, 128), scales(1, 128)
        ps.encode_act(x.to(t).cuda(), c, s)
        o = torch.empty(1, 128, dtype=t, device="cuda")
        ps.decode_act(c, s, o)
        assert o[0, :3].isnan().all() and (o[0, 3:] == 0).all()
    x[0, :4] = torch.tensor([7e4, 1e6, -1e6, 6.4e4])           # coded as 69632 or more, but the last: 2^16 in every scale
    c, s = codes(1, 128), scales(1, 128)
    ps.encode_act(x.cuda(), c, s)
    o = torch.empty(1, 128, dtype=torch.float16, device="cuda")
    ps.decode_act(c, s, o)
    assert o[0, 1:4].tolist() == [math.inf, -math.inf, 65504.0] and torch.equal(o.cpu(), want_of(c, s, "f16").half())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_the_largest_values(ps, dtype, act):
    """Backward from codes of the largest values: f is a or 0 there and f' 1 or 0, so every result is known."""
    kind = {"silu": ps.ACT_SILU, "gelu": ps.ACT_GELU, "gelu_tanh": ps.ACT_GELU_TANH}[act]
    a = top(dtype)
    b = torch.zeros_like(a)
    b[0, 40:48], b[1, 199] = 0.5, -0.25
    saved = [codes(*a.shape), scales(*a.shape), codes(*a.shape), scales(*a.shape)]
    out = torch.empty_like(a, device="cuda")
    ps.glu_forward(a.cuda(), out, kind, saved[0], saved[1], b=b.cuda(), b_code=saved[2], b_scale=saved[3])
    d = torch.full_like(a, 0.25).cuda()
    da, db, again = (torch.empty_like(d) for _ in range(3))
    ps.glu_backward(d, kind, saved[0], saved[1], da, b_code=saved[2], b_scale=saved[3], db=db, out=again)
    va, vb = want_of(saved[0], saved[1], dtype), b.double()
    large = va.abs() > 1e3                                      # f' is 1 or 0 in every type
    assert large[0, 40:47].all() and large[1, 199] and int(large.sum()) == 8
    t = lambda v: v[large].to(DT[dtype])  # noqa: E731
    assert torch.equal(da.cpu()[large], t(0.25 * vb * (va > 0)))
    assert torch.equal(db.cpu()[large], t(0.25 * va.clamp(min=0)))
    assert torch.equal(again.cpu()[large], t(va.clamp(min=0) * vb))
    # one input alone
    ps.glu_backward(d, kind, saved[0], saved[1], da, out=again)
    assert torch.equal(da.cpu()[large], t(0.25 * (va > 0)))
    assert torch.equal(again.cpu()[large], t(va.clamp(min=0)))


@pytest.mark.parametrize("t,n,k", [(1, 8, 200), (64, 40, 256), (200, 33, 330), (1030, 12, 300), (700, 300, 20), (192, 1024, 1152)])
def test_weight_gradients_of_the_largest_values(ps, t, n, k):
    """One token alone has a gradient for each row of dw, so that dw is its z: rows that end a step or a tile, and
    those that whole steps take. In fp16 z is code times scale, or one step less for powers of two in blocks whose scales
    reach the border, and finite."""
    dtype, f = "f16", torch.finfo(torch.float16)
    x = top(dtype)[0, 40:48].repeat(t, -(-k // 8))[:, :k].contiguous()
    x[:, 1::5] *= 0.001                                         # smaller values beside the largest
    c, s = codes(t, k), scales(t, k)
    ps.encode_act(x.cuda(), c, s)
    dy = torch.zeros(t, n, dtype=torch.float16)
    at = [(i * 37 + t - 1) % t for i in range(n)]
    dy[at, range(n)] = 1.0
    w, b = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    for db in (None, b):
        ps.linear_wgrad(dy.cuda(), c, w, scale=s, db=db)
        z, got = want_of(c, s, dtype)[at], w.cpu().double()
        assert got.isfinite().all()
        same = got == z.half().double()
        power = (torch.frexp(z.abs())[0] == 0.5) & (s.cpu()[at].repeat_interleave(128, 1)[:, :k] >= 256)
        assert (same | (power & (got == z * (1 - f.eps / 2)))).all()
        assert (got.abs() == f.max).any()
    assert (b == dy.double().sum(0).cuda()).all()


def test_fp16_weight_gradients_of_wider_values(ps):
    """Saved values beyond fp16 are infinite in a product with an fp16 dy, not cut to its largest value."""
    x = torch.zeros(1, 128)
    x[0, :4] = torch.tensor([1e6, 8e4, 65e3, 5e4])
    c, s = codes(1, 128), scales(1, 128)
    ps.encode_act(x.cuda(), c, s)
    w = torch.empty(8, 128, device="cuda")
    ps.linear_wgrad(torch.ones(1, 8, dtype=torch.float16, device="cuda"), c, w, scale=s)
    z = ref.value(c, s)[0]
    assert (w[:, :2] == math.inf).all() and (w[:, 2] == 65504).all() and (w[:, 3].cpu() == z[3]).all() and (w[:, 4:] == 0).all()
