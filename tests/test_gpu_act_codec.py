"""GPU tests of the activation codec and the feed-forward activations against
64 bits (act_ref)."""
import math

import pytest
import torch

import act_ref as ref
from act_util import DT, E4M3, Padded, acts, codes, gen, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


SHAPES = [(1, 1), (1, 128), (3, 8), (2, 127), (5, 129), (7, 255), (1, 12288), (33, 1001), (64, 512), (257, 136), (2, 65536)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1), (8, 8)])
def test_codec(ps, dtype, rows, cols, pad, shift):
    g = gen(rows * 31 + cols)
    x = acts(g, rows, cols, dtype)
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0
    a = Padded(rows, cols, dtype, pad, shift, x)
    c, s = codes(rows, cols), scales(rows, cols)
    ps.encode_act(a.m, c, s)
    v, want = ref.encode(x.double())
    assert torch.equal(ref.dec(s), want)
    assert torch.equal(ref.value(c), v)
    o = Padded(rows, cols, dtype, pad, shift)
    ps.decode_act(c, s, o.m)
    assert torch.equal(o.m.cpu(), ref.value(c, s).to(DT[dtype]))
    assert o.outside_is_untouched()


@pytest.mark.parametrize("dtype", list(DT))
def test_codec_values_at_the_borders(ps, dtype):
    """Blocks of zeros, of the type's smallest and largest values, next to a change of scale, with and of
    non-finite values."""
    f = torch.finfo(DT[dtype])
    rows = [torch.zeros(128), torch.full((128,), f.max), torch.full((128,), -f.smallest_normal),
            torch.full((128,), f.smallest_normal * f.eps), torch.full((128,), 448.0), torch.full((128,), 450.0),
            torch.linspace(-448, 448, 128), torch.tensor([448 * (1 + f.eps)] * 128), torch.tensor([math.nan] * 128),
            torch.tensor([math.inf] * 128), torch.tensor([-0.0] * 128)]
    for at, bad in ((0, math.inf), (17, -math.inf), (127, math.nan)):
        r = torch.linspace(-3, 3, 128)
        r[at] = bad
        rows.append(r)
    x = torch.stack(rows).to(DT[dtype])
    c, s = codes(*x.shape), scales(*x.shape)
    ps.encode_act(x.cuda(), c, s)
    v, want = ref.encode(x.double())
    assert torch.equal(ref.dec(s), want)
    got = ref.value(c)
    assert torch.equal(got.isnan(), v.isnan())
    assert torch.equal(got.nan_to_num(), v.nan_to_num())
    o = torch.empty_like(x, device="cuda")
    ps.decode_act(c, s, o)
    assert torch.equal(o.cpu().nan_to_num(), ref.value(c, s).to(DT[dtype]).nan_to_num())


def test_decode_reads_the_whole_scale(ps):
    """A scale that is no power of two counts as it is."""
    c = torch.arange(256, dtype=torch.uint8).repeat(2, 1).cuda()
    s = torch.tensor([[0.3, 7.7], [1e-3, 2.0 / 3]], device="cuda")
    o = torch.empty(2, 256, device="cuda")
    ps.decode_act(c, s, o)
    want = c.cpu().view(E4M3).float() * s.cpu().repeat_interleave(128, 1)
    assert torch.equal(o.cpu().nan_to_num(), want.nan_to_num())


def test_codec_past_32_bit_offsets(ps):
    """More than 2^31 values: the first and last rows, and some between."""
    rows, cols = 33000, 65544
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 16383, 32767, 32768, rows - 1]
    part = acts(gen(5), len(at), cols, "bf16")
    x[at] = part.cuda()
    c, s = codes(rows, cols), scales(rows, cols)
    ps.encode_act(x, c, s)
    v, want = ref.encode(part.double())
    assert torch.equal(ref.value(c[at]), v) and torch.equal(ref.dec(s[at]), want)
    x.zero_()
    ps.decode_act(c, s, x)
    assert torch.equal(x[at].cpu(), (v * want.repeat_interleave(128, 1)[:, :cols]).bfloat16())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 129, 0), (17, 1001, 5), (64, 640, 0), (1, 11008, 0)])
def test_glu(ps, dtype, act, gated, rows, cols, pad):
    g = gen(rows + cols)
    kind = {"silu": ps.ACT_SILU, "gelu": ps.ACT_GELU, "gelu_tanh": ps.ACT_GELU_TANH}[act]
    xa, xb = (acts(g, rows, cols, dtype, 0.3).clamp(-9, 9) for _ in range(2))
    k = 2 if gated else 1
    both = Padded(rows, k * cols, dtype, pad, 1)                     # a and b are halves of one matrix
    a, b = both.m[:, :cols], both.m[:, cols:] if gated else None
    a.copy_(xa)
    if gated:
        b.copy_(xb)
    out = Padded(rows, cols, dtype, pad)
    c = [(codes(rows, cols), scales(rows, cols)) for _ in range(k)]
    saved = dict(a_code=c[0][0], a_scale=c[0][1])
    if gated:
        saved.update(b_code=c[1][0], b_scale=c[1][1])
    ps.glu_forward(a, out.m, kind, b=b, **saved)
    want, err = ref.glu(act, xa.double(), xb.double() if gated else None)
    ref.check(out.m, want, err, "out")
    assert out.outside_is_untouched() and both.outside_is_untouched()
    for x, (code, scale) in zip((xa, xb), c):
        v, s = ref.encode(x.double())
        assert torch.equal(ref.value(code), v) and torch.equal(ref.dec(scale), s)
    alone = Padded(rows, cols, dtype, 1)
    ps.glu_forward(a, alone.m, kind, b=b)                             # nothing saved: the same output
    assert torch.equal(alone.m, out.m)

    d = acts(g, rows, cols, dtype, 0.2)
    va, vb = ref.value(*c[0]), ref.value(*c[1]) if gated else None
    refs, errs = ref.glu_back(act, d.double(), va, vb)
    dd = Padded(rows, cols, dtype, pad, 0, d)
    for again in (False, True):
        grads = Padded(rows, k * cols, dtype, pad, 1)
        o = Padded(rows, cols, dtype, 2)
        ps.glu_backward(dd.m, kind, da=grads.m[:, :cols], db=grads.m[:, cols:] if gated else None,
                        out=o.m if again else None, **saved)
        ref.check(grads.m[:, :cols], refs[0], errs[0], "da")
        if gated:
            ref.check(grads.m[:, cols:], refs[1], errs[1], "db")
        if again:
            ref.check(o.m, refs[2], errs[2], "out again")
        assert grads.outside_is_untouched() and o.outside_is_untouched()
    for into in ("da", "db")[:k]:                                     # a gradient takes the place of dout
        here, other = Padded(rows, cols, dtype, pad, 0, d), Padded(rows, cols, dtype)
        ps.glu_backward(here.m, kind, da=here.m if into == "da" else other.m,
                        db=None if not gated else other.m if into == "da" else here.m, **saved)
        assert torch.equal(here.m, grads.m[:, :cols] if into == "da" else grads.m[:, cols:])


@pytest.mark.parametrize("act", [0, 1, 2])
def test_glu_of_large_and_non_finite_values(ps, act):
    """Large inputs saturate without NaN; NaN and infinities in a reach the output's and gradient's own elements only."""
    x = torch.zeros(2, 256, device="cuda")
    x[0, :6] = torch.tensor([1e30, -1e30, 3e38, -3e38, 100.0, -100.0])
    x[1, 5], x[1, 7] = math.nan, math.inf
    out, c, s = torch.empty_like(x), codes(2, 256), scales(2, 256)
    ps.glu_forward(x, out, act, a_code=c, a_scale=s)
    assert out[0].isfinite().all()
    assert torch.equal(out[0, :6].cpu(), torch.tensor([1e30, 0, 3e38, 0, 100.0, 0]))
    assert out[1, 5].isnan() and out[1, 7] == math.inf and int(out[1].isfinite().sum()) == 254
    d = torch.ones_like(x)
    da = torch.empty_like(x)
    ps.glu_backward(d, act, c, s, da)
    # 3e38 sets the block's scale to 2^120, where the code of 1e30 (less than 2^-20 of a scale) is 0: the slope there is 1/2
    assert torch.equal(da[0, :4].cpu(), torch.tensor([0.5, 0.5, 1, 0]))
    assert sorted(da[1].isnan().nonzero().flatten().tolist()) == [5, 7]


def test_no_rows(ps):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    c, s = codes(0, 256), scales(0, 256)
    ps.encode_act(x, c, s)
    ps.decode_act(c, s, x)
    ps.glu_forward(x, x.clone(), ps.ACT_SILU, a_code=c, a_scale=s)
    ps.glu_backward(x, ps.ACT_SILU, c, s, x.clone())


def test_refusals_of_the_binding(ps):
    x = torch.zeros(4, 256, device="cuda")
    c, s = codes(4, 256), scales(4, 256)
    for bad, says in ((dict(code=c[:3]), "code"), (dict(scale=s[:, :1]), "scale"), (dict(code=c.view(torch.float8_e5m2)), "code"),
                      (dict(x=x.double()), "dtype"), (dict(x=x.t()), "contiguous"), (dict(x=torch.zeros(4, 512, device="cuda")[:, ::2]), "contiguous"),
                      (dict(x=x[0]), "dimensions"), (dict(scale=s.cpu()), "scale"), (dict(code=None), "needed")):
        a = dict(x=x, code=c, scale=s)
        a.update(bad)
        with pytest.raises(ValueError, match=says):
            ps.encode_act(a["x"], a["code"], a["scale"])
    with pytest.raises(ps.PSError, match="overlap"):
        ps.glu_forward(x, x, ps.ACT_SILU)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_over_their_whole_range(ps, act):
    """fp32 against 64 bits from where f leaves 0 to where it is a; its tails go to 0 and a."""
    kind = {"silu": ps.ACT_SILU, "gelu": ps.ACT_GELU, "gelu_tanh": ps.ACT_GELU_TANH}[act]
    end = 80.0 if act == "silu" else 12.5 if act == "gelu" else 8.5     # f(-end) is above 2^-126
    a = torch.linspace(-end, end, 1 << 16, device="cuda").view(64, 1024)
    out = torch.empty_like(a)
    ps.glu_forward(a, out, kind)
    want, err = ref.glu(act, a.double().cpu(), None)
    ref.check(out, want, err, act)
    a = torch.tensor([[0.0, -0.0, 200.0, 1e30, 3e38, -200.0, -1e30, -3e38]], device="cuda")
    out = torch.empty_like(a)
    ps.glu_forward(a, out, kind)
    assert torch.equal(out, a.clamp(min=0))
