"""GPU tests of the weight gradient from 8-bit inputs against 64 bits (act_ref)."""
import math

import pytest
import torch

import act_ref as ref
from act_util import DT, E4M3, Padded, acts, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


def inputs(t, n, k, dtype, scaled, seed=0):
    g = gen(seed + t + 3 * n + 7 * k)
    dy = acts(g, t, n, dtype, 0.3)
    x = acts(g, t, k, "f32", 0.3)
    v, s = ref.encode(x.double())
    if not scaled:
        v, s = ref.grid(x.double().clamp(-30, 30)), None
    return dy, v.to(E4M3).cuda(), None if s is None else s.float().cuda(), g


def run(ps, t, n, k, dtype="bf16", dw="f32", scaled=True, db=False, mul=False, add=False, accumulate=False, pad=0, seed=0):
    dy, code, scale, g = inputs(t, n, k, dtype, scaled, seed)
    m = torch.randn(k, generator=g) if mul else None
    a = torch.randn(k, generator=g) if add else None
    start = acts(g, n, k, dw, 0.1)
    w = Padded(n, k, dw, pad, 1, start if accumulate else None)
    b = torch.full((n,), 3.0, device="cuda") if db else None
    d = Padded(t, n, dtype, pad, 1, dy)
    ps.linear_wgrad(d.m, code, w.m, scale=scale, db=b, mul=None if m is None else m.cuda(), add=None if a is None else a.cuda(),
                    accumulate=accumulate)
    want, e, wb, eb = ref.wgrad(dy.double(), ref.value(code, scale), None if m is None else m.double(),
                                None if a is None else a.double())
    if accumulate:
        want = want + start.double()
        e = e + ref.F * want.abs()
        wb, eb = wb + 3.0, eb + ref.F * (wb.abs() + 3)
    ref.check(w.m, want, e, "dw")
    assert w.outside_is_untouched()
    if db:
        ref.check(b, wb, eb, "db")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 64, 64), (2, 17, 300), (31, 32, 256), (33, 33, 33), (64, 128, 128), (77, 129, 130),
                                   (100, 16, 1001), (129, 1001, 16), (500, 300, 8), (513, 24, 24), (700, 257, 511),
                                   (1000, 130, 1100), (2049, 1025, 1030), (1024, 1024, 1024), (3000, 64, 2048), (96, 1500, 1100)])
@pytest.mark.parametrize("scaled", [True, False])
def test_products(ps, dtype, t, n, k, scaled):
    run(ps, t, n, k, dtype, scaled=scaled)


@pytest.mark.parametrize("dw", list(DT))
@pytest.mark.parametrize("t,n,k", [(70, 40, 200), (1300, 200, 136), (600, 1030, 1025), (900, 20, 700)])
@pytest.mark.parametrize("opts", [dict(db=True), dict(mul=True), dict(add=True), dict(db=True, mul=True, add=True),
                                  dict(accumulate=True), dict(db=True, mul=True, add=True, accumulate=True)], ids=str)
def test_epilogue(ps, dw, t, n, k, opts):
    run(ps, t, n, k, dw=dw, pad=3, scaled=False, **opts)


def test_all_codes_and_every_place(ps):
    """Whole numbers whose sums are exact in fp32: a product of one-hot tokens puts each value in its own place."""
    t, n, k = 512, 272, 256
    code = torch.arange(256, dtype=torch.uint8).repeat(t, 1).cuda()
    code = torch.where((code & 0x7F) == 0x7F, 0, code)
    dy = torch.zeros(t, n, dtype=torch.bfloat16)
    for i in range(n):
        dy[(i * 37) % t, i] = float(1 + i % 5)
    w = torch.empty(n, k, device="cuda")
    ps.linear_wgrad(dy.cuda(), code, w)
    want = torch.tensor([float(1 + i % 5) for i in range(n)])[:, None] * code[0].cpu().view(E4M3).float()[None]
    assert torch.equal(w.cpu(), want)
    code = torch.randint(0, 256, (t, k), generator=gen(1), dtype=torch.uint8)
    code = torch.where((code & 0x7F) == 0x7F, 0, code)
    dy = torch.zeros(t, n, dtype=torch.bfloat16)
    for i in range(n):
        dy[(i * 37 + 5) % t, i] = 2.0
    ps.linear_wgrad(dy.cuda(), code.cuda(), w)
    assert torch.equal(w.cpu(), 2 * code.view(E4M3).float()[[(i * 37 + 5) % t for i in range(n)]])


def test_whole_scales_count(ps):
    """Scales that are no power of two: z is their product rounded to dy's type."""
    t, n, k = 40, 8, 200
    dy, code, scale, _ = inputs(t, n, k, "bf16", True)
    scale = scale * 0.7
    w = torch.empty(n, k, device="cuda")
    ps.linear_wgrad(dy.cuda(), code, w, scale=scale)
    z = (ref.value(code).float() * scale.cpu().repeat_interleave(128, 1)[:, :k]).bfloat16().double()
    want, e, _, _ = ref.wgrad(dy.double(), z, None, None)
    ref.check(w, want, e)


def test_no_tokens(ps):
    dy, code = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=E4M3, device="cuda")
    w, b = torch.full((8, 16), 2.0, device="cuda"), torch.full((8,), 2.0, device="cuda")
    ps.linear_wgrad(dy, code, w, db=b, accumulate=True)
    assert (w == 2).all() and (b == 2).all()
    ps.linear_wgrad(dy, code, w, db=b, add=torch.ones(16, device="cuda"))
    assert (w == 0).all() and (b == 0).all()


def test_non_finite_values_stay_in_their_row_or_column(ps):
    """Also where the row's neighbours in memory are NaN: columns next to the matrix, and rows behind it."""
    t, n, k = 100, 70, 90
    dy, code, scale, _ = inputs(t, n, k, "bf16", True)
    wide = torch.full((t + 9, n + 11), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:t, :n] = dy.cuda()
    w = torch.empty(n, k, device="cuda")
    ps.linear_wgrad(wide[:t, :n], code, w, scale=scale)
    assert w.isfinite().all()
    dy[3, 60] = math.inf
    code.view(torch.uint8)[50, 20] = 0x7F
    ps.linear_wgrad(dy.cuda(), code, w, scale=scale)
    bad = ~w.isfinite().cpu()
    assert bad[60].all() and bad[:, 20].all()
    bad[60], bad[:, 20] = False, False
    assert not bad.any()


def test_same_results_every_time(ps):
    dy, code, scale, _ = inputs(3000, 96, 640, "bf16", True)
    first = None
    for _ in range(3):
        w, b = torch.empty(96, 640, device="cuda"), torch.empty(96, device="cuda")
        size = ps.linear_wgrad_workspace_size(3000, 96, 640)
        ps.linear_wgrad(dy.cuda(), code, w, scale=scale, db=b, workspace=torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
        first = first or (w, b)
        assert torch.equal(w, first[0]) and torch.equal(b, first[1])


def test_past_32_bit_offsets(ps):
    """dy of more than 2^31 elements: tokens far apart count, each in its place."""
    t, n, k = 270_000, 8192, 64
    dy = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    code = torch.zeros(t, k, dtype=torch.uint8, device="cuda")
    g = gen(9)
    at = [0, 7, 131_071, 131_072, 262_143, 262_150, t - 1]
    rows, vals = acts(g, len(at), n, "bf16", 0.1), torch.randint(0, 120, (len(at), k), generator=g, dtype=torch.uint8)
    dy[at] = rows.cuda()
    code[at] = vals.cuda()
    w, b = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    ps.linear_wgrad(dy, code, w, db=b)
    want, e, wb, eb = ref.wgrad(rows.double(), vals.view(E4M3).double(), None, None)
    ref.check(w, want, e)
    ref.check(b, wb, eb)


def test_refusals_of_the_binding(ps):
    dy, code, scale, _ = inputs(16, 8, 128, "bf16", True)
    dy, w = dy.cuda(), torch.empty(8, 128, device="cuda")
    for change, says in ((dict(dw=w.t()), "dw"), (dict(dw=w.double()), "dtype"), (dict(code=code[:15]), "code"),
                         (dict(scale=scale.double()), "scale"), (dict(mul=torch.ones(127).cuda()), "mul"), (dict(db=torch.ones(9).cuda()), "db"),
                         (dict(add=torch.ones(128)), "add"), (dict(dy=dy[0]), "dimensions")):
        a = dict(dy=dy, code=code, dw=w, scale=scale)
        a.update(change)
        with pytest.raises(ValueError, match=says):
            ps.linear_wgrad(**a)
    with pytest.raises(ps.PSError, match="dy_type"):
        ps.linear_wgrad(dy.float(), code, w, scale=scale)
    dy, code, scale, _ = inputs(1024, 8, 128, "bf16", True)      # tokens enough to be split
    assert ps.linear_wgrad_workspace_size(1024, 8, 128) > 0
    with pytest.raises(ps.PSError, match="workspace"):
        ps.linear_wgrad(dy.cuda(), code, w, scale=scale, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
