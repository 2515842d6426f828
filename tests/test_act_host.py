"""Host-side checks of the activation checkpoints that need no GPU: record
layouts, refusals (all before any device call), and the reference's gradients
against differences."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import act_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
M = 1 << 20


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


def test_records_match_the_header(ps, tmp_path):
    recs = {"ps_block_norm": ps.CBlockNorm, "ps_block_norm_fwd": ps.CBlockNormFwd, "ps_block_norm_bwd": ps.CBlockNormBwd,
            "ps_linear_wgrad_args": ps.CLinearWgrad}
    lines = ['#include <stdio.h>', '#include "ps.h"', "int main(void) {"]
    for rec, cls in recs.items():
        lines.append(f'  printf("%zu", sizeof({rec}));')
        lines += [f'  printf(" %zu", offsetof({rec}, {f[0]}));' for f in cls._fields_]
        lines.append('  printf("\\n");')
    lines.append('  printf("%d %d %d %d %d %d\\n", PS_ACT_BLOCK, PS_NORM_MAX_COLS, PS_NORM_GATE_BY_SEG, PS_NORM_MOD_BY_SEG,'
                 ' PS_NORM_MUL_PLUS_ONE, PS_ACT_GELU_TANH);')
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    for line, cls in zip(out, recs.values()):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert [int(x) for x in out[-1].split()] == [ps.ACT_BLOCK, ps.NORM_MAX_COLS, ps.NORM_GATE_BY_SEG, ps.NORM_MOD_BY_SEG,
                                                 ps.NORM_MUL_PLUS_ONE, ps.ACT_GELU_TANH]


def _refused(ps, status, got, says):
    assert status == got, (got, ps.last_error())
    assert says in ps.last_error(), ps.last_error()


@pytest.mark.parametrize("change,status,says", [
    (dict(type=3), 1, "type"), (dict(rows=-1), 3, "rows"), (dict(rows=1 << 31), 3, "rows"), (dict(cols=-1), 3, "cols"),
    (dict(cols=(1 << 24) + 1), 3, "cols"), (dict(rows=1 << 30, cols=1024, ld=1024), 3, "blocks"), (dict(ld=999), 3, "apart"),
    (dict(x=None), 1, "x is NULL"), (dict(code=None), 1, "code is NULL"), (dict(scale=None), 1, "scale is NULL"),
    (dict(x=M + 1), 2, "x is not"), (dict(scale=9 * M + 2), 2, "scale is not"), (dict(code=M + 2000), 1, "overlap"),
    (dict(scale=M), 1, "overlap"),
])
def test_codec_refusals(ps, change, status, says):
    a = dict(x=M, type=1, rows=100, cols=1000, ld=1000, code=5 * M, scale=9 * M)
    a.update(change)
    _refused(ps, status, ps.lib().ps_encode_act(a["x"], a["type"], a["rows"], a["cols"], a["ld"], a["code"], a["scale"], None),
             says)
    _refused(ps, status, ps.lib().ps_decode_act(a["code"], a["scale"], a["x"], a["type"], a["rows"], a["cols"], a["ld"], None),
             says)


def test_empty_matrices_need_no_arrays(ps):
    for rows, cols in ((0, 100), (100, 0), (0, 0)):
        assert ps.lib().ps_encode_act(None, 1, rows, cols, cols, None, None, None) == 0
        assert ps.lib().ps_decode_act(None, None, None, 1, rows, cols, cols, None) == 0
        assert ps.lib().ps_glu_forward(rows, cols, 1, 0, None, 0, None, 0, None, 0, None, None, None, None, None) == 0
        assert ps.lib().ps_glu_backward(rows, cols, 1, 0, None, 0, None, None, None, None, None, 0, None, 0, None, 0, None) == 0


GLU = dict(rows=100, cols=1000, type=1, act=0, a=M, lda=2000, b=M + 2000, ldb=2000, out=3 * M, ldo=1000, a_code=5 * M,
           a_scale=6 * M, b_code=7 * M, b_scale=8 * M)


@pytest.mark.parametrize("change,status,says", [
    (dict(type=-1), 1, "type"), (dict(act=3), 1, "activation"), (dict(rows=-5), 3, "rows"), (dict(a=None), 1, "a is NULL"),
    (dict(out=None), 1, "out is NULL"), (dict(lda=5), 3, "apart"), (dict(a_code=None), 1, "a_code is NULL"),
    (dict(b_scale=None), 1, "b_scale is NULL"), (dict(b=None), 1, "need b"), (dict(out=M), 1, "overlap"),
    (dict(out=M + 2000, ldo=2000), 1, "overlap"), (dict(out=M + 1998, ldo=2000, b=20 * M), 1, "overlap"),
    (dict(b_code=5 * M + 99999), 1, "overlap"), (dict(b=M + 2001), 2, "b is not"),
])
def test_glu_forward_refusals(ps, change, status, says):
    a = dict(GLU, **change)
    _refused(ps, status, ps.lib().ps_glu_forward(*a.values(), None), says)


GLUB = dict(rows=100, cols=1000, type=1, act=0, dout=3 * M, ldd=1000, a_code=5 * M, a_scale=6 * M, b_code=7 * M,
            b_scale=8 * M, da=M, lda=2000, db=M + 2000, ldb=2000, out=10 * M, ldo=1000)


@pytest.mark.parametrize("change,status,says", [
    (dict(act=-1), 1, "activation"), (dict(dout=None), 1, "dout is NULL"), (dict(da=None), 1, "da is NULL"),
    (dict(db=None), 1, "db is NULL"), (dict(b_code=None, b_scale=None), 1, "db needs"), (dict(b_code=None), 1, "b_code is NULL"),
    (dict(a_scale=None), 1, "a_scale is NULL"), (dict(da=M, db=M), 1, "overlap"), (dict(da=3 * M, lda=1000, db=3 * M, ldb=1000), 1, "overlap"),
    (dict(da=3 * M + 2, lda=1000), 1, "overlap"), (dict(out=3 * M), 1, "overlap"), (dict(out=5 * M), 1, "overlap"),
])
def test_glu_backward_refusals(ps, change, status, says):
    a = dict(GLUB, **change)
    _refused(ps, status, ps.lib().ps_glu_backward(*a.values(), None), says)


def _norm(ps, **kw):
    a = dict(rows=100, cols=1000, post_eps=1e-6, pre_eps=1e-6, residual_scale=1.0, branch_scale=1.0, type=1, vec_type=1,
             post_norm=1, pre_norm=1, post_weight=20 * M, mul=21 * M)
    a.update(kw)
    return ps.CBlockNorm(**a)


NORMS = [
    (dict(type=7), 1, "type"), (dict(vec_type=7), 1, "vec_type"), (dict(pre_norm=0), 1, "pre_norm"),
    (dict(post_norm=3), 1, "post_norm"), (dict(flags=8), 1, "flags"), (dict(pre_eps=-1.0), 1, "eps"),
    (dict(post_eps=math.nan), 1, "eps"), (dict(residual_scale=math.inf), 1, "scale"), (dict(branch_scale=math.nan), 1, "scale"),
    (dict(rows=-1), 3, "rows"), (dict(cols=16385), 4, "cols"), (dict(n_segs=-1), 3, "n_segs"), (dict(n_segs=65536, seg_start=M), 3, "n_segs"),
    (dict(n_segs=3), 1, "together"), (dict(seg_start=40 * M), 1, "together"), (dict(flags=1), 1, "segments"),
    (dict(flags=2), 1, "segments"), (dict(post_norm=0), 1, "post_weight"), (dict(flags=4, mul=None), 1, "MUL_PLUS_ONE"),
]


def _fwd(ps, rec, **kw):
    a = dict(x=M, ldx=1000, y=2 * M, ldy=1000, h=3 * M, ldh=1000, n=4 * M, ldn=1000, h_code=5 * M, h_rstd=6 * M,
             y_code=7 * M, y_rstd=8 * M)
    a.update(kw)
    return ps.lib().ps_block_norm_forward(rec, ps.CBlockNormFwd(**a), None)


def _bwd(ps, rec, **kw):
    a = dict(dn=M, lddn=1000, dh=2 * M, lddh=1000, dx=3 * M, lddx=1000, dy=4 * M, lddy=1000, h_code=5 * M, h_rstd=6 * M,
             y_code=7 * M, y_rstd=8 * M, d_post_weight=9 * M, d_mul=10 * M, workspace=64 * M, workspace_bytes=1 << 30)
    a.update(kw)
    return ps.lib().ps_block_norm_backward(rec, ps.CBlockNormBwd(**a), None)


@pytest.mark.parametrize("change,status,says", NORMS)
def test_block_norm_refusals(ps, change, status, says):
    _refused(ps, status, _fwd(ps, _norm(ps, **change)), says)
    _refused(ps, status, _bwd(ps, _norm(ps, **change)), says)
    size = ctypes.c_size_t(5)
    _refused(ps, status, ps.lib().ps_block_norm_workspace_size(_norm(ps, **change), size), says)
    assert size.value == 0


@pytest.mark.parametrize("norm,change,status,says", [
    ({}, dict(x=None), 1, "x is NULL"), ({}, dict(n=None), 1, "n is NULL"), ({}, dict(h=None), 1, "h is NULL"),
    ({}, dict(ldy=5), 3, "apart"), ({}, dict(y=None), 1, "h needs y"), ({}, dict(y=None, h=None), 1, "needs y"),
    ({}, dict(n=M), 1, "overlap"), ({}, dict(h=2 * M), 1, "overlap"), ({}, dict(h=M, ldh=1001), 1, "overlap"),
    ({}, dict(h=4 * M), 1, "overlap"), ({}, dict(y_scale=9 * M), 1, "without a post_norm"),
    (dict(post_norm=0, post_weight=None), {}, 1, "need a post_norm or a gate"),
    (dict(post_norm=0, post_weight=None, gate=30 * M), {}, 1, "y_rstd needs"),
    (dict(post_norm=0, post_weight=None, gate=30 * M), dict(y_rstd=None), 1, "y_scale is NULL"),
    (dict(post_norm=0, post_weight=None, gate=30 * M), dict(y_rstd=None, y_code=None, y_scale=9 * M), 1, "needs y_code"),
    (dict(post_weight=20 * M + 1), {}, 2, "post_weight"), (dict(mul=4 * M), {}, 1, "overlap"),
    ({}, dict(h_rstd=6 * M + 2), 2, "h_rstd"),
])
def test_block_norm_forward_refusals(ps, norm, change, status, says):
    _refused(ps, status, _fwd(ps, _norm(ps, **norm), **change), says)


@pytest.mark.parametrize("norm,change,status,says", [
    ({}, dict(dn=None), 1, "dn is NULL"), ({}, dict(dx=None), 1, "dx is NULL"), ({}, dict(h_code=None), 1, "h_code"),
    ({}, dict(h_rstd=None), 1, "h_rstd"), ({}, dict(y_code=None), 1, "y_code"), ({}, dict(y_rstd=None), 1, "y_rstd"),
    (dict(post_norm=0, post_weight=None, gate=30 * M), dict(d_post_weight=None), 1, "y_scale"),
    (dict(post_weight=None), {}, 1, "d_post_weight"), (dict(mul=None), {}, 1, "d_mul"), ({}, dict(d_add=11 * M), 1, "d_add"),
    ({}, dict(d_gate=11 * M), 1, "d_gate"), ({}, dict(dy=None), 1, "d_post_weight"), ({}, dict(reserved=1), 1, "reserved"),
    ({}, dict(accumulate=2), 1, "accumulate"), ({}, dict(workspace_bytes=100), 7, "workspace"),
    ({}, dict(workspace=None), 1, "workspace"), ({}, dict(workspace=64 * M + 8), 2, "workspace"),
    ({}, dict(workspace=3 * M), 1, "overlap"), ({}, dict(dx=2 * M, dy=2 * M), 1, "overlap"), ({}, dict(dx=M, dy=M), 1, "overlap"),
    ({}, dict(dx=2 * M + 2), 1, "overlap"), ({}, dict(d_mul=9 * M), 1, "overlap"), ({}, dict(lddx=999), 3, "apart"),
])
def test_block_norm_backward_refusals(ps, norm, change, status, says):
    _refused(ps, status, _bwd(ps, _norm(ps, **norm), **change), says)


WG = dict(tokens=500, out_features=100, in_features=1000, dy=M, lddy=100, code=3 * M, scale=5 * M, dw=7 * M, lddw=1000,
          db=9 * M, workspace=64 * M, workspace_bytes=1 << 30, dy_type=1, dw_type=0)


@pytest.mark.parametrize("change,status,says", [
    (dict(tokens=-1), 3, "tokens"), (dict(out_features=-1), 3, "out_features"), (dict(in_features=1 << 25), 3, "in_features"),
    (dict(out_features=1 << 20, in_features=1 << 20), 3, "2^36"), (dict(tokens=1 << 30, in_features=1024), 3, "blocks"),
    (dict(dy_type=0), 4, "dy_type"), (dict(dy_type=5), 1, "dy_type"), (dict(dw_type=3), 1, "dw_type"),
    (dict(reserved=1), 1, "reserved"), (dict(accumulate=-1), 1, "accumulate"), (dict(dy=None), 1, "dy is NULL"),
    (dict(code=None), 1, "code is NULL"), (dict(dw=None), 1, "dw is NULL"), (dict(lddy=99), 3, "apart"), (dict(lddw=99), 3, "apart"),
    (dict(workspace_bytes=16), 7, "workspace"), (dict(workspace=None), 1, "workspace"), (dict(dw=3 * M), 1, "overlap"),
    (dict(db=7 * M), 1, "overlap"), (dict(mul=7 * M), 1, "overlap"), (dict(dw=7 * M + 2), 2, "dw is not"),
    (dict(workspace=M), 1, "overlap"),
])
def test_wgrad_refusals(ps, change, status, says):
    a = ps.CLinearWgrad(**dict(WG, **change))
    _refused(ps, status, ps.lib().ps_linear_wgrad(a, None), says)


def test_null_records(ps):
    L = ps.lib()
    _refused(ps, 1, L.ps_block_norm_forward(None, None, None), "norm is NULL")
    _refused(ps, 1, L.ps_block_norm_forward(_norm(ps), None, None), "io is NULL")
    _refused(ps, 1, L.ps_block_norm_backward(_norm(ps), None, None), "io is NULL")
    _refused(ps, 1, L.ps_block_norm_workspace_size(_norm(ps), None), "bytes is NULL")
    _refused(ps, 1, L.ps_linear_wgrad(None, None), "args is NULL")
    _refused(ps, 1, L.ps_linear_wgrad_workspace_size(1, 1, 1, None), "bytes is NULL")


def test_binding_refuses_tensors_without_a_gpu(ps):
    x, code = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8)
    for call in (lambda: ps.encode_act(x, code, torch.zeros(4, 2)), lambda: ps.glu_forward(x, x.clone(), ps.ACT_SILU),
                 lambda: ps.block_norm_forward(ps.BlockNorm(), x, x.clone()),
                 lambda: ps.linear_wgrad(x.bfloat16(), code, torch.zeros(256, 256))):
        with pytest.raises(ValueError, match="GPU"):
            call()


# --------------------------------------------------------------------------- the reference itself

@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_reference_slopes_are_differences(name):
    a = torch.linspace(-9, 9, 181, dtype=torch.float64)
    d = 1e-5
    f = lambda v: ref.act(name, v)[0]  # noqa: E731
    assert torch.allclose(ref.act(name, a)[1], (f(a + d) - f(a - d)) / (2 * d), rtol=1e-8, atol=1e-9)


@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("ada", [False, True])
def test_reference_gradients_are_differences(pre, post, gated, ada):
    """The backward formulas from exact normalised values, against central differences of the forward pass."""
    g = torch.Generator().manual_seed(len(pre + post) * 4 + gated * 2 + ada)
    rows, cols = 5, 7
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    starts = [0, 2, 2, 5]
    per = (3, cols) if ada else (cols,)
    c = dict(pre=pre, post=post, pre_eps=0.1, post_eps=0.2, alpha=1.3, beta=0.7, plus_one=ada, branch=True,
             seg=ref.segments(starts, rows), w1=rand(cols) if post != "none" else None, gate=rand(*per) if gated else None,
             mul=rand(*per), add=rand(*per) if ada else None)
    x, y, dn, dh = (rand(rows, cols) for _ in range(4))
    f = ref.forward(c, x, y)
    yh = f["y_hat"][0] if post != "none" else y
    got = ref.backward(c, dn, dh, f["h_hat"][0], f["h_rstd"][0], yh, f["y_rstd"][0] if post != "none" else None)

    def loss(**change):
        k = {**c, **{n: v for n, v in change.items() if n not in ("x", "y")}}
        o = ref.forward(k, change.get("x", x), change.get("y", y))
        return (o["n"][0] * dn).sum() + (o["h"][0] * dh).sum()
    d = 1e-6
    for name, key, v in (("dx", "x", x), ("dy", "y", y), ("d_post_weight", "w1", c["w1"]), ("d_gate", "gate", c["gate"]),
                         ("d_mul", "mul", c["mul"]), ("d_add", "add", c["add"])):
        if v is None:
            continue
        num = torch.zeros_like(v)
        for i in range(v.numel()):
            e = torch.zeros(v.numel(), dtype=torch.float64)
            e[i] = d
            e = e.view(v.shape)
            num.view(-1)[i] = (loss(**{key: v + e}) - loss(**{key: v - e})) / (2 * d)
        assert torch.allclose(got[name][0], num, rtol=1e-6, atol=1e-7), name


def test_reference_encode_is_the_nearest_code():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[every.isfinite()].unique()
    x = torch.linspace(-460, 460, 4001, dtype=torch.float64).clamp(-448, 448)
    near = (x[:, None] - every[None]).abs().amin(1)
    assert torch.equal((ref.grid(x) - x).abs(), near)
    x = torch.tensor([[1.0, -3.0, math.inf, math.nan, 0.0, 448.0 * 4]], dtype=torch.float64)
    v, s = ref.encode(x)
    assert s.item() == 4.0 and v[0, 2:4].isnan().all() and v[0, 5] == 448 and v[0, 1] == -0.75


def test_a_call_with_every_array_is_checked_whole(ps):
    """The call with the most arrays: each is held against all others, the last one (the workspace) too."""
    rec = _norm(ps, n_segs=3, seg_start=40 * M, gate=41 * M, add=42 * M, flags=7)
    every = dict(d_gate=43 * M, d_add=44 * M)
    for at in (M, 5 * M, 9 * M, 40 * M, 41 * M, 42 * M, 43 * M, 44 * M):
        _refused(ps, 1, _bwd(ps, rec, workspace=at, **every), "overlap")


def test_norm_rows_have_a_limit(ps):
    rec = ps.CBlockNorm(rows=(1 << 30) + 1, cols=1, type=1, vec_type=0, pre_norm=1)
    _refused(ps, 3, ps.lib().ps_block_norm_forward(rec, ps.CBlockNormFwd(), None), "2^30")
    _refused(ps, 3, ps.lib().ps_block_norm_backward(rec, ps.CBlockNormBwd(), None), "2^30")
    _refused(ps, 3, ps.lib().ps_block_norm_workspace_size(rec, ctypes.c_size_t(0)), "2^30")


@pytest.mark.parametrize("how", ["deepcopy", "pickle", "replace"])
def test_a_copied_norm_has_vectors_of_its_own(ps, how):
    """A used norm keeps the addresses of its vectors; a copy must not take them over."""
    import copy
    import dataclasses
    import pickle
    norm = ps.BlockNorm(mul=torch.ones(8), gate=torch.ones(8), post_norm=ps.NORM_RMS)
    first = norm._record(2, 8, torch.bfloat16, torch.device("cpu"))
    assert first.mul == norm.mul.data_ptr()
    if how == "deepcopy":
        other = copy.deepcopy(norm)
    elif how == "pickle":
        other = pickle.loads(pickle.dumps(norm))
    else:
        other = dataclasses.replace(norm, mul=torch.ones(8), gate=torch.ones(8))
    rec = other._record(3, 8, torch.bfloat16, torch.device("cpu"))
    assert (rec.rows, rec.mul, rec.gate) == (3, other.mul.data_ptr(), other.gate.data_ptr())
    assert other.mul.data_ptr() != norm.mul.data_ptr() and rec.post_norm == ps.NORM_RMS
    assert norm == norm and norm != other and len({norm, other}) == 2
