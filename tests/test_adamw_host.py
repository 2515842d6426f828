"""Host-side checks of the AdamW plan and the e4m3 codec that need no GPU:
record layouts, refusals (all before any device call) and the numpy
reference's own pins."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import adamw_ref as ref
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


def test_records_match_the_header(ps, tmp_path):
    recs = {"ps_adamw_tensor": ps.CAdamWTensor, "ps_adamw_control": ps.CAdamWControl}
    lines = ['#include <stdio.h>', '#include "ps.h"', "int main(void) {"]
    for rec, cls in recs.items():
        lines.append(f'  printf("%zu", sizeof({rec}));')
        lines += [f'  printf(" %zu", offsetof({rec}, {f[0]}));' for f in cls._fields_]
        lines.append('  printf("\\n");')
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    for line, cls in zip(out, recs.values()):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert ctypes.sizeof(ps.CAdamWControl) == 64


def _rec(ps, n=1000, **kw):
    base = dict(param=1 << 20, grad=2 << 20, m=3 << 20, v=4 << 20, numel=n, param_type=ps.TYPE_F32,
                grad_type=ps.TYPE_BF16, copy_type=ps.TYPE_BF16, state_type=ps.STATE_F32, group=0)
    base.update(kw)
    return ps.CAdamWTensor(**base)


def _size(ps, recs):
    arr, out = (ps.CAdamWTensor * max(1, len(recs)))(*recs), ctypes.c_size_t(0)
    return ps.lib().ps_adamw_workspace_size(arr, len(recs), ctypes.byref(out)), out.value


def _create(ps, recs, ws=1 << 30, size=1 << 24):
    arr, h = (ps.CAdamWTensor * max(1, len(recs)))(*recs), ctypes.c_void_p()
    return ps.lib().ps_adamw_plan_create(arr, len(recs), ws, size, None, ctypes.byref(h)), h


E8 = dict(state_type=1, m_scale=5 << 20, v_scale=6 << 20)
BF = dict(param_type=1, residual=7 << 20)


@pytest.mark.parametrize("change,status,says", [
    (dict(numel=-1), 3, "numel"),
    (dict(numel=(1 << 40) + 1), 3, "numel"),
    (dict(numel=1 << 36), 3, "too large"),
    (dict(reserved=1), 1, "reserved"),
    (dict(grad_type=3), 1, "grad_type"),
    (dict(grad_type=-1), 1, "grad_type"),
    (dict(param_type=2), 4, "param_type"),
    (dict(param_type=5), 1, "param_type"),
    (dict(state_type=2), 1, "state_type"),
    (dict(group=16), 1, "group"),
    (dict(group=-1), 1, "group"),
    (dict(grad=(2 << 20) + 8), 2, "grad"),
    (dict(param=(1 << 20) + 4), 2, "param"),
    (dict(m=0), 1, "m is NULL"),
    (dict(v=0), 1, "v is NULL"),
    (dict(m=(3 << 20) + 2), 2, "m is not"),
    (dict(residual=7 << 20), 1, "no residual"),
    (dict(copy=8 << 20, copy_type=0), 1, "copy_type"),
    (dict(copy=(8 << 20) + 8), 2, "copy"),
    (dict(BF, copy=8 << 20), 1, "no copy"),
    (dict(BF, residual=(7 << 20) + 2), 2, "residual"),
    (dict(E8, m_scale=0), 1, "m_scale"),
    (dict(E8, v_scale=(6 << 20) + 2), 2, "v_scale"),
])
def test_bad_tensors_are_refused(ps, change, status, says):
    got, _ = _size(ps, [_rec(ps), _rec(ps, **change)])
    assert got == status and says in ps.last_error()
    assert "tensor 1" in ps.last_error() or says == "too large"
    assert _create(ps, [_rec(ps), _rec(ps, **change)])[0] == status


def test_lists_and_workspaces_are_checked(ps):
    L = ps.lib()
    size = ctypes.c_size_t(0)
    assert L.ps_adamw_workspace_size(None, 2, ctypes.byref(size)) == 1
    assert L.ps_adamw_workspace_size(None, -1, ctypes.byref(size)) == 1
    assert L.ps_adamw_workspace_size(None, 0, None) == 1
    st, empty = _size(ps, [])
    assert st == 0 and empty >= 64
    st, need = _size(ps, [_rec(ps)])
    assert st == 0 and need > empty
    # a tensor without elements is passed by, its pointers unread
    assert _size(ps, [_rec(ps, numel=0, param=3, m=0, grad=5)])[0] == 0
    assert _create(ps, [_rec(ps)], size=need - 1)[0] == 7
    assert _create(ps, [_rec(ps)], ws=None, size=need)[0] == 7
    assert _create(ps, [_rec(ps)], ws=(1 << 30) + 128)[0] == 2
    assert L.ps_adamw_plan_create(None, 0, 1 << 30, 1 << 24, None, None) == 1


@pytest.mark.parametrize("recs", [
    [{}, {}],                                                     # the same tensor twice
    [{}, dict(param=9 << 20, m=10 << 20, v=(4 << 20) + 3984)],     # 16 bytes shared with the first v
    [dict(m=(1 << 20) + 3984)],                                    # m begins inside param
    [dict(E8, v_scale=(5 << 20) + 12)],                            # 4 scales each, one of them shared
    [dict(BF, residual=(1 << 20) + 1984)],
    [dict(grad=(1 << 20) + 16)],                                   # gradient inside its own parameter
    [{}, dict(param=9 << 20, m=10 << 20, v=11 << 20, grad=(3 << 20) + 16)],
])
def test_overlapping_arrays_are_refused(ps, recs):
    assert _create(ps, [_rec(ps, **r) for r in recs])[0] == 1
    assert "overlap" in ps.last_error()


def test_workspace_inside_an_array_is_refused(ps):
    assert _create(ps, [_rec(ps, n=1 << 20, param=1 << 30, m=1 << 31, v=1 << 32)], ws=(1 << 30) + 4096)[0] == 1
    assert "workspace" in ps.last_error()


@pytest.mark.parametrize("grad,refused", [((1 << 30) + 256, True), ((1 << 30) - 1008, True), ((1 << 30) - 2000, False)])
def test_gradients_inside_the_workspace_are_refused(ps, grad, refused):
    """1000 bf16 gradients behind, across and before the workspace's start; also where only the gradient counts. The
    second tensor has a fault of its own, found later, so that no list gets to a device call."""
    later = _rec(ps, param=(1 << 30) + 4096, m=9 << 20, v=10 << 20)
    for first in (_rec(ps, grad=grad), _rec(ps, grad=grad, param=0)):
        assert _create(ps, [first, later])[0] == 1
        assert ("grad overlaps the workspace" if refused else "the workspace overlaps an array of tensor 1") in ps.last_error()


def test_calls_without_a_plan_are_refused(ps):
    L = ps.lib()
    h = ps.HParams().c()
    assert L.ps_adamw_step(None, ctypes.byref(h), 1, 1, 0, 0, None) == 1
    assert L.ps_adamw_grad_norm(None, 1.0, 1.0, None) == 1
    assert L.ps_adamw_set_grads(None, None, 0, None) == 1
    assert L.ps_adamw_plan_destroy(None) == 0


def test_codec_arguments(ps):
    L = ps.lib()
    for f, order in ((L.ps_encode_fp8, (0, 1, 2)), (L.ps_decode_fp8, (1, 2, 0))):
        good = (1 << 20, 2 << 20, 3 << 20)                        # x, code, scale
        call = lambda a, n=10, kind=0: f(a[order[0]], a[order[1]], a[order[2]], n, kind, None)  # noqa: E731
        assert call(good, kind=2) == 1
        assert call(good, n=-1) == 3
        assert call(good, n=(1 << 40) + 1) == 3
        for i in range(3):
            assert call(tuple(0 if j == i else p for j, p in enumerate(good))) == 1
            assert call(tuple(p + 2 if j == i else p for j, p in enumerate(good))) == 2
        assert call((0, 0, 0), n=0) == 0


def test_binding_refuses_wrong_tensors(ps):
    torch = pytest.importorskip("torch")
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt)  # noqa: E731
    T = ps.AdamWTensor
    bad = [
        T(None, None),
        T(f(8), f(9), f(8), f(8)),
        T(f(8), f(8, torch.float64), f(8), f(8)),
        T(f(8, torch.float16), f(8), f(8), f(8)),
        T(f(8), f(8)),
        T(f(8), f(8), f(8), f(8, torch.uint8)),
        T(f(8), f(8), f(8, torch.uint8), f(8, torch.uint8)),
        T(f(8), f(8), f(8), f(8), f(1), f(1)),
        T(f(300), f(300), f(300, torch.uint8), f(300, torch.uint8), f(1), f(1)),
        T(f(8), f(8), f(8), f(8), copy=f(8)),
        T(f(16)[::2], f(8), f(8), f(8)),
        T(f(8, torch.bfloat16), f(8), f(8), f(8), residual=f(8)),
    ]
    for t in bad:
        with pytest.raises(ValueError):
            ps.AdamWPlan([t])
    with pytest.raises(ValueError, match="not on a GPU"):
        ps.AdamWPlan([T(f(8), f(8), f(8), f(8))])
    for x, c, s in ((f(8), f(8), f(1)), (f(8), f(8, torch.uint8), f(2)), (f(8, torch.float64), f(8, torch.uint8), f(1)),
                    (f(16)[::2], f(8, torch.uint8), f(1))):
        with pytest.raises(ValueError):
            ps.encode_fp8(x, c, s, 0)
        with pytest.raises(ValueError):
            ps.decode_fp8(c, s, x, 0)


@pytest.mark.parametrize("dtype", ["float8_e4m3fnuz", "float8_e5m2", "float8_e5m2fnuz", "float8_e8m0fnu", "bool"])
def test_binding_refuses_bytes_that_are_no_e4m3_codes(ps, dtype):
    """Other 8-bit floats have another bias or other places; their bytes would be moments of other values."""
    torch = pytest.importorskip("torch")
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt)  # noqa: E731
    other, code = f(8, torch.uint8).view(getattr(torch, dtype)), f(8, torch.uint8)
    for m, v in ((other, code), (code, other), (other, other)):
        with pytest.raises(ValueError, match="dtype"):
            ps.AdamWPlan([ps.AdamWTensor(f(8), f(8), m, v, f(1), f(1))])
    for call in (lambda: ps.encode_fp8(f(8), other, f(1), 0), lambda: ps.decode_fp8(other, f(1), f(8), 0)):
        with pytest.raises(ValueError, match="dtype"):
            call()


@pytest.mark.parametrize("dtype", ["float8_e4m3fn", "uint8", "int8"])
def test_binding_takes_e4m3_codes_and_plain_bytes(ps, dtype):
    torch = pytest.importorskip("torch")
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt)  # noqa: E731
    code = f(8, torch.uint8).view(getattr(torch, dtype))
    with pytest.raises(ValueError, match="not on a GPU"):
        ps.AdamWPlan([ps.AdamWTensor(f(8), f(8), code, code.clone(), f(1), f(1))])
    with pytest.raises(ValueError, match="not on a GPU"):
        ps.decode_fp8(code, f(1), f(8), 0)


# ---- the numpy reference itself ----

def test_reference_codes_equal_torch():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    fine = ~np.isnan(want)
    assert list(codes[~fine]) == [127, 255]
    assert np.array_equal(ref.e4m3_value(codes)[fine].view(np.uint32), want[fine].view(np.uint32))
    rng = np.random.default_rng(1)
    mids = ref.MIDS.astype(np.float32)
    y = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(1000)),
                        ref.VALUES.astype(np.float32), np.exp(rng.uniform(-20, 6.1, 20000)).astype(np.float32)])
    y = np.concatenate([y, -y])
    assert np.array_equal(ref.e4m3_code(y), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scale_is_the_smallest_power_of_two():
    top = np.concatenate([np.float32(448) * 2.0 ** np.arange(-117, 110, 7), np.float32(449) * 2.0 ** np.arange(-117, 110, 7),
                          [0.0, 1e-45, 1e-38, 3e38]]).astype(np.float32)
    s = ref.block_scale(top).astype(np.float64)
    assert np.all(top <= 448 * s) and np.all((s == 2.0 ** -126) | (top > 224 * s))
    # the bit form that kernels use: a carry out of the mantissa bits above 1.75
    e = np.maximum(((top.view(np.uint32).astype(np.int64) + 0x1FFFFF) >> 23) - 8, 1)
    assert np.array_equal(s, 2.0 ** (e - 127.0))


def test_reference_stochastic_cut_is_unbiased():
    """The mean over all 2^16 random values is y to within one unit of its last kept place / 2^16, plus the
    rounding of y + 2^-6 below the normal range (2^-30)."""
    bits = np.arange(65536)
    for y in (0.0, 2.0 ** -12, 0.003, 2.0 ** -6, 0.017, 1.0, 1.06, 3.3, 223.0, 447.9, 448.0):
        y = np.float32(y)
        q = ref.stochastic_cut(np.full(65536, y), bits)
        place = 2.0 ** (max(np.floor(np.log2(y)) if y else -6, -6) - 3)
        assert set(np.unique(q)) <= set(ref.VALUES.astype(np.float32))
        assert abs(q.astype(np.float64).mean() - float(y)) <= place / 65536 + 2.0 ** -30


def test_reference_update_against_the_oracle_step():
    """fp32 moments and weights: the contract without fma stays within a few roundings of the oracle's step."""
    rng = np.random.default_rng(2)
    n = 4096
    w, g = rng.normal(0, 0.02, n).astype(np.float32), rng.normal(0, 1e-3, n).astype(np.float32)
    m, v = rng.normal(0, 1e-4, n).astype(np.float32), (rng.normal(0, 1e-3, n) ** 2).astype(np.float32)
    for algo in (0, 1):
        hp = oracle.HParams(algo=algo, lr=1e-3, weight_decay=0.1)
        c = oracle.coeffs(hp, 7)
        w32, m32, v32, _ = ref.update(w, g, m, v, c, 1.0, algo == 1, np.float32)
        w64, m64, v64, _ = ref.update(w, g, m, v, c, 1.0, algo == 1, np.float64)
        h = 2.0 ** -24
        big_m = np.abs(c["B1"] * m) + np.abs(c["C1"] * g)
        assert np.all(np.abs(m32 - m64) <= 3 * h * big_m) and np.all(np.abs(v32 - v64) <= 4 * h * v64)
        # u: m (3 h of its terms), r and d (5 h), quotient and factor (3 h); w' rounds the difference once
        scale = np.abs(c["A"] if algo == 0 else c["AG"] + c["AM"]) * (big_m + np.abs(g)) / (np.sqrt(v64) * c["RS2"])
        assert np.all(np.abs(w32 - w64) <= 16 * h * scale + 2 * h * np.abs(w64))


@pytest.mark.parametrize("algo", [0, 1])
def test_reference_update_is_the_optimizers_of_torch(algo):
    """Twenty steps of the formula in 64 bits against torch.optim.AdamW and NAdam (decoupled decay). The scalars are
    rounded to fp32: m, v and their roots are off by at most 2^-24 for each of the scalars that make them (2 in m and in
    v a step, relative), the update by 2^-24 for each of its four more, so by (2 + 1 + 4) 2^-24 relative to its terms, and a
    step's terms are at most lr (1 + wd |w|) times |m^| / sqrt(v^) <= 10, or 20 with the gradient's own term."""
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    n, lr, wd, steps = 500, 1e-2, 0.1, 20
    w = rng.normal(0, 0.5, n)
    t = torch.tensor(w, requires_grad=True)
    opt = torch.optim.NAdam([t], lr=lr, weight_decay=wd, decoupled_weight_decay=True, momentum_decay=4e-3) if algo else \
        torch.optim.AdamW([t], lr=lr, weight_decay=wd)
    m, v = np.zeros(n), np.zeros(n)
    hp = oracle.HParams(algo=algo, lr=lr, weight_decay=wd)
    for step in range(1, steps + 1):
        g = rng.normal(0, 1e-2, n)
        t.grad = torch.tensor(g)
        opt.step()
        w, m, v, _ = ref.update(w, g, m, v, oracle.coeffs(hp, step), 1.0, algo == 1, np.float64)
        bound = step * 7 * 2.0 ** -24 * lr * (20 + wd * np.abs(w))
        assert np.all(np.abs(w - t.detach().numpy()) <= bound), step
