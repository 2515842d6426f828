"""GPU tests of the block norms at the widths where a kernel's shape changes:
whole waves of columns (multiples of 512) over many rows of a strip, one part a
lane up to 8192 columns, several above."""
import pytest
import torch

from test_gpu_block_norm import ADA, Case, ps  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    dict(rows=9000, cols=512, post="rms"), dict(rows=9000, cols=512, branch=False, pre="layer", add=True),
    dict(rows=2500, cols=1024, starts=[0, 7, 7, 1200, 2477], **ADA), dict(rows=5000, cols=1536, post="layer", gate=True, pad=8),
    dict(rows=700, cols=2560, gate=True, pre="layer"), dict(rows=1200, cols=4096, post="rms", beta=0.5),
    dict(rows=600, cols=5120, starts=[0, 250, 560], post="rms", **ADA), dict(rows=40, cols=4097, post="rms"),
    dict(rows=20, cols=5001, post="layer", gate=True, pre="layer", pad=1), dict(rows=9, cols=7681, gate=True),
    dict(rows=9, cols=8191, branch=False), dict(rows=530, cols=8192, post="rms"), dict(rows=5, cols=8193, gate=True),
    dict(rows=300, cols=9001, starts=[0, 100, 290], post="rms", **ADA), dict(rows=270, cols=12288, post="layer", gate=True),
    dict(rows=7, cols=12280, branch=False, pre="layer"), dict(rows=260, cols=16383, starts=[0, 120, 260], post="rms", **ADA),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['rows']}x{c['cols']}-{c.get('post')}-{c.get('branch', True)}")
def test_forward_and_backward(ps, case, dtype):  # noqa: F811
    t = Case(ps, dtype=dtype, **case)
    t.forward().check_forward()
    t.backward().check_backward()
    t.backward(with_dh=False).check_backward(with_dh=False)


@pytest.mark.parametrize("case", [dict(rows=3000, cols=1024, post="rms"), dict(rows=600, cols=5120, gate=True),
                                  dict(rows=300, cols=9001, post="rms", gate=True)], ids=str)
def test_outputs_in_place_of_inputs(ps, case):  # noqa: F811
    """dx in dh or dn and dy in the other; without dh, either in dn."""
    t = Case(ps, **case).forward()
    for with_dh in (True, False):
        t.backward(with_dh=with_dh)
        want = t.dx.m.clone(), t.dy.m.clone(), {k: v.clone() for k, v in t.g.items()}
        for which in (0, 1):
            dn, dh = t.mat(t.dn), t.mat(t.dh) if with_dh else None
            other = dh or t.mat()
            t.backward(with_dh=with_dh, dn=dn, dh=dh, dx=other if which else dn, dy=dn if which else other)
            assert torch.equal(t.dx.m, want[0]) and torch.equal(t.dy.m, want[1])
            assert all(torch.equal(t.g[k], v) for k, v in want[2].items())
