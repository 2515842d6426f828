"""The AdamW step's square root and quotient against the library's, value by
value on the GPU (tests/kernels/probe_adamw.hip)."""
import ctypes
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

PROBE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kernels", "libps_probe.so")
U32, VP = ctypes.c_uint32, ctypes.c_void_p


@pytest.fixture(scope="module")
def probe():
    L = ctypes.CDLL(PROBE)
    L.probe_root_diff.argtypes = [U32, U32, VP, VP]
    L.probe_quotient_diff.argtypes = [ctypes.c_int, ctypes.c_int, U32, U32, VP, VP]
    return L


def run(f, *args):
    out = torch.zeros(1, dtype=torch.int64, device="cuda")
    assert f(*args, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    return int(out)


def test_every_root_from_2_to_the_minus_100(probe):
    """All 1.9e9 finite values from 2^-100 on, and the two zeros."""
    first = (127 - 100) << 23
    assert run(probe.probe_root_diff, first, 0x7F800000 - first) == 0
    assert run(probe.probe_root_diff, 0, 1) == 0 and run(probe.probe_root_diff, 0x80000000, 1) == 0


@pytest.mark.parametrize("ea,ed", [(0, 0), (-60, 59), (57, -60), (-60, -60), (57, 59), (-20, -3), (5, -40)])
def test_quotients_over_every_divisor_mantissa(probe, ea, ed):
    """2^23 divisors with 32 numerators each, half of them next to a rounding border."""
    assert run(probe.probe_quotient_diff, ea, ed, 32, 1 + ea + 64 * ed & 0xFFFF) == 0
