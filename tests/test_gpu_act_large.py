"""GPU tests of the activation checkpoints where a call's lanes, and its bytes,
pass 32 bits: more workgroups than one dimension of a grid holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def _ramp(n, dtype):
    """1 .. 8 over and over: whole in every type, and in a code with any power-of-two scale."""
    return (torch.arange(8, device="cuda", dtype=dtype) + 1).repeat((n + 7) // 8)[:n]


def test_codec_of_more_blocks_than_a_grid_dimension(ps):
    rows = (1 << 29) + 5
    x = _ramp(rows, torch.bfloat16).view(rows, 1)
    code = torch.full((rows, 1), 127, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(rows, 1, device="cuda")
    ps.encode_act(x, code, scale)
    # x / s in 256 .. 448: s is 2^(e - 8) for x = 2^e .. 1.75 * 2^e
    assert torch.equal(scale[:8].flatten().cpu(), torch.tensor([2.0 ** (e - 8) for e in (0, 1, 1, 2, 2, 2, 2, 3)]))
    assert torch.equal(scale, scale[:8].flatten().repeat(rows // 8 + 1)[:rows].view(rows, 1))
    back = torch.zeros_like(x)
    ps.decode_act(code, scale, back)
    assert torch.equal(back, x)


def test_activation_of_more_blocks_than_a_grid_dimension(ps):
    rows = (1 << 28) + 5
    a = _ramp(rows, torch.bfloat16).view(rows, 1)
    out, da = torch.zeros_like(a), torch.zeros_like(a)
    code = torch.full((rows, 1), 127, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(rows, 1, device="cuda")
    ps.glu_forward(a, out, ps.ACT_SILU, code, scale)
    ps.glu_backward(a, ps.ACT_SILU, code, scale, da)
    z = torch.arange(1, 9, dtype=torch.float64)
    q = torch.sigmoid(z)
    for got, want in ((out, z * q), (da, z * (q + z * q * (1 - q)))):
        eight = got[:8].flatten().double().cpu()
        # one rounding to bf16, and some of fp32
        assert ((eight - want).abs() <= want * (2 ** -8 + 2 ** -20)).all()
        assert torch.equal(got, got[:8].flatten().repeat(rows // 8 + 1)[:rows].view(rows, 1))


@pytest.mark.parametrize("rows,cols", [((1 << 26) + 5, 8), ((1 << 25) + 3, 1032)])
def test_norm_of_more_rows_than_a_grid_dimension(ps, rows, cols):
    eight = _ramp(8, torch.bfloat16)
    x = eight.repeat((cols + 7) // 8)[:cols].expand(rows, cols).contiguous()
    x[1::2] *= 2                                             # rms norms see no scale
    n, rstd = torch.zeros_like(x), torch.zeros(rows, device="cuda")
    ps.block_norm_forward(ps.BlockNorm(pre_eps=0.0), x, n, h_rstd=rstd)
    z = torch.arange(1, 9, dtype=torch.float64)
    want = z / z.square().mean().sqrt()
    assert ((n[0, :8].double().cpu() - want).abs() <= want * (2 ** -8 + 2 ** -20)).all()
    for i in range(0, rows, 1 << 22):                        # in parts: comparisons of it all take as much again
        assert torch.equal(n[i:i + (1 << 22)], n[0].expand_as(n[i:i + (1 << 22)]))
    assert torch.equal(rstd[0::2], rstd[0].expand_as(rstd[0::2]))
    assert torch.equal(rstd[1::2], (rstd[0] / 2).expand_as(rstd[1::2]))
