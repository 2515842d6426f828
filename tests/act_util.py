"""Inputs and poisoned buffers of the activation checkpoints' GPU tests."""
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
POISON = -7.5       # what outputs and the space between their rows hold before a call


def gen(seed):
    return torch.Generator().manual_seed(seed)


def acts(g, rows, cols, dtype, spread=0.6):
    """Activations: rows and channels of different size, some channels large."""
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    wide = torch.exp(spread * torch.randn(1, cols, generator=g))
    wide[torch.rand(1, cols, generator=g) < 0.02] *= 20
    return (x * wide).to(DT[dtype])


class Padded:
    """A matrix on the GPU inside a poisoned allocation: `pad` columns after each row, `shift` elements before."""

    def __init__(self, rows, cols, dtype, pad=0, shift=0, fill=None):
        dtype = DT.get(dtype, dtype)
        self.base = torch.full((shift + max(rows, 1) * (cols + pad) + 64,), POISON, dtype=torch.float32).to(dtype).cuda()
        self.m = self.base[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.dtype = dtype
        if fill is not None:
            self.m.copy_(fill)

    def outside_is_untouched(self):
        """All but the matrix still holds the poison."""
        seen = self.base.clone()
        rows, cols = self.m.shape
        if rows and cols:
            torch.as_strided(seen, self.m.shape, self.m.stride(), self.m.storage_offset()).fill_(POISON)
        return bool((seen.float() == torch.tensor(POISON).to(self.dtype).float()).all())


def codes(rows, cols):
    return torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda").view(E4M3)


def scales(rows, cols):
    return torch.full((rows, -(-cols // 128)), POISON, device="cuda")
