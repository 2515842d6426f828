"""The polynomial that GELU's kernel takes for Phi, as it stands in the source,
against 64 bits."""
import os
import re

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_coefficients():
    """t P(t), t = 1 / (1 + 0.35 z), in exact arithmetic with the fp32 coefficients: within one rounding of fp32
    (2^-24) of Phi(-z) exp(z^2 / 2) up to z = 14.5, and within 5.93e-8."""
    src = open(os.path.join(ROOT, "precision_state_amd", "csrc", "k_act.hip")).read()
    found = re.search(r"kP\[\] = \{(.*?)\};", src, re.S).group(1)
    p = [float(torch.tensor(float(c.strip().rstrip("f")), dtype=torch.float32)) for c in found.split(",")]
    assert len(p) == 9
    z = torch.linspace(0, 14.5, 200001, dtype=torch.float64)
    t = 1 / (1 + 0.35 * z)
    w = sum(c * t ** (i + 1) for i, c in enumerate(p))
    off = (w / (0.5 * torch.special.erfcx(z / 2 ** 0.5)) - 1).abs().max()
    assert off < 2.0 ** -24 and off < 5.93e-8, float(off)
