"""Plain references of the AdamW plan's operators in numpy, written from the
formulas of include/ps.h. Arithmetic on float32 arrays rounds every operation
once, as the step's contract says, so the float32 reference is bit-exact; the
same functions on float64 arrays give the formula in 64 bits."""
import numpy as np

BLOCK = 256


def e4m3_values():
    """The values of the codes 0 .. 126 (sign 0; 127 is NaN)."""
    k = np.arange(127)
    e, f = k >> 3, k & 7
    return np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))


VALUES = e4m3_values()
MIDS = (VALUES[1:] + VALUES[:-1]) / 2


def e4m3_code(y):
    """Codes of y, |y| <= 448: nearest value, ties to the even code."""
    a = np.abs(y).astype(np.float64)
    k = np.searchsorted(MIDS, a, side="left")              # ties stay below
    tie = (k < 126) & (MIDS[np.minimum(k, 125)] == a) & (k % 2 == 1)
    k = k + tie
    return (k | (np.signbit(y).astype(np.int64) << 7)).astype(np.uint8)


def e4m3_value(code):
    code = np.asarray(code, np.uint8)
    v = VALUES[np.minimum(code & 127, 126)]
    return np.where(code & 128, -v, v).astype(np.float32)


def blocks_of(n):
    return (n + BLOCK - 1) // BLOCK


def per_block_max(x):
    n = x.size
    y = np.zeros(blocks_of(n) * BLOCK, x.dtype)
    y[:n] = np.abs(x)
    return y.reshape(-1, BLOCK).max(1)


def spread(s, n):
    return np.repeat(s, BLOCK)[:n]


def block_scale(top):
    """Smallest power of two s >= 2^-126 with top <= 448 s."""
    top = top.astype(np.float64)
    m, e = np.frexp(top)                                    # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = np.where(m <= 0.875, e - 9, e - 8)
    return np.ldexp(1.0, np.where(top == 0, -126, np.maximum(e, -126))).astype(np.float32)


def stochastic_cut(y, bits):
    """float32 y >= 0 cut to e4m3's places after adding bits / 2^16 of the last one."""
    small = y < np.float32(2.0 ** -6)
    z = np.where(small, y + np.float32(2.0 ** -6), y).astype(np.float32)
    u = (z.view(np.uint32) + (bits.astype(np.uint32) << np.uint32(4))) & np.uint32(0xFFF00000)
    q = u.view(np.float32)
    return np.where(small, q - np.float32(2.0 ** -6), q).astype(np.float32)


def second_code(r, scale, bits=None):
    y = (r / scale).astype(np.float32)                      # by a power of two: exact
    if bits is not None:
        y = stochastic_cut(y, bits)
    return e4m3_code(np.where(r > 0, np.maximum(y, np.float32(2.0 ** -9)), y))


def encode(x, signed):
    y = x if signed else np.sqrt(x)
    s = block_scale(per_block_max(y))
    t = spread(s, x.size)
    return (e4m3_code(y / t) if signed else second_code(y, t)), s


def decode(code, scale, signed):
    x = e4m3_value(code) * spread(scale, code.size)
    return x if signed else x * x


def update(w, g, m0, v0, c, mul, nadam, T):
    """The element formula in type T: (w', m, v, r). c: the fp32 step scalars by name."""
    k = {a: T(b) for a, b in c.items()}
    w, g, m0, v0 = (a.astype(T) for a in (w, g, m0, v0))
    g = g * T(mul)
    m = k["B1"] * m0 + k["C1"] * g
    v = k["B2"] * v0 + k["C2"] * (g * g)
    r = np.sqrt(v)
    d = r * k["RS2"] + k["EPS"]
    u = (k["AG"] * g + k["AM"] * m) / d if nadam else k["A"] * (m / d)
    u = u + k["CWD"] * w
    return w - u, m, v, r


def bf16_to_f32(b):
    return (b.astype(np.uint32) << np.uint32(16)).view(np.float32)


def bf16_round(x):
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
