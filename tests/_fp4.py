"""Microscaled values in 64 bits, for the tests of MXFP4 and of checkpoints in 8 bits: the definitions, one value
after the other, sharing no code with the library."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:-1])
E5M2 = np.array([(m / 4 * 2.0 ** -14 if e == 0 else (1 + m / 4) * 2.0 ** (e - 15)) for e in range(31) for m in range(4)])
TABLES = {"e2m1": E2M1, "e4m3": E4M3, "e5m2": E5M2}
NAN_CODE = {"e2m1": 7, "e4m3": 0x7F, "e5m2": 0x7F}
SIGN_BIT = {"e2m1": 3, "e4m3": 7, "e5m2": 7}


def f64(t):
    return t.detach().double().cpu().numpy()


def quantize(x, fmt):
    """x [R, K] (64 bits) -> (codes [R, 32 G], scale codes [R, G]): the least power of two that holds the group, the
    nearest value of the format, ties to the even code."""
    table = TABLES[fmt]
    R, K = x.shape
    G = -(-K // 32)
    g = np.zeros((R, G * 32))
    g[:, :K] = x
    neg = np.signbit(g).reshape(R, G, 32)
    g = g.reshape(R, G, 32)
    bad = ~np.isfinite(g).all(2)
    a = np.abs(np.where(bad[:, :, None], 0, g))
    amax = a.max(2)
    e = np.full((R, G), -127)
    for i in range(-126, 128):
        e = np.where(amax > table[-1] * 2.0 ** (i - 1), i, e)
    v = a * 2.0 ** -e.astype(float)[:, :, None]
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)   # table[hi - 1] < v <= table[hi]
    lo = hi - 1
    down, up = v - table[lo], table[hi] - v
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(bad[:, :, None], NAN_CODE[fmt], code)
    code = code | (neg.astype(int) << SIGN_BIT[fmt])
    return code.reshape(R, G * 32).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales, K, fmt):
    """64-bit values [R, K] of codes and scale codes."""
    bit, n = SIGN_BIT[fmt], len(TABLES[fmt])
    table = np.concatenate([TABLES[fmt], np.full((1 << bit) - n, np.nan)])
    if fmt == "e5m2":
        table[0x7C] = np.inf
    v = table[codes & ((1 << bit) - 1)] * (1.0 - 2.0 * (codes >> bit))
    s = 2.0 ** (scales.astype(float) - 127)
    s[scales == 255] = np.nan
    return (v.reshape(len(codes), -1, 32) * s[:, :, None]).reshape(len(codes), -1)[:, :K]


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], 2).reshape(len(q), -1)


def tiled(s, rows=None):
    """Scale codes [R, G] in the order of the tensor cores, element by element; padding 0."""
    R, G = s.shape
    out = np.zeros((-(-R // 128), -(-G // 4), 512), np.uint8)
    r, g = np.meshgrid(np.arange(R), np.arange(G), indexing="ij")
    out[r // 128, g // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + g % 4] = s
    return out.reshape(-1)


def bf16(x):
    """64-bit values to bf16, nearest even, once (as a tensor on the CPU)."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    unit = 2.0 ** (np.maximum(e, -125) - 8.0)
    with np.errstate(invalid="ignore"):
        r = np.where(np.isfinite(x), np.round(x / unit) * unit, x)
    return torch.from_numpy(r).to(torch.bfloat16)


def random_operand(rng, R, K, lo=125, hi=128):
    """(codes, scale codes) of a random operand; with scales of so few powers of two the products of up to 4096
    terms are exact in FP32, in whatever order they are summed."""
    G = -(-K // 32)
    codes = rng.integers(0, 16, (R, 32 * G)).astype(np.uint8)
    codes[:, K:] = 0
    return codes, rng.integers(lo, hi + 1, (R, G)).astype(np.uint8)
