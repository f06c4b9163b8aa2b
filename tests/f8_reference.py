"""Plain 64-bit references of the 8-bit floating-point operators and the norms
before the 8-bit products (numpy), written from their definitions, and the
error bounds their tests use."""
import numpy as np

from i8_reference import EPS, TINY, group_slots, silu, torch_dtype  # noqa: F401  (shared with the integer operators)

BLOCK = 128
# the value of every code; 0x7F and 0xFF are NaN
_m = np.arange(256) & 7
_e = (np.arange(256) >> 3) & 15
VALUES = np.where(_e == 0, _m * 2.0 ** -9, (8 + _m) * 2.0 ** (_e - 10.0)) * np.where(np.arange(256) < 128, 1.0, -1.0)
VALUES[[0x7F, 0xFF]] = np.nan
POSITIVE = VALUES[:127]  # ascending: a code is its number's place
MIDDLES = (POSITIVE[1:] + POSITIVE[:-1]) / 2


def blocks(n):
    return -(-n // BLOCK)


def codes_of(t):
    """The codes of a float8 tensor."""
    import torch
    return t.cpu().view(torch.uint8).numpy()


def tensor_of(codes):
    """A float8 tensor on the GPU of codes."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(codes).astype(np.uint8)).view(torch.float8_e4m3fn).cuda()


def nearest(t):
    """fp64 numbers to the nearest e4m3 numbers, in the middle to the even code."""
    size = np.minimum(np.abs(t), 448.0)
    at = np.searchsorted(MIDDLES, size, side="left")  # middles below the number
    tie = (at < len(MIDDLES)) & (MIDDLES[np.minimum(at, len(MIDDLES) - 1)] == size)
    return np.copysign(POSITIVE[at + (tie & (at % 2 == 1))], t)


def quant(x):
    """x [rows][k] fp64 -> values of the codes [rows][k], fp32 scales [blocks][rows] as fp64."""
    rows, k = x.shape
    codes, scales = np.zeros(x.shape), np.zeros((blocks(k), rows))
    for b in range(blocks(k)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        with np.errstate(invalid="ignore", over="ignore"):
            s = (np.abs(part).max(1) / 448.0).astype(np.float32).astype(np.float64)
        s[~np.isfinite(part).all(1)] = np.nan
        scales[b] = s
        for m in range(rows):
            if s[m] > 0:
                codes[m, b * BLOCK:(b + 1) * BLOCK] = nearest(part[m] / s[m])
    return codes, scales


def product(codes, scales, w, w_scale):
    """One matrix (values of its codes): y in fp64, and the sum of its terms' magnitudes."""
    y, size = 0.0, 0.0
    for b in range(scales.shape[0]):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        s = scales[b][:, None] * np.repeat(w_scale[:, b].astype(np.float64), BLOCK)[None, :w.shape[0]]
        y = y + s * (codes[:, at] @ w[:, at].T)
        size = size + np.abs(s) * (np.abs(codes[:, at]) @ np.abs(w[:, at]).T)
    return y, size


def sum_error(size, kb, parts=16):
    """Of the fp32 sum: 128 additions inside a block (products of two codes are exact; a whole step each, should the
    matrix units cut bits off), the two scales' product, an addition for each block and for each part of K that was
    summed by itself, at most 16 of them."""
    return size * (128 * 2.0 ** -23 + (kb + parts + 2) * 2.0 ** -24) * 1.001


def cut(size, dtype):
    """Outputs of 16 bits may come from the matrix units' 8-bit products: of 8 neighbouring products, 7 may lose what is
    below 2^-13 of the power of two at or under the largest, which is at most their sum."""
    return 0.0 if dtype == "f32" else 7 * 2.0 ** -13 * size


def product_bound(y, size, kb, dtype):
    """The sum's error, then the output's rounding."""
    e = sum_error(size, kb) + cut(size, dtype)
    return e + (np.abs(y) + e) * EPS[dtype] * 1.001 + TINY[dtype]


def swiglu_bound(g, g_size, u, u_size, kb, dtype):
    """The slope of silu is at most 1.1; its own steps are at most 11 roundings for every gate."""
    dg, du = sum_error(g_size, kb) + cut(g_size, dtype), sum_error(u_size, kb) + cut(u_size, dtype)
    e = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du
    return e + (np.abs(silu(g) * u) + e) * (11 * 2.0 ** -24 + EPS[dtype]) * 1.001 + TINY[dtype] + 2.0 ** -126


def norm(h, t, gain, eps):
    """g as stored (fp32), and v in fp64; rows that are not finite come out as NaN."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        g = h.astype(np.float32) if t is None else (h.astype(np.float64) + t).astype(np.float32)
        v = g.astype(np.float64)
        inv = 1.0 / np.sqrt((v * v).sum(1, keepdims=True) / v.shape[1] + np.float64(np.float32(eps)))
        v = np.where(np.isfinite(g).all(1, keepdims=True), v * inv, np.nan)
        return g, v if gain is None else v * gain.astype(np.float64)[None, :]
