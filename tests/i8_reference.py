"""Plain 64-bit references of the routing and 8-bit integer operators (numpy),
written from their definitions, and the error bounds their tests use."""
import numpy as np

EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half a step, relative
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half the smallest subnormal


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def quant(x):
    """x [rows][k] (fp64 values of the input) -> codes, fp32 scales as fp64."""
    codes, scales = np.zeros(x.shape), np.zeros(x.shape[0])
    for m, row in enumerate(x):
        if not np.isfinite(row).all():
            scales[m] = np.nan
            continue
        scales[m] = np.float64(np.float32(np.abs(row).max() / 127.0))
        if scales[m] > 0:
            codes[m] = np.clip(np.rint(row / scales[m]), -127, 127)
    return codes, scales


def product(codes, scales, w, w_scale):
    """One matrix: the exact sums times both scales, fp64."""
    return (codes @ w.astype(np.float64).T) * scales[:, None] * w_scale.astype(np.float64)[None, :]


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def product_bound(y, dtype):
    """The sum to fp32, the two scales' product and the last product: a rounding each; then the output's."""
    return np.abs(y) * (3 * 2.0 ** -24 + EPS[dtype]) * 1.001 + TINY[dtype]


def swiglu_bound(g, u, dtype):
    """g and u carry 3 roundings each; g's grow by the condition of silu, at most 1 + |g|; the exponential (2 steps
    of its own), the sum, the quotient and the product add 2 + 1 + 1 + 1 roundings, an exponent's argument none."""
    h = silu(g) * u
    return np.abs(h) * ((3 * (1 + np.abs(g)) + 3 + 7) * 2.0 ** -24 + EPS[dtype]) * 1.001 + TINY[dtype] + 2.0 ** -126


def route(logits, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """Row by row, as the definition reads."""
    rows, E = logits.shape
    idx, gate = np.full((rows, top_k), -1, np.int32), np.zeros((rows, top_k))
    size = E // groups
    for r in range(rows):
        l = np.minimum(logits[r].astype(np.float64), np.finfo(np.float32).max)
        cand = ~np.isnan(l) & (l != -np.inf)
        if bias is not None:
            cand &= ~np.isnan(bias) & (bias != -np.inf)
        if not cand.any():
            continue
        with np.errstate(over="ignore", invalid="ignore", under="ignore"):
            if score == "softmax":
                e = np.where(cand, np.exp(np.where(cand, l - l[cand].max(), 0.0)), 0.0)
                s = e / e.sum()
            else:
                s = np.where(cand, 1.0 / (1.0 + np.exp(-np.where(cand, l, 0.0))), 0.0)
        c = s if bias is None else s + bias.astype(np.float64)
        if groups > 1:
            worth = []
            for g in range(groups):
                mine = sorted((c[e] for e in range(g * size, (g + 1) * size) if cand[e]), reverse=True)[:group_top]
                worth.append(sum(mine) if mine else -np.inf)
            stay = [g for g in sorted(range(groups), key=lambda g: (-worth[g], g)) if worth[g] > -np.inf][:top_groups]
            cand &= np.isin(np.arange(E) // size, stay)
        key = l if bias is None else c
        best = sorted((e for e in range(E) if cand[e]), key=lambda e: (-key[e], e))[:top_k]
        idx[r, :len(best)] = best
        g = s[best]
        if renorm:
            g = g / g.sum() if g.sum() > 0 else np.zeros_like(g)
        gate[r, :len(best)] = g * scale
    return idx, gate


def group_slots(idx, E):
    flat = idx.reshape(-1)
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1))])
    return order.astype(np.int32), offsets.astype(np.int32)
