"""The e4m3 tile kernels at sizes that run their steady loops, the hand-over to
what is left of K, and their way from one tile to the next, to the last bit."""
import numpy as np
import pytest

import f8_reference as ref
import memory_bound_mxfp4_amd as moe
from test_gpu_f8 import _idx

pytestmark = pytest.mark.gpu

# rows, columns of all matrices together, K.  256 x 256 tiles, more than one a workgroup: K of 1 stage to several rounds
# of the loop, last rows that fill 1 to 4 quarters of a tile, columns that end inside one, at an odd number, at a tile.
DENSE = [(3338, 7200, 112), (3428, 7200, 240), (3478, 7168, 384), (3578, 7200, 528), (3338, 7168, 640), (3840, 7200, 784),
         (3428, 7200, 1040), (3478, 7202, 656), (2314, 6144, 1040),
         # two 128 x 128 tiles to a CU
         (1200, 4096, 528), (1300, 6000, 656), (1700, 5000, 784), (900, 5000, 1040),
         # one to a CU: on from tile to tile, and one tile a workgroup
         (1078, 6000, 3216), (700, 7200, 3344), (1090, 6002, 3408), (600, 6000, 1040), (1000, 2050, 1168), (1000, 2048, 2176),
         # 64 x 128 and 64 x 64 tiles, two groups of waves
         (500, 3000, 1600), (250, 6000, 1680), (500, 2998, 2064), (500, 2048, 2064), (500, 800, 3344)]
# tokens (a quarter of them padding; of one slot each: none, all experts with as many), slots each, experts, columns of
# all matrices together, K, rows by slot
GROUPED = [(2200, 2, 8, 6080, 528, False), (2200, 2, 8, 6080, 384, True), (2180, 2, 8, 6080, 656, True), (2190, 2, 8, 6080, 1040, False),
           (960, 2, 16, 4000, 528, False), (100, 2, 8, 6400, 528, True), (100, 2, 8, 6400, 784, False), (200, 3, 3, 6400, 1296, False),
           (214, 2, 8, 4000, 1168, True), (106, 4, 16, 4000, 2064, False), (40, 2, 3, 6400, 1680, True), (40, 3, 2, 4000, 2064, False),
           (950, 2, 2, 400, 2064, True), (108, 2, 8, 4000, 1680, True), (272, 1, 2, 8960, 1296, True), (268, 1, 2, 8704, 1424, False)]


def slots_of(tokens, top_k, E):
    """The experts of the slots of a case."""
    if top_k == 1:
        return (np.arange(tokens, dtype=np.int32) * 7 % E).reshape(tokens, 1).astype(np.int32)
    return _idx(tokens, top_k, E, tokens)


def _pick(gen, shape, values):
    import torch
    v = torch.tensor(values, device="cuda")
    return v[torch.randint(len(values), shape, generator=gen, device="cuda")]


def _operands(gen, m, n, k, lead, swiglu):
    """Codes and scales of few bits, so that every sum in fp32 is exact in any order. With SwiGLU the gates lie above 32,
    where silu(g) is g in fp32."""
    kb = ref.blocks(k)
    parts = (2,) if swiglu else ()
    x = _pick(gen, (m, k), [0.0, 1.0, 2.0] if swiglu else [0.0, 1.0, -1.0, 2.0])
    w = _pick(gen, lead + parts + (n, k), [0.0, 1.0, -1.0, 0.5])
    xs = _pick(gen, (kb, m), [0.25, 0.5, 1.0, 2.0, 4.0])
    ws = _pick(gen, lead + parts + (ref.blocks(n), kb), [0.25, 0.5, 1.0, 2.0, 4.0])
    if swiglu:
        x[:, :32], xs[0] = 1.0, 2.0
        w[..., 0, :, :] = w[..., 0, :, :].abs()
        w[..., 0, :, :32], ws[..., 0, :, 0] = 1.0, 1.0
    return x, w, xs, ws


def _product(x, xs, w, ws):
    """x [m][k], xs [blocks][m], one matrix w [n][k], ws [blocks][blocks], in 64 bits."""
    k, n = x.shape[1], w.shape[0]
    wide = x.double() * xs.double().t().repeat_interleave(ref.BLOCK, 1)[:, :k]
    matrix = w.double() * ws.double().repeat_interleave(ref.BLOCK, 0)[:n].repeat_interleave(ref.BLOCK, 1)[:, :k]
    return (wide @ matrix.t()).float()


def _once(exact, out):
    """Numbers of 64 bits to 16 in one rounding: first to fp32 towards 0 with the last bit set where anything was cut off,
    which keeps them on their side of every middle."""
    import torch
    f = exact.float()
    bits = f.view(torch.int32) - (f.double().abs() > exact.abs()).int()
    return (bits | (f.double() != exact).int()).view(torch.float32).to(out)


def _want(x, xs, w, ws, swiglu, out):
    """The output, and what else it may be: the two sums' product is one of fp32, which the compiler rounds to fp16 by
    way of fp32 or at once (where their product lies within half a last place of fp32 of a middle, these two differ)."""
    if not swiglu:
        y = _product(x, xs, w, ws).to(out)
        return y, y
    g, u = _product(x, xs, w[0], ws[0]), _product(x, xs, w[1], ws[1])
    assert bool((g > 32.0).all())
    y = (g * u).to(out)
    return y, y if out == g.dtype else _once(g.double() * u.double(), out)


def _e4m3(v):
    import torch
    return v.to(torch.float8_e4m3fn)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("m,n,k", DENSE)
def test_gemm_loops(m, n, k, swiglu, out):
    import torch
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    n, dtype = n // 2 if swiglu else n, ref.torch_dtype(out)
    x, w, xs, ws = _operands(gen, m, n, k, (), swiglu)
    want = _want(x, xs, w, ws, swiglu, dtype)
    y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
    for _ in range(2):
        moe.gemm_f8(_e4m3(x), _e4m3(w), ws, x_scale=xs, swiglu=swiglu, out=y[:m])
        assert bool(((y[:m] == want[0]) | (y[:m] == want[1])).all())
        assert bool((y[m] == 7.0).all())


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("tokens,top_k,E,n,k,by_slot", GROUPED)
def test_experts_loops(tokens, top_k, E, n, k, by_slot, swiglu, out):
    import torch
    gen = torch.Generator("cuda").manual_seed(tokens + n + k)
    n, dtype, slots = n // 2 if swiglu else n, ref.torch_dtype(out), tokens * top_k
    idx = torch.from_numpy(slots_of(tokens, top_k, E)).cuda()
    x, w, xs, ws = _operands(gen, slots if by_slot else tokens, n, k, (E,), swiglu)
    flat = idx.reshape(-1)
    want = torch.zeros(2, slots, n, dtype=dtype, device="cuda")
    for e in range(E):
        mine = torch.nonzero(flat == e).flatten()
        rows = mine if by_slot else mine // top_k
        want[0, mine], want[1, mine] = _want(x[rows], xs[:, rows], w[e], ws[e], swiglu, dtype)
    groups = moe.moe_group_slots(idx, E)
    y = torch.full((slots + 1, n), 7.0, dtype=dtype, device="cuda")
    for _ in range(2):
        moe.experts_gemm_f8(_e4m3(x), groups, _e4m3(w), ws, x_scale=xs, swiglu=swiglu, out=y[:slots])
        assert bool(((y[:slots] == want[0]) | (y[:slots] == want[1])).all())
        assert bool((y[slots] == 7.0).all())
