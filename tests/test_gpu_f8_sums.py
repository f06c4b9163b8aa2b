"""How exact the sums of the e4m3 products are: fp32 where the outputs are, and
where a call has few rows; with the matrix units' 8-bit products no further off
than documented, and on normal values far less."""
import pytest

import f8_reference as ref
import memory_bound_mxfp4_amd as moe
from test_f8_plan import KINDS, _plan

# rows, n: one size for every kernel of 16-bit outputs at K 256, and of fp32 ones
SIZES = [(4, 300), (16, 300), (60, 300), (400, 800), (300, 5000), (500, 4000), (1000, 2048), (1000, 2100), (1300, 6000),
         (3338, 7168)]


def _e4m3(v):
    import torch
    return v.to(torch.float8_e4m3fn)


def test_sizes_reach_every_kernel():
    for wide in (False, True):
        assert {_plan(m, 1, False, n, 256, False, wide).kind for m, n in SIZES} == KINDS[wide]


def _large_and_small(m, n, apart):
    """65536 + 30 - 65536 in every output; `apart`: the large ones in groups of 8 of their own, or all in one."""
    import torch
    x, w = torch.zeros(m, 256, device="cuda"), torch.zeros(n, 256, device="cuda")
    for k, (a, b) in zip((0, 1, 130) if apart else (0, 1, 2), ((256.0, 256.0), (5.0, 6.0), (256.0, -256.0))):
        x[:, k], w[:, k] = a, b
    return _e4m3(x), _e4m3(w), torch.ones(2, m, device="cuda"), torch.ones(ref.blocks(n), 2, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("m,n", SIZES)
def test_a_small_product_beside_large_ones(m, n, apart):
    import torch
    x, w, xs, ws = _large_and_small(m, n, apart)
    for out in ("bf16", "f16", "f32"):
        y = moe.gemm_f8(x, w, ws, x_scale=xs, out_dtype=ref.torch_dtype(out))
        if out == "f32" or m <= 16:
            assert bool((y == 30.0).all()), out
        else:  # of 8 products the others may each lose what is below 2^-13 of the largest: here one of them, 30
            assert bool(((y >= 30.0 - 2.0 ** -13 * 65536) & (y <= 30.0)).all()), out


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SIZES)
def test_normal_values_lose_little(m, n):
    """Codes of normal values in one block, and the same products, of the other sign and in another order, in the next:
    what is left of the sum is what was lost on the way. Of 8 neighbouring products of normal values (unit variance) the
    largest is some 2.5, so bits below 2^-12 are cut off; a product has its last bit 2^-7 under its first at the most, so
    only those under 2^-6, one in 20 (the integral of K0 up to there), lose anything, evenly below 2^-12 and to either
    side: of two blocks thirteen losses of 2^-12 / sqrt(3), 5.1e-4 beside a sum of 11.3 from 128 terms, 4.5e-5
    (measured: 1.6e-5). Sums of a block that were rounded to bf16 would leave some 1.6e-3, to fp16 2e-4."""
    import torch
    gen = torch.Generator("cuda").manual_seed(m + n)
    a = _e4m3(torch.randn(m, 128, device="cuda", generator=gen) * 64.0).float()
    b = _e4m3(torch.randn(n, 128, device="cuda", generator=gen) * 64.0).float()
    order = torch.randperm(128, device="cuda", generator=gen)
    x, w = torch.cat([a, a[:, order]], 1), torch.cat([b, -b[:, order]], 1)
    xs, ws = torch.ones(2, m, device="cuda"), torch.ones(ref.blocks(n), 2, device="cuda")
    size = float((a.double() @ b.double().t()).square().mean().sqrt())
    for out in ("bf16", "f16", "f32"):
        y = moe.gemm_f8(_e4m3(x), _e4m3(w), ws, x_scale=xs, out_dtype=ref.torch_dtype(out)).double()
        lost = float(y.square().mean().sqrt()) / size
        # fp32: 256 additions, each off by a last place, at the most, of a partial sum that is on average no larger than `size`
        limit = 256 * 2.0 ** -23 if out == "f32" or m <= 16 else 5e-5
        print(f"{m} x {n}, {out}: {lost:.2e} of a block's sum")
        assert lost <= limit, out
