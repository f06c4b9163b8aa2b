"""The e4m3 operators and the norms with codes out where offsets pass 32 bits: rows, matrices, outputs and codes of
more than 4 GiB, checked at their beginning, around the border and at their end, to the last bit."""
import pytest

import memory_bound_mxfp4_amd as moe

pytestmark = pytest.mark.gpu


def _few(shape, gen):
    """e4m3 numbers of few bits, whose sums are exact in any order."""
    import torch
    return torch.randint(-2, 3, shape, generator=gen, device="cuda", dtype=torch.int8).to(torch.float8_e4m3fn)


def _places(count, size):
    """Some of `count` rows of `size` bytes: the first, around each 4 GiB, the last."""
    at = [range(0, 20), range(count - 300, count)]
    for border in range(1, count * size // 2 ** 32 + 1):
        row = border * 2 ** 32 // size
        at.append(range(max(0, row - 10), min(count, row + 10)))
    return sorted({i for r in at for i in r})


def _scales(blocks, rows, gen):
    import torch
    return 2.0 ** torch.randint(-1, 2, (blocks, rows), generator=gen, device="cuda").float()


def _want(x, xs, w, ws):
    """Rows of x by rows of w with a scale for each block of both, in 64 bits."""
    wide = x.double() * xs.double().t().repeat_interleave(128, 1)
    return (wide @ (w.double() * ws.double().repeat_interleave(128, 1)).t()).float()


@pytest.mark.parametrize("m,n,k,out", [(1100000, 64, 4096, "bfloat16"), (1200000, 2048, 128, "bfloat16"), (1200000, 2048, 128, "float32"),
                                       (20, 1 << 20, 4224, "bfloat16"), (300, 1 << 20, 4224, "bfloat16")])
def test_gemm_past_32_bits(m, n, k, out):
    import torch
    gen, dtype = torch.Generator("cuda").manual_seed(m + n), getattr(torch, out)
    x, w = _few((m, k), gen), _few((n, k), gen)
    xs, ws = _scales(k // 128, m, gen), _scales(k // 128, n // 128 if n >= 128 else 1, gen).t().contiguous()
    y = moe.gemm_f8(x, w, ws, x_scale=xs, out_dtype=dtype)
    rows = torch.tensor(_places(m, max(k, n * y.element_size())) if m > 1000 else range(m), device="cuda")
    cols = torch.tensor(_places(n, k) if n > 100000 else range(n), device="cuda")
    want = _want(x[rows], xs[:, rows], w[cols], ws[cols // 128])
    assert torch.equal(y[rows][:, cols], want.to(dtype))


@pytest.mark.parametrize("tokens", [6, 700])
def test_experts_past_32_bits(tokens):
    import torch
    E, n, k = 300, 4096, 4096
    gen = torch.Generator("cuda").manual_seed(tokens)
    x, w = _few((tokens, k), gen), torch.empty(E, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        w[e] = _few((n, k), gen)
    xs, ws = _scales(k // 128, tokens, gen), _scales(E * n // 128, k // 128, gen).view(E, n // 128, k // 128)
    idx = torch.stack([torch.arange(tokens, device="cuda") % 3, 296 + torch.arange(tokens, device="cuda") % 4], 1).int()
    y = moe.experts_gemm_f8(x, moe.moe_group_slots(idx, E), w, ws, x_scale=xs, out_dtype=torch.float32).view(tokens, 2, n)
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        assert torch.equal(y[t, j], _want(x[t], xs[:, t], w[e], ws[e].repeat_interleave(128, 0)))


@pytest.mark.parametrize("f8", [True, False])
def test_codes_past_32_bits(f8):
    """More than 2^32 elements in, out and of codes: rows are those of a call of their own."""
    import torch
    rows, k = 600000, 8192
    gen = torch.Generator("cuda").manual_seed(1)
    some = torch.randn(1000, k, device="cuda", generator=gen)
    x = torch.empty(rows, k, device="cuda")
    x.view(600, 1000, k).copy_(some)
    x[-1] *= 3.0
    at = torch.tensor(_places(rows, k), device="cuda")
    norm = moe.residual_add_rmsnorm_f8 if f8 else moe.residual_add_rmsnorm_i8
    for call in ([moe.quant_rows_f8] if f8 else []) + [norm]:
        q, s = call(x)
        want, ws = call(x[at])
        assert torch.equal(q[at].view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(s[..., at], ws)
        del q, s, want, ws
