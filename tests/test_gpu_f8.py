"""GPU parity of the 8-bit floating-point operators (row quantiser, product,
the experts' products) and of the norms before the 8-bit products against
plain 64-bit references, and a run of them together as a layer."""
import numpy as np
import pytest

import f8_reference as ref
import memory_bound_mxfp4_amd as moe

pytestmark = pytest.mark.gpu


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _x(rows, k, dtype, seed, sigma=1.0):
    """Random rows as a GPU tensor of the type, and their values in fp64."""
    import torch
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(rows, k, generator=g) * sigma).to(ref.torch_dtype(dtype))
    return t.cuda(), t.double().numpy()


def _w(shape, seed):
    """Codes of every size (uint8) [..][n][k], and block scales [..][blocks of n][blocks of k]."""
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 127, shape).astype(np.uint8) | (rng.integers(0, 2, shape) * 128).astype(np.uint8)
    scale = shape[:-2] + (ref.blocks(shape[-2]), ref.blocks(shape[-1]))
    return w, (rng.uniform(0.5, 1.5, scale) * 1e-3).astype(np.float32)


def _close(y, want, bound, what=""):
    y = y.double().cpu().numpy()
    bad = ~(np.abs(y - want) <= bound)
    bad &= ~(np.isnan(y) & np.isnan(want))
    assert not bad.any(), (what, np.argwhere(bad)[:4], y[bad][:4], want[bad][:4], bound[bad][:4])


def _same_codes(q, s, codes, scales):
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scales, equal_nan=True)
    got = ref.VALUES[ref.codes_of(q)]
    assert np.array_equal(got, codes), (np.argwhere(got != codes)[:4], got[got != codes][:4], codes[got != codes][:4])


# ---- rows to codes ----------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 7168), (3, 5), (7, 16), (5, 130), (2, 1000), (300, 257), (9, 2048),
                                    (16, 128), (17, 384), (33, 20001), (2, 65536)])
def test_quant_rows(dtype, rows, k):
    x, v = _x(rows, k, dtype, rows * 7 + k, sigma=3.0)
    _same_codes(*moe.quant_rows_f8(x), *ref.quant(v))


def _borders(dtype):
    """Blocks with quotients on, next to and far from the middles between two codes, at scales of every kind."""
    import torch
    mids = torch.from_numpy(np.concatenate([ref.MIDDLES, [448.0]]))
    rows = []
    for scale in (1.0, 0.5, 3.0 / 7.0, 2.0 ** -120, 2.0 ** 100, 1.0 + 2.0 ** -23, 1.9999999):
        for step in (0.0, 2.0 ** -23, -2.0 ** -23, 2.0 ** -12, -2.0 ** -12):
            row = mids * scale * (1.0 + step)
            row[-1] = 448.0 * scale
            rows.append(row)
            rows.append(-row)
    rows.append(torch.zeros(127))
    tiny = torch.zeros(127)
    tiny[5] = 2.0 ** -149                                  # a scale that rounds to 0
    rows.append(tiny)
    rows.append(torch.arange(127) * 2.0 ** -149)           # subnormals, a scale far from amax / 448
    rows.append(torch.arange(127) * 10 * 2.0 ** -149)
    rows.append((torch.arange(127) - 60) * 2.0 ** -126)
    rows.append(torch.linspace(-1, 1, 127) * 3e38)
    rows.append(torch.full((127,), -0.0))
    x = torch.stack([r.double() for r in rows]).to(ref.torch_dtype(dtype))
    return torch.where(torch.isinf(x), torch.zeros_like(x), x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quant_rows_borders(dtype):
    x = _borders(dtype)
    codes, scales = ref.quant(x.double().numpy())
    _same_codes(*moe.quant_rows_f8(x.cuda()), codes, scales)
    import torch
    wide = torch.zeros(x.shape[0], 128, dtype=x.dtype)     # the same blocks by 16-byte loads
    wide[:, :127] = x
    codes, scales = ref.quant(wide.double().numpy())
    _same_codes(*moe.quant_rows_f8(wide.cuda()), codes, scales)


def test_quant_rows_of_every_bf16():
    """Every finite bf16 number beside one that makes the scale 1, and beside a larger one."""
    import torch
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every.float()) & (every.float().abs() <= 448.0)]
    x = torch.zeros(-(-len(every) // 127), 128, dtype=torch.bfloat16)
    flat = torch.zeros(x.shape[0] * 127, dtype=torch.bfloat16)
    flat[:len(every)] = every
    x[:, 1:] = flat.view(-1, 127)
    for most in (448.0, 2.0 ** 9, 1000.0):
        x[:, 0] = most
        _same_codes(*moe.quant_rows_f8(x.cuda()), *ref.quant(x.double().numpy()))


def test_quant_rows_of_nan_and_infinity():
    import torch
    x = torch.randn(5, 300)
    x[1, 299], x[2, 0], x[3, 130] = float("nan"), float("inf"), float("-inf")
    for dtype in ("bf16", "f16", "f32"):
        q, s = moe.quant_rows_f8(x.to(ref.torch_dtype(dtype)).cuda())
        bad = torch.isnan(s).cpu()
        want = torch.zeros(3, 5, dtype=torch.bool)
        want[2, 1] = want[0, 2] = want[1, 3] = True
        assert torch.equal(bad, want)
        codes = ref.codes_of(q) & 0x7F
        assert not codes[1, 256:].any() and not codes[2, :128].any() and not codes[3, 128:256].any()
        assert codes[1, :256].any() and codes[2, 128:].any() and codes[3, 256:].any() and codes[0].any() and codes[4].any()


def test_quant_rows_strides():
    import torch
    for dtype in ("bf16", "f32"):
        wide, v = _x(6, 700, dtype, 3)
        for part, pv in ((wide[:, 1:302], v[:, 1:302]), (wide[::2, 8:520], v[::2, 8:520]), (wide[:, 3:4], v[:, 3:4])):
            _same_codes(*moe.quant_rows_f8(part), *ref.quant(pv))
    q = torch.full((4, 64), 9, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((4,), 9.0, device="cuda")
    x, v = _x(2, 64, "bf16", 1)
    moe.quant_rows_f8(x, q=q[:2], scale=s[:2].view(1, 2))
    assert (q.view(torch.uint8)[2:] == 9).all() and (s[2:] == 9).all()


# ---- the norms ----------------------------------------------------------------------------------------------------


def _check_norm(q, s, v, f8, out=None):
    """Scales and codes of v in 64 bits: v is known to some 2^-50, so a scale may be either neighbour of a border that
    near, and so may a code be whose quotient is that near to a middle."""
    near = 2.0 ** -44
    got = s.cpu().numpy().astype(np.float64)
    rows, k = v.shape
    edges = range(0, k, ref.BLOCK) if f8 else [0]
    got = got if f8 else got[None, :]
    codes = ref.VALUES[ref.codes_of(q)] if f8 else q.cpu().numpy().astype(np.float64)
    for b, at in enumerate(edges):
        part = v[:, at:at + ref.BLOCK] if f8 else v
        mine = codes[:, at:at + ref.BLOCK] if f8 else codes
        most = np.abs(part).max(1) / (448.0 if f8 else 127.0)
        with np.errstate(over="ignore"):
            low, high = ((most * (1 + d)).astype(np.float32).astype(np.float64) for d in (-near, near))
        bad = ~(np.isfinite(part).all(1) & np.isfinite(high))
        assert np.isnan(got[b][bad]).all() and (mine[bad] == 0).all()
        ok = ~bad
        assert ((got[b] == low) | (got[b] == high))[ok].all(), (b, got[b][ok], low[ok])
        assert (mine[ok & (got[b] == 0)] == 0).all()
        use = ok & (got[b] > 0)
        t = part[use] / got[b][use][:, None]
        if f8:
            choice = [ref.nearest(t * (1 + d)) for d in (-near, near)]
        else:
            choice = [np.clip(np.rint(t * (1 + d)), -127, 127) for d in (-near, near)]
        wrong = (mine[use] != choice[0]) & (mine[use] != choice[1])
        assert not wrong.any(), (b, np.argwhere(wrong)[:4], mine[use][wrong][:4], choice[0][wrong][:4])
    if out is not None:
        _close(out, v, np.abs(v) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133)  # to fp32, then to bf16: half a step each


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (1, 7168), (3, 5), (5, 64), (2, 127), (9, 128), (4, 136), (17, 1000), (70, 257),
                                         (300, 512), (40, 2048), (2, 4104), (3, 8192), (2, 8200), (2, 16384), (2, 20001), (1, 65536)])
def test_norm(f8, dtype, rows, hidden):
    import torch
    call = moe.residual_add_rmsnorm_f8 if f8 else moe.residual_add_rmsnorm_i8
    h, hv = _x(rows, hidden, "f32", rows + hidden, sigma=3.0)
    t, tv = _x(rows, hidden, dtype, hidden, sigma=2.0)
    gain = (np.random.default_rng(hidden).uniform(0.5, 1.5, hidden) * np.where(np.arange(hidden) % 7, 1, -1)).astype(np.float32)
    use_gain, use_out = (rows + hidden) % 3 > 0, hidden % 2 == 0 or rows > 9
    out = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda") if use_out else None
    g, v = ref.norm(hv, tv, gain if use_gain else None, 1e-5)
    dev_gain = _dev(gain) if use_gain else None
    total = torch.full_like(h, 7.0)
    q, s = call(h, t, gain=dev_gain, eps=1e-5, h_out=total, out=out)
    assert np.array_equal(total.cpu().numpy(), g) and np.array_equal(h.double().cpu().numpy(), hv)
    _check_norm(q, s, v, f8, out)
    kept = h.clone()
    q2, s2 = call(kept, t, gain=dev_gain, eps=1e-5)                       # in place
    assert torch.equal(kept, total) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    q3, s3 = call(total, gain=dev_gain, eps=1e-5)                         # nothing to add
    assert torch.equal(q3.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s3, s)


@pytest.mark.parametrize("f8", [True, False])
def test_norm_strides(f8):
    import torch
    call = moe.residual_add_rmsnorm_f8 if f8 else moe.residual_add_rmsnorm_i8
    wide, hv = _x(6, 900, "f32", 5)
    add, tv = _x(6, 900, "f16", 6)
    for a, b in ((0, 512), (1, 302), (4, 260), (8, 9)):
        g, v = ref.norm(hv[::2, a:b], tv[1::2, a:b], None, 1e-6)
        total = torch.full((4, b - a), 9.0, device="cuda")
        q, s = call(wide[::2, a:b], add[1::2, a:b], h_out=total[:3])
        assert np.array_equal(total[:3].cpu().numpy(), g) and (total[3] == 9.0).all()
        _check_norm(q, s, v, f8)


@pytest.mark.parametrize("f8", [True, False])
@pytest.mark.parametrize("hidden", [200, 256, 9000])
def test_norm_bad_rows(f8, hidden):
    """Rows with a NaN or an infinity, rows of zeros, sums that overflow, and gains that are not finite."""
    import torch
    call = moe.residual_add_rmsnorm_f8 if f8 else moe.residual_add_rmsnorm_i8
    h = torch.randn(8, hidden, generator=torch.Generator().manual_seed(1))
    t = torch.zeros(8, hidden)
    h[1, 3], h[2, hidden - 1], h[3, 0] = float("nan"), float("inf"), float("-inf")
    h[4] = 0.0
    h[5], t[5, 9] = 3e38, 3e38
    h[6] *= 1e37
    h[7] *= 1e-30
    out = torch.empty(8, hidden, dtype=torch.bfloat16, device="cuda")
    for eps in (1e-6, 0.0):
        g, v = ref.norm(h.numpy(), t.double().numpy(), None, eps)
        q, s = call(h.cuda(), t.cuda(), eps=eps, out=out)
        _check_norm(q, s, v, f8, out)
        bad = torch.isnan(s).all(0) if f8 else torch.isnan(s)
        assert bad.tolist() == [False, True, True, True, eps == 0.0, True, False, False]
    gain = torch.ones(hidden)
    gain[150] = float("inf")
    g, v = ref.norm(h.numpy()[:1], None, gain.numpy(), 1e-6)
    q, s = call(h[:1].cuda(), gain=gain.cuda())
    _check_norm(q, s, v, f8)
    assert torch.isnan(s).sum() == 1


# ---- the dense product --------------------------------------------------------------------------------------------

SHAPES = [(1, 1, 16), (1, 16, 64), (1, 640, 7168), (2, 33, 48), (3, 17, 80), (5, 100, 1040), (16, 33, 256), (17, 100, 272),
          (31, 64, 4096), (64, 96, 528), (65, 130, 1040), (100, 515, 336), (129, 257, 528), (256, 256, 128), (300, 512, 64),
          (257, 1030, 400), (513, 770, 144), (1000, 1111, 272)]


def _want(codes, scales, w, ws, swiglu, out):
    """The product in 64 bits and the bound of its error."""
    kb = scales.shape[0]
    if swiglu:
        (g, gs), (u, us) = (ref.product(codes, scales, ref.VALUES[w[p]], ws[p]) for p in (0, 1))
        return ref.silu(g) * u, ref.swiglu_bound(g, gs, u, us, kb, out)
    y, size = ref.product(codes, scales, ref.VALUES[w], ws)
    return y, ref.product_bound(y, size, kb, out)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm(m, n, k, swiglu):
    kinds = ["bf16", "f16", "f32"]
    dtype, out = kinds[(m + n) % 3], kinds[(n + k // 16) % 3]
    x, v = _x(m, k, dtype, m + 3 * n + k)
    w, ws = _w((2, n, k) if swiglu else (n, k), k + n)
    ws *= np.float32(0.05)  # sums of some 10: inside fp16
    y = moe.gemm_f8(x, ref.tensor_of(w), _dev(ws), swiglu=swiglu, out_dtype=ref.torch_dtype(out))
    _close(y, *_want(*ref.quant(v), w, ws, swiglu, out))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m", [1, 20, 150])
def test_gemm_types(dtype, out, m):
    n, k = 200, 320
    x, v = _x(m, k, dtype, m)
    w, ws = _w((n, k), 8)
    y = moe.gemm_f8(x, ref.tensor_of(w), _dev(ws), out_dtype=ref.torch_dtype(out))
    _close(y, *_want(*ref.quant(v), w, ws, False, out))


@pytest.mark.parametrize("m", [1, 4, 40, 300])
@pytest.mark.parametrize("n,k", [(150, 416), (260, 1024)])
def test_gemm_of_codes(m, n, k):
    """Rows that are codes already, rows apart, and the same answer as from the float rows."""
    import torch
    x, v = _x(m, k, "bf16", m)
    w, ws = _w((n, k), 2)
    q, s = moe.quant_rows_f8(x)
    wide = torch.full((m, k + 48), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # NaN between the rows
    wide.view(torch.uint8)[:, :k] = q.view(torch.uint8)
    a = moe.gemm_f8(wide[:, :k], ref.tensor_of(w), _dev(ws), x_scale=s, out_dtype=torch.float32)
    b = moe.gemm_f8(q, ref.tensor_of(w), _dev(ws), x_scale=s, out_dtype=torch.float32)
    assert torch.equal(a, b)
    y = moe.gemm_f8(x, ref.tensor_of(w), _dev(ws), out_dtype=torch.float32)
    want, bound = _want(*ref.quant(v), w, ws, False, "f32")
    _close(a, want, bound)
    _close(y, want, bound)


@pytest.mark.parametrize("m", [1, 17, 200])
def test_gemm_float_rows_apart(m):
    x, v = _x(m, 300, "f32", m)
    w, ws = _w((70, 96), 4)
    _close(moe.gemm_f8(x[:, 5:101], ref.tensor_of(w), _dev(ws)), *_want(*ref.quant(v[:, 5:101]), w, ws, False, "bf16"))


@pytest.mark.parametrize("m", [1, 16, 130])
def test_gemm_longest_rows(m):
    """K at its limit, every code at its end and every product of one sign: the largest sums there are."""
    import torch
    n, k = 40, 65536
    q = torch.full((m, k), 448.0, device="cuda").to(torch.float8_e4m3fn)
    w = torch.full((n, k), 448.0, device="cuda").to(torch.float8_e4m3fn)
    w[::2] = (-w[::2].float()).to(torch.float8_e4m3fn)
    xs, ws = torch.rand(512, m, device="cuda") + 0.5, torch.rand(1, 512, device="cuda") + 0.5
    y = moe.gemm_f8(q, w, ws, x_scale=xs, out_dtype=torch.float32)
    want = (xs.double().t() @ ws[0].double() * 448.0 * 448.0 * 128).cpu().numpy()[:, None] * np.where(np.arange(n) % 2, 1.0, -1.0)
    _close(y, want, ref.product_bound(want, np.abs(want), 512, "f32"))


# sizes that reach every kernel, beside SHAPES
ALL_KERNELS = [(1, 300, 656), (12, 300, 656), (12, 5000, 400), (24, 300, 656), (60, 200, 7184), (60, 1000, 1040), (60, 5000, 272),
               (500, 400, 7184), (500, 800, 7184), (300, 2500, 272), (300, 5000, 272), (1000, 2050, 272), (1500, 7000, 144),
               (2040, 8100, 272), (2100, 3600, 400)]


def _exact_inputs(m, n, k, lead, seed):
    """Codes and scales of few bits: every sum in fp32, in any order and however products are aligned, is exact."""
    rng = np.random.default_rng(seed)
    kb = ref.blocks(k)
    x = rng.choice([0.0, 1.0, -1.0, 2.0], (m, k))
    w = rng.choice([0.0, 1.0, -1.0, 0.5], lead + (n, k))
    xs, ws = 2.0 ** rng.integers(-2, 3, (kb, m)), 2.0 ** rng.integers(-2, 3, lead + (ref.blocks(n), kb))
    return x, w, xs, ws


def _e4m3(v):
    import torch
    return torch.from_numpy(np.ascontiguousarray(v)).float().to(torch.float8_e4m3fn).cuda()


def _rounded(y, out):
    import torch
    return torch.from_numpy(np.ascontiguousarray(y)).float().to(ref.torch_dtype(out)).cuda()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("m,n,k", ALL_KERNELS)
def test_gemm_exact(m, n, k, swiglu, out):
    """Each row, column and block of K with its own scale, to the last bit. With SwiGLU the gates lie above 32, where
    silu(g) is g in fp32."""
    import torch
    x, w, xs, ws = _exact_inputs(m, n, k, (2,) if swiglu else (), m + n)
    if swiglu:
        x[:, 32:] = 0.0                                     # short sums, whose product fits
        x[:, :32], w[0, :, :32], xs[0], ws[0, :, 0] = 1.0, 1.0, np.maximum(xs[0], 1.0), 2.0
        w[0, :, 32:] = 0.0
    y = moe.gemm_f8(_e4m3(x), _e4m3(w), _dev(ws.astype(np.float32)), x_scale=_dev(xs.astype(np.float32)), swiglu=swiglu,
                    out_dtype=ref.torch_dtype(out))
    if swiglu:
        want = ref.product(x, xs, w[0], ws[0])[0] * ref.product(x, xs, w[1], ws[1])[0]
    else:
        want = ref.product(x, xs, w, ws)[0]
    assert torch.equal(y, _rounded(want, out))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("by_slot", [False, True])
@pytest.mark.parametrize("tokens,top_k,E,n,k", [(1, 4, 8, 300, 272), (9, 3, 16, 600, 400), (60, 4, 3, 300, 656), (300, 4, 8, 520, 272),
                                                (300, 4, 8, 1200, 272), (130, 4, 16, 1947, 1216), (700, 4, 4, 1100, 400),
                                                (2000, 2, 2, 2100, 272)])
def test_experts_exact(tokens, top_k, E, n, k, by_slot, out):
    import torch
    idx = _idx(tokens, top_k, E, tokens)
    rows = tokens * top_k if by_slot else tokens
    x, w, xs, ws = _exact_inputs(rows, n, k, (E,), tokens)
    groups = moe.moe_group_slots(_dev(idx), E)
    y = moe.experts_gemm_f8(_e4m3(x), groups, _e4m3(w), _dev(ws.astype(np.float32)), x_scale=_dev(xs.astype(np.float32)),
                            out_dtype=ref.torch_dtype(out))
    flat = idx.reshape(-1)
    want = np.zeros((tokens * top_k, n))
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        from_rows = mine if by_slot else mine // top_k
        want[mine] = ref.product(x[from_rows], xs[:, from_rows], w[e], ws[e])[0]
    assert torch.equal(y, _rounded(want, out))


@pytest.mark.parametrize("m", [1, 3, 90, 300])
def test_gemm_bad_and_empty_rows(m):
    """A row with a NaN gives a row of NaN and no other; so does a NaN among the codes of a matrix row, and a scale
    that is one its block's rows; a row of zeros gives zeros."""
    import torch
    n, k = 300, 144
    x, _ = _x(m, k, "f32", 1)
    w, ws = _w((2, n, k), 2)
    if m > 2:
        x[1, 5] = float("nan")
        x[2] = 0.0
        y = moe.gemm_f8(x, ref.tensor_of(w[0]), _dev(ws[0]), out_dtype=torch.float32)
        assert torch.isnan(y[1]).all() and not torch.isnan(y[[0, 2]]).any() and (y[2] == 0).all()
        h = moe.gemm_f8(x * 3e4, ref.tensor_of(w), _dev(ws), swiglu=True, out_dtype=torch.float32)
        assert torch.isnan(h[1]).all() and torch.isfinite(h[0]).all() and (h[2] == 0).all()
    w[0, 7, 143] = 0x7F
    w[0, 9, 0] = 0xFF
    y = moe.gemm_f8(x, ref.tensor_of(w[0]), _dev(ws[0]), out_dtype=torch.float32)[:1]
    assert torch.isnan(y).nonzero()[:, 1].tolist() == [7, 9]
    ws[0, 1, 1] = np.nan
    y = moe.gemm_f8(x, ref.tensor_of(w[0]), _dev(ws[0]), out_dtype=torch.float32)[:1]
    assert torch.isnan(y).nonzero()[:, 1].tolist() == [7, 9] + list(range(128, 256))


def test_gemm_leaves_the_rest_alone():
    import torch
    for m, n in ((1, 50), (20, 50), (70, 260), (300, 300)):
        x, _ = _x(m, 160, "bf16", m)
        w, ws = _w((n, 160), n)
        flat = torch.full((m * n + 512,), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.gemm_f8(x, ref.tensor_of(w), _dev(ws), out=flat[:m * n].view(m, n))
        assert (flat[m * n:] == 77.0).all() and not (flat[:m * n] == 77.0).all()


# ---- products by expert -------------------------------------------------------------------------------------------


def _idx(tokens, top_k, E, seed, empty=True):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:top_k] if top_k <= E else rng.integers(0, E, top_k) for _ in range(tokens)])
    if empty and tokens > 3:
        idx[tokens - tokens // 4:] = -1
        idx[0, top_k - 1] = E + 3  # no expert either
    return idx.astype(np.int32)


def _experts_case(tokens, top_k, E, n, k, swiglu, by_slot, dtype, out, idx=None, codes_in=False):
    idx = _idx(tokens, top_k, E, tokens + E) if idx is None else idx
    slots = tokens * top_k
    x, v = _x(slots if by_slot else tokens, k, dtype, tokens + n)
    w, ws = _w((E, 2, n, k) if swiglu else (E, n, k), E + n)
    ws *= np.float32(0.05)
    groups = moe.moe_group_slots(_dev(idx), E)
    codes, scales = ref.quant(v)
    xs = None
    if codes_in:
        x, xs = moe.quant_rows_f8(x)
    y = moe.experts_gemm_f8(x, groups, ref.tensor_of(w), _dev(ws), x_scale=xs, swiglu=swiglu, out_dtype=ref.torch_dtype(out))
    want, bound = np.zeros((slots, n)), np.zeros((slots, n))
    flat = idx.reshape(-1)
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        if len(mine):
            rows = mine if by_slot else mine // top_k
            want[mine], bound[mine] = _want(codes[rows], scales[:, rows], w[e], ws[e], swiglu, out)
    _close(y, want, bound)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("by_slot", [False, True])
@pytest.mark.parametrize("tokens,top_k,E,n,k", [(1, 1, 1, 16, 16), (1, 4, 16, 50, 272), (5, 2, 4, 33, 144), (8, 16, 32, 64, 512),
                                                (40, 3, 5, 140, 160), (100, 8, 16, 96, 256), (300, 2, 3, 270, 272), (700, 2, 2, 520, 144)])
def test_experts(tokens, top_k, E, n, k, by_slot, swiglu):
    kinds = ["bf16", "f16", "f32"]
    _experts_case(tokens, top_k, E, n, k, swiglu, by_slot, kinds[(tokens + n) % 3], kinds[(n + k // 16) % 3],
                  codes_in=(tokens + top_k) % 2 == 0)


# with SwiGLU, to every kernel: tokens, top_k, experts, n, k, rows by slot
SWIGLU_EXPERTS = [(9, 3, 16, 300, 400, False), (60, 4, 3, 500, 656, True), (100, 4, 8, 550, 656, False), (300, 4, 8, 600, 272, True),
                  (258, 2, 16, 985, 1168, False), (700, 4, 4, 550, 400, True), (2000, 2, 2, 1050, 272, False), (1000, 4, 8, 1500, 272, False)]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,top_k,E,n,k,by_slot", SWIGLU_EXPERTS)
def test_experts_swiglu(tokens, top_k, E, n, k, by_slot, out):
    _experts_case(tokens, top_k, E, n, k, True, by_slot, "bf16", out, codes_in=tokens % 200 == 0)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("idx", [[5], [0, 3, 5, 2], [1, -1, 1, 4], [-1, -1], [2] * 20, list(range(6)) * 8])
def test_experts_of_one_token(idx, swiglu):
    """One token: distinct experts, one that comes twice, none, more slots than a tile."""
    _experts_case(1, len(idx), 6, 50, 272, swiglu, False, "bf16", "f32", idx=np.array([idx], np.int32))


@pytest.mark.parametrize("tokens", [30, 600])
def test_experts_all_on_one(tokens):
    """Every token takes one expert, all others are empty."""
    _experts_case(tokens, 1, 40, 130, 144, False, False, "bf16", "f32", idx=np.full((tokens, 1), 17, np.int32))


# ---- the chain ------------------------------------------------------------------------------------------------------


class _Layer:
    """Norm, routed experts and a shared expert, with a program's own buffers."""

    def __init__(self, tokens, hidden, inter, E, top_k, seed=0):
        import torch
        self.E, self.k, self.tokens = E, top_k, tokens
        sets = [_w(s, seed + i) for i, s in enumerate(((E, 2, inter, hidden), (E, hidden, inter), (2, inter, hidden), (hidden, inter)))]
        self.host = [(w, s * np.float32(0.2)) for w, s in sets]
        self.w1, self.w2, self.v1, self.v2 = ((ref.tensor_of(w), _dev(s)) for w, s in self.host)
        self.gain = _dev(np.random.default_rng(seed).uniform(0.5, 1.5, hidden).astype(np.float32))
        empty = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")
        self.total = empty(tokens, hidden, dtype=torch.float32)
        self.x, self.xs = empty(tokens, hidden, dtype=torch.float8_e4m3fn), empty(ref.blocks(hidden), tokens, dtype=torch.float32)
        self.idx, self.gate = empty(tokens, top_k, dtype=torch.int32), empty(tokens, top_k, dtype=torch.float32)
        self.groups = moe.alloc_slot_groups(tokens, top_k, E)
        self.h, self.y = empty(tokens * top_k, inter), empty(tokens * top_k, hidden)
        self.hs, self.ys = empty(tokens, inter), empty(tokens, hidden, dtype=torch.float32)
        size = max(moe.experts_gemm_f8_workspace_size(self.groups, tokens, inter, hidden, True, torch.float8_e4m3fn),
                   moe.experts_gemm_f8_workspace_size(self.groups, tokens * top_k, hidden, inter, False, torch.bfloat16),
                   moe.gemm_f8_workspace_size(tokens, inter, hidden, True, torch.float8_e4m3fn),
                   moe.gemm_f8_workspace_size(tokens, hidden, inter, False, torch.bfloat16))
        self.ws = empty(size, dtype=torch.uint8)

    def __call__(self, logits, h, t, out, stream=None):
        moe.residual_add_rmsnorm_f8(h, t, gain=self.gain, h_out=self.total, q=self.x, scale=self.xs, stream=stream)
        moe.moe_route(logits, self.k, idx=self.idx, gate=self.gate, stream=stream)
        moe.moe_group_slots(self.idx, self.E, groups=self.groups, stream=stream)
        moe.experts_gemm_f8(self.x, self.groups, *self.w1, x_scale=self.xs, swiglu=True, out=self.h, ws=self.ws, stream=stream)
        moe.experts_gemm_f8(self.h, self.groups, *self.w2, out=self.y, ws=self.ws, stream=stream)
        moe.gemm_f8(self.x, *self.v1, x_scale=self.xs, swiglu=True, out=self.hs, ws=self.ws, stream=stream)
        moe.gemm_f8(self.hs, *self.v2, out=self.ys, ws=self.ws, stream=stream)
        moe.moe_combine(self.y, self.gate, residual=self.ys, out=out, stream=stream)
        return out


def _layer_inputs(tokens, hidden, E, seed):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((tokens, E)) * 1.7).astype(np.float32)
    if tokens > 2:
        logits[tokens - 2:] = -np.inf  # padded rows
    h, hv = _x(tokens, hidden, "f32", seed, sigma=2.0)
    t, tv = _x(tokens, hidden, "bf16", seed + 1)
    return logits, h, t, hv, tv


@pytest.mark.parametrize("tokens,hidden,inter", [(1, 512, 256), (7, 256, 144), (150, 272, 144)])
def test_layer(tokens, hidden, inter):
    """Stage by stage: each stage's output against the 64-bit form of what the stage before left."""
    import torch
    E, k = 16, 4
    layer = _Layer(tokens, hidden, inter, E, k)
    logits, h, t, hv, tv = _layer_inputs(tokens, hidden, E, tokens)
    out = torch.empty(tokens, hidden, device="cuda")
    layer(_dev(logits), h, t, out)
    g, v = ref.norm(hv, tv, layer.gain.cpu().numpy(), 1e-6)
    assert np.array_equal(layer.total.cpu().numpy(), g)
    _check_norm(layer.x, layer.xs, v, True)
    codes, scales = ref.VALUES[ref.codes_of(layer.x)], layer.xs.cpu().numpy().astype(np.float64)
    flat = layer.idx.cpu().numpy().reshape(-1)
    (w1, s1), (w2, s2), (v1, t1), (v2, t2) = layer.host

    def by_expert(codes, scales, w, s, n, div, swiglu):
        want, bound = np.zeros((len(flat), n)), np.zeros((len(flat), n))
        for e in range(E):
            mine = np.flatnonzero(flat == e)
            if len(mine):
                want[mine], bound[mine] = _want(codes[mine // div], scales[:, mine // div], w[e], s[e], swiglu, "bf16")
        return want, bound

    _close(layer.h, *by_expert(codes, scales, w1, s1, inter, k, True), "FC1")
    _close(layer.y, *by_expert(*ref.quant(layer.h.double().cpu().numpy()), w2, s2, hidden, 1, False), "FC2")
    _close(layer.hs, *_want(codes, scales, v1, t1, True, "bf16"), "shared FC1")
    _close(layer.ys, *_want(*ref.quant(layer.hs.double().cpu().numpy()), v2, t2, False, "f32"), "shared FC2")
    y, gate = layer.y.double().cpu().numpy().reshape(tokens, k, hidden), layer.gate.double().cpu().numpy()[:, :, None]
    want = layer.ys.double().cpu().numpy() + (y * gate).sum(1)
    size = np.abs(layer.ys.double().cpu().numpy()) + (np.abs(y) * gate).sum(1)
    _close(out, want, size * (k + 1) * 2.0 ** -24 * 1.001 + 2.0 ** -149, "sum")


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_layer_in_a_graph_and_on_another_stream(tokens):
    """Captured once and replayed on new inputs, with the program's own eager work in between; and eagerly on a side
    stream: the same bits as an eager run."""
    import torch
    hidden, inter, E, k = 256, 128, 16, 4
    layer, check = _Layer(tokens, hidden, inter, E, k), _Layer(tokens, hidden, inter, E, k)
    ins = [_layer_inputs(tokens, hidden, E, 50 + i) for i in range(4)]
    logits, h, t, out = _dev(ins[0][0]), ins[0][1].clone(), ins[0][2].clone(), torch.empty(tokens, hidden, device="cuda")
    want = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(logits, h, t, out)
    s.synchronize()
    check(logits, h, t, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer(logits, h, t, out)
    for lg, hi, ti, _, _ in ins + ins[:2]:
        logits.copy_(_dev(lg))
        h.copy_(hi)
        t.copy_(ti)
        torch.cuda.synchronize()
        graph.replay()
        check(logits, h, t, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(layer.total, check.total)


def test_two_streams_at_once():
    """Two layers with their own buffers on two streams: each has the bits of a run alone."""
    import torch
    hidden, inter, E, k, tokens = 256, 128, 16, 4, 200
    layers = [_Layer(tokens, hidden, inter, E, k, seed=i) for i in range(2)]
    ins = [_layer_inputs(tokens, hidden, E, i) for i in range(2)]
    dev = [(_dev(i[0]), i[1], i[2]) for i in ins]
    alone = [l(*d, torch.empty(tokens, hidden, device="cuda")).clone() for l, d in zip(layers, dev)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty(tokens, hidden, device="cuda") for _ in range(2)]
    for _ in range(5):
        for l, d, s, o in zip(layers, dev, streams, outs):
            l(*d, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, outs))


def test_memory_of_a_call_on_another_stream():
    """A call given a stream makes its outputs and workspace there: what the current stream allocates and writes while
    that stream still works never lands in them."""
    import torch
    m, n, k, top_k, E = 48, 512, 1024, 2, 4
    x, _ = _x(m, k, "f32", 1)
    t, _ = _x(m, k, "bf16", 2)
    w, ws = _w((E, n, k), 3)
    w, ws = ref.tensor_of(w), _dev(ws)
    groups = moe.moe_group_slots(_dev(_idx(m, top_k, E, 4)), E)

    kept = []  # a buffer of the caller's is the caller's to keep while the stream works

    def run(stream):
        q, qs = moe.quant_rows_f8(x, stream=stream)
        h = torch.empty_like(x)
        kept.append(h)
        nq, ns = moe.residual_add_rmsnorm_f8(x, t, h_out=h, stream=stream)
        iq, s = moe.residual_add_rmsnorm_i8(x, t, h_out=h, stream=stream)
        return (q, qs, nq, ns, iq, s, moe.gemm_f8(x, w[0], ws[0], stream=stream),
                moe.experts_gemm_f8(x, groups, w, ws, stream=stream),
                moe.gemm_f8(nq, w[0], ws[0], x_scale=ns, out_dtype=torch.bfloat16, stream=stream))

    want = [v.clone() for v in run(None)]
    need = moe.gemm_f8_workspace_size(m, n, k, False, torch.float32)
    torch.cuda.synchronize()
    for as_int in (False, True):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the calls below wait behind this
        got = run(side.cuda_stream if as_int else side)
        trash = [torch.full((size,), 0x55, dtype=torch.uint8, device="cuda")
                 for size in (need, m * k, 4 * m, 1 << 16, 1 << 12) for _ in range(4)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert all(bool((v == 0x55).all()) for v in trash)


@pytest.mark.parametrize("f8", [True, False])
def test_norm_of_more_rows_than_a_launch_takes(f8):
    """2^21 + 37 rows go in two launches: the last rows and those around the border are those of a call of their own."""
    import torch
    rows, hidden = (1 << 21) + 37, 8
    call = moe.residual_add_rmsnorm_f8 if f8 else moe.residual_add_rmsnorm_i8
    h = torch.randn(rows, hidden, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    q, s = call(h)
    for lo, hi in [(0, 100), ((1 << 21) - 50, (1 << 21) + 10), (rows - 60, rows)]:
        want, ws = call(h[lo:hi].clone())
        assert torch.equal(q[lo:hi].view(torch.uint8), want.view(torch.uint8))
        assert torch.equal((s[:, lo:hi] if f8 else s[lo:hi]), ws)


@pytest.mark.parametrize("m,n,k,out", [(40, 300, 272, "bf16"), (600, 520, 272, "bf16"), (600, 520, 272, "f32")])
def test_experts_of_a_groups_buffer_that_holds_anything(m, n, k, out):
    """Whatever a groups buffer holds, nothing outside the output is written, and a right one then gives right bits."""
    import torch
    top_k, E = 4, 8
    x, _ = _x(m, k, "bf16", 1)
    w, ws = _w((E, n, k), 2)
    w, ws = ref.tensor_of(w), _dev(ws)
    groups = moe.moe_group_slots(_dev(_idx(m, top_k, E, 3)), E)
    dtype = getattr(torch, {"bf16": "bfloat16", "f32": "float32"}[out])
    want = moe.experts_gemm_f8(x, groups, w, ws, out_dtype=dtype)
    right = groups.buffer.clone()
    block = torch.empty(64 + m * top_k + 64, n, dtype=dtype, device="cuda")
    y = block[64:-64]
    gen = torch.Generator("cuda").manual_seed(4)
    for fill in (0, 0xFF, 0x7F, 0x01, None):
        if fill is None:
            groups.buffer.view(torch.uint8).random_(0, 256, generator=gen)
        else:
            groups.buffer.view(torch.uint8).fill_(fill)
        block.fill_(7)
        moe.experts_gemm_f8(x, groups, w, ws, out=y)
        torch.cuda.synchronize()
        assert bool((block[:64] == 7).all()) and bool((block[-64:] == 7).all())
    groups.buffer.copy_(right)
    moe.experts_gemm_f8(x, groups, w, ws, out=y)
    assert torch.equal(y, want)


def test_norm_feeds_the_integer_product():
    """residual_add_rmsnorm_i8 leaves what gemm_i8 takes."""
    import torch
    import i8_reference as ref8
    h, hv = _x(20, 256, "f32", 1)
    t, tv = _x(20, 256, "bf16", 2)
    q, s = moe.residual_add_rmsnorm_i8(h, t)
    w = np.random.default_rng(3).integers(-127, 128, (48, 256)).astype(np.int8)
    ws = np.full(48, 1e-3, np.float32)
    y = moe.gemm_i8(q, _dev(w), _dev(ws), x_scale=s, out_dtype=torch.float32)
    want = ref8.product(q.cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64), w, ws)
    _close(y, want, ref8.product_bound(want, "f32"))
