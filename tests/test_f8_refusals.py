"""The 8-bit floating-point entry points and the norms before the 8-bit
products turn bad arguments down on the host, before anything is enqueued (no
GPU needed), and the binding checks what the C interface cannot see."""
import ctypes

import pytest

import memory_bound_mxfp4_amd as moe

P = ctypes.c_void_p
BF16, F32, F16, I8, F8 = moe.MOE_DTYPE_BF16, moe.MOE_DTYPE_F32, moe.MOE_DTYPE_F16, moe.MOE_DTYPE_I8, moe.MOE_DTYPE_F8
INVALID, UNSUPPORTED, SMALL = moe.MOE_ERR_INVALID_ARGUMENT, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE_TOO_SMALL


def test_quant_refusals():
    f = moe.load().quant_rows_f8
    x, q, s = P(0x1000), P(0x2000), P(0x3000)
    for args in ((None, BF16, 64, 1, 64, q, s), (x, BF16, 64, 1, 64, None, s), (x, BF16, 64, 1, 64, q, None),
                 (x, F8, 64, 1, 64, q, s), (x, I8, 64, 1, 64, q, s), (x, BF16, 63, 2, 64, q, s), (x, BF16, 64, 0, 64, q, s),
                 (x, BF16, 64, 1, 0, q, s), (P(0x1001), BF16, 64, 1, 64, q, s), (P(0x1002), F32, 64, 1, 64, q, s),
                 (x, BF16, 64, 1, 64, q, P(0x3002))):
        assert f(*args, None) == INVALID, args
    assert f(x, BF16, 65537, 1, 65537, q, s, None) == UNSUPPORTED
    assert f(x, BF16, 64, 1 << 24, 64, q, s, None) == UNSUPPORTED
    x = P(0x10000)                                                          # 4 rows of 160 fp32: 2560 bytes, 640 codes, 32 of scales
    for q, s in ((0x10000 + 2556, 0x30000), (0x10000 - 639, 0x30000), (0x20000, 0x10000 + 2556), (0x20000, 0x10000 - 28),
                 (0x20000, 0x20000 + 636), (0x20000, 0x20000 - 28)):
        assert f(x, F32, 160, 4, 160, P(q), P(s), None) == INVALID, (hex(q), hex(s))


def _gemm(**over):
    a = dict(x=P(0x1000), xd=BF16, stride=64, xs=None, m=4, k=64, w=P(0x2000), ws=P(0x3000), n=32, swiglu=0,
             y=P(0x4000), yd=BF16, work=P(0x10000), size=1 << 20)
    a.update(over)
    return moe.load().gemm_f8(a["x"], a["xd"], a["stride"], a["xs"], a["m"], a["k"], a["w"], a["ws"], a["n"], a["swiglu"],
                              a["y"], a["yd"], a["work"], a["size"], None)


BAD_PRODUCT = [
    dict(x=None), dict(w=None), dict(ws=None), dict(y=None), dict(m=0), dict(n=0), dict(k=0), dict(k=8), dict(k=40),
    dict(stride=48), dict(swiglu=2), dict(xd=7), dict(xd=I8), dict(xd=I8, xs=P(0x5000)), dict(yd=F8), dict(yd=I8), dict(yd=5),
    dict(xd=F8), dict(xs=P(0x5000)), dict(xd=F8, xs=P(0x5000), stride=72), dict(xd=F8, xs=P(0x5000), x=P(0x1008)),
    dict(xd=F8, xs=P(0x5002)), dict(x=P(0x1001)), dict(w=P(0x2008)), dict(y=P(0x4008)), dict(ws=P(0x3002)), dict(work=None),
    dict(work=P(0x10010))]


@pytest.mark.parametrize("over", BAD_PRODUCT, ids=str)
def test_gemm_invalid(over):
    assert _gemm(**over) == INVALID


def test_gemm_unsupported_and_workspace():
    assert _gemm(k=65552, stride=65552) == UNSUPPORTED
    assert _gemm(n=(1 << 20) + 1) == UNSUPPORTED
    assert _gemm(m=1 << 24) == UNSUPPORTED
    need = moe.load().gemm_f8_workspace_size(4, 32, 64, 0, BF16)
    assert need > 0 and _gemm(size=need - 1) == SMALL
    assert moe.load().gemm_f8_workspace_size(0, 32, 64, 0, BF16) == 0


def _experts(**over):
    a = dict(x=P(0x1000), xd=BF16, stride=64, xs=None, rows=4, k=64, g=P(0x20000), gb=1 << 20, tokens=4, top_k=2, E=8,
             w=P(0x2000), ws=P(0x3000), n=32, swiglu=0, y=P(0x4000), yd=BF16, work=P(0x10000), size=1 << 20)
    a.update(over)
    if "m" in over:
        a["rows"] = over["m"]
    return moe.load().experts_gemm_f8(a["x"], a["xd"], a["stride"], a["xs"], a["rows"], a["k"], a["g"], a["gb"],
                                      a["tokens"], a["top_k"], a["E"], a["w"], a["ws"], a["n"], a["swiglu"], a["y"],
                                      a["yd"], a["work"], a["size"], None)


@pytest.mark.parametrize("over", BAD_PRODUCT + [
    dict(g=None), dict(g=P(0x20080)), dict(rows=5), dict(rows=2), dict(tokens=0), dict(top_k=0), dict(top_k=65),
    dict(E=0), dict(E=4097)], ids=str)
def test_experts_invalid(over):
    assert _experts(**over) == INVALID


def test_experts_workspaces():
    lib = moe.load()
    assert _experts(gb=lib.moe_slot_groups_size(4, 2, 8) - 1) == SMALL
    assert _experts(size=lib.experts_gemm_f8_workspace_size(4, 2, 8, 4, 32, 64, 0, BF16) - 1) == SMALL
    assert lib.experts_gemm_f8_workspace_size(4, 65, 8, 4, 32, 64, 0, BF16) == 0


FAR = dict(x=P(0x100000), w=P(0x200000), ws=P(0x300000), y=P(0x400000), work=P(0x500000))


def test_product_outputs_over_inputs():
    """The output over the rows, the matrix, the scales, the workspace or the groups; the workspace over any of them."""
    lib = moe.load()
    over = dict(FAR, k=144, stride=144, n=160)                              # 4 rows of 288 bytes, 2 x 2 blocks of scales, 1280 bytes of y
    need = lib.gemm_f8_workspace_size(4, 160, 144, 0, BF16)
    x_end, w_end, s_end = 0x100000 + 4 * 288, 0x200000 + 160 * 144, 0x300000 + 16
    for at in (0x100000, x_end - 16, 0x100000 - 1264, 0x200000, w_end - 16, 0x200000 - 1264, 0x300000, 0x300000 - 1264,
               0x500000, 0x500000 + need - 16, 0x500000 - 1264):
        assert _gemm(**{**over, "y": P(at)}) == INVALID, hex(at)
    for at in (0x100000, 0x100000 - 256, 0x100400, 0x200000, w_end - 256, 0x300000, 0x400000, 0x400400):
        assert _gemm(**{**over, "work": P(at)}) == INVALID, hex(at)
    codes = {**over, "xd": F8, "xs": P(0x600000)}                           # 2 x 4 scales
    for at in (0x600000, 0x600010, 0x600000 - 1264):
        assert _gemm(**{**codes, "y": P(at)}) == INVALID, hex(at)
    two = {**over, "swiglu": 1}
    assert _gemm(**{**two, "y": P(w_end + 160 * 144 - 16)}) == INVALID
    assert _gemm(**{**two, "y": P(s_end)}) == INVALID
    for at in (0x100000, 0x200000, 0x300000):                               # one row
        assert _gemm(**{**over, "m": 1, "y": P(at)}) == INVALID, hex(at)

    need = lib.experts_gemm_f8_workspace_size(4, 2, 8, 4, 160, 144, 0, BF16)
    groups = lib.moe_slot_groups_size(4, 2, 8)
    far = {**over, "g": P(0x700000), "gb": groups}
    for at in (0x100000, 0x200000 + 8 * 160 * 144 - 16, 0x300000 + 8 * 16 - 16, 0x500000 + need - 16, 0x700000, 0x700000 + groups - 16):
        assert _experts(**{**far, "y": P(at)}) == INVALID, hex(at)
    for at in (0x100000, 0x200000 + 8 * 160 * 144 - 256, 0x300000, 0x700000, 0x700000 + groups - 256):
        assert _experts(**{**far, "work": P(at)}) == INVALID, hex(at)
    for at in (0x100000, 0x200000, 0x300000, 0x700000):
        assert _experts(**{**far, "rows": 1, "tokens": 1, "y": P(at)}) == INVALID, hex(at)


def _norm(f8=True, **over):
    a = dict(h=P(0x10000), hs=160, t=P(0x20000), td=BF16, ts=160, gain=P(0x30000), rows=4, hidden=160, eps=1e-6,
             h_out=P(0x40000), out=P(0x50000), q=P(0x60000), scale=P(0x70000))
    a.update(over)
    f = moe.load().residual_add_rmsnorm_f8 if f8 else moe.load().residual_add_rmsnorm_i8
    return f(a["h"], a["hs"], a["t"], a["td"], a["ts"], a["gain"], a["rows"], a["hidden"], a["eps"], a["h_out"], a["out"],
             a["q"], a["scale"], None)


@pytest.mark.parametrize("f8", [True, False])
def test_norm_refusals(f8):
    for over in (dict(h=None), dict(q=None), dict(scale=None), dict(rows=0), dict(hidden=0), dict(hs=159), dict(ts=159),
                 dict(td=I8), dict(td=F8), dict(td=9), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                 dict(t=None), dict(h_out=None), dict(h=P(0x10002)), dict(t=P(0x20001)), dict(t=P(0x20002), td=F32),
                 dict(gain=P(0x30002)), dict(h_out=P(0x40002)), dict(out=P(0x50001)), dict(scale=P(0x70002))):
        assert _norm(f8, **over) == INVALID, over
    assert _norm(f8, hidden=65537, hs=65537, ts=65537) == UNSUPPORTED
    assert _norm(f8, rows=1 << 24) == UNSUPPORTED


@pytest.mark.parametrize("f8", [True, False])
def test_norm_outputs_over_inputs(f8):
    """4 rows of 160: 2560 bytes of h and h_out, 1280 of t and out, 640 of codes, 640 of the gain."""
    for name, size in (("out", 1280), ("q", 640), ("scale", 32 if f8 else 16), ("h_out", 2560)):
        for base, length in ((0x10000, 2560), (0x20000, 1280), (0x30000, 640)):
            for at in (base + length - 4, base - size + 4):
                assert _norm(f8, **{name: P(at)}) == INVALID, (name, hex(at))
    assert _norm(f8, h_out=P(0x10004)) == INVALID
    assert _norm(f8, h_out=P(0x10000), hs=164) == INVALID                   # in place, but its rows lie apart
    outs = dict(h_out=(0x40000, 2560), out=(0x50000, 1280), q=(0x60000, 640), scale=(0x70000, 32 if f8 else 16))
    for one, (base, length) in outs.items():
        for other in outs:
            if other != one:
                assert _norm(f8, **{other: P(base + length - 4)}) == INVALID, (one, other)


def test_binding_checks():
    """What the binding sees and the C interface cannot: types, shapes, strides and devices of tensors."""
    import torch
    e4m3 = torch.float8_e4m3fn
    x, w, s = torch.zeros(4, 64), torch.zeros(32, 64).to(e4m3), torch.zeros(1, 1)
    h, t = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (
            lambda: moe.gemm_f8(x, w, s),                                  # on the CPU
            lambda: moe.gemm_f8(x.double(), w, s),                         # type of x
            lambda: moe.gemm_f8(x.to(torch.int8), w, s, x_scale=torch.zeros(1, 4)),
            lambda: moe.gemm_f8(x.to(torch.float8_e5m2), w, s, x_scale=torch.zeros(1, 4)),
            lambda: moe.gemm_f8(x, w.float(), s),                          # type of w
            lambda: moe.gemm_f8(x, w.view(torch.int8), s),
            lambda: moe.gemm_f8(x, w, s.double()),
            lambda: moe.gemm_f8(x, w[:, :48], s),                          # k of w, and not contiguous
            lambda: moe.gemm_f8(x, w, torch.zeros(1, 2)),                  # blocks of the scales
            lambda: moe.gemm_f8(x, w, torch.zeros(32, 1)),
            lambda: moe.gemm_f8(x, w, s, swiglu=True),                     # w needs two matrices
            lambda: moe.gemm_f8(x, w, s, x_scale=torch.zeros(1, 4)),       # scales of rows that are no codes
            lambda: moe.gemm_f8(x.to(e4m3), w, s),                         # codes without scales
            lambda: moe.gemm_f8(x.to(e4m3), w, s, x_scale=torch.zeros(4, 1)),  # scales the other way round
            lambda: moe.gemm_f8(x.t(), w, s),                              # elements apart
            lambda: moe.gemm_f8(x, w, s, out=torch.zeros(4, 31)),
            lambda: moe.gemm_f8(x, w, s, out=torch.zeros(4, 32), out_dtype=torch.float16),
            lambda: moe.gemm_f8(x, w, s, out_dtype=e4m3),
            lambda: moe.quant_rows_f8(x, q=torch.zeros(4, 64)),
            lambda: moe.quant_rows_f8(x, scale=torch.zeros(4, 1)),
            lambda: moe.quant_rows_f8(x.to(e4m3)),
            lambda: moe.quant_rows_f8(x[:1].expand(4, 64)),                # rows on top of each other
            lambda: moe.residual_add_rmsnorm_f8(h, t),                     # on the CPU
            lambda: moe.residual_add_rmsnorm_f8(t, t),                     # type of h
            lambda: moe.residual_add_rmsnorm_f8(h, t[:3]),
            lambda: moe.residual_add_rmsnorm_f8(h, t.to(torch.int8)),
            lambda: moe.residual_add_rmsnorm_f8(h, h_out=torch.zeros(4, 64)),
            lambda: moe.residual_add_rmsnorm_f8(torch.zeros(4, 80)[:, :64], t),   # in place needs rows one after another
            lambda: moe.residual_add_rmsnorm_f8(h, t, gain=torch.zeros(63)),
            lambda: moe.residual_add_rmsnorm_f8(h, t, gain=torch.zeros(64, dtype=torch.bfloat16)),
            lambda: moe.residual_add_rmsnorm_f8(h, t, out=torch.zeros(4, 64)),
            lambda: moe.residual_add_rmsnorm_f8(h, t, q=torch.zeros(4, 64, dtype=torch.int8)),
            lambda: moe.residual_add_rmsnorm_i8(h, t, q=torch.zeros(4, 64).to(e4m3)),
            lambda: moe.residual_add_rmsnorm_i8(h, t, scale=torch.zeros(1, 4)),
    ):
        with pytest.raises(ValueError):
            call()
    groups = moe.alloc_slot_groups(4, 2, 8, device="cpu")
    wide, scales = torch.zeros(8, 32, 64).to(e4m3), torch.zeros(8, 1, 1)
    with pytest.raises(ValueError):
        moe.experts_gemm_f8(torch.zeros(5, 64), groups, wide, scales)
    with pytest.raises(ValueError):
        moe.experts_gemm_f8(x, groups, wide[:7], scales[:7])


def test_sizes_past_32_bits():
    """Sizes whose low 32 bits would pass are turned down by the binding."""
    import torch
    big = (1 << 32) + 4
    rows = torch.zeros(1, dtype=torch.bfloat16).expand(big, 1)
    w = torch.zeros(32, 16).to(torch.float8_e4m3fn)
    for call in (
            lambda: moe.quant_rows_f8(rows),
            lambda: moe.quant_rows_f8(rows.t()),
            lambda: moe.residual_add_rmsnorm_f8(torch.zeros(1).expand(big, 1)),
            lambda: moe.gemm_f8(torch.zeros(4, 16), w[:1, :1].expand(big, 16), torch.zeros(1, 1)),
            lambda: moe.gemm_f8_workspace_size(big, 32, 64, False, torch.bfloat16),
            lambda: moe.experts_gemm_f8_workspace_size(moe.SlotGroups(4, 2, 8, None, None, None), 4, big, 64, False,
                                                       torch.bfloat16),
    ):
        with pytest.raises(ValueError):
            call()
