"""Four-bit rows and weights, their dispatch and their products.

The quantisation is defined to the bit (nearest codes, ties to even, with the named
32-bit steps), so codes, scale bytes and values have to be equal to a search over the
code values in 64 bits. Products are held to the formulas in 64 bits: with v = 2^-23 a sum
of K products is off by (K + 2) v times the sum of magnitudes and the tensor scales by
2 v; activations and the rounding to 16 bits as for the products of wider types."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, TINY, ACT_ERR = 2.0 ** -23, 2.0 ** -25, 2.0 ** -17
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FMTS = ["nv", "mx", "e8m0"]
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def rand(seed, *shape, dtype=torch.float32, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * gain).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def group(fmt):
    return 16 if fmt == "nv" else 32


def pieces(H, fmt):
    return -(-(H // group(fmt)) // 16)


def two(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


E4M3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119],
                    dtype=torch.float64)


def nearest(v, table):
    hi = torch.searchsorted(table, v.contiguous()).clamp_(1, table.numel() - 1)
    down, up = v - table[hi - 1], table[hi] - v
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x, fmt, ts=None):
    """(codes [R, H / 2], scale bytes [pieces, R, 16], values [R, H] in 64 bits); ts: one for each row."""
    R, H = x.shape
    g = group(fmt)
    f32 = lambda t: t.float().double()
    v = x.double().reshape(R, H // g, g)
    amax = v.abs().amax(2)
    bad = ~torch.isfinite(amax)
    amax = torch.where(bad, 0.0, amax)
    if fmt == "nv":
        t = torch.ones(R, 1, dtype=torch.float64, device=DEV) if ts is None else ts.double().reshape(-1, 1).expand(R, 1)
        byte = nearest(f32(amax / f32(6.0 * t)).clamp(max=448.0), E4M3.to(DEV))
        d = f32(E4M3.to(DEV)[byte] * t)
        byte = torch.where(bad, 0x7F, byte)
    else:
        e = (amax.clamp(min=2.0 ** -149).view(torch.int64) >> 52) - 1025
        if fmt == "e8m0":
            e = torch.where(6.0 * two(e) >= amax, e, e + 1)
        e = e.clamp(-127, 127)
        d = two(e)
        byte = torch.where(bad, 255, e + 127)
    v = torch.where(bad[:, :, None], 0.0, v)
    r = torch.where(d[:, :, None] > 0, f32(v / torch.where(d > 0, d, 1.0)[:, :, None]), 0.0)
    code = nearest(r.abs().clamp(max=6.0), torch.tensor(CODES, dtype=torch.float64, device=DEV))
    val = torch.tensor(CODES, dtype=torch.float64, device=DEV)[code] * torch.sign(r) * d[:, :, None]
    val = torch.where(bad[:, :, None], math.nan, val)
    code = (code + 8 * (torch.signbit(r) & ((code > 0) | torch.signbit(r)))).to(torch.uint8).reshape(R, H // 2, 2)
    sc = torch.zeros(R, pieces(H, fmt) * 16, dtype=torch.uint8, device=DEV)
    sc[:, :H // g] = byte.to(torch.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), sc.reshape(R, -1, 16).transpose(0, 1).contiguous(), val.reshape(R, H)


def same_codes(a, b):
    """Equal but for the sign of zeros, which are equal values."""
    za, zb = [torch.stack([t & 15, t >> 4], -1) for t in (a, b)]
    return bool(((za == zb) | ((za & 7 == 0) & (zb & 7 == 0))).all())


def inputs(seed, R, H, dtype):
    """Rows with outliers, and groups that are zero, tiny, huge, or of one magnitude."""
    x = rand(seed, R, H)
    x = torch.where(torch.rand(R, H, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)) < 0.02, x * 50, x)
    if R > 4:
        x[1] = 0
        x[2] *= 1e-6
        x[3] = x[3].sign() * 0.75
        x[4] = (x[4] * 4).round() / 4     # many ties
    return x.to(dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,H", [(1, 64), (3, 128), (5, 192), (33, 512), (17, 576), (7, 1024), (130, 2048), (64, 7168), (3, 32768), (700, 320)])
def test_quant_and_back(dev, R, H, fmt):
    for n, dtype in enumerate(DT.values()):
        x = inputs(R + n, R, H + 16, dtype)[:, :H]
        for ts in ([None] if fmt != "nv" else [None, (x.abs().amax().float() / 2688)[None].contiguous(), torch.full((1,), 0.0137, device=DEV)]):
            q, sc, val = quantise(x, fmt, ts)
            o = dev.quant_fp4(x, fmt=fmt, tensor_scale=ts)
            assert torch.equal(o["scales"], sc) and same_codes(o["xq"], q)
            for out in DT.values():
                back = dev.dequant_fp4(o["xq"], o["scales"], fmt=fmt, tensor_scale=ts, dtype=out)
                assert torch.equal(back, val.float().to(out))


@pytest.mark.parametrize("fmt", FMTS)
def test_every_magnitude(dev, fmt):
    """bf16 and float32 values over the whole range of exponents, zeros and subnormal numbers among them."""
    bits = torch.arange(0, 1 << 16, device=DEV, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).reshape(-1, 64)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    for v in (x, x.float() * 1.0000001, x[:, torch.randperm(64, device=DEV, generator=torch.Generator(DEV).manual_seed(1))]):
        for ts in ([None] if fmt != "nv" else [None, torch.full((1,), 3.7e-5, device=DEV), torch.full((1,), 2.0 ** -100, device=DEV),
                                               torch.full((1,), 1.1e30, device=DEV)]):
            q, sc, val = quantise(v, fmt, ts)
            o = dev.quant_fp4(v, fmt=fmt, tensor_scale=ts)
            assert torch.equal(o["scales"], sc) and same_codes(o["xq"], q)
            assert torch.equal(dev.dequant_fp4(o["xq"], o["scales"], fmt=fmt, tensor_scale=ts, dtype=torch.float32), val.float())


def test_every_border(dev):
    """Quotients on and next to the borders between codes, for divisors of 24 bits."""
    H, n = 1024, 400
    d = (rand(1, n).abs() + 0.5) * torch.exp2(torch.arange(n, device=DEV) % 41 - 20.0)
    b = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device=DEV).repeat(H // 8)
    for ts in d.tolist():
        t = torch.full((1,), ts, device=DEV)
        x = b * t
        x = torch.stack([x, -x, torch.nextafter(x, torch.full_like(x, 1e30)), torch.nextafter(x, torch.zeros_like(x))])
        x[:, ::16] = 6.0 * t  # scale 1 in every group
        q, sc, _ = quantise(x, "nv", t)
        o = dev.quant_fp4(x, tensor_scale=t)
        assert torch.equal(o["scales"], sc) and same_codes(o["xq"], q)


@pytest.mark.parametrize("fmt", FMTS)
def test_not_finite(dev, fmt):
    x = rand(1, 12, 128)
    x[1, 5], x[2, 40], x[3, 127] = math.nan, math.inf, -math.inf
    for dtype in DT.values():
        q, sc, val = quantise(x.to(dtype), fmt)
        o = dev.quant_fp4(x.to(dtype), fmt=fmt)
        assert torch.equal(o["scales"], sc) and same_codes(o["xq"], q)
        back = dev.dequant_fp4(o["xq"], o["scales"], fmt=fmt, dtype=torch.float32)
        assert torch.equal(torch.isnan(back), torch.isnan(val)) and torch.isnan(back).sum() == 3 * group(fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_by_name(dev, fmt):
    """Only the rows asked for are read or written, each way to name them."""
    R, H, L = 60, 320, 4
    x = rand(2, R, H, dtype=torch.bfloat16)
    keep = torch.rand(R, device=DEV, generator=torch.Generator(DEV).manual_seed(3)) < 0.5
    slab = torch.arange(R, device=DEV) % (R // L) < i32([0, 15, 3, 9]).repeat_interleave(R // L)
    for rows, how in ((torch.arange(R, device=DEV) < 23, dict(d_num_live=i32([23]))), (keep, dict(m_indices=torch.where(keep, 2, -1).to(torch.int32))),
                      (slab, dict(masked_m=i32([0, 15, 3, 9]), cap=R // L)), (torch.zeros(R, dtype=torch.bool, device=DEV), dict(d_num_live=i32([0])))):
        args = dict(tensor_scale=None, n_scales=1, d_num_live=None, m_indices=None, masked_m=None, cap=0) | how
        xn = torch.where(rows[:, None], x, math.nan)
        xq, sc = torch.full((R, H // 2), 7, dtype=torch.uint8, device=DEV), torch.full((pieces(H, fmt), R, 16), 7, dtype=torch.uint8, device=DEV)
        st = i32([0])
        assert dev.moe_quant_fp4(xn, H, torch.bfloat16, R, H, fmt, *args.values(), xq, sc, R, st) == dev.MOE_OK
        q, s, val = quantise(x, fmt)
        assert same_codes(xq[rows], q[rows]) and torch.equal(sc[:, rows], s[:, rows])
        assert (xq[~rows] == 7).all() and (sc[:, ~rows] == 7).all()
        out = torch.full((R, H), 9.0, device=DEV, dtype=torch.bfloat16)
        assert dev.moe_dequant_fp4(xq, sc, R, R, H, fmt, *args.values(), out, H, torch.bfloat16, st) == dev.MOE_OK
        assert torch.equal(out[rows], val[rows].float().bfloat16()) and (out[~rows] == 9).all()
        assert dev.moe_status_sync(st) == dev.MOE_OK
    o = dev.quant_fp4(x, fmt=fmt, num_live=i32([R + 1]))
    assert dev.moe_status_sync(o["status"]) == dev.MOE_ERR_LIVE_OVERFLOW
    o = dev.quant_fp4(x.view(L, R // L, H), fmt=fmt, masked_m=i32([0, 15, 3, 9]))
    assert o["xq"].shape == (L, R // L, H // 2) and same_codes(o["xq"].view(R, -1)[slab], q[slab])


def test_a_scale_for_each_expert(dev):
    L, N, K = 3, 40, 192
    w = rand(3, L, N, K) * torch.tensor([1.0, 0.01, 30.0], device=DEV)[:, None, None]
    ts = (w.abs().amax((1, 2)) / 2688).contiguous()
    o = dev.quant_fp4(w.view(L * N, K), tensor_scale=ts)
    q, sc, val = quantise(w.view(L * N, K), "nv", ts.repeat_interleave(N))
    assert torch.equal(o["scales"], sc) and same_codes(o["xq"], q)
    assert torch.equal(dev.dequant_fp4(o["xq"], o["scales"], tensor_scale=ts, dtype=torch.float32), val.float())


# ---------------------------------------------------------------------------
# Dispatch
# ---------------------------------------------------------------------------

DISPATCH = [  # T, H, E, L, K, block, dtype
    (1, 64, 8, 8, 2, 1, "bf16"), (16, 256, 8, 8, 2, 128, "fp32"), (128, 7168, 256, 32, 8, 128, "bf16"), (255, 320, 64, 64, 8, 16, "fp16"),
    (2048, 128, 16, 16, 1, 8, "bf16"), (300, 1024, 64, 64, 7, 128, "bf16"), (1000, 2048, 256, 256, 8, 128, "bf16"), (777, 576, 40, 7, 6, 16, "fp32"),
    (4096, 512, 300, 300, 4, 1, "fp16"), (100, 32768, 32, 32, 32, 8, "bf16"), (70, 32768, 1000, 1000, 32, 1, "fp32"),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(DISPATCH)))
def test_dispatch(dev, case, fmt):
    """The layout of the unquantised permute, and each kept slot's row quantised as alone."""
    T, H, E, L, K, block, name = DISPATCH[case]
    x = inputs(case, T, H + 16, DT[name])[:, :H]
    g = torch.Generator(DEV).manual_seed(case)
    ids = torch.randint(0, E, (T, K), device=DEV, dtype=torch.int32, generator=g)
    ids[torch.rand(T, K, device=DEV, generator=g) < 0.1] = -1
    w = rand(case, T, K)
    ts = (x.abs().amax().float() / 2688)[None].contiguous() if fmt == "nv" and case % 2 else None
    for n in (None, T, T // 2):
        live = None if n is None else i32([n])
        d = dev.dispatch_fp4(x, ids, w, E, L, block_e=block, fmt=fmt, tensor_scale=ts, num_tokens=live)
        p = dev.permute(x.contiguous(), ids, w, E, L, block_e=block, num_tokens=live)
        assert dev.moe_status_sync(d["status"]) == dev.MOE_OK
        for k in ("m_indices", "src2dst", "counts", "starts", "psum", "total"):
            assert torch.equal(d[k], p[k]), k
        t, k = torch.nonzero(d["src2dst"] >= 0, as_tuple=True)
        rows = d["src2dst"][t, k].long()
        q = dev.quant_fp4(x, fmt=fmt, tensor_scale=ts)
        assert torch.equal(d["xq"][rows], q["xq"][t]) and torch.equal(d["scales"][:, rows], q["scales"][:, t])
        assert torch.equal(d["row_weights"][rows], w[t, k])


@pytest.mark.parametrize("T", [100, 700])
def test_dispatch_leaves_padding(dev, T):
    H, E, K, block = 192, 12, 3, 64
    x, ids, w = rand(1, T, H), torch.randint(0, E, (T, K), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(2)), rand(3, T, K)
    bound = dev.moe_compact_bound(T * K, E, block)
    xq, sc = torch.full((bound, H // 2), 7, dtype=torch.uint8, device=DEV), torch.full((1, bound + 5, 16), 7, dtype=torch.uint8, device=DEV)
    v = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    mi, s2d, counts, starts, psum, total, st = v(bound), v(T * K), v(E), v(E), v(E), v(1), v(1)
    ws = dev.Workspace(T, K, E, DEV)
    assert dev.moe_dispatch_fp4(x, H, torch.float32, T, None, H, ids, w, K, E, E, block, "nv", None, xq, sc, bound + 5, mi, bound, s2d, counts,
                                starts, psum, total, None, ws.buf, ws.nbytes, st) == dev.MOE_OK
    assert dev.moe_status_sync(st) == dev.MOE_OK and (mi >= 0).sum() == T * K
    assert (xq[mi < 0] == 7).all() and (sc[:, :bound][:, mi < 0] == 7).all() and (sc[:, bound:] == 7).all()


def test_empty_dispatch(dev):
    e = torch.empty(0, 64, device=DEV)
    d = dev.dispatch_fp4(e, torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV), 4, 4)
    assert d["bound"] == 0 and (d["counts"] == 0).all() and int(d["total"]) == 0


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

def phi(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    return v.clamp_min(0) if name == "relu" else v


def segments(counts, align, gap=0):
    starts, ends, at = [], [], 0
    for c in counts:
        starts.append(at)
        ends.append(at + c)
        at += -(-c // align) * align + gap
    return starts, ends, max(at, 1)


def weights(dev, seed, L, Nw, K, fmt):
    w = rand(seed, L, Nw, K, gain=K ** -0.5)
    ts = (w.abs().amax((1, 2)) / 2688).contiguous() if fmt == "nv" else None
    o = dev.quant_fp4(w.view(L * Nw, K), fmt=fmt, tensor_scale=ts)
    val = quantise(w.view(L * Nw, K), fmt, None if ts is None else ts.repeat_interleave(Nw))[2]
    return o["xq"].view(L, Nw, K // 2), o["scales"], ts, val.view(L, Nw, K)


def check(out, xv, wv, bias, res, seg, N, act, gated, tiny=TINY):
    """Every real row within the bound; every other row as it was (9)."""
    hs, K = torch.finfo(out.dtype).eps / 2, xv.shape[1]
    real = torch.zeros(out.shape[0], dtype=torch.bool, device=DEV)
    for e, (lo, hi) in enumerate(seg):
        if hi <= lo:
            continue
        real[lo:hi] = True
        P = xv[lo:hi] @ wv[e].t()
        err = (K + 4) * V * (xv[lo:hi].abs() @ wv[e].abs().t())
        if bias is not None:
            P = P + bias[e].double()
            err = err + V * P.abs()
        a = phi(act, P[:, :N])
        ea = 1.13 * err[:, :N] + ACT_ERR * (a.abs() + err[:, :N]) * (act != "none")
        if gated:
            u, eu = P[:, N:], err[:, N:]
            want, bound = a * u, ea * u.abs() + a.abs() * eu + ea * eu + V * (a * u).abs()
        else:
            want, bound = a, ea
        if res is not None:
            want = want + res[lo:hi].double()
            bound = bound + V * want.abs()
        assert ((out[lo:hi].double() - want).abs() <= hs * want.abs() + bound * (1 + hs) + tiny).all()
    assert (out[~real] == 9).all()


SHAPES = [  # counts per expert, align, K, N
    ([1], 1, 64, 64), ([1], 1, 128, 8), ([5], 1, 192, 136), ([16, 1], 16, 256, 128), ([0, 3, 0, 17], 8, 320, 264), ([208, 207, 209], 1, 576, 128),
    ([0, 0, 0], 8, 64, 64), ([700], 128, 2048, 1408), ([31, 600, 0, 129, 64], 16, 512, 384), ([40] * 33, 8, 1088, 72), ([130, 7], 128, 4160, 256),
]
EPI = [  # act, gated, bias, residual
    ("none", False, False, False), ("relu", False, True, True), ("silu", True, True, False), ("gelu", True, False, True), ("silu", False, False, True),
]


@pytest.mark.parametrize("fmt", ["nv", "e8m0", "mx"])
@pytest.mark.parametrize("epi", range(len(EPI)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_product(dev, shape, epi, fmt):
    counts, align, K, N = SHAPES[shape]
    act, gated, has_b, has_r = EPI[epi]
    N = max(16, N // 16 * 16) if gated else N
    starts, ends, R = segments(counts, align, gap=shape % 3)
    L, Nw = len(counts), 2 * N if gated else N
    seg = list(zip(starts, ends))
    real = torch.zeros(R, dtype=torch.bool, device=DEV)
    for lo, hi in seg:
        real[lo:hi] = True
    x = rand(1, R, K)
    x[~real] = math.nan  # rows of no expert hold anything: scales and codes of NaN here
    xts = torch.full((1,), 0.01, device=DEV) if fmt == "nv" else None
    q = dev.quant_fp4(x, fmt=fmt, tensor_scale=xts)
    xv = quantise(x, fmt, xts)[2]
    w, wsc, wts, wv = weights(dev, 2, L, Nw, K, fmt)
    bias = rand(3, L, Nw) if has_b else None
    dtype = torch.float16 if epi % 2 else torch.bfloat16
    res = rand(4, R, N + 3, dtype=dtype)[:, :N] if has_r else None
    st = i32([0])
    call = lambda: dev.expert_matmul_fp4(q["xq"], w, q["scales"], wsc, fmt=fmt, starts=i32(starts), psum=i32(ends), x_tscale=xts, w_tscale=wts,
                                         bias=bias, act=act, gated=gated, residual=res, out=torch.full((R, N), 9.0, device=DEV, dtype=dtype), status=st)
    out = call()
    assert dev.moe_status_sync(st) == dev.MOE_OK
    check(out, xv, wv, bias, res, seg, N, act, gated)
    assert torch.equal(out, call())


@pytest.mark.parametrize("fmt", ["nv", "e8m0"])
@pytest.mark.parametrize("R", [1, 2, 15, 16, 17, 100, 128, 129, 208, 209, 300, 1000])
@pytest.mark.parametrize("K,N", [(64, 8), (2048, 264), (7168, 1024), (4672, 128)])
def test_product_dense(dev, R, K, N, fmt):
    """One matrix: few rows take the reduction in runs; any row stride."""
    x = rand(R, R, K)
    q = dev.quant_fp4(x, fmt=fmt)
    wide = torch.zeros(R, K // 2 + 48, dtype=torch.uint8, device=DEV)
    wide[:, :K // 2] = q["xq"]
    w, wsc, wts, wv = weights(dev, 2, 1, N, K, fmt)
    bias, res = rand(3, N), rand(4, R, N, dtype=torch.bfloat16)
    out = dev.expert_matmul_fp4(wide[:, :K // 2], w[0], q["scales"], wsc, fmt=fmt, w_tscale=wts, bias=bias, residual=res)
    check(out, quantise(x, fmt)[2], wv, bias[None], res, [(0, R)], N, "none", False)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("gated,act,dtype", [(True, "silu", torch.bfloat16), (True, "gelu", torch.float16), (False, "relu", torch.float16)])
@pytest.mark.parametrize("R,K,N", [(1, 64, 16), (2, 1024, 48), (3, 1088, 112), (4, 2048, 7168), (4, 7168, 32), (4, 14336, 16), (5, 2048, 64),
                                   (1, 40960, 16), (2, 4096, 256), (2, 65536, 16)])
def test_product_of_few_rows(dev, R, K, N, gated, act, dtype, fmt):
    """One or two rows of one matrix, with every part of the epilogue; just more rows, and rows too long for it."""
    Nw = 2 * N if gated else N
    x = rand(R, R, K)
    xts = torch.full((1,), 0.02, device=DEV) if fmt == "nv" else None
    q = dev.quant_fp4(x, fmt=fmt, tensor_scale=xts)
    w, wsc, wts, wv = weights(dev, 2, 1, Nw, K, fmt)
    bias, res = rand(3, 1, Nw), rand(4, R, N + 5, dtype=dtype)[:, 3:N + 3]
    call = lambda: dev.expert_matmul_fp4(q["xq"], w, q["scales"], wsc, fmt=fmt, x_tscale=xts, w_tscale=wts, bias=bias, act=act, gated=gated,
                                         residual=res, out_dtype=dtype)
    out = call()
    check(out, quantise(x, fmt, xts)[2], wv, bias, res, [(0, R)], N, act, gated)
    assert torch.equal(out, call())


def test_few_rows_not_a_number(dev):
    R, K, N = 2, 512, 72
    x = rand(1, R, K)
    x[1, 100] = math.nan
    w = rand(2, N, K, gain=K ** -0.5)
    w[5, 7] = math.inf
    q, wq = dev.quant_fp4(x), dev.quant_fp4(w)
    out = dev.expert_matmul_fp4(q["xq"], wq["xq"], q["scales"], wq["scales"])
    bad = torch.zeros(R, N, dtype=torch.bool, device=DEV)
    bad[1], bad[:, 5] = True, True
    assert torch.equal(torch.isnan(out), bad) and torch.isfinite(out[~bad]).all()


def test_product_of_slabs(dev):
    L, cap, K, N = 5, 48, 576, 96
    m = i32([0, 48, 5, 17, 1])
    x = rand(1, L, cap, K)
    q = dev.quant_fp4(x, masked_m=m)
    w, wsc, wts, wv = weights(dev, 2, L, 2 * N, K, "nv")
    st = i32([0])
    out = dev.expert_matmul_fp4(q["xq"], w, q["scales"], wsc, masked_m=m, w_tscale=wts, act="silu", gated=True,
                                out=torch.full((L, cap, N), 9.0, device=DEV, dtype=torch.bfloat16), status=st)
    assert dev.moe_status_sync(st) == dev.MOE_OK
    check(out.view(L * cap, N), quantise(x.view(L * cap, K), "nv")[2], wv, None, None, [(e * cap, e * cap + int(c)) for e, c in enumerate(m.tolist())],
          N, "silu", True)


def test_exact_products(dev):
    """Small whole numbers: every sum is exact, so every element and scale is where it belongs."""
    for fmt, K in (("nv", 1024), ("e8m0", 1024), ("nv", 64), ("mx", 320)):
        R, N, g = 150, 136, group(fmt)
        gen = torch.Generator(DEV).manual_seed(K)
        ri = lambda n, *s: torch.randint(0, n, s, device=DEV, generator=gen)
        def make(rows):
            code = ri(16, rows, K)
            byte = ri(4, rows, K // g) * 8 + 0x28 if fmt == "nv" else ri(4, rows, K // g) + 126    # 2^-2 .. 2, 2^-1 .. 4
            sc = torch.zeros(rows, pieces(K, fmt) * 16, dtype=torch.uint8, device=DEV)
            sc[:, :K // g] = byte.to(torch.uint8)
            d = torch.exp2((byte >> 3).double() - 7) if fmt == "nv" else torch.exp2(byte.double() - 127)
            v = torch.tensor(CODES + [-c for c in CODES], dtype=torch.float64, device=DEV)[code].view(rows, K // g, g) * d.round(decimals=6)[:, :, None]
            c8 = code.to(torch.uint8).view(rows, K // 2, 2)
            return (c8[:, :, 0] | (c8[:, :, 1] << 4)).contiguous(), sc.view(rows, -1, 16).transpose(0, 1).contiguous(), v.view(rows, K)
        xq, xs, xv = make(R)
        wq, ws, wv = make(N)
        # sums are multiples of 2^-6 below 2^18 (K * 36 * 16 / 4): 24 bits hold them, and adding them one
        # matrix of single rows at a time keeps the 16-bit output exact too
        P = xv @ wv.t()
        assert P.abs().max() < 2.0 ** 18
        out = dev.expert_matmul_fp4(xq, wq, xs, ws, fmt=fmt, bias=None, out_dtype=torch.bfloat16)
        assert torch.equal(out, P.float().to(torch.bfloat16))


def test_not_a_number_stays_in_its_row(dev):
    R, K, N = 40, 512, 72
    x = rand(1, R, K)
    x[7, 100] = math.nan
    q = dev.quant_fp4(x)
    w, wsc, wts, wv = weights(dev, 2, 1, N, K, "nv")
    out = dev.expert_matmul_fp4(q["xq"], w, q["scales"], wsc, w_tscale=wts)
    assert torch.isnan(out[7]).all() and torch.isfinite(out[:7]).all() and torch.isfinite(out[8:]).all()


@pytest.mark.parametrize("bad", [([0, 10], [20, 30]), ([0, 20], [20, 41]), ([-1, 20], [10, 30]), ([0, 20], [10, 15])])
def test_bad_segments(dev, bad):
    """Segments that share rows, leave the rows or go backwards are flagged and count as empty."""
    L, R, K, N = 2, 40, 256, 64
    q = dev.quant_fp4(rand(1, R, K))
    w, wsc, wts, wv = weights(dev, 2, L, N, K, "nv")
    st = i32([0])
    out = dev.expert_matmul_fp4(q["xq"], w, q["scales"], wsc, starts=i32(bad[0]), psum=i32(bad[1]), w_tscale=wts,
                                out=torch.full((R, N), 9.0, device=DEV, dtype=torch.bfloat16), status=st)
    assert dev.moe_status_sync(st) == dev.MOE_ERR_BAD_LAYOUT
    good = [(a, b) if 0 <= a <= b <= R and not (i == 1 and bad[0][1] < bad[1][0]) else (0, 0) for i, (a, b) in enumerate(zip(*bad))]
    check(out, quantise(rand(1, R, K), "nv")[2], wv, None, None, good, N, "none", False)


def test_captured_chain(dev):
    """Dispatch, both products and the combine in one graph, replayed with other tokens and routing."""
    T, H, F, E, k = 300, 512, 256, 8, 3
    x, ids, tw = rand(1, T, H, dtype=torch.bfloat16), torch.zeros(T, k, dtype=torch.int32, device=DEV), rand(2, T, k)
    up, ups, upt, _ = weights(dev, 3, E, 2 * F, H, "nv")
    dn, dns, dnt, _ = weights(dev, 4, E, H, F, "nv")
    ws = dev.Workspace(T, k, E, DEV)

    def step():
        d = dev.dispatch_fp4(x, ids, tw, E, E, block_e=16, workspace=ws)
        seg = dict(starts=d["starts"], psum=d["psum"], status=d["status"])
        a = dev.expert_matmul_fp4(d["xq"], up, d["scales"], ups, w_tscale=upt, act="silu", gated=True, **seg)
        q = dev.quant_fp4(a, m_indices=d["m_indices"])
        y = dev.expert_matmul_fp4(q["xq"], dn, q["scales"], dns, w_tscale=dnt, **seg)
        return dev.combine(y, d["src2dst"], tw, status=d["status"]), d["status"]

    def fill(seed):
        x.copy_(rand(seed, T, H, dtype=torch.bfloat16))
        ids.copy_(torch.randint(0, E, (T, k), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(seed)))

    fill(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, st = step()
    for seed in (5, 6):
        fill(seed)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, step()[0]) and dev.moe_status_sync(st) == dev.MOE_OK and torch.isfinite(got).all()


def far_rows(R, W, dtype):
    """Zeros of R rows of W elements whose starts are more than 2^31 elements apart (memory of them is needed all the same)."""
    ld = 2 ** 31 + 64
    return torch.zeros((R - 1) * ld + W, dtype=dtype, device=DEV).as_strided((R, W), (ld, 1))


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_far_apart(dev, fmt):
    """Offsets that 32 bits do not hold: of rows, of outputs and of residual rows, and of pieces of scales."""
    R, K, N = 3, 1024, 48
    near = rand(1, R, K, dtype=torch.bfloat16)
    x = far_rows(R, K, torch.bfloat16)
    x.copy_(near)
    q, sc, val = quantise(near, fmt)
    o = dev.quant_fp4(x, fmt=fmt)
    assert torch.equal(o["scales"], sc) and same_codes(o["xq"], q)
    ids = i32([[0, 1], [1, 0], [1, 1]])
    d = dev.dispatch_fp4(x, ids, torch.ones(R, 2, device=DEV), 2, 2, block_e=1, fmt=fmt)
    rows = d["src2dst"].long()
    assert all(same_codes(d["xq"][rows[:, k]], o["xq"]) for k in range(2))
    x.zero_()
    assert dev.dequant_fp4(o["xq"], o["scales"], fmt=fmt, out=x) is x
    assert torch.equal(x, val.float().to(torch.bfloat16))
    w, wsc, wts, wv = weights(dev, 2, 1, N, K, fmt)
    del x
    ld = 2 ** 27 + 8  # of scales: with two pieces or more, the second is 2^31 bytes on
    far = torch.zeros(pieces(K, fmt), ld, 16, dtype=torch.uint8, device=DEV)
    far[:, :R] = sc
    res, out = far_rows(R, N, torch.bfloat16), far_rows(R, N, torch.bfloat16)
    res.copy_(rand(4, R, N, dtype=torch.bfloat16))
    wide = far_rows(R, K // 2, torch.uint8)
    wide.copy_(o["xq"])
    for n in (R, 2):  # (two rows take no tensor cores)
        out.fill_(9)
        dev.expert_matmul_fp4(wide[:n], w, far, wsc, fmt=fmt, w_tscale=wts, residual=res[:n], out=out[:n])
        check(out, val, wv, None, res, [(0, n)], N, "none", False)


# ---------------------------------------------------------------------------
# Signs of zeros, and tensors of zeros
# ---------------------------------------------------------------------------

def codes_by_search(x, fmt, ts):
    """The four-bit elements (sign and magnitude, one a byte) and the scale bytes of float32 rows, by the
    definition: the nearest of all values, the even code among two as near, on the host. ts [R]."""
    values = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])

    def nearest_of(v, table):
        off = np.abs(table - np.minimum(v, table[-1])[..., None].astype(np.float64))
        best = off == off.min(-1, keepdims=True)
        even = best & (np.arange(len(table)) % 2 == 0)
        return np.where(even.any(-1), even.argmax(-1), best.argmax(-1))

    R, H = x.shape
    g = group(fmt)
    v = x.reshape(R, H // g, g)
    bad = ~np.isfinite(v).all(2)
    amax = np.abs(np.where(bad[:, :, None], np.float32(0), v)).max(2)
    with np.errstate(all="ignore"):
        if fmt == "nv":
            t = np.float32(ts)[:, None]
            byte = nearest_of(np.where(amax > 0, amax / (np.float32(6) * t), np.float32(0)), values)
            d = np.float32(values[byte]) * t
            q = np.where(d[:, :, None] > 0, v / d[:, :, None], np.float32(0))
        else:
            e = np.frexp(np.float64(amax))[1] - 3
            if fmt == "e8m0":
                e = e + (6 * np.ldexp(1.0, e) < amax)
            e = np.clip(np.where(amax > 0, e, -127), -127, 127)
            byte, d = e + 127, np.ldexp(1.0, e)
            q = np.float64(v) / d[:, :, None]
        code = nearest_of(np.where(bad[:, :, None], 0, np.abs(q)), np.array(CODES))
    code = code | np.where((d[:, :, None] > 0) & np.signbit(v), 8, 0)
    code = np.where(bad[:, :, None], 0, code)
    return code.reshape(R, H).astype(np.uint8), np.where(bad, 0x7F if fmt == "nv" else 0xFF, byte).astype(np.uint8)


def elements(xq):
    """Packed pairs, one element a byte."""
    return torch.stack([xq & 15, xq >> 4], -1).flatten(-2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DT.values()), ids=list(DT))
def test_codes_to_the_sign_of_zeros(dev, dtype, fmt):
    """Every bit of every element and scale, zeros of both signs and values that round to them included,
    alone and dispatched."""
    R, H = 48, 192
    x = rand(7, R, H)
    x[:, 3::7], x[:, 5::11] = -0.0, 0.0
    x[4:8] = -x[4:8].abs() * 10.0 ** -torch.arange(H, device=DEV).remainder(9).float()   # down to where a group's scale makes them zeros
    x[8, :64], x[9] = -0.0, -0.0
    x[10] = torch.where(rand(8, H) < 0, -6.0, 0.25)                    # ties between zero and the first code
    x[11, 40], x[12, 70], x[13] = math.nan, -math.inf, x[13] * 1e-38   # (subnormal numbers in float32)
    x[14, ::16], x[14, 1::16] = 3.0, -1e-30
    x = x.to(dtype)
    for ts in ([None] if fmt != "nv" else [None, 0.0137, 2.0 ** -100, 2.0 ** -130, 1.1e30, 2.0 ** 110]):
        t = None if ts is None else torch.full((1,), ts, device=DEV)
        code, byte = codes_by_search(x.float().cpu().numpy(), fmt, np.full(R, 1.0 if ts is None else ts, np.float32))
        o = dev.quant_fp4(x, fmt=fmt, tensor_scale=t)
        assert np.array_equal(o["scales"].transpose(0, 1).reshape(R, -1)[:, :H // group(fmt)].cpu().numpy(), byte)
        assert np.array_equal(elements(o["xq"]).cpu().numpy(), code)
        for n in (R, 700):  # both forms of the dispatch
            y = x.repeat(-(-n // R), 1)[:n].contiguous()
            ids = torch.arange(n * 4, device=DEV, dtype=torch.int32).view(n, 4) % 5
            d = dev.dispatch_fp4(y, ids, torch.ones(n, 4, device=DEV), 5, 5, block_e=1, fmt=fmt, tensor_scale=t)
            rows = d["src2dst"].long()
            for k in (0, 3):
                assert np.array_equal(elements(d["xq"][rows[:, k]]).cpu().numpy(), code[np.arange(n) % R])


@pytest.mark.parametrize("dtype", list(DT.values()), ids=list(DT))
def test_tensor_of_zeros(dev, dtype):
    """amax / 2688 of a tensor of zeros is 0: scales, elements and values are zeros, and so are products."""
    L, N, K, R = 3, 16, 192, 5
    w = rand(1, L, N, K)
    w[1] = 0.0
    w[1, :, ::3] = -0.0
    w = w.to(dtype)
    ts = (w.abs().amax((1, 2)).float() / 2688).contiguous()
    assert ts[1] == 0
    o = dev.quant_fp4(w.view(L * N, K), tensor_scale=ts)
    q, sc, val = quantise(w.view(L * N, K), "nv", torch.where(ts > 0, ts, 1.0).repeat_interleave(N))
    assert torch.equal(o["scales"], sc) and same_codes(o["xq"], q) and (o["scales"][:, N:2 * N] == 0).all()
    assert torch.equal(dev.dequant_fp4(o["xq"], o["scales"], tensor_scale=ts, dtype=torch.float32), val.float())
    bias = rand(2, L, N)
    xr = rand(3, L * R, K)
    x = dev.quant_fp4(xr)
    seg = [(e * R, e * R + R) for e in range(L)]
    out = dev.expert_matmul_fp4(x["xq"], o["xq"].view(L, N, K // 2), x["scales"], o["scales"], starts=i32([a for a, _ in seg]), w_tscale=ts,
                                psum=i32([b for _, b in seg]), bias=bias)
    check(out, quantise(xr, "nv")[2], val.view(L, N, K), bias, None, seg, N, "none", False)
    assert torch.equal(out[R:2 * R], bias[1].bfloat16().expand(R, N))
    one = dev.expert_matmul_fp4(x["xq"][:2], o["xq"].view(L, N, K // 2)[1], x["scales"], o["scales"][:, N:2 * N].contiguous(),
                                w_tscale=ts[1:2], bias=bias[1])
    assert torch.equal(one, bias[1].bfloat16().expand(2, N))
    zero = torch.zeros(1, device=DEV)  # the rows too, alone and dispatched
    rows = torch.zeros(700, K, dtype=dtype, device=DEV)
    rows[:, ::2] = -0.0
    z = dev.quant_fp4(rows, tensor_scale=zero)
    assert (z["scales"] == 0).all() and (z["xq"] == 0).all()
    for n in (40, 700):
        d = dev.dispatch_fp4(rows[:n], i32([[0, 1, 2, 3]]).repeat(n, 1), torch.ones(n, 4, device=DEV), 4, 4, block_e=1, tensor_scale=zero)
        assert (d["scales"] == 0).all() and (d["xq"] == 0).all()


def test_status_of_the_values_of_rows(dev):
    """A live count that is too large is flagged in the caller's status word; where there is none the call makes none."""
    R, H = 20, 128
    o = dev.quant_fp4(rand(1, R, H))
    st, n, out = i32([0]), i32([R + 1]), torch.empty(R, H, dtype=torch.bfloat16, device=DEV)
    dev.dequant_fp4(o["xq"], o["scales"], num_live=n, status=st, out=out)
    assert dev.moe_status_sync(st) == dev.MOE_ERR_LIVE_OVERFLOW
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    assert dev.dequant_fp4(o["xq"], o["scales"], num_live=n, out=out) is out
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("R,K,N,gated", [(1, 4096, 10240, False), (1, 10240, 2048, False), (2, 2048, 14336, False), (2, 7168, 2048, True),
                                         (1, 64, 40000, False), (2, 512, 32768, False), (1, 24576, 64, False)])
def test_few_rows_of_large_matrices(dev, R, K, N, gated, fmt):
    """Where the tensor cores are faster one or two rows take them too: the same sums, to the last bits that
    a residual of the rounded output leaves, as of the same rows given as a segment."""
    Nw = 2 * N if gated else N
    # (magnitudes from group to group so far apart that sums in 24 bits depend on their order)
    far = lambda seed, n: rand(seed, n, K) * torch.exp2(rand(seed + 9, n, K // 32, gain=3.0)).repeat_interleave(32, 1)
    q, w = dev.quant_fp4(far(R, R), fmt=fmt), dev.quant_fp4(far(2, Nw) * K ** -0.5, fmt=fmt)
    call = lambda **o: dev.expert_matmul_fp4(q["xq"], w["xq"], q["scales"], w["scales"], fmt=fmt, gated=gated, act="silu" if gated else "none",
                                             out_dtype=torch.float16, **o)
    less = -call()
    assert torch.equal(call(residual=less), call(residual=less, starts=i32([0]), psum=i32([R])))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_product_of_the_most_experts(dev, fmt):
    """1024 experts, whose lists leave the least room for stages, and tiles of the most rows."""
    L, K, N = 1024, 1088, 16
    counts = [e % 3 for e in range(L)]
    counts[5], counts[700], counts[1023] = 208, 417, 208
    starts, ends, R = segments(counts, 1)
    x = rand(1, R, K)
    q = dev.quant_fp4(x, fmt=fmt)
    w, wsc, wts, wv = weights(dev, 2, L, 2 * N, K, fmt)
    st = i32([0])
    out = dev.expert_matmul_fp4(q["xq"], w, q["scales"], wsc, fmt=fmt, starts=i32(starts), psum=i32(ends), w_tscale=wts, act="silu", gated=True, status=st)
    assert dev.moe_status_sync(st) == dev.MOE_OK
    check(out, quantise(x, fmt)[2], wv, None, None, list(zip(starts, ends)), N, "silu", True)
