"""The experts' products with bias, activation, gate and residual, and their
gradients, against the formulas in 64 bits.

Bounds, with v = 2^-23 (one step of a 32-bit accumulation, twice the half step,
as tensor cores may truncate): a sum of K products is off by (K + 2) v times the
sum of magnitudes; the activations' slopes are below 1.13 and their own error
(__expf to about 2 + 1.2 |x| ulp, normcdff 5 ulp) below 2^-17 relative to the
magnitudes that enter; the rounding to 16 bits adds half a step, and 2^-25 covers
fp16's smallest numbers. Gradients carry one more half step for the rounding of
the pre-activations' gradient."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, TINY, ACT_ERR = 2.0 ** -23, 2.0 ** -25, 2.0 ** -17


def rand(seed, *shape, dtype=torch.float32, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * gain).to(dtype)


def phi(name, v):
    """(activation, slope) in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if name == "gelu":
        c = 0.5 * torch.erfc(-v / math.sqrt(2.0))
        return v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return v.clamp_min(0), (v > 0).double()
    return v, torch.ones_like(v)


def segments(counts, align, gap=0):
    """Segment starts and ends of rows padded to `align` (and `gap` rows between), and R."""
    starts, ends, at = [], [], 0
    for c in counts:
        starts.append(at)
        ends.append(at + c)
        at += -(-c // align) * align + gap
    return starts, ends, max(at, 1)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def quant(x):
    """e4m3 codes, packed scale words, leading dimension and the values they stand for."""
    R, K = x.shape
    v = x.reshape(R, K // 128, 128)
    m, e = torch.frexp(v.abs().amax(2).clamp_min(1e-10))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    q = (v * torch.exp2(-e.float())[:, :, None]).to(torch.float8_e4m3fn)
    val = (q.double() * torch.exp2(e.double())[:, :, None]).reshape(R, K)
    G = K // 128
    G4, ld = (G + 3) // 4, (R + 3) // 4 * 4
    b = torch.full((ld, G4 * 4), 0xFF, dtype=torch.uint8, device=DEV)   # bytes past the last group are never used
    b[:R, :G] = (e + 127).to(torch.uint8)
    return q.reshape(R, K), b.view(torch.int32).t().contiguous(), ld, val


SHAPES = [  # counts per expert, align, K, N
    ([1], 1, 64, 64), ([1], 1, 8, 8), ([5], 1, 72, 136), ([16, 1], 16, 128, 128), ([0, 3, 0, 17], 8, 200, 264),
    ([256, 255, 257], 1, 136, 128), ([0, 0, 0], 8, 64, 64), ([700], 128, 2048, 1408), ([31, 600, 0, 129, 64], 16, 512, 384),
    ([40] * 33, 8, 256, 72),
]
EPI = [  # act, gated, bias, residual, pre
    ("none", False, False, False, False), ("relu", False, True, True, True), ("silu", True, True, False, True),
    ("gelu", False, True, False, False), ("gelu", True, False, True, False), ("silu", False, False, False, True),
    ("relu", True, True, True, True),
]


def check_forward(out, pre, xv, wv, bias, res, seg, N, act, gated, dtype):
    """Every real row within the bound; every other row as it was (9)."""
    hs = torch.finfo(dtype).eps / 2
    K = xv.shape[1]
    real = torch.zeros(out.shape[0], dtype=torch.bool, device=DEV)
    for e, (lo, hi) in enumerate(seg):
        if hi <= lo:
            continue
        real[lo:hi] = True
        P = xv[lo:hi] @ wv[e].t()
        err = (K + 2) * V * (xv[lo:hi].abs() @ wv[e].abs().t())
        if bias is not None:
            P = P + bias[e].double()
            err = err + V * P.abs()
        if pre is not None:
            assert ((pre[lo:hi].double() - P).abs() <= hs * P.abs() + err * (1 + hs) + TINY).all()
        a, _ = phi(act, P[:, :N])
        ea = 1.13 * err[:, :N] + ACT_ERR * (a.abs() + err[:, :N]) * (act != "none")
        if gated:
            u, eu = P[:, N:], err[:, N:]
            want, bound = a * u, ea * u.abs() + a.abs() * eu + ea * eu + V * (a * u).abs()
        else:
            want, bound = a, ea
        if res is not None:
            want = want + res[lo:hi].double()
            bound = bound + V * want.abs()
        assert ((out[lo:hi].double() - want).abs() <= hs * want.abs() + bound * (1 + hs) + TINY).all()
    assert (out[~real] == 9).all() and (pre is None or (pre[~real] == 9).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("epi", range(len(EPI)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_forward(dev, shape, epi, dtype):
    counts, align, K, N = SHAPES[shape]
    act, gated, has_b, has_r, has_p = EPI[epi]
    if gated:
        N = max(16, N // 16 * 16)
    starts, ends, R = segments(counts, align, gap=shape % 3)
    L, Nw = len(counts), 2 * N if gated else N
    x = rand(1, R, K + 8, dtype=dtype)[:, :K]
    w = rand(2, L, Nw, K, dtype=dtype, gain=K ** -0.5)
    bias = rand(3, L, Nw) if has_b else None
    res = rand(4, R, N + 3, dtype=dtype)[:, :N] if has_r else None
    seg = list(zip(starts, ends))
    for lo in range(R):  # rows of no expert hold NaN
        if not any(a <= lo < b for a, b in seg):
            x[lo] = float("nan")
    out = torch.full((R, N), 9.0, device=DEV, dtype=dtype)
    pre = torch.full((R, Nw), 9.0, device=DEV, dtype=dtype) if has_p else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda o: dev.expert_matmul(x, w, i32(starts), i32(ends), bias=bias, act=act, gated=gated, residual=res,
                                       out=o, pre=pre, status=st)
    call(out)
    assert dev.moe_status_sync(st) == dev.MOE_OK
    check_forward(out, pre, x.double(), w.double(), bias, res, seg, N, act, gated, dtype)
    again = call(torch.full_like(out, 9.0))
    assert torch.equal(out, again)


@pytest.mark.parametrize("R", [1, 2, 15, 16, 17, 100, 300, 1000])
@pytest.mark.parametrize("K,N", [(64, 8), (2048, 264), (136, 1024)])
def test_forward_dense(dev, R, K, N):
    x, w = rand(1, R, K, dtype=torch.bfloat16), rand(2, N, K, dtype=torch.bfloat16, gain=K ** -0.5)
    b, res = rand(3, N), rand(4, R, N, dtype=torch.bfloat16)
    out = dev.expert_matmul(x, w, bias=b, residual=res)
    check_forward(out, None, x.double(), w[None].double(), b[None], res, [(0, R)], N, "none", False, torch.bfloat16)


@pytest.mark.parametrize("R", [1, 9, 33, 64, 130, 256, 300])
@pytest.mark.parametrize("K,N", [(1024, 256), (7168, 1160), (2056, 64)])
def test_few_tiles_split_the_reduction(dev, R, K, N):
    """One dense matrix with few rows: runs of the reduction on several pairs, joined in a fixed order."""
    x, w = rand(1, R, K, dtype=torch.bfloat16), rand(2, N, K, dtype=torch.bfloat16, gain=K ** -0.5)
    b = rand(3, N)
    pre = torch.full((R, N), 9.0, device=DEV, dtype=torch.bfloat16)
    out = dev.expert_matmul(x, w, bias=b, act="gelu", pre=pre)
    check_forward(out, pre, x.double(), w[None].double(), b[None], None, [(0, R)], N, "gelu", False, torch.bfloat16)
    assert torch.equal(out, dev.expert_matmul(x, w, bias=b, act="gelu", pre=pre))
    dout = rand(4, R, N, dtype=torch.bfloat16)
    dx = dev.expert_matmul_grad(dout, x, w, need=("dx",))["dx"].double()
    want = dout.double() @ w.double()
    mag = dout.double().abs() @ w.double().abs()
    assert ((dx - want).abs() <= 2.0 ** -8 * want.abs() + (N + 4) * V * mag).all()


@pytest.mark.parametrize("R", [1, 40, 200])
@pytest.mark.parametrize("K,N,gated", [(2048, 512, False), (7168, 128, True), (2176, 64, False)])
def test_few_tiles_split_the_reduction_e4m3(dev, R, K, N, gated):
    Nw = 2 * N if gated else N
    q, sc, ld, xv = quant(rand(1, R, K))
    wq, wsc, ldw, wv = quant(rand(2, Nw, K, gain=K ** -0.5))
    out = dev.expert_matmul(q, wq, act="silu", gated=gated, x_scales=sc, ld_xs=ld, w_scales=wsc, ld_ws=ldw)
    check_forward(out, None, xv, wv[None], None, None, [(0, R)], N, "silu", gated, torch.bfloat16)


FP8 = [  # counts, align, K, N, gated
    ([1], 1, 128, 64, False), ([3, 0, 30], 4, 512, 128, True), ([225, 224], 1, 640, 136, False), ([449], 1, 1152, 64, True),
    ([4] * 32, 128, 7168, 256, True), ([100, 0, 300], 128, 2048, 384, True),
]


@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts,align,K,N,gated", FP8)
def test_forward_e4m3(dev, counts, align, K, N, gated, odt):
    starts, ends, R = segments(counts, align)
    L, Nw = len(counts), 2 * N if gated else N
    q, sc, ld, xv = quant(rand(1, R, K) * torch.exp2(torch.randint(-6, 7, (R, 1), device=DEV).float()))
    wq, wsc, ldw, wv = quant(rand(2, L * Nw, K, gain=K ** -0.5))
    bias = rand(3, L, Nw)
    seg = list(zip(starts, ends))
    for lo in range(R):
        if not any(a <= lo < b for a, b in seg):
            q.view(torch.uint8)[lo] = 0x7F
            sc[:, lo] = -1
    out = torch.full((R, N), 9.0, device=DEV, dtype=odt)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev.expert_matmul(q, wq.view(L, Nw, K), i32(starts), i32(ends), bias=bias, act="silu" if gated else "none", gated=gated,
                      x_scales=sc, ld_xs=ld, w_scales=wsc, ld_ws=ldw, out=out, out_dtype=odt, status=st)
    assert dev.moe_status_sync(st) == dev.MOE_OK
    check_forward(out, None, xv, wv.view(L, Nw, K), bias, None, seg, N, "silu" if gated else "none", gated, odt)


def test_forward_on_a_dispatch(dev):
    """e4m3 rows of both dispatch layouts through the same product: equal rows, equal results."""
    T, H, E, L, K, N = 64, 512, 16, 8, 4, 128
    x = rand(1, T, H, dtype=torch.bfloat16)
    rng = np.random.default_rng(0)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)).to(DEV)
    tw = torch.softmax(rand(2, T, K), 1)
    w = rand(3, L * 2 * N, H, dtype=torch.bfloat16, gain=H ** -0.5)
    wq = dev.quant_group(w)
    kw = dict(act="silu", gated=True, w_scales=wq["scales"], ld_ws=wq["ld_s"])
    c = dev.dispatch_compact(x, ids, tw, E, L, block_e=128)
    m = dev.dispatch_masked(x, ids, tw, E, L, T)
    w3 = wq["xq"].view(L, 2 * N, H)
    yc = dev.expert_matmul(c["xq"], w3, c["starts"], c["psum"], x_scales=c["scales"], ld_xs=c["ld_s"], **kw)
    ym = dev.expert_matmul(m["xq"], w3, masked_m=m["masked_m"], x_scales=m["scales"], ld_xs=m["ld_s"], **kw)
    a = dev.combine(yc, c["src2dst"], tw)
    b = dev.combine(ym.view(-1, N), m["src2dst"], tw)
    assert torch.equal(a, b) and torch.isfinite(a.float()).all() and (a != 0).any()


def test_offsets_past_32_bits(dev):
    """Rows whose element offsets pass 2^31 (2.6e9 elements of output, of the gradient and of sorted rows)."""
    R, K, N = 640_000, 64, 4096
    x, w = rand(1, R, K, dtype=torch.bfloat16), rand(2, N, K, dtype=torch.bfloat16, gain=0.125)
    out = dev.expert_matmul(x, w)
    dx = dev.expert_matmul_grad(out, x, w, need=("dx",))["dx"]
    for lo in (0, 524_288 - 8, R - 16):       # the first rows, around element 2^31, the last rows
        sl = slice(lo, lo + 16)
        want = x[sl].double() @ w.double().t()
        err = (K + 2) * V * (x[sl].double().abs() @ w.double().abs().t())
        assert ((out[sl].double() - want).abs() <= 2.0 ** -8 * want.abs() + err * 1.01).all()
        want, mag = out[sl].double() @ w.double(), out[sl].double().abs() @ w.double().abs()
        assert ((dx[sl].double() - want).abs() <= 2.0 ** -8 * want.abs() + (N + 2) * V * mag).all()
    del out, dx
    T, H, k = 40_000, 8192, 8
    x = rand(3, T, H, dtype=torch.bfloat16)
    ids = torch.arange(T * k, device=DEV, dtype=torch.int32).reshape(T, k) % k
    p = dev.permute(x, ids, torch.ones(T, k, device=DEV), k, k, block_e=1)
    for t in (0, 20_000, T - 1):
        assert all(torch.equal(p["xs"][r], x[t]) for r in p["src2dst"][t].tolist())
    back = dev.permute_grad(p["xs"], p["src2dst"])
    assert torch.equal(back, (x.float() * k).bfloat16())


@pytest.mark.parametrize("begin,end", [([0, 10], [4, 21]), ([-1, 4], [3, 8]), ([0, 6], [4, 5])])
def test_bad_segments_are_flagged(dev, begin, end):
    """A segment outside the rows counts as empty and is flagged; the others are computed."""
    x, w = rand(1, 20, 64, dtype=torch.bfloat16), rand(2, 2, 64, 64, dtype=torch.bfloat16)
    out = torch.full((20, 64), 9.0, device=DEV, dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev.expert_matmul(x, w, i32(begin), i32(end), out=out, status=st)
    assert dev.moe_status_sync(st) == dev.MOE_ERR_BAD_LAYOUT
    for e, (lo, hi) in enumerate(zip(begin, end)):
        if 0 <= lo <= hi <= 20:
            want = (x[lo:hi].double() @ w[e].double().t()).bfloat16()
            assert (out[lo:hi].double() - want.double()).abs().max() <= 0.05 * want.double().abs().max()
    assert (out[8 if begin[0] < 0 else 4:] == 9).all() or begin[0] < 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("act,gated", [("none", False), ("silu", True), ("gelu", False), ("relu", True), ("gelu", True)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_gradients(dev, shape, act, gated, dtype):
    counts, align, K, N = SHAPES[shape]
    if gated:
        N = max(16, N // 16 * 16)
    starts, ends, R = segments(counts, align, gap=shape % 3)
    L, Nw = len(counts), 2 * N if gated else N
    seg = list(zip(starts, ends))
    x, dout = rand(1, R, K + 8, dtype=dtype)[:, :K], rand(2, R, N + 8, dtype=dtype)[:, :N]
    w = rand(3, L, Nw, K, dtype=dtype, gain=K ** -0.5)
    pre = rand(4, R, Nw, dtype=dtype)
    for r in range(R):
        if not any(a <= r < b for a, b in seg):
            x[r] = dout[r] = pre[r] = float("nan")
    dx = torch.full((R, K), 9.0, device=DEV, dtype=dtype)
    dwt = torch.float32 if shape % 2 else dtype
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda d: dev.expert_matmul_grad(dout, x, w, i32(starts), i32(ends), pre=pre, act=act, gated=gated, dx=d,
                                            need=("dx", "dw", "dbias"), dw_dtype=dwt, status=st)
    o = call(dx)
    assert dev.moe_status_sync(st) == dev.MOE_OK
    hs, hw = torch.finfo(dtype).eps / 2, torch.finfo(dwt).eps / 2
    real = torch.zeros(R, dtype=torch.bool, device=DEV)
    for e, (lo, hi) in enumerate(seg):
        if hi <= lo:
            assert (o["dw"][e] == 0).all() and (o["dbias"][e] == 0).all()
            continue
        real[lo:hi] = True
        g, p, n = dout[lo:hi].double(), pre[lo:hi].double(), hi - lo
        a, d = phi(act, p[:, :N])
        dP = torch.cat([g * d * p[:, N:], g * a], 1) if gated else g * d
        # the 32-bit gradient of P (slopes are below 1.13, relative error as above), then its rounding
        if act == "none" and not gated:
            e32, e16 = torch.zeros_like(dP), torch.zeros_like(dP)
        else:
            m = torch.cat([(g * p[:, N:]).abs() * 1.13, (g * p[:, :N]).abs()], 1) if gated else g.abs() * 1.13
            e32 = ACT_ERR * m
            e16 = e32 + hs * (dP.abs() + e32) + TINY
        for got, A, B, eA, h, steps in (
                (o["dx"][lo:hi], dP, w[e].double(), e16, hs, Nw),
                (o["dw"][e], dP.t(), x[lo:hi].double(), e16.t(), hw, n)):
            want, mag = A @ B, A.abs() @ B.abs()
            bound = eA @ B.abs() + (steps + 2) * V * (mag + eA @ B.abs())
            assert ((got.double() - want).abs() <= h * want.abs() + bound * (1 + h) + TINY).all()
        bound = e32.sum(0) + (n + 2) * V * (dP.abs() + e32).sum(0)
        assert ((o["dbias"][e].double() - dP.sum(0)).abs() <= bound).all()
    assert (dx[~real] == 9).all()
    again = call(torch.full_like(dx, 9.0))
    for k in ("dx", "dw", "dbias"):
        assert torch.equal(o[k], again[k]), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts,align,K,N", [([1], 1, 64, 64), ([3, 0, 40, 128], 8, 512, 128), ([70] * 9, 1, 136, 320)])
def test_few_rows_keep_the_gradients_rounding(dev, counts, align, K, N, dtype):
    """While R <= 128 L the rounding of the pre-activations' gradient is carried along: what is lost of it is its
    second rounding (half a step squared), so dx and dw are off by little more than their own rounding."""
    starts, ends, R = segments(counts, align)
    assert R <= 128 * len(counts)
    x, dout = rand(1, R, K, dtype=dtype), rand(2, R, N, dtype=dtype)
    w, pre = rand(3, len(counts), 2 * N, K, dtype=dtype, gain=K ** -0.5), rand(4, R, 2 * N, dtype=dtype)
    o = dev.expert_matmul_grad(dout, x, w, i32(starts), i32(ends), pre=pre, act="silu", gated=True,
                               dx=torch.zeros_like(x))
    hs = torch.finfo(dtype).eps / 2
    for e, (lo, hi) in enumerate(zip(starts, ends)):
        if hi <= lo:
            continue
        g, p = dout[lo:hi].double(), pre[lo:hi].double()
        a, d = phi("silu", p[:, :N])
        dP = torch.cat([g * d * p[:, N:], g * a], 1)
        m = torch.cat([(g * p[:, N:]).abs() * 1.13, (g * p[:, :N]).abs()], 1)
        err = ACT_ERR * m + hs * hs * dP.abs() + TINY
        for got, A, B, eA, steps in ((o["dx"][lo:hi], dP, w[e].double(), err, 4 * N),
                                     (o["dw"][e], dP.t(), x[lo:hi].double(), err.t(), 2 * (hi - lo))):
            want, mag = A @ B, A.abs() @ B.abs()
            bound = eA @ B.abs() + (steps + 2) * V * (mag + eA @ B.abs())
            assert ((got.double() - want).abs() <= hs * want.abs() + bound * (1 + hs) + TINY).all()


def test_gradients_of_slabs_equal_those_of_segments(dev):
    L, cap, K, N = 5, 48, 128, 64
    m = [0, 48, 17, 1, 30]
    x, dout = rand(1, L, cap, K, dtype=torch.bfloat16), rand(2, L, cap, N, dtype=torch.bfloat16)
    pre, w = rand(3, L, cap, N, dtype=torch.bfloat16), rand(4, L, N, K, dtype=torch.bfloat16)
    starts = [e * cap for e in range(L)]
    ends = [s + c for s, c in zip(starts, m)]
    kw = dict(act="silu", need=("dx", "dw", "dbias"))
    z = lambda *s: torch.zeros(*s, device=DEV, dtype=torch.bfloat16)
    a = dev.expert_matmul_grad(dout, x, w, masked_m=i32(m), pre=pre, dx=z(L, cap, K), **kw)
    b = dev.expert_matmul_grad(dout.view(-1, N), x.view(-1, K), w, i32(starts), i32(ends), pre=pre.view(-1, N),
                               dx=z(L * cap, K), **kw)
    for k in ("dx", "dw", "dbias"):
        assert torch.equal(a[k].reshape(b[k].shape), b[k]), k


def test_gradients_against_differences(dev):
    """<c, out> by central differences in 64 bits along one direction of x, w and bias."""
    counts, K, N = [7, 0, 20], 64, 32
    starts, ends, R = segments(counts, 8)
    x, w = rand(1, R, K, dtype=torch.float16), rand(2, 3, 2 * N, K, dtype=torch.float16, gain=0.125)
    b, c = rand(3, 3, 2 * N), rand(4, R, N, dtype=torch.float16)
    dirs = [rand(5, R, K, dtype=torch.float64), rand(6, 3, 2 * N, K, dtype=torch.float64), rand(7, 3, 2 * N, dtype=torch.float64)]

    def f(h):
        xx, ww, bb = (v.double() + h * d for v, d in zip((x, w, b), dirs))
        total = 0
        for e, (lo, hi) in enumerate(zip(starts, ends)):
            P = xx[lo:hi] @ ww[e].t() + bb[e]
            total = total + (c[lo:hi].double() * phi("gelu", P[:, :N])[0] * P[:, N:]).sum()
        return total

    h = 1e-4
    want = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
    pre = torch.zeros(R, 2 * N, device=DEV, dtype=torch.float16)
    kw = dict(act="gelu", gated=True)
    dev.expert_matmul(x, w, i32(starts), i32(ends), bias=b, pre=pre, **kw)
    g = dev.expert_matmul_grad(c, x, w, i32(starts), i32(ends), pre=pre, dx=torch.zeros_like(x), dw_dtype=torch.float32,
                               need=("dx", "dw", "dbias"), **kw)
    parts = [(g[k].double() * d) for k, d in zip(("dx", "dw", "dbias"), dirs)]
    got, mag = sum(p.sum() for p in parts), sum(p.abs().sum() for p in parts)
    # roundings of pre, dP and dx to fp16 (2^-11 each): at most four of them on any path
    assert (got - want).abs() <= 4 * 2.0 ** -11 * mag


def test_graph_replay_with_other_counts(dev):
    """Captured once, replayed with other segment ends: the tile list is formed on the device."""
    L, K, N, R = 6, 256, 192, 600
    x, w = rand(1, R, K, dtype=torch.bfloat16), rand(2, L, N, K, dtype=torch.bfloat16, gain=0.06)
    starts = i32([0, 100, 200, 300, 400, 500])
    ends = i32([10, 100, 300, 301, 433, 600])
    out, st = torch.zeros(R, N, device=DEV, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32, device=DEV)
    pre, dw = torch.zeros_like(out), torch.zeros_like(w)
    ws = dev.GradWorkspace(R, L, N, torch.bfloat16, DEV)

    def step():
        dev.expert_matmul(x, w, starts, ends, act="silu", out=out, pre=pre, status=st)
        return dev.expert_matmul_grad(out, x, w, starts, ends, pre=pre, act="silu", dw=dw, need=("dw",), workspace=ws,
                                      status=st)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for e in ([0, 100, 200, 300, 400, 500], [100, 200, 300, 400, 500, 600], [1, 180, 216, 400, 499, 501]):
        ends.copy_(i32(e))
        out.zero_(), pre.zero_()
        graph.replay()
        torch.cuda.synchronize()
        a, b = out.clone(), dw.clone()
        out.zero_(), pre.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, dw)
    assert dev.moe_status_sync(st) == dev.MOE_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("R,K,N", [(5, 2048, 64), (300, 136, 128)])
def test_nan_reaches_its_row_alone(dev, R, K, N, act, gated, dtype):
    """A NaN in one row (or one expert's weight row) shows in what depends on it and
    nowhere else; no activation turns it into a number."""
    Nw, bad, feature = 2 * N if gated else N, R // 2, 3
    x, w = rand(1, R, K, dtype=dtype), rand(2, 2, Nw, K, dtype=dtype, gain=K ** -0.5)
    half = R // 2 + 1  # expert 0 owns the bad row
    seg = (i32([0, half]), i32([half, R]))
    call = lambda a, b: dev.expert_matmul(a, b, *seg, act=act, gated=gated).clone()
    clean = call(x, w)
    xb, wb = x.clone(), w.clone()
    xb[bad, K - 1] = float("nan")
    got = call(xb, w)
    rows = torch.arange(R, device=DEV) == bad
    assert got[rows].isnan().all() and torch.equal(got[~rows], clean[~rows])
    wb[1, feature, 0] = float("nan")
    got = call(x, wb)
    hit = torch.zeros(R, N, dtype=torch.bool, device=DEV)
    hit[half:, feature] = True
    assert got[hit].isnan().all() and torch.equal(got[~hit], clean[~hit])
    if act == "none" and not gated:
        return
    dout, pre = rand(3, R, N, dtype=dtype), rand(4, R, Nw, dtype=dtype)
    grad = lambda p: dev.expert_matmul_grad(dout, x, w, *seg, pre=p, act=act, gated=gated)
    g = grad(pre)
    g = {k: g[k].clone() for k in ("dx", "dw")}
    pb = pre.clone()
    pb[bad, feature] = float("nan")
    b = grad(pb)
    if act == "relu" and not gated:  # the slope of relu is a number at NaN
        return
    assert b["dx"][rows].isnan().all() and torch.equal(b["dx"][~rows], g["dx"][~rows])
    hit = torch.zeros(2, Nw, dtype=torch.bool, device=DEV)
    hit[0, feature] = act in ("silu", "gelu")  # the others' slope at NaN is 1: dout * up
    if gated:
        hit[0, N + feature] = True
    same = ~hit
    same[0, feature] = False
    assert b["dw"][hit].isnan().all() and torch.equal(b["dw"][same], g["dw"][same])


def check_gradients(o, dout, pre, x, w, seg, N, act, gated, dw_dtype, carried=()):
    """dx, dw and dbias of every expert's rows within the bounds of test_gradients; rows of no expert as they were (9).
    `carried`: those of dx and dw that carry the rounding of the pre-activations' gradient along, which is then off
    by its second rounding (half a step squared) only."""
    dtype, Nw = x.dtype, w.shape[1]
    hs, hw = torch.finfo(dtype).eps / 2, torch.finfo(dw_dtype).eps / 2
    real = torch.zeros(x.shape[0], dtype=torch.bool, device=DEV)
    for e, (lo, hi) in enumerate(seg):
        if hi <= lo:
            assert all((o[k][e] == 0).all() for k in ("dw", "dbias") if o[k] is not None)
            continue
        real[lo:hi] = True
        g, n = dout[lo:hi].double(), hi - lo
        if act == "none" and not gated:
            dP = g
            e32 = e16 = torch.zeros_like(dP)
        else:
            p = pre[lo:hi].double()
            a, d = phi(act, p[:, :N])
            dP = torch.cat([g * d * p[:, N:], g * a], 1) if gated else g * d
            m = torch.cat([(g * p[:, N:]).abs() * 1.13, (g * p[:, :N]).abs()], 1) if gated else g.abs() * 1.13
            e32 = ACT_ERR * m
            e16 = e32 + hs * (dP.abs() + e32) + TINY
        e48 = e32 + hs * hs * (dP.abs() + e32) + TINY
        for k, A, B, h, steps in (("dx", dP, w[e].double(), hs, Nw), ("dw", dP.t(), x[lo:hi].double(), hw, n)):
            if o[k] is None:
                continue
            got, eA, terms = o[k][lo:hi] if k == "dx" else o[k][e], e48 if k in carried else e16, 2 if k in carried else 1
            eA = eA.t() if k == "dw" else eA
            want, mag = A @ B, A.abs() @ B.abs()
            bound = eA @ B.abs() + (terms * steps + 2) * V * (mag + eA @ B.abs())
            assert ((got.double() - want).abs() <= h * want.abs() + bound * (1 + h) + TINY).all(), e
        if o["dbias"] is not None:
            bound = e32.sum(0) + (n + 2) * V * (dP.abs() + e32).sum(0)
            assert ((o["dbias"][e].double() - dP.sum(0)).abs() <= bound).all(), e
    if o["dx"] is not None:
        assert (o["dx"][~real] == 9).all()


def valid_segments(begin, end, R):
    """The segments that count: inside the rows, and without a row of an earlier one that is."""
    inside = [0 <= lo <= hi <= R for lo, hi in zip(begin, end)]
    seg, bad = [], False
    for e, (lo, hi) in enumerate(zip(begin, end)):
        shares = any(inside[f] and max(lo, begin[f]) < min(hi, end[f]) for f in range(e))
        ok = inside[e] and not shares
        bad |= not ok
        seg.append((lo, hi) if ok else (0, 0))
    return seg, bad


LISTS = [  # begin, end, R, K, N
    ([0, 10], [4, 21], 20, 64, 64), ([-1, 4], [3, 8], 20, 64, 64), ([0, 6], [4, 5], 20, 64, 64),    # outside the rows
    ([10, 0], [20, 10], 20, 64, 64), ([7, 20, 3], [12, 20, 7], 20, 136, 64),                        # in another order
    ([0, 5], [10, 15], 20, 64, 64), ([5, 0], [15, 10], 20, 64, 64), ([0, 4, 2], [8, 4, 12], 20, 64, 64),
    ([0, 0, 0], [40, 40, 40], 40, 2048, 64), ([0] * 9, [300] * 9, 300, 1024, 128),                  # with split reductions
    ([0, 8, 6, 12], [8, 9, 10, 20], 20, 128, 64), ([0, 0, 30], [0, 30, 300], 300, 64, 264),
    (list(range(0, 1200, 3)), list(range(4, 1204, 3)), 1300, 64, 16),                               # each overlaps the next
]


@pytest.mark.parametrize("begin,end,R,K,N", LISTS)
def test_segments_that_do_not_fit_count_as_empty(dev, begin, end, R, K, N):
    """Segments outside the rows, or with rows of an earlier one, are flagged and nothing of them is read or written;
    all others are computed, in any order."""
    L, dtype = len(begin), torch.bfloat16
    seg, bad = valid_segments(begin, end, R)
    x, w = rand(1, R, K, dtype=dtype), rand(2, L, N, K, dtype=dtype, gain=K ** -0.5)
    bias, dout = rand(3, L, N), rand(4, R, N, dtype=dtype)
    out, pre = (torch.full((R, N), 9.0, device=DEV, dtype=dtype) for _ in range(2))
    want = dev.MOE_ERR_BAD_LAYOUT if bad else dev.MOE_OK
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev.expert_matmul(x, w, i32(begin), i32(end), bias=bias, act="silu", out=out, pre=pre, status=st)
    assert dev.moe_status_sync(st) == want
    check_forward(out, pre, x.double(), w.double(), bias, None, seg, N, "silu", False, dtype)
    for act in ("silu", "none"):
        st.zero_()
        dx = torch.full((R, K), 9.0, device=DEV, dtype=dtype)
        o = dev.expert_matmul_grad(dout, x, w, i32(begin), i32(end), pre=pre, act=act, dx=dx, status=st,
                                   need=("dx", "dw", "dbias"))
        assert dev.moe_status_sync(st) == want
        check_gradients(o, dout, pre, x, w, seg, N, act, False, dtype)
        st.zero_()
        alone = dev.expert_matmul_grad(dout, x, w, i32(begin), i32(end), pre=pre, act=act, status=st, need=("dbias",))
        assert dev.moe_status_sync(st) == want and torch.equal(alone["dbias"], o["dbias"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts", [[100, 60, 0, 3], [512, 0, 0, 0], [128] * 4, [0, 0, 0, 0], [513, 0, 0, 0]])
def test_gradients_do_not_depend_on_the_buffer(dev, counts, dtype):
    """The rows held decide how exact dx and dw are: the same batch in a larger buffer, or in slabs, gives equal bits,
    and up to 128 rows an expert the rounding of the pre-activations' gradient is carried along in each."""
    L, K, N = 4, 136, 64
    tight, ends, R = segments(counts, 1)
    rows = rand(1, R, K, dtype=dtype), rand(2, R, N, dtype=dtype), rand(3, R, 2 * N, dtype=dtype)
    w = rand(4, L, 2 * N, K, dtype=dtype, gain=K ** -0.5)
    got = []
    for room in (R, 4 * 128, 4 * 128 + 1, 9000):  # rows of the buffer
        if room < R:
            continue
        x, dout, pre = (torch.full((room, t.shape[1]), float("nan"), device=DEV, dtype=dtype) for t in rows)
        for big, t in zip((x, dout, pre), rows):
            big[:R] = t
        dx = torch.full((room, K), 9.0, device=DEV, dtype=dtype)
        o = dev.expert_matmul_grad(dout, x, w, i32(tight), i32(ends), pre=pre, act="silu", gated=True, dx=dx)
        check_gradients(o, dout, pre, x, w, list(zip(tight, ends)), N, "silu", True, dtype,
                        ("dx", "dw") if sum(counts) <= 128 * L else ())
        got.append((o["dx"][:R], o["dw"]))
    for cap in (max(max(counts), 1), 4000):
        slabs = [torch.full((L, cap, t.shape[1]), float("nan"), device=DEV, dtype=dtype) for t in rows]
        for e, (lo, hi) in enumerate(zip(tight, ends)):
            for big, t in zip(slabs, rows):
                big[e, :hi - lo] = t[lo:hi]
        dx = torch.full((L, cap, K), 9.0, device=DEV, dtype=dtype)
        o = dev.expert_matmul_grad(slabs[1], slabs[0], w, masked_m=i32(counts), pre=slabs[2], act="silu", gated=True, dx=dx)
        flat = got[0][0].clone()
        for e, (lo, hi) in enumerate(zip(tight, ends)):
            flat[lo:hi] = o["dx"][e, :hi - lo]
        got.append((flat, o["dw"]))
    for dx, dw in got[1:]:
        assert torch.equal(dx, got[0][0]) and torch.equal(dw, got[0][1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("act,gated", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("counts,K,N", [([300, 0, 170], 136, 128), ([700], 264, 64), ([257, 640], 64, 320)])
def test_weight_gradients_in_fp32_carry_the_rounding(dev, counts, K, N, act, gated, dtype):
    """With any number of rows: in 32 bits dw has no rounding of its own, so it is given none of the pre-activations'
    gradient's either. dx is the same beside a dw of either type."""
    starts, ends, R = segments(counts, 1)
    L, Nw = len(counts), 2 * N if gated else N
    x, dout, pre = rand(1, R, K, dtype=dtype), rand(2, R, N, dtype=dtype), rand(3, R, Nw, dtype=dtype)
    w = rand(4, L, Nw, K, dtype=dtype, gain=K ** -0.5)
    call = lambda t, **k: dev.expert_matmul_grad(dout, x, w, i32(starts), i32(ends), pre=pre, act=act, gated=gated,
                                                 dw_dtype=t, **k)
    o = call(torch.float32, need=("dx", "dw", "dbias"))
    seg = list(zip(starts, ends))
    check_gradients(o, dout, pre, x, w, seg, N, act, gated, torch.float32, ("dw",))
    alone, half = call(torch.float32, need=("dw",)), call(dtype)
    assert torch.equal(alone["dw"], o["dw"]) and torch.equal(half["dx"], o["dx"])
    check_gradients(half, dout, pre, x, w, seg, N, act, gated, dtype)


def test_a_reduction_of_seconds_is_waited_for(dev):
    """dW over 1.2e9 rows: the epilogue waits longer than a single step may take. The few rows that are not zero hold
    small whole numbers, so the sums are exact."""
    R, K, N = 1_200_000_000, 8, 8
    x, dout = (torch.zeros(R, 8, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    at = torch.tensor([0, 63, 64, 999_999_937, 1 << 30, R - 1], device=DEV)
    vx, vd = (torch.randint(-3, 4, (at.numel(), 8), device=DEV).bfloat16() for _ in range(2))
    x[at], dout[at] = vx, vd
    w, st = torch.zeros(N, K, device=DEV, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32, device=DEV)
    o = dev.expert_matmul_grad(dout, x, w, need=("dw",), dw_dtype=torch.float32, status=st)
    assert dev.moe_status_sync(st) == dev.MOE_OK
    assert torch.equal(o["dw"], vd.float().t() @ vx.float())


def test_a_wait_that_ran_out_is_the_gravest_status(dev):
    """The status word's bits, set from the host: a timeout comes before a bad layout and the rest."""
    for bits, want in ((8, dev.MOE_ERR_TIMEOUT), (15, dev.MOE_ERR_TIMEOUT), (12, dev.MOE_ERR_TIMEOUT), (7, dev.MOE_ERR_BAD_LAYOUT),
                       (3, dev.MOE_ERR_LIVE_OVERFLOW), (1, dev.MOE_ERR_OVERFLOW), (0, dev.MOE_OK)):
        assert dev.moe_status_sync(i32([bits])) == want


# Several hundred tiles, so that every pair of CTAs takes some one after the other: both accumulators and their hand-back,
# the ring and the scale words going on from tile to tile, and tiles of every height beside each other.

def ragged(seed, L, most):
    """Counts per expert: none, whole blocks of 64 rows, and any other number up to `most`."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, most + 1, L)
    c[::5] = 64 * rng.integers(0, most // 64 + 1, c[::5].size)
    c[rng.integers(0, L, 2)] = 0
    return c.tolist()


def padded(R, seg):
    """Whether a row is of no expert."""
    pad = torch.ones(R, dtype=torch.bool, device=DEV)
    for lo, hi in seg:
        pad[lo:hi] = False
    return pad


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("act,gated,residual", [("silu", True, False), ("gelu", False, True), ("relu", True, True)])
def test_forward_of_many_tiles(dev, act, gated, residual, dtype):
    L, K, N = 48, 200, 528
    starts, ends, R = segments(ragged(1, L, 700), 8, gap=1)
    seg, Nw = list(zip(starts, ends)), 2 * N if gated else N
    x, w = rand(1, R, K, dtype=dtype), rand(2, L, Nw, K, dtype=dtype, gain=K ** -0.5)
    bias, res = rand(3, L, Nw), rand(4, R, N, dtype=dtype) if residual else None
    x[padded(R, seg)] = float("nan")
    out, pre = torch.full((R, N), 9.0, device=DEV, dtype=dtype), torch.full((R, Nw), 9.0, device=DEV, dtype=dtype)
    call = lambda o: dev.expert_matmul(x, w, i32(starts), i32(ends), bias=bias, act=act, gated=gated, residual=res, out=o, pre=pre)
    call(out)
    check_forward(out, pre, x.double(), w.double(), bias, res, seg, N, act, gated, dtype)
    assert torch.equal(out, call(torch.full_like(out, 9.0)))


@pytest.mark.parametrize("L,most,K,N,gated", [(40, 700, 1152, 272, True), (64, 480, 512, 392, False), (256, 12, 640, 128, True)])
def test_forward_of_many_tiles_e4m3(dev, L, most, K, N, gated):
    starts, ends, R = segments(ragged(2, L, max(most, 64)) if most >= 64 else [int(c) for c in np.arange(L) % (most + 1)], 4)
    seg, Nw = list(zip(starts, ends)), 2 * N if gated else N
    q, sc, ld, xv = quant(rand(1, R, K) * torch.exp2(torch.randint(-6, 7, (R, 1), device=DEV).float()))
    wq, wsc, ldw, wv = quant(rand(2, L * Nw, K, gain=K ** -0.5))
    pad = padded(R, seg)
    q.view(torch.uint8)[pad] = 0x7F
    sc[:, :R][:, pad] = -1
    out = torch.full((R, N), 9.0, device=DEV, dtype=torch.bfloat16)
    call = lambda o: dev.expert_matmul(q, wq.view(L, Nw, K), i32(starts), i32(ends), act="silu", gated=gated, x_scales=sc,
                                       ld_xs=ld, w_scales=wsc, ld_ws=ldw, out=o)
    call(out)
    check_forward(out, None, xv, wv.view(L, Nw, K), None, None, seg, N, "silu", gated, torch.bfloat16)
    assert torch.equal(out, call(torch.full_like(out, 9.0)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("L,most,K,N,act,gated", [(48, 600, 520, 264, "silu", True), (96, 128, 520, 264, "gelu", False),
                                                  (96, 200, 520, 272, "silu", True), (48, 600, 520, 520, "none", False)])
def test_gradients_of_many_tiles(dev, L, most, K, N, act, gated, dtype):
    """With one term and with two (most <= 200: at most 128 rows an expert on average)."""
    N = N // 16 * 16 if gated else N
    counts = ragged(3, L, most)
    starts, ends, R = segments(counts, 8, gap=3)
    seg, Nw = list(zip(starts, ends)), 2 * N if gated else N
    x, dout, pre = rand(1, R, K, dtype=dtype), rand(2, R, N, dtype=dtype), rand(3, R, Nw, dtype=dtype)
    w = rand(4, L, Nw, K, dtype=dtype, gain=K ** -0.5)
    for t in (x, dout, pre):
        t[padded(R, seg)] = float("nan")
    two = sum(counts) <= 128 * L
    assert two == (most <= 200)
    for dwt in (dtype, torch.float32):
        call = lambda: dev.expert_matmul_grad(dout, x, w, i32(starts), i32(ends), pre=pre, act=act, gated=gated, dw_dtype=dwt,
                                              dx=torch.full((R, K), 9.0, device=DEV, dtype=dtype), need=("dx", "dw", "dbias"))
        o = call()
        check_gradients(o, dout, pre, x, w, seg, N, act, gated, dwt, ("dx", "dw") if two else ("dw",) if dwt is torch.float32 else ())
        again = call()
        assert all(torch.equal(o[k], again[k]) for k in ("dx", "dw", "dbias"))
