"""Norms around a block with gate, residual scale and residual sum, and their
gradients, against the formulas in 64 bits.

Bounds, with u = 2^-24: a row sum adds at most 16 terms per thread, 5 shuffle
steps and 16 warps (64 steps cover it, as does its square root's rsqrtf of 2
ulp), and each factor of a product one more; C = 128 steps of u on the sum of
magnitudes therefore cover every 32-bit result, and the rounding to the type
adds half a step. Sums over T tokens add T steps."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
IDS = ["bf16", "fp16", "fp32"]
U, C, TINY = 2.0 ** -24, 128, 2.0 ** -25
EPS = 1e-6


def rand(seed, *shape, dtype=torch.float32, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * gain).to(dtype)


def make(T, H, dtype, gate, post, pre, y=True):
    s = dict(x=rand(1, T, H + 16, dtype=dtype, gain=2.0)[:, :H])
    s["y"] = rand(2, T, H + 8, dtype=dtype)[:, :H] if y else None
    s["w_post"] = 1 + rand(3, H, gain=0.3) if y and post else None
    s["w_pre"] = 1 + rand(4, H, gain=0.3) if pre else None
    s["gate"] = {"none": None, "channel": rand(5, H), "token": rand(6, T)}[gate] if y else None
    return s


def gate64(s, mode):
    if s["gate"] is None:
        return torch.ones(1, dtype=torch.float64, device=DEV)
    return s["gate"].double()[:, None] if mode == "token" else s["gate"].double()


def rms64(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


CASES = [  # T, H, gate, post, pre
    (1, 64, "none", True, True), (1, 7168, "channel", True, True), (3, 8, "token", True, True),
    (37, 1000, "channel", True, False), (129, 2048, "token", False, True), (64, 4104, "channel", False, True),
    (500, 512, "none", True, True), (33, 8192, "token", True, True), (700, 136, "channel", True, True),
    (20, 5496, "none", False, True),
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,H,mode,post,pre", CASES)
def test_forward(dev, dtype, T, H, mode, post, pre):
    s = make(T, H, dtype, mode, post, pre)
    o = dev.block_norm(s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], scale=0.37, w_pre=s["w_pre"], eps=EPS,
                       save_rstd=True)
    torch.cuda.synchronize()
    hs = torch.finfo(dtype).eps / 2
    x, y = s["x"].double(), s["y"].double()
    n = y
    if post:
        n = y * rms64(y) * s["w_post"].double()
        assert ((o["rstd_post"].double() - rms64(y)[:, 0]).abs() <= C * U * rms64(y)[:, 0]).all()
    add = 0.37 * gate64(s, mode) * n
    xo = x + add
    err = C * U * add.abs() + U * xo.abs()
    assert ((o["x"].double() - xo).abs() <= hs * xo.abs() + err * (1 + hs) + TINY).all()
    if pre:
        r = rms64(xo)
        h = xo * r * s["w_pre"].double()
        rel = err.norm(dim=1, keepdim=True) / xo.norm(dim=1, keepdim=True) + C * U
        assert ((o["rstd_pre"].double() - r[:, 0]).abs() <= (rel * r)[:, 0]).all()
        bound = err * (r * s["w_pre"].double()).abs() + rel * h.abs()
        assert ((o["h"].double() - h).abs() <= hs * h.abs() + bound * (1 + hs) + TINY).all()
    else:
        assert o["h"] is None


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_forward_norm_alone(dev, dtype):
    """Without a block output: h = rms(x) * w_pre and the stream is passed on."""
    s = make(77, 1240, dtype, "none", False, True, y=False)
    o = dev.block_norm(s["x"], w_pre=s["w_pre"], eps=EPS)
    x = s["x"].double()
    h = x * rms64(x) * s["w_pre"].double()
    hs = torch.finfo(dtype).eps / 2
    assert o["x"] is s["x"]
    assert ((o["h"].double() - h).abs() <= (hs + 2 * C * U) * h.abs() + TINY).all()


def grads64(s, mode, scale, dxo, dh, rx, ry):
    """The gradients and, beside each, the sum of magnitudes its 32-bit error is measured against."""
    x = s["x"].double()
    g = dxo.double() if dxo is not None else torch.zeros_like(x)
    G = g.abs()
    o = {}
    if s["w_pre"] is not None:
        r, d, w = rx.double()[:, None], dh.double(), s["w_pre"].double()
        xh, t = x * r, d * w
        g = g + r * (t - xh * (t * xh).mean(1, keepdim=True))
        G = G + r * (t.abs() + xh.abs() * (t * xh).abs().mean(1, keepdim=True))
        o["dw_pre"] = ((d * xh).sum(0), (d * xh).abs().sum(0))
    o["dx"] = (g, G)
    if s["y"] is not None:
        y, gt = s["y"].double(), gate64(s, mode)
        post = s["w_post"] is not None
        r = ry.double()[:, None] if post else torch.ones_like(x[:, :1])
        w = s["w_post"].double() if post else torch.ones_like(x[0])
        yh = y * r
        u, Um = scale * gt * g, abs(scale) * gt.abs() * G
        dim = 1 if mode == "token" else 0
        if mode != "none":
            o["dgate"] = ((scale * g * yh * w).sum(dim), (abs(scale) * G * (yh * w).abs()).sum(dim))
        if post:
            o["dw_post"] = ((u * yh).sum(0), (Um * yh.abs()).sum(0))
            t, tm = u * w, Um * w.abs()
            o["dy"] = (r * (t - yh * (t * yh).mean(1, keepdim=True)),
                       r * (tm + yh.abs() * (tm * yh.abs()).mean(1, keepdim=True)))
        else:
            o["dy"] = (u, Um)
    return o


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,H,mode,post,pre", CASES)
def test_gradients(dev, dtype, T, H, mode, post, pre):
    s = make(T, H, dtype, mode, post, pre)
    dxo, dh = rand(7, T, H + 8, dtype=dtype)[:, :H], (rand(8, T, H, dtype=dtype) if pre else None)
    rx = rms64(s["x"].double())[:, 0].float() if pre else None
    ry = rms64(s["y"].double())[:, 0].float() if post else None
    call = lambda: dev.block_norm_grad(dxo, dh, s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], scale=0.37,
                                       w_pre=s["w_pre"], rstd_pre=rx, rstd_post=ry)
    o = call()
    torch.cuda.synchronize()
    hs = torch.finfo(dtype).eps / 2
    want = grads64(s, mode, 0.37, dxo, dh, rx, ry)
    for k, (v, mag) in want.items():
        got = o[k].double()
        if k in ("dx", "dy"):
            bound = hs * v.abs() + 2 * C * U * mag * (1 + hs) + TINY
        else:
            bound = (2 * C + T) * U * mag
        assert ((got - v).abs() <= bound).all(), k
    assert {k for k, v in o.items() if v is not None} == set(want)
    again = call()
    for k in want:
        assert torch.equal(o[k], again[k]), k


def test_gradients_without_a_stream_gradient(dev):
    """dx_out None counts as zeros."""
    s = make(40, 264, torch.float32, "channel", True, True)
    dh = rand(8, 40, 264)
    rx, ry = rms64(s["x"].double())[:, 0].float(), rms64(s["y"].double())[:, 0].float()
    kw = dict(w_post=s["w_post"], gate=s["gate"], scale=2.0, w_pre=s["w_pre"], rstd_pre=rx, rstd_post=ry)
    a = dev.block_norm_grad(None, dh, s["x"], s["y"], **kw)
    b = dev.block_norm_grad(torch.zeros(40, 264, device=DEV), dh, s["x"], s["y"], **kw)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_no_tokens(dev):
    """T = 0: the sums over tokens are written as zeros."""
    H = 256
    s = make(0, H, torch.bfloat16, "channel", True, True)
    z = torch.empty(0, device=DEV)
    o = dev.block_norm_grad(s["x"], s["x"], s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"],
                            rstd_pre=z, rstd_post=z)
    f = dev.block_norm(s["x"], s["y"], w_post=s["w_post"], w_pre=s["w_pre"])
    torch.cuda.synchronize()
    assert f["h"].shape == (0, H)
    for k in ("dw_pre", "dw_post", "dgate"):
        assert (o[k] == 0).all(), k


def test_gradients_against_differences(dev):
    """Central differences of <a, x'> + <b, h> in 64 bits along one direction of every input."""
    T, H, sc = 9, 168, 0.6
    for mode in ("channel", "token", "none"):
        s = make(T, H, torch.float32, mode, True, True)
        a, b = rand(11, T, H), rand(12, T, H)
        dirs = {k: rand(20 + i, *s[k].shape, dtype=torch.float64) for i, k in enumerate(s) if s[k] is not None}

        def f(h):
            v = {k: s[k].double() + h * dirs[k] for k in dirs}
            gt = 1.0 if mode == "none" else (v["gate"][:, None] if mode == "token" else v["gate"])
            x = v["x"] + sc * gt * v["y"] * rms64(v["y"]) * v["w_post"]
            return (a.double() * x).sum() + (b.double() * x * rms64(x) * v["w_pre"]).sum()

        h = 1e-4
        want = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)   # error of order h^4
        o = dev.block_norm(s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], scale=sc, w_pre=s["w_pre"], eps=EPS,
                           save_rstd=True)
        g = dev.block_norm_grad(a, b, o["x"], s["y"], w_post=s["w_post"], gate=s["gate"], scale=sc, w_pre=s["w_pre"],
                                rstd_pre=o["rstd_pre"], rstd_post=o["rstd_post"])
        names = {"x": "dx", "y": "dy", "w_post": "dw_post", "w_pre": "dw_pre", "gate": "dgate"}
        got = sum((g[names[k]].double() * dirs[k]).sum() for k in dirs)
        mag = sum((g[names[k]].double() * dirs[k]).abs().sum() for k in dirs)
        assert (got - want).abs() <= 1e-5 * mag, mode


def test_as_many_tokens_as_channels(dev):
    """T = H: a named mode, or a 2-D gate, gives its own result; [T, 1] is the form without a name."""
    n, dtype = 96, torch.float32
    s = make(n, n, dtype, "token", True, True)
    for mode, two_d in (("token", s["gate"][:, None]), ("channel", s["gate"][None])):
        kw = dict(w_post=s["w_post"], scale=0.37, w_pre=s["w_pre"])
        call = lambda **k: dev.block_norm(s["x"], s["y"], eps=EPS, save_rstd=True, **kw, **k)
        grad = lambda f, **k: dev.block_norm_grad(s["x"], f["h"], f["x"], s["y"], rstd_pre=f["rstd_pre"],
                                                  rstd_post=f["rstd_post"], **kw, **k)
        f, f2 = call(gate=s["gate"], gate_mode=mode), call(gate=two_d)
        g, g2 = grad(f, gate=s["gate"], gate_mode=mode), grad(f, gate=two_d)
        y, w = s["y"].double(), s["w_post"].double()
        x = s["x"].double() + 0.37 * gate64(s, mode) * rms64(y) * y * w
        bound = C * U * (s["x"].double().abs() + (x - s["x"].double()).abs()) + U * x.abs()
        assert ((f["x"].double() - x).abs() <= bound).all()
        for k in f:
            assert torch.equal(f[k], f2[k]), k
        for k in g:
            assert torch.equal(g[k], g2[k].view_as(g[k])), k


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_a_gate_per_token_may_start_at_any_float(dev, dtype):
    """A batch's part of a longer gate: the same results as from a copy of it, also without tokens."""
    T, H = 21, 136
    s = make(T, H, dtype, "token", True, True)
    longer = torch.cat([rand(9, 3), s["gate"], rand(10, 2)])
    kw = dict(w_post=s["w_post"], scale=0.37, w_pre=s["w_pre"])
    for first in (1, 2, 3):
        longer[first:first + T] = s["gate"]
        part = longer[first:first + T]
        assert part.data_ptr() % 16 != 0
        a, b = (dev.block_norm(s["x"], s["y"], gate=g, save_rstd=True, **kw) for g in (s["gate"], part))
        c, d = (dev.block_norm_grad(s["x"], a["h"], a["x"], s["y"], gate=g, rstd_pre=a["rstd_pre"],
                                    rstd_post=a["rstd_post"], **kw) for g in (s["gate"], part))
        for u, v in ((a, b), (c, d)):
            assert all(torch.equal(u[k], v[k]) for k in u)
    e = make(0, H, dtype, "token", True, True)
    z = torch.empty(0, device=DEV)
    o = dev.block_norm_grad(e["x"], e["x"], e["x"], e["y"], gate=e["gate"], rstd_pre=z, rstd_post=z, **kw)
    torch.cuda.synchronize()
    assert all((o[k] == 0).all() for k in ("dw_pre", "dw_post")) and o["dgate"].shape == (0,)


@pytest.mark.parametrize("mode", ["none", "channel", "token"])
@pytest.mark.parametrize("sx", [1e-13, 1.0, 1e15])
@pytest.mark.parametrize("sy", [1e-13, 1.0, 1e15])
def test_gradients_of_very_small_and_large_rows(dev, sx, sy, mode):
    """Rows whose reciprocal root, cubed, is out of fp32's range; every gradient is an ordinary number. Small rows
    come with eps = 0. The same bounds as at ordinary sizes."""
    T, H = 19, 264
    s = make(T, H, torch.float32, mode, True, True)
    s["x"], s["y"] = s["x"] * sx, s["y"] * sy
    dxo, dh = rand(7, T, H, gain=1.0 / sx), rand(8, T, H)
    rx, ry = (torch.rsqrt((s[k].double() ** 2).mean(1)).float() for k in ("x", "y"))
    o = dev.block_norm_grad(dxo, dh, s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], scale=0.37, w_pre=s["w_pre"],
                            rstd_pre=rx, rstd_post=ry)
    torch.cuda.synchronize()
    want = grads64(s, mode, 0.37, dxo, dh, rx, ry)
    assert {k for k, v in o.items() if v is not None} == set(want)
    for k, (v, mag) in want.items():
        bound = (2 * C + T) * U * mag + (U * v.abs() if k in ("dx", "dy") else 0)
        assert torch.isfinite(o[k]).all() and ((o[k].double() - v).abs() <= bound).all(), k


# More rows than the grid holds: the second row of a pair, the walk over the rows and the ring's wrap. `H` in 16-byte
# vectors: one per thread and up to 2048 (rings of three slots, of one, and 1024 threads).
LONG = [  # T, vectors, gate, post, pre
    (20011, 17, "token", True, True), (20011, 64, "channel", True, True), (3001, 155, "token", False, True),
    (2501, 896, "channel", True, True), (1201, 897, "none", True, False), (1001, 1024, "token", True, True),
    (999, 1025, "channel", True, True), (701, 2048, "token", True, True), (650, 2048, "channel", False, True),
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,vectors,mode,post,pre", LONG)
def test_more_rows_than_the_grid(dev, dtype, T, vectors, mode, post, pre):
    H = vectors * 16 // torch.finfo(dtype).bits * 8
    test_forward(dev, dtype, T, H, mode, post, pre)
    test_gradients(dev, dtype, T, H, mode, post, pre)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,vectors", [(20011, 17), (2501, 896), (701, 2048)])
def test_more_rows_than_the_grid_without_a_block_output(dev, dtype, T, vectors):
    """One tensor a row in the ring, and two backward."""
    H = vectors * 16 // torch.finfo(dtype).bits * 8
    s = make(T, H, dtype, "none", False, True, y=False)
    o = dev.block_norm(s["x"], w_pre=s["w_pre"], eps=EPS, save_rstd=True)
    x, dh = s["x"].double(), rand(8, T, H, dtype=dtype)
    h, hs = x * rms64(x) * s["w_pre"].double(), torch.finfo(dtype).eps / 2
    assert ((o["h"].double() - h).abs() <= (hs + 2 * C * U) * h.abs() + TINY).all()
    g = dev.block_norm_grad(None, dh, s["x"], w_pre=s["w_pre"], rstd_pre=o["rstd_pre"])
    for k, (v, mag) in grads64(s, "none", 1.0, None, dh, o["rstd_pre"], None).items():
        bound = hs * v.abs() + 2 * C * U * mag * (1 + hs) + TINY if k == "dx" else (2 * C + T) * U * mag
        assert ((g[k].double() - v).abs() <= bound).all(), k
