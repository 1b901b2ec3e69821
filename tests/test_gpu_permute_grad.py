"""Rows sorted by expert without quantisation (permute), the way back in every
type (combine), and the gradients of both, against the CPU oracle's layout and
plain sums in 64 bits.

Bounds: a copy is exact; a product is off by 2^-24 before its rounding to the
type (half a step, eps / 2); a sum of n terms in fp32 by n * 2^-24 of the sum of
magnitudes. The dot products of combine_grad add at most 16 terms per thread
(rows up to 8192 elements of 16 bits), 5 shuffle steps and 16 warps: 64 steps
cover them. 2^-25 is half of fp16's smallest step."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
IDS = ["bf16", "fp16", "fp32"]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def routing(seed, T, E, K):
    """Ids in [-1, E) with repeats inside a token, and weights, some of them negative."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(-1, E, size=(T, K)).astype(np.int32)
    return ids, rng.standard_normal((T, K)).astype(np.float32)


def oracle_layout(ref, ids, L, b, n_live=None):
    """The oracle's compact layout (its dispatch of zero rows of 128 elements)."""
    T, K = ids.shape
    n = T if n_live is None else n_live
    bound = ref.compact_bound(T * K, L, b)
    xq = np.zeros((max(bound, 1), 128), np.uint8)
    sc, ld = ref.scale_buffer("u8", max(bound, 1), 1, fill=0)
    mi, s2d = np.zeros(max(bound, 1), np.int32), np.zeros((T, K), np.int32)
    c, s, p = (np.zeros(L, np.int32) for _ in range(3))
    t = np.zeros(1, np.int32)
    ref.dispatch_compact(np.zeros((T, 128), np.uint16), T, n, 128, ids, np.zeros((T, K), np.float32), K, L, b,
                         128, "u8", xq, sc, ld, mi, bound, s2d, c, s, p, t)
    return dict(bound=bound, m_indices=mi[:bound], src2dst=s2d, counts=c, starts=s, psum=p, total=t)


def rand(seed, *shape, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


PERMUTE = [  # T, H, E, L, K, block
    (1, 64, 1, 1, 1, 1), (1, 7168, 256, 256, 8, 128), (16, 256, 8, 8, 2, 128), (128, 7168, 256, 32, 8, 128),
    (203, 1000, 17, 9, 3, 16), (256, 128, 4, 4, 8, 1),      # the largest one-launch sizes
    (257, 136, 4, 4, 8, 8), (1777, 2048, 64, 64, 6, 64),    # two launches
    (3001, 72, 300, 300, 5, 7), (700, 24584, 8, 3, 4, 128), (40, 32768, 8, 8, 2, 4),
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,H,E,L,K,b", PERMUTE)
def test_permute_rows_and_layout(dev, ref, dtype, T, H, E, L, K, b):
    ids, w = routing(T + K, T, E, K)
    want = oracle_layout(ref, ids, L, b)
    ldx = H + 16  # a padded row stride
    xb = rand(1, T, ldx, dtype=dtype)
    x = xb[:, :H]
    out = torch.full((want["bound"], H), 7.0, device=DEV, dtype=dtype)
    rw = torch.full((want["bound"],), 7.0, device=DEV)
    o = dev.permute(x, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), E, L, block_e=b, out=out,
                    row_weights=rw)
    torch.cuda.synchronize()
    for k in ("m_indices", "src2dst", "counts", "starts", "psum", "total"):
        assert np.array_equal(o[k].cpu().numpy(), want[k]), k
    exp = torch.full_like(out, 7.0)
    exp_rw = torch.full_like(rw, 7.0)
    s2d = torch.from_numpy(want["src2dst"]).to(DEV).long()
    kept = s2d >= 0
    tok = torch.arange(T, device=DEV)[:, None].expand(T, K)
    exp[s2d[kept]] = x[tok[kept]]
    exp_rw[s2d[kept]] = torch.from_numpy(w).to(DEV)[kept]
    assert torch.equal(out, exp) and torch.equal(rw, exp_rw)
    assert dev.moe_status_sync(o["status"]) == dev.MOE_OK


@pytest.mark.parametrize("T,n", [(100, 0), (100, 37), (100, 200), (900, 0), (900, 411), (900, 5000)])
def test_permute_live_count(dev, ref, T, n):
    """Tokens past a device-side live count take no row; a count above T is clamped and flagged."""
    H, E, K, b = 512, 16, 4, 8
    ids, w = routing(5, T, E, K)
    want = oracle_layout(ref, ids, E, b, min(n, T))
    x = rand(2, T, H, dtype=torch.bfloat16)
    x[min(n, T):] = float("nan")
    out = torch.zeros(want["bound"], H, device=DEV, dtype=torch.bfloat16)
    o = dev.permute(x, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), E, E, block_e=b, out=out,
                    num_tokens=torch.tensor([n], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for k in ("m_indices", "src2dst", "counts", "psum"):
        assert np.array_equal(o[k].cpu().numpy(), want[k]), k
    assert torch.isfinite(out.float()).all()
    assert dev.moe_status_sync(o["status"]) == (dev.MOE_ERR_LIVE_OVERFLOW if n > T else dev.MOE_OK)


def test_permute_empty(dev):
    o = dev.permute(torch.empty(0, 64, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV),
                    torch.empty(0, 2, device=DEV), 4, 4)
    torch.cuda.synchronize()
    assert o["bound"] == 0 and o["counts"].tolist() == [0] * 4 and o["total"].tolist() == [0]


BACK = [  # T, H, R rows offered, K
    (1, 8, 3, 1), (1, 7168, 64, 8), (5, 128, 40, 3), (129, 1000, 900, 6), (64, 4104, 4000, 32),
    (700, 2048, 5000, 7), (33, 8192, 400, 8), (9, 32768, 100, 4),
]


def back_inputs(seed, T, H, R, K, dtype):
    """Distinct rows for the slots, about a fifth of them dropped, one token with none."""
    rng = np.random.default_rng(seed)
    row = np.full(T * K, -1, np.int32)
    n = min(R, T * K)
    pick = rng.permutation(T * K)[:max(1, int(n * 0.8))]
    row[pick] = rng.permutation(R)[:pick.size]
    row = row.reshape(T, K)
    if T > 1:
        row[rng.integers(T)] = -1
    return torch.from_numpy(row).to(DEV), rand(seed, T, K, dtype=torch.float32)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T,H,R,K", BACK)
def test_combine_and_its_gradients(dev, dtype, T, H, R, K):
    row, w = back_inputs(T + H, T, H, R, K, dtype)
    y = rand(3, R, H + 8, dtype=dtype)[:, :H]
    dout = rand(4, T, H + 16, dtype=dtype)[:, :H]
    out = dev.combine(y, row, w)
    dy = torch.full((R, H), 5.0, device=DEV, dtype=dtype)
    g = dev.combine_grad(dout, y, row, w, dy=dy)
    dx = dev.permute_grad(y, row)
    torch.cuda.synchronize()
    hs, tiny, u = half_step(dtype), 2.0 ** -25, 2.0 ** -24
    kept = (row >= 0)
    at = row.clamp_min(0).long()
    terms = y[at].double() * kept[:, :, None]                         # [T, K, H]
    for got, wt in ((out, w.double()), (dx, torch.ones_like(w).double())):
        ref64 = torch.einsum("tk,tkh->th", wt, terms)
        mag = torch.einsum("tk,tkh->th", wt.abs(), terms.abs())
        assert ((got.double() - ref64).abs() <= hs * ref64.abs() + (K + 1) * u * mag * (1 + hs) + tiny).all()
    dy64 = w.double()[:, :, None] * dout.double()[:, None, :]
    want = torch.full((R, H), 5.0, device=DEV, dtype=torch.float64)
    want[row[kept].long()] = dy64[kept]
    owned = torch.zeros(R, dtype=torch.bool, device=DEV)
    owned[row[kept].long()] = True
    assert (dy[~owned] == 5.0).all()
    assert ((dy.double() - want).abs() <= (hs + 2 * u) * want.abs() + tiny).all()
    dw64 = torch.einsum("th,tkh->tk", dout.double(), terms)
    mag = torch.einsum("th,tkh->tk", dout.double().abs(), terms.abs())
    steps = 64 if H * y.element_size() <= 16384 else 256
    assert ((g["dweights"].double() - dw64).abs() <= steps * u * mag).all()
    assert (g["dweights"][~kept] == 0).all()
    assert dev.moe_status_sync(g["status"]) == dev.MOE_OK
    # the halves alone, and the same bits on a second call
    a = dev.combine_grad(dout, y, row, w, need_dy=False)
    b = dev.combine_grad(dout, y, row, w, need_dweights=False, dy=torch.full_like(dy, 5.0))
    torch.cuda.synchronize()
    assert a["dy"] is None and torch.equal(a["dweights"], g["dweights"])
    assert b["dweights"] is None and torch.equal(b["dy"], dy)


def test_combine_grad_against_differences(dev):
    """<c, combine(y + h v, w + h u)> by central differences in 64 bits against the gradients."""
    T, H, R, K = 13, 264, 60, 4
    row, w = back_inputs(8, T, H, R, K, torch.float32)
    y, c = rand(5, R, H, dtype=torch.float32), rand(6, T, H, dtype=torch.float32)
    v, u = rand(7, R, H, dtype=torch.float64), rand(8, T, K, dtype=torch.float64)
    kept, at = (row >= 0).double(), row.clamp_min(0).long()

    def f(h):
        return (c.double() * torch.einsum("tk,tkh->th", (w.double() + h * u) * kept, (y.double() + h * v)[at])).sum()

    h = 1e-3   # the function is quadratic in h: central differences are exact but for rounding
    want = (f(h) - f(-h)) / (2 * h)
    g = dev.combine_grad(c, y, row, w, dy=torch.zeros_like(y))
    got = (g["dy"].double() * v).sum() + (g["dweights"].double() * u).sum()
    mag = (g["dy"].double() * v).abs().sum() + (g["dweights"].double() * u).abs().sum()
    assert (got - want).abs() <= 1e-6 * mag


def test_combine_grad_flags_a_row_past_the_buffer(dev):
    T, H, R, K = 6, 64, 10, 2
    row = torch.arange(T * K, dtype=torch.int32, device=DEV).reshape(T, K)   # 10 and 11 are past R
    y, d = rand(1, R, H, dtype=torch.float32), rand(2, T, H, dtype=torch.float32)
    g = dev.combine_grad(d, y, row, dy=torch.zeros_like(y))
    assert dev.moe_status_sync(g["status"]) == dev.MOE_ERR_BAD_LAYOUT
    assert (g["dweights"].reshape(-1)[R:] == 0).all()
    assert torch.equal(g["dy"], d.repeat_interleave(K, 0)[:R])


def test_live_count_leaves_the_rest_alone(dev):
    T, H, R, K, n = 50, 128, 200, 3, 17
    row, w = back_inputs(3, T, H, R, K, torch.bfloat16)
    y, d = rand(1, R, H, dtype=torch.bfloat16), rand(2, T, H, dtype=torch.bfloat16)
    live = torch.tensor([n], dtype=torch.int32, device=DEV)
    full = dev.combine_grad(d, y, row, w, dy=torch.zeros_like(y))
    cut = row.clone()
    cut[n:] = -1
    want = dev.combine_grad(d, y, cut, w, dy=torch.zeros_like(y))
    got = dev.combine_grad(d, y, row, w, num_tokens=live, dy=torch.zeros_like(y))
    assert torch.equal(got["dy"], want["dy"]) and torch.equal(got["dweights"][:n], full["dweights"][:n])


def test_round_trip_under_a_graph_on_another_stream(dev):
    """permute -> combine -> gradients captured once and replayed with new routing."""
    T, H, E, K = 300, 1024, 8, 8
    x = rand(1, T, H, dtype=torch.bfloat16)
    d = rand(2, T, H, dtype=torch.bfloat16)
    ids0, w0 = routing(1, T, E, K)
    ids, w = torch.from_numpy(ids0).to(DEV), torch.from_numpy(w0).to(DEV)
    bound = dev.moe_compact_bound(T * K, E, 16)
    xs, dy = (torch.zeros(bound, H, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    ws = dev.Workspace(T, K, E, DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        o = dev.permute(x, ids, w, E, E, block_e=16, workspace=ws, status=st, out=xs)
        back = dev.combine(xs, o["src2dst"], w, status=st)
        g = dev.combine_grad(d, xs, o["src2dst"], w, status=st, dy=dy)
        return back, g["dweights"], dev.permute_grad(dy, o["src2dst"], status=st)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2, 3):
        i, ww = routing(seed, T, E, K)
        ids.copy_(torch.from_numpy(i))
        w.copy_(torch.from_numpy(ww))
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(mine, want):
            assert torch.equal(a, b)
    assert dev.moe_status_sync(st) == dev.MOE_OK
