"""The router's choice, its losses and their gradients, against the formulas in 64 bits.

Bounds, with u = 2^-23: the fast exponential is off by (3 + 1.2 |x|) u relative, the
fast quotient by 2 u, the fast logarithm by 2^-21.4 or 3 u, a sum of 32 values a lane and
5 steps of the warp by 19 u. With |x| at most D (the largest magnitude or spread of a
row's logits) a score, normalised or not, is off by B = (40 + 2.4 D) u relative. A
gradient's terms are products of up to four such values, so each is off by 4 B of its
magnitude. The reference's own steps in 64 bits are off by 2^-53 of what they add up, which
is at most a row's magnitudes: 2^-48 of those covers 32 of them, where a gradient is 0 but
for them. The rounding of a 16-bit output adds half a step, and 2^-25 covers fp16's
smallest numbers."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -23
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = [(1, 1, 1), (1, 256, 8), (3, 2, 2), (5, 31, 4), (300, 32, 32), (77, 33, 5), (129, 64, 6), (40, 77, 1), (333, 128, 9),
         (64, 200, 31), (500, 256, 8), (31, 300, 10), (17, 513, 8), (9, 1024, 32)]


def rand(seed, *shape, dtype=torch.float32, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * gain).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def spread(l):
    """D: largest magnitude or spread of the finite logits."""
    f = l.double()[torch.isfinite(l)]
    return float(max(f.max() - f.min(), f.abs().max())) if f.numel() else 0.0


def rel(l):
    return (40 + 2.4 * spread(l)) * U


def score(l, kind):
    return torch.softmax(l, 1) if kind == "softmax" else torch.sigmoid(l)


def choose(l, K, bias, kind):
    """The choice by repeated search on the host: ids, -1 where none is left."""
    d = l.double()
    key = (d if bias is None else score(d, kind) + bias.double()).clone()
    key = torch.where(torch.isnan(key) | (d == -math.inf) | torch.isnan(d), -math.inf, key)
    ids = torch.full((l.shape[0], K), -1, dtype=torch.int64, device=l.device)
    index = torch.arange(l.shape[1], device=l.device)
    for k in range(K):
        best = key.max(1, keepdim=True).values
        at = torch.where(key == best, index, l.shape[1]).min(1).values
        some = best[:, 0] > -math.inf
        ids[:, k] = torch.where(some, at, -1)
        key.scatter_(1, at[:, None], -math.inf)
    return ids


def weights(l, ids, kind, renorm, scale):
    w = torch.where(ids >= 0, score(l.double(), kind).gather(1, ids.clamp_min(0)), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
        w = torch.where(ids >= 0, w, 0.0)
    return scale * w


def check_route(dev, l, K, bias, kind, renorm, scale=1.0):
    o = dev.route(l, K, bias=bias, score=kind, renorm=renorm, scale=scale)
    ids = choose(l, K, bias, kind)
    assert torch.equal(o["topk_ids"].long(), ids)
    want = weights(l, ids, kind, renorm, scale)
    assert ((o["topk_weights"].double() - want).abs() <= rel(l) * want.abs() + 1e-37).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased,renorm", [(False, True), (True, True), (False, False), (True, False)])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_route(dev, T, E, K, biased, renorm, kind):
    for n, dtype in enumerate(DT.values()):
        l = rand(T + n, T, E + 5, dtype=dtype, gain=1.5)[:, 2:E + 2]  # rows that start anywhere
        check_route(dev, l, K, rand(9, E, gain=0.1) if biased else None, kind, renorm, scale=2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_and_masks(dev, biased, kind):
    """Few distinct values; rows with fewer experts than slots, and none at all."""
    T, E, K = 200, 100, 6
    l = rand(1, T, E).mul(2).round()
    l[:50] = 1.25
    for t in range(50, 120):
        l[t, t - 50:] = -math.inf
    l[120:130, ::2] = -math.inf
    l[130:135, 3:] = -0.0
    l[130:135, :3] = 0.0
    bias = rand(2, E).round() * 0.5 if biased else None
    check_route(dev, l, K, bias, kind, kind == "sigmoid")
    o = dev.route(l[50:51], K, score=kind)  # nothing left at all
    assert (o["topk_ids"] == -1).all() and (o["topk_weights"] == 0).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(40, 8), (256, 8), (1024, 31), (64, 32)])
def test_near_keys_are_told_apart(dev, E, K, kind):
    """The bias undoes the scores but for what 32 bits leave of them."""
    l = rand(3, 1, E).repeat(50, 1)
    s = score(l.double(), kind)[0]
    bias = (0.75 - s).float()
    key = s + bias.double()
    assert key.max() - key.min() < 2.0 ** -23
    check_route(dev, l, K, bias, kind, True)


def test_not_a_number(dev):
    l = rand(4, 6, 64)
    l[0, 5] = math.nan
    l[1, 7] = math.inf
    l[2] = math.nan
    for kind in ("softmax", "sigmoid"):
        o = dev.route(l, 4, score=kind, renorm=False)
        ids = choose(l, 4, None, kind)
        assert torch.equal(o["topk_ids"].long(), ids) and ids[1, 0] == 7 and (ids[0] != 5).all() and (ids[2] == -1).all()
        w = o["topk_weights"]
        assert torch.isnan(w[:2]).all() if kind == "softmax" else torch.isfinite(w).all()
        assert (w[2] == 0).all() and torch.isfinite(w[3:]).all()


def test_far_logits(dev):
    """Scores that leave the range of a float: sigmoids of very negative logits keep their ratios."""
    l = rand(5, 40, 32, gain=3.0)
    for shift in (-200.0, -80.0, 80.0, 3000.0):
        for kind in ("softmax", "sigmoid"):
            check_route(dev, l + shift, 5, None, kind, True)


@pytest.mark.parametrize("n", [0, 1, 13, 40])
def test_live_tokens(dev, n):
    T, E, K = 40, 64, 4
    l = rand(6, T, E)
    st = i32([0])
    ids, w = torch.full((T, K), 7, dtype=torch.int32, device=DEV), torch.full((T, K), 7.0, device=DEV)
    assert dev.moe_route(l, E, torch.float32, T, i32([n]), E, K, "softmax", None, True, 1.0, ids, w, st) == dev.MOE_OK
    assert torch.equal(ids[:n].long(), choose(l[:n], K, None, "softmax")) and (ids[n:] == 7).all() and (w[n:] == 7).all()
    assert dev.moe_status_sync(st) == dev.MOE_OK
    dev.route(l, K, num_tokens=i32([T + 1]), status=st)
    assert dev.moe_status_sync(st) == dev.MOE_ERR_LIVE_OVERFLOW


# ---------------------------------------------------------------------------
# Losses
# ---------------------------------------------------------------------------

def losses(l, ids, spans, kind):
    """(balance, z, counts, sums of p) in 64 bits, differentiable."""
    E, K = l.shape[1], ids.shape[1]
    dead = (l == -math.inf).all(1)
    safe = torch.where(dead[:, None], torch.zeros_like(l), l)
    sg = torch.sigmoid(safe)
    p = torch.softmax(safe, 1) if kind == "softmax" else sg / sg.sum(1, keepdim=True)
    p = torch.where(dead[:, None], torch.zeros_like(p), p)
    lse = torch.where(dead, torch.zeros_like(l[:, 0]), torch.logsumexp(safe, 1))
    Q, N = sum(b > a for a, b in spans), sum(b - a for a, b in spans)
    balance, z, counts, sums = l.sum() * 0 if torch.isfinite(l).all() else 0.0, 0.0, [], []
    for a, b in spans:
        flat = ids[a:b].reshape(-1).long()
        n = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        counts.append(n)
        sums.append(p[a:b].sum(0))
        if b > a:
            balance = balance + (n.double() * sums[-1]).sum() * E / (K * (b - a) ** 2) / Q
            z = z + (lse[a:b] ** 2).sum() / N
    return balance, z, torch.stack(counts), torch.stack(sums), lse


GROUPS = [  # tokens, groups
    (1, None), (7, None), (300, None), (5000, None), (50, [(0, 50)]), (50, [(0, 0), (3, 3), (3, 10), (10, 11), (20, 50), (50, 50)]),
    (900, [(i * 30, i * 30 + i) for i in range(30)]), (40, [(40, 40)]), (0, None), (3000, [(0, 1), (1, 2999), (2999, 3000)]),
    (2000, [(i, i + 1) for i in range(0, 2000, 2)]),
]


def groups(spans, T):
    return (None, None, [(0, T)]) if spans is None else (i32([a for a, _ in spans]), i32([b for _, b in spans]), spans)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(1, 1), (33, 4), (64, 6), (256, 8), (1000, 32)])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_balance_loss(dev, case, E, K, kind):
    T, spans = GROUPS[case]
    begin, end, spans = groups(spans, T)
    for n, dtype in enumerate(DT.values()):
        l = rand(case + n, T, E + 3, dtype=dtype, gain=2.0)[:, 1:E + 1]
        ids = torch.randint(-1, E + 1, (T, K), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(case))
        o = dev.balance_loss(l, ids, begin, end, score=kind)
        again = dev.balance_loss(l, ids, begin, end, score=kind)
        balance, z, counts, sums, lse = losses(l.double(), ids, spans, kind)
        assert torch.equal(o["counts"].long(), counts)
        # parts of at most 304 CTAs, of at most T / (8 * 304) + 1 tokens a warp and 8 warps
        B = rel(l) if T else 0.0
        depth = (T // 2432 + 1 + 8 + 304) * U / 2
        assert ((o["prob_sums"].double() - sums).abs() <= (B + depth) * sums).all()
        assert abs(float(o["loss"][0]) - float(balance)) <= (B + depth + 64 * U) * abs(float(balance))
        top = float(lse.abs().max()) if T else 0.0
        assert abs(float(o["loss"][1]) - float(z)) <= 2 * top * (B + 2.0 ** -21 + top * U) + (depth + 64 * U) * float(z)
        for k in ("loss", "counts", "prob_sums"):
            assert torch.equal(o[k], again[k])  # deterministic
        if begin is not None:
            assert dev.moe_status_sync(o["status"]) == dev.MOE_OK


def test_one_workspace_serves_every_batch(dev):
    """The same workspace, used by larger and smaller calls in turn, on a stream of its own."""
    s = torch.cuda.Stream()
    ws = dev.BalanceWorkspace(256, 8, DEV)
    want = []
    for T, E, Q in [(3000, 256, 8), (5, 17, 1), (900, 64, 3), (3000, 256, 8)]:
        l, ids = rand(T, T, E), torch.randint(0, E, (T, 4), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(T))
        b = i32([q * (T // Q) for q in range(Q)])
        want.append((l, ids, b, b + T // Q, dev.balance_loss(l, ids, b, b + T // Q)))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = [dev.balance_loss(l, ids, b, e, workspace=ws) for l, ids, b, e, _ in want]
    s.synchronize()
    for g, (*_, w) in zip(got, want):
        assert all(torch.equal(g[k], w[k]) for k in ("loss", "counts", "prob_sums"))


@pytest.mark.parametrize("spans", [[(0, 10), (9, 20)], [(0, 41)], [(-1, 5)], [(5, 3)], [(20, 30), (0, 10)], [(0, 10), (30, 20), (25, 40)]])
def test_groups_out_of_order(dev, spans):
    """Groups that share tokens, leave the batch or go backwards: flagged, all empty."""
    T, E, K = 40, 16, 2
    l, ids = rand(1, T, E), torch.zeros(T, K, dtype=torch.int32, device=DEV)
    begin, end, _ = groups(spans, T)
    o = dev.balance_loss(l, ids, begin, end)
    assert dev.moe_status_sync(o["status"]) == dev.MOE_ERR_BAD_LAYOUT
    assert (o["loss"] == 0).all() and (o["counts"] == 0).all() and (o["prob_sums"] == 0).all()
    st = i32([0])
    g = dev.route_grad(l, ids, dloss=torch.ones(2, device=DEV), counts=torch.ones_like(o["counts"]), seq_begin=begin, seq_end=end, status=st)
    assert dev.moe_status_sync(st) == dev.MOE_ERR_BAD_LAYOUT and (g == 0).all()


def test_losses_of_masked_and_dead_rows(dev):
    T, E, K, n = 64, 48, 3, 50
    l = rand(8, T, E)
    l[:, 40:] = -math.inf
    l[3] = -math.inf
    ids = torch.randint(0, 40, (T, K), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(1))
    l[n:] = math.nan  # not live: never read
    for kind in ("softmax", "sigmoid"):
        o = dev.balance_loss(l, ids, score=kind, num_tokens=i32([n]))
        balance, z, counts, sums, _ = losses(l[:n].double(), ids[:n], [(0, n)], kind)
        assert torch.equal(o["counts"].long(), counts)
        assert ((o["prob_sums"].double() - sums).abs() <= (rel(l) + 320 * U) * sums).all()
        assert abs(float(o["loss"][0] - balance)) <= 1e-4 * float(balance) and abs(float(o["loss"][1] - z)) <= 1e-4 * float(z)
        dl = dev.route_grad(l, ids, dweights=torch.ones(T, K, device=DEV), dloss=torch.ones(2, device=DEV), counts=o["counts"],
                            score=kind, renorm=False, num_tokens=i32([n]))
        assert (dl[n:] == 0).all() and torch.isfinite(dl).all() and (dl[:, 40:] == 0).all() and (dl[3] == 0).all()
    l[7, 1] = math.nan
    assert torch.isnan(dev.balance_loss(l[:n], ids[:n])["loss"]).all()


# ---------------------------------------------------------------------------
# Gradients
# ---------------------------------------------------------------------------

def magnitudes(l, ids, dw, dloss, counts, spans, kind, renorm, scale):
    """Sum of the magnitudes of the terms of every gradient, in 64 bits."""
    E, K = l.shape[1], ids.shape[1]
    soft, sg = torch.softmax(l, 1), torch.sigmoid(l)
    p = soft if kind == "softmax" else sg / sg.sum(1, keepdim=True)
    mag = torch.zeros_like(l)
    if dloss is not None:
        Q, N = sum(b > a for a, b in spans), sum(b - a for a, b in spans)
        lse = torch.logsumexp(l, 1, keepdim=True)
        for q, (a, b) in enumerate(spans):
            if b > a:
                g = (dloss[0] * E / (Q * K * (b - a) ** 2)).abs() * counts[q].double()
                mag[a:b] += p[a:b] * (g + (p[a:b] * g).sum(1, keepdim=True)) + (2 * dloss[1] / N).abs() * (lse.abs() + 1)[a:b] * soft[a:b]
    if dw is not None:
        ok = (ids >= 0) & (ids < E)
        at = ids.long().clamp(0, E - 1)
        s = torch.where(ok, (soft if kind == "softmax" else sg).gather(1, at), 0.0)
        u = s / s.sum(1, keepdim=True).clamp_min(1e-300) if renorm else s
        t = scale * u * (dw.double().abs() + (u * dw.double().abs()).sum(1, keepdim=True))
        mag.scatter_add_(1, at, torch.where(ok, t, 0.0))
        if not renorm and kind == "softmax":
            mag += scale * soft * (u * dw.double().abs()).sum(1, keepdim=True)
    return mag


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("parts", ["weights", "losses", "both"])
@pytest.mark.parametrize("case,E,K", [(0, 8, 2), (1, 33, 5), (2, 64, 6), (3, 256, 8), (5, 77, 4), (6, 1024, 32), (7, 16, 2),
                                      (9, 200, 8), (10, 130, 3)])
def test_route_grad(dev, case, E, K, parts, kind, renorm):
    T, spans = GROUPS[case]
    begin, end, spans = groups(spans, T)
    for n, (name, dtype) in enumerate(DT.items()):
        l = rand(case + n, T, E + 3, dtype=dtype, gain=2.0)[:, 1:E + 1]
        ids = choose(l + rand(1, T, E), K, None, "softmax").to(torch.int32).contiguous()
        ids[::3, K - 1] = -1
        dw = rand(11, T, K) if parts != "losses" else None
        dloss = rand(12, 2) if parts != "weights" else None
        counts = dev.balance_loss(l, ids, begin, end, score=kind)["counts"] if dloss is not None else None
        g = dev.route_grad(l, ids, dweights=dw, dloss=dloss, counts=counts, seq_begin=begin, seq_end=end, score=kind, renorm=renorm,
                           scale=1.5)
        leaf = l.double().requires_grad_()
        total = leaf.sum() * 0
        if dw is not None:
            s = torch.where(ids >= 0, score(leaf, kind).gather(1, ids.long().clamp_min(0)), 0.0)
            total = total + 1.5 * ((s / s.sum(1, keepdim=True).clamp_min(1e-300) if renorm else s) * dw).sum()
        if dloss is not None:
            balance, z, *_ = losses(leaf, ids, spans, kind)
            total = total + dloss[0].double() * balance + dloss[1].double() * z
        total.backward()
        mag = magnitudes(l.double(), ids, dw, dloss.double() if dloss is not None else None, counts, spans, kind, renorm, 1.5)
        hs, own = torch.finfo(dtype).eps / 2, 2.0 ** -48 * mag.sum(1, keepdim=True)
        assert ((g.double() - leaf.grad).abs() <= 4 * rel(l) * mag + own + hs * leaf.grad.abs() * (1 + hs) + (2.0 ** -25 if name == "fp16" else 1e-37)).all()


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(dev, kind, renorm):
    """dlogits along random directions against differences of the forward calls. The step h
    leaves an error of h^2 / 6 times the third derivative (the sums' magnitude G at most, as
    scores' derivatives are below 1), and of 2^-22 F / h from F, the forward values' size."""
    T, E, K, h = 24, 40, 4, 2.0 ** -6
    l, dw, dloss = rand(1, T, E), rand(2, T, K, gain=0.3), torch.tensor([0.7, 0.2], device=DEV)
    ids = dev.route(l, K)["topk_ids"]
    counts = dev.balance_loss(l, ids, score=kind)["counts"]
    g = dev.route_grad(l, ids, dweights=dw, dloss=dloss, counts=counts, score=kind, renorm=renorm, scale=2.0).double()

    def value(x):  # the weights of the same choice: a bias that leaves no other
        lone = torch.full_like(x, -math.inf).scatter_(1, ids.long(), x.gather(1, ids.long()))
        if kind == "softmax" and not renorm:
            s = torch.softmax(x.double(), 1).gather(1, ids.long())
            w = 2.0 * s
        else:
            o = dev.route(lone, K, score=kind, renorm=renorm, scale=2.0)
            w = torch.zeros_like(x).scatter_(1, o["topk_ids"].long(), o["topk_weights"]).gather(1, ids.long()).double()
        loss = dev.balance_loss(x, ids, score=kind)["loss"].double()
        return float((w * dw).sum() + (loss * dloss).sum())

    for seed in range(5):
        d = rand(20 + seed, T, E)
        d = d / d.norm()
        diff = (value(l + h * d) - value(l - h * d)) / (2 * h)
        F = float(2 * dw.abs().sum() + 0.7 + 0.2 * 30)
        assert abs(diff - float((g * d).sum())) <= h * h * float(2 * dw.abs().max() + 2) + 64 * U * F / h


def test_gradient_with_an_expert_twice(dev):
    T, E, K = 33, 20, 4
    l, dw = rand(1, T, E), rand(2, T, K)
    ids = torch.randint(0, 4, (T, K), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(3))
    for kind, renorm in [("softmax", True), ("sigmoid", False)]:
        leaf = l.double().requires_grad_()
        s = score(leaf, kind).gather(1, ids.long())
        ((s / s.sum(1, keepdim=True) if renorm else s) * dw).sum().backward()
        g = dev.route_grad(l, ids, dweights=dw, score=kind, renorm=renorm)
        mag = magnitudes(l.double(), ids, dw, None, None, None, kind, renorm, 1.0)
        assert ((g.double() - leaf.grad).abs() <= 4 * rel(l) * mag + 2.0 ** -48 * mag.sum(1, keepdim=True)).all()
        assert torch.equal(g, dev.route_grad(l, ids, dweights=dw, score=kind, renorm=renorm))


def test_many_tokens(dev):
    """More tokens than the grids hold at once."""
    T, E, K = 70001, 64, 4
    l = rand(1, T, E, dtype=torch.bfloat16)
    check_route(dev, l, K, rand(2, E, gain=0.1), "sigmoid", True)
    ids = dev.route(l, K)["topk_ids"]
    dw = rand(3, T, K)
    g = dev.route_grad(l, ids, dweights=dw)
    leaf = l.double().requires_grad_()
    s = torch.softmax(leaf.gather(1, ids.long()), 1)
    (s * dw).sum().backward()
    mag = magnitudes(l.double(), ids, dw, None, None, None, "softmax", True, 1.0)
    assert ((g.double() - leaf.grad).abs() <= 4 * rel(l) * mag + 2.0 ** -48 * mag.sum(1, keepdim=True) + 2.0 ** -8 * leaf.grad.abs()).all()


def test_rows_far_apart(dev):
    """Rows of logits and of the gradient more than 2^31 elements apart."""
    T, E, K, ld = 3, 40, 4, 2 ** 31 + 5
    near = rand(1, T, E + 5, dtype=torch.bfloat16)[:, :E]  # (odd strides both: the same lanes read the same elements)
    l = torch.zeros((T - 1) * ld + E, dtype=torch.bfloat16, device=DEV).as_strided((T, E), (ld, 1))
    l.copy_(near)
    a, b = dev.route(l, K), dev.route(near, K)
    assert torch.equal(a["topk_ids"], b["topk_ids"]) and torch.equal(a["topk_weights"], b["topk_weights"])
    a, b = dev.balance_loss(l, b["topk_ids"]), dev.balance_loss(near, b["topk_ids"])
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["prob_sums"], b["prob_sums"])
    ids, dw, dl = dev.route(near, K)["topk_ids"], rand(2, T, K), torch.ones(2, device=DEV)
    g = [dev.route_grad(t, ids, dweights=dw, dloss=dl, counts=b["counts"]) for t in (l, near)]
    assert torch.equal(*g)


def test_captured_and_replayed(dev):
    """The router's calls in one graph, replayed with other logits, groups and live counts."""
    T, E, K, Q = 256, 64, 4, 3
    l, n, begin, end = rand(1, T, E), i32([T]), i32([0, 100, 100]), i32([100, 100, 256])
    dw, dloss = rand(2, T, K), torch.tensor([1.0, 0.1], device=DEV)
    ws, st = dev.BalanceWorkspace(E, Q, DEV), i32([0])

    def step():
        r = dev.route(l, K, num_tokens=n, status=st)
        b = dev.balance_loss(l, r["topk_ids"], begin, end, num_tokens=n, workspace=ws, status=st)
        g = dev.route_grad(l, r["topk_ids"], dweights=dw, dloss=dloss, counts=b["counts"], seq_begin=begin, seq_end=end,
                           num_tokens=n, status=st)
        return r["topk_ids"], r["topk_weights"], b["loss"], b["counts"], b["prob_sums"], g

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed, live, b, e in [(5, 256, [0, 90, 100], [90, 90, 256]), (6, 120, [10, 50, 110], [50, 100, 120]), (7, 0, [0, 0, 0], [0, 0, 0])]:
        l.copy_(rand(seed, T, E))
        n.fill_(live)
        begin.copy_(i32(b))
        end.copy_(i32(e))
        graph.replay()
        got = [t.clone() for t in out]
        want = step()
        assert torch.equal(got[0][:live], want[0][:live]) and torch.equal(got[1][:live], want[1][:live])
        assert all(torch.equal(x, y) for x, y in zip(got[2:], want[2:]))
        assert dev.moe_status_sync(st) == dev.MOE_OK


# ---------------------------------------------------------------------------
# Rows that are not numbers, and gradients where scores leave the range of a float
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [1, 33, 64, 256])
@pytest.mark.parametrize("row,want", [("nan", math.nan), ("nan and -inf", math.nan), ("inf", math.inf), ("inf and nan", math.nan),
                                      ("one nan", math.nan), ("-inf", None)])
def test_z_loss_of_rows_that_are_not_numbers(dev, row, want, E, kind):
    """The z loss holds what logsumexp of such a row is; a row of -inf alone has no part in it."""
    T, K = 40, 1
    l = rand(1, T, E)
    l[11] = {"nan": math.nan, "nan and -inf": -math.inf, "inf": math.inf, "inf and nan": math.inf, "one nan": 0.0, "-inf": -math.inf}[row]
    if row in ("nan and -inf", "inf and nan", "one nan"):
        l[11, E // 2] = math.nan
    ids = torch.zeros(T, K, dtype=torch.int32, device=DEV)
    got = float(dev.balance_loss(l, ids, score=kind)["loss"][1])
    if want is None:
        z = float((torch.logsumexp(torch.cat([l[:11], l[12:]]).double(), 1) ** 2).sum() / T)
        assert abs(got - z) <= 1e-4 * z  # (the rows' own error; what is tested is which rows count)
    else:
        assert got == want or (math.isnan(got) and math.isnan(want))


def closed(l, ids, dw, dloss, counts, spans, kind, renorm, scale):
    """(gradient, sum of the magnitudes of its terms, what exponentials below 2^-126 may add), in
    64 bits from logarithms of the scores, so that no score leaves the range."""
    E, K = l.shape[1], ids.shape[1]
    soft = kind == "softmax"
    ls = torch.log_softmax(l, 1) if soft else torch.nn.functional.logsigmoid(l)
    rest = torch.ones_like(l) if soft else torch.sigmoid(-l)
    p, sm, lse = torch.softmax(ls, 1), torch.softmax(l, 1), torch.logsumexp(l, 1, keepdim=True)
    # sums of scores are at least the largest one's: a sigmoid where that is above e^-20, else 1
    lost = lambda top: 2.0 ** -126 / torch.where((top >= -20) & (not soft), torch.sigmoid(top), 1.0)
    g, mag, low = torch.zeros_like(l), torch.zeros_like(l), torch.zeros_like(l)
    if dloss is not None:
        Q, N = sum(b > a for a, b in spans), sum(b - a for a, b in spans)
        f = lost(l.max(1, keepdim=True).values)
        for q, (a, b) in enumerate(spans):
            if b > a:
                c = dloss[0] * E / (Q * K * (b - a) ** 2) * counts[q].double()
                P, r = p[a:b], rest[a:b]
                g[a:b] += P * (c - (P * c).sum(1, keepdim=True)) * r + 2 * dloss[1] / N * lse[a:b] * sm[a:b]
                mag[a:b] += P * (c.abs() + (P * c.abs()).sum(1, keepdim=True)) * r + (2 * dloss[1] / N).abs() * (lse.abs() + 1)[a:b] * sm[a:b]
                low[a:b] += 4 * E * f[a:b] * c.abs().max() + 2.0 ** -126 * (2 * dloss[1] / N).abs() * (lse.abs() + 1)[a:b]
    if dw is not None:
        at = ids.long()
        a, r, d = ls.gather(1, at), rest.gather(1, at), dw.double()
        u = torch.softmax(a, 1) if renorm else a.exp()
        f = 4 * K * scale * (lost(l.gather(1, at).max(1, keepdim=True).values) if renorm else 2.0 ** -126) * d.abs().max(1, keepdim=True).values
        if renorm:
            t, m = scale * u * (d - (u * d).sum(1, keepdim=True)) * r, scale * u * (d.abs() + (u * d.abs()).sum(1, keepdim=True)) * r
        else:
            t, m = scale * u * d * r, scale * u * d.abs() * r
        g.scatter_add_(1, at, t)
        mag.scatter_add_(1, at, m)
        low += f
        if soft and not renorm:
            g -= scale * p * (u * d).sum(1, keepdim=True)
            mag += scale * p * (u * d.abs()).sum(1, keepdim=True)
    return g, mag, low


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("shift", [-200.0, -80.0, -61.0, -60.0, -59.0, -21.0, -20.0, -19.0, 80.0])
@pytest.mark.parametrize("parts", ["weights", "losses"])
def test_gradient_of_far_logits(dev, parts, shift, kind, renorm):
    """Every logit far from zero, only the chosen ones, or only the others: losses and gradients
    where sigmoids become exponentials, on both sides of that border."""
    T, E, K = 60, 48, 4
    l = rand(5, T, E, gain=2.0)
    ids = choose(rand(6, T, E), K, None, "softmax").to(torch.int32).contiguous()
    chosen = torch.zeros(T, E, dtype=torch.bool, device=DEV).scatter_(1, ids.long(), True)
    moved = torch.ones(T, E, dtype=torch.bool, device=DEV)
    moved[20:40], moved[40:] = chosen[20:40], ~chosen[40:]
    l = torch.where(moved, l + shift, l).contiguous()
    spans = [(0, 10), (10, 33), (33, 60)]
    begin, end = i32([a for a, _ in spans]), i32([b for _, b in spans])
    d = l.double()
    o = dev.balance_loss(l, ids, begin, end, score=kind)
    balance, z, counts, sums, lse = losses(d, ids, spans, kind)
    B, depth = rel(l), 320 * U
    assert torch.equal(o["counts"].long(), counts)
    assert ((o["prob_sums"].double() - sums).abs() <= (B + depth) * sums + T * 2.0 ** -126 / 2.0 ** -29).all()  # (e^-20 > 2^-29)
    assert abs(float(o["loss"][0] - balance)) <= (B + depth + 64 * U) * float(balance) + 2.0 ** -30
    top = float(lse.abs().max())
    assert abs(float(o["loss"][1] - z)) <= 2 * top * (B + 2.0 ** -21 + top * U) + (depth + 64 * U) * float(z)
    dw = rand(11, T, K) if parts == "weights" else None
    dloss = torch.tensor([30.0, 0.5], device=DEV) if parts == "losses" else None
    g = dev.route_grad(l, ids, dweights=dw, dloss=dloss, counts=o["counts"] if dloss is not None else None, seq_begin=begin, seq_end=end,
                       score=kind, renorm=renorm, scale=1.5)
    want, mag, low = closed(d, ids, dw, None if dloss is None else dloss.double(), counts, spans, kind, renorm, 1.5)
    own = 2.0 ** -48 * mag.sum(1, keepdim=True)
    assert ((g.double() - want).abs() <= 4 * B * mag + own + low + 1e-37).all()
    if parts == "losses":  # the balance loss alone: the z loss's gradient is far larger where logits are
        dloss = torch.tensor([30.0, 0.0], device=DEV)
        g = dev.route_grad(l, ids, dloss=dloss, counts=o["counts"], seq_begin=begin, seq_end=end, score=kind, renorm=renorm)
        want, mag, low = closed(d, ids, None, dloss.double(), counts, spans, kind, renorm, 1.0)
        assert ((g.double() - want).abs() <= 4 * B * mag + 2.0 ** -48 * mag.sum(1, keepdim=True) + low + 1e-37).all()


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("part", ["weights", "balance", "z"])
def test_each_gradient_against_differences(dev, part, kind, renorm):
    """Every part of the gradient alone, along itself, against differences of the forward calls.

    With d the unit vector along the gradient, the difference over a step h is |g| but for three
    errors: what the step cuts off (taken from the formulas in 64 bits, with the same d and h), the
    forward values' rounding over h, and the gradient's own rounding. Together they may be a
    twentieth of |g| at most, so that a gradient of zero, of half its size or of the other sign
    fails."""
    T, E, K, h, scale = 8, 16, 4, 0.5, 2.0
    l, dw = rand(1, T, E), rand(2, T, K)
    cols = torch.tensor([3, 7, 8, 14], device=DEV)
    bias = torch.zeros(E, device=DEV).index_fill_(0, cols, 10.0)  # chooses these whatever the logits
    ids = cols.to(torch.int32).repeat(T, 1).contiguous()
    picked = torch.randint(0, E, (T, K), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(3))  # of the losses
    counts = dev.balance_loss(l, picked, score=kind)["counts"]
    c = {"weights": [0.0, 0.0], "balance": [1.0, 0.0], "z": [0.0, 1.0]}[part]
    args = dict(dweights=dw) if part == "weights" else dict(dloss=torch.tensor(c, device=DEV), counts=counts)
    g = dev.route_grad(l, ids if part == "weights" else picked, score=kind, renorm=renorm, scale=scale, **args).double()
    size = float(g.norm())
    d = g / size

    def forward(x):  # the calls' value, and a bound on its rounding
        if part == "weights":
            o = dev.route(x, K, bias=bias, score=kind, renorm=renorm, scale=scale)
            assert torch.equal(o["topk_ids"].sort(1).values, ids)
            w = torch.zeros(T, E, device=DEV).scatter_(1, o["topk_ids"].long(), o["topk_weights"])[:, cols].double()
            return float((w * dw).sum()), rel(x) * float((w * dw).abs().sum())
        o = dev.balance_loss(x, picked, score=kind)["loss"]
        depth, top = (1 + 8 + 304) * U / 2, float(torch.logsumexp(x.double(), 1).abs().max())
        if part == "balance":
            return float(o[0]), (rel(x) + depth + 64 * U) * float(o[0])
        return float(o[1]), 2 * top * (rel(x) + 2.0 ** -21 + top * U) + (depth + 64 * U) * float(o[1])

    def formula(x):
        if part == "weights":
            s = score(x, kind)[:, cols]
            return (scale * (s / s.sum(1, keepdim=True) if renorm else s) * dw.double()).sum()
        return losses(x, picked, [(0, T)], kind)[0 if part == "balance" else 1]

    x0, x1 = (l.double() - h * d).float(), (l.double() + h * d).float()
    moved = x1.double() - x0.double()  # the step as it is after its rounding
    leaf = l.double().requires_grad_()
    slope, = torch.autograd.grad(formula(leaf), leaf)
    along = float((slope * moved).sum())
    cut = abs(float(formula(x1.double()) - formula(x0.double())) - along)
    (f0, e0), (f1, e1) = forward(x0), forward(x1)
    mag = magnitudes(l.double(), ids if part == "weights" else picked, dw if part == "weights" else None,
                     None if part == "weights" else torch.tensor(c, device=DEV, dtype=torch.float64), counts, [(0, T)], kind, renorm, scale)
    tol = cut + e0 + e1 + float((4 * rel(l) * mag * moved.abs()).sum())
    assert tol <= 0.05 * 2 * h * size
    assert abs((f1 - f0) - float((g * moved).sum())) <= tol


@pytest.mark.parametrize("top", [-100.0, -61.0, -59.0, -40.0, -21.0, -20.5, -20.0, -19.5, -5.0])
def test_sigmoid_ratios_of_spread_logits(dev, top):
    """Renormalised sigmoids far below zero and far apart: every ratio above 2^-126 e^20 is there, in the
    weights, their gradient, the probabilities and theirs."""
    T, E, K = 30, 40, 6
    l = top - rand(1, T, E).abs() * 15.0
    l[:, 7] = top
    o = dev.route(l, K, score="sigmoid", scale=2.0)
    ids = choose(l, K, None, "sigmoid")
    assert torch.equal(o["topk_ids"].long(), ids)
    low = 2.0 ** -126 * math.exp(20.0)
    d = torch.nn.functional.logsigmoid(l.double())
    want = 2.0 * torch.softmax(d.gather(1, ids), 1)
    assert ((o["topk_weights"].double() - want).abs() <= rel(l) * want + 2.0 * low).all()
    p, b = torch.softmax(d, 1).sum(0), dev.balance_loss(l, o["topk_ids"], score="sigmoid")
    assert ((b["prob_sums"][0].double() - p).abs() <= (rel(l) + 320 * U) * p + T * low).all()
    dw, dloss = rand(3, T, K), torch.tensor([30.0, 0.0], device=DEV)
    for kw in (dict(dweights=dw), dict(dloss=dloss, counts=b["counts"])):
        g = dev.route_grad(l, o["topk_ids"], score="sigmoid", scale=2.0, **kw)
        want, mag, less = closed(l.double(), o["topk_ids"], kw.get("dweights"), dloss.double() if "dloss" in kw else None, b["counts"], [(0, T)],
                                 "sigmoid", True, 2.0)
        assert ((g.double() - want).abs() <= 4 * rel(l) * mag + 2.0 ** -48 * mag.sum(1, keepdim=True) + less + 1e-37).all()
