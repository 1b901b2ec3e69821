"""Cases of the MoE-block operators: what each reads and computes, in plain torch and through the package.

Four groups of calls, as one MoE block makes them:
  permute / permute_grad / combine_grad   tokens sorted by expert and back, and the gradients of both
  expert_matmul / expert_matmul_grad      the experts' product with bias, activation, gate and residual
  block_norm / block_norm_grad            the norms before and after the block, with gate and residual scale

With ``own`` false, ``run`` computes an operator from elementary torch operations in 32 bits; with
``own`` true it makes the package's calls. Buffers that an operator leaves unwritten in part (padding
rows) are zeroed once when the state is made, so whole outputs can be compared.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode batch on one of eight ranks: 32 of 256 experts are local; launch latency counts
        dict(name="permute_decode", op="permute", T=128, H=7168, E=256, L=32, topk=8, block=128, skew=0.0, dtype="bf16"),
        # a prefill batch with every expert local and the skew of real routers; bandwidth counts
        dict(name="permute_prefill", op="permute", T=8192, H=7168, E=256, L=256, topk=8, block=128, skew=1.2, dtype="bf16"),
        # gradient of the way back in fp32: odd token count, top-6, segments of 16 rows
        dict(name="back_grad_fp32", op="sort_grad", T=1777, H=2048, E=64, L=64, topk=6, block=16, skew=0.7, dtype="fp32"),
        # gradients of the way there and back in a training step of a prefill-sized batch
        dict(name="back_grad_train", op="sort_grad", T=8192, H=7168, E=256, L=256, topk=8, block=128, skew=1.2, dtype="bf16"),
        # one token through a dense output projection with bias and residual: weights are all the traffic
        dict(name="dense_one_token", op="matmul", T=1, E=1, L=1, topk=1, block=1, K=2048, N=7168, act="none", gated=False,
             bias=True, residual=True, dtype="bf16"),
        # decode on one rank, e4m3 rows and weights as the dispatch writes them: a few rows per expert
        dict(name="experts_decode_fp8", op="matmul", T=128, E=256, L=32, topk=8, block=128, K=7168, N=2048, act="silu",
             gated=True, bias=False, residual=False, dtype="e4m3"),
        # prefill over 64 experts in e4m3: the tensor cores count
        dict(name="experts_prefill_fp8", op="matmul", T=4096, E=64, L=64, topk=8, block=128, K=7168, N=2048, act="silu",
             gated=True, bias=False, residual=False, dtype="e4m3"),
        # a training step's first product: bias, gated activation, pre-activations kept; ragged segments
        dict(name="experts_train", op="matmul", T=8191, E=16, L=16, topk=2, block=8, K=2048, N=1408, act="silu",
             gated=True, bias=True, residual=False, dtype="bf16"),
        # its gradients: rows, weights and bias
        dict(name="experts_train_grad", op="matmul_grad", T=8191, E=16, L=16, topk=2, block=8, K=2048, N=1408, act="silu",
             gated=True, bias=True, residual=False, dtype="bf16"),
        # one token between two blocks while decoding
        dict(name="norm_one_token", op="norm", T=1, H=7168, gate="channel", post=True, pre=True, scale=0.5, dtype="bf16"),
        # the same for a prefill batch, with a gate per token
        dict(name="norm_prefill", op="norm", T=8192, H=7168, gate="token", post=True, pre=True, scale=1.0, dtype="bf16"),
        # the gradients of a training step, with a gate per channel
        dict(name="norm_train_grad", op="norm_grad", T=8192, H=7168, gate="channel", post=True, pre=True, scale=0.25,
             dtype="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A size in [lo, hi], spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(max(round(v / step) * step, lo), hi))


def draw(rng):
    while True:
        op = rng.choice(["permute", "sort_grad", "matmul", "matmul", "matmul_grad", "norm", "norm_grad"])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if op in ("permute", "sort_grad"):
            E = _spread(rng, 1, 256)
            c = dict(op=op, T=_spread(rng, 1, 8192), H=_spread(rng, 64, 7168, 8), E=E, L=rng.choice([E, E, max(1, E // 8)]),
                     topk=min(E, rng.randint(1, 8)), block=rng.choice([1, 8, 16, 64, 128]), skew=rng.choice([0.0, 0.7, 1.2]),
                     dtype=dtype)
        elif op in ("matmul", "matmul_grad"):
            E = rng.choice([1, _spread(rng, 1, 64), _spread(rng, 8, 256)])
            dtype = rng.choice(["bf16", "fp16", "e4m3"]) if op == "matmul" else rng.choice(["bf16", "fp16"])
            K = _spread(rng, 128, 7168, 128) if dtype == "e4m3" else _spread(rng, 64, 7168, 8)
            gated = rng.random() < 0.5
            c = dict(op=op, T=_spread(rng, 1, 8192), E=E, L=rng.choice([E, max(1, E // 8)]), topk=min(E, rng.choice([1, 2, 8])),
                     block=rng.choice([1, 8, 16, 128]), K=K, N=_spread(rng, 64, 2048 if gated else 7168, 16), gated=gated,
                     act=rng.choice(["silu", "gelu", "relu"] if gated else ["none", "silu", "gelu", "relu"]),
                     bias=rng.random() < 0.5, residual=rng.random() < 0.4 and op == "matmul", dtype=dtype)
        else:
            post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
            c = dict(op=op, T=_spread(rng, 1, 8192), H=_spread(rng, 64, 7168, 8), gate=rng.choice(["none", "channel", "token"]),
                     post=post, pre=pre, scale=rng.choice([1.0, 0.5, 0.2]), dtype=dtype)
        w = work(c)
        if w["flops"] > 1.9e12 or w["bytes"] > 2.0e9:
            continue
        if 3072 not in (c.get("H"), c.get("K"), c.get("N"), 2 * c.get("N", 0), c["T"], c["T"] * c.get("topk", 1)):
            return c


def _rows(c):
    """Expected kept slots of a case."""
    return max(1.0, c["T"] * c["topk"] * c["L"] / c["E"])


def _elem(c):
    return {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}[c["dtype"]]


def work(c):
    op, T, es = c["op"], c["T"], _elem(c)
    if op == "permute":
        A, row = _rows(c), c["H"] * es
        return {"bytes": int(T * row + A * row + 12 * T * c["topk"] + 8 * A), "flops": 0}
    if op == "sort_grad":  # reads dout, y and the gradient of the sorted rows; writes dy, dweights, dx
        A, row = _rows(c), c["H"] * es
        return {"bytes": int(2 * T * row + 3 * A * row + 12 * T * c["topk"]), "flops": int(4 * A * c["H"])}
    if op in ("matmul", "matmul_grad"):
        A, K, N = _rows(c), c["K"], c["N"]
        Nw = 2 * N if c["gated"] else N
        active = c["L"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** T) if c["topk"] < c["E"] else c["L"]
        wbytes = max(1.0, active) * Nw * K * es
        if op == "matmul":
            out = A * N * 2 * (2 if c["residual"] else 1)
            keep = A * Nw * 2 if _keeps(c) else 0
            return {"bytes": int(wbytes + A * K * es + out + keep), "flops": int(2 * A * Nw * K)}
        return {"bytes": int(wbytes + c["L"] * Nw * K * es + 2 * A * K * es + A * (N + Nw) * es), "flops": int(4 * A * Nw * K)}
    H = c["H"]
    if op == "norm":
        return {"bytes": int(T * H * es * (1 + (2 if c["post"] else 0) + (1 if c["pre"] else 0)) + 8 * T), "flops": int(10 * T * H)}
    n = 2 + (2 if c["post"] else 0) + (2 if c["pre"] else 0)
    return {"bytes": int(T * H * es * n + 8 * T), "flops": int(20 * T * H)}


def _keeps(c):
    """Whether the pre-activations are kept for a backward pass."""
    return c["dtype"] != "e4m3" and c["act"] != "none" and c["T"] > 64


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, gain=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * gain).to(dtype)


def _routing(c, g, skew=0.0):
    """topk distinct experts per token by Gumbel top-k over a popularity of rank^-skew, and softmax weights."""
    T, E, k = c["T"], c["E"], c["topk"]
    pop = -skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    pop = pop[torch.randperm(E, device="cuda", generator=g)]
    u = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-20, 1.0 - 1e-7)
    ids = (pop - torch.log(-torch.log(u))).topk(k, dim=1).indices.to(torch.int32).contiguous()
    w = torch.softmax(_randn(g, T, k), dim=1)
    return ids, w.contiguous()


def _bound(A, L, b):
    n = min(A, L)
    return b * (n + (A - n) // b)


def _layout(ids, L, b):
    """counts, starts, psum [L] of the compact layout and the row of every slot (-1 when not local)."""
    flat = ids.reshape(-1).to(torch.int64)
    local = (flat >= 0) & (flat < L)
    key = torch.where(local, flat, torch.full_like(flat, L))
    counts = (key[:, None] == torch.arange(L, device=key.device)[None, :]).sum(0)
    aligned = (counts + b - 1) // b * b
    starts = torch.cumsum(aligned, 0) - aligned
    order = torch.sort(key, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    first = torch.cat([first, counts.sum()[None]])
    starts1 = torch.cat([starts, torch.zeros_like(starts[:1])])
    skey = key[order]
    rank = torch.arange(flat.numel(), device=key.device) - first[skey]
    row = torch.empty_like(flat)
    row[order] = torch.where(skey < L, starts1[skey] + rank, torch.full_like(skey, -1))
    return counts, starts, starts + counts, aligned.sum(), row.reshape(ids.shape)


def _quant(x):
    """Rows in e4m3 with one power-of-two scale per 128 elements: (codes, exponents)."""
    R, K = x.shape
    v = x.reshape(R, K // 128, 128)
    m, e = torch.frexp(v.abs().amax(2).clamp_min(1e-10))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    q = (v * torch.exp2(-e.float())[:, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(R, K), e


def _pack(e):
    """Exponents [R, G] as packed scale words [G4, R rounded up to 4], four groups in a word."""
    R, G = e.shape
    G4, ld = (G + 3) // 4, (R + 3) // 4 * 4
    b = torch.zeros(ld, G4 * 4, dtype=torch.uint8, device=e.device)
    b[:R, :G] = (e + 127).to(torch.uint8)
    return b.view(torch.int32).t().contiguous(), ld


def _weights(c, g):
    """The experts' weights [L, Nw, K], made expert by expert: (tensor, packed scales, exponents, ld)."""
    L, K, Nw = c["L"], c["K"], c["N"] * (2 if c["gated"] else 1)
    if c["dtype"] != "e4m3":
        w = torch.empty(L, Nw, K, device="cuda", dtype=DT[c["dtype"]])
        for e in range(L):
            w[e] = _randn(g, Nw, K, gain=K ** -0.5)
        return w, None, None, 0
    w = torch.empty(L, Nw, K, device="cuda", dtype=torch.float8_e4m3fn)
    ex = torch.empty(L, Nw, K // 128, device="cuda", dtype=torch.int32)
    for e in range(L):
        w[e], ex[e] = _quant(_randn(g, Nw, K, gain=K ** -0.5))
    sc, ld = _pack(ex.reshape(L * Nw, -1))
    return w, sc, ex, ld


def prepare(c, seed):
    g, op, dev = _gen(seed), c["op"], "cuda"
    s = {"case": dict(c)}
    if op == "permute":
        dt = DT[c["dtype"]]
        s["x"] = _randn(g, c["T"], c["H"], dtype=dt)
        s["ids"], s["w"] = _routing(c, g, c["skew"])
        R = _bound(c["T"] * c["topk"], c["L"], c["block"])
        s["R"], s["xs"] = R, torch.zeros(R, c["H"], device=dev, dtype=dt)
        s["rw"] = torch.zeros(R, device=dev)
        if own:
            import combine_fp8_quant_gb300 as mp
            s["ws"] = mp.Workspace(c["T"], c["topk"], c["L"], dev)
            s["st"] = torch.zeros(1, dtype=torch.int32, device=dev)
    elif op == "sort_grad":
        dt = DT[c["dtype"]]
        ids, s["w"] = _routing(c, g, c["skew"])
        s["R"] = R = max(1, _bound(c["T"] * c["topk"], c["L"], c["block"]))
        s["s2d"] = _layout(ids, c["L"], c["block"])[4].to(torch.int32)
        s["dout"] = _randn(g, c["T"], c["H"], dtype=dt)
        s["y"] = _randn(g, R, c["H"], dtype=dt)
        s["dxs"] = _randn(g, R, c["H"], dtype=dt)
        s["dy"] = torch.zeros(R, c["H"], device=dev, dtype=dt)
        if own:
            s["st"] = torch.zeros(1, dtype=torch.int32, device=dev)
    elif op in ("matmul", "matmul_grad"):
        T, L, K, N, b = c["T"], c["L"], c["K"], c["N"], c["block"]
        Nw = 2 * N if c["gated"] else N
        dt = torch.bfloat16 if c["dtype"] == "e4m3" else DT[c["dtype"]]
        if c["E"] == 1:  # dense: every row is the one expert's
            R, s["starts"], s["psum"], s["seg"] = T, None, None, [(0, T)]
        else:
            counts, starts, psum, _, _ = _layout(_routing(c, g)[0], L, b)
            R = max(1, _bound(T * c["topk"], L, b))
            s["starts"], s["psum"] = starts.to(torch.int32), psum.to(torch.int32)
            s["seg"] = list(zip(starts.tolist(), psum.tolist()))  # the host's copy of the plan
        real = torch.zeros(R, dtype=torch.bool, device=dev)
        for lo, hi in s["seg"]:
            real[lo:hi] = True
        x = _randn(g, R, K)
        if c["dtype"] == "e4m3":
            q, s["xe"] = _quant(x)
            q.view(torch.uint8)[~real] = 0x7F  # padding rows hold whatever was there: NaN here
            s["x"], (s["xsc"], s["ldx"]) = q, _pack(s["xe"])
        else:
            s["x"] = x.to(dt).masked_fill_(~real[:, None], float("nan"))
        s["wt"], s["wsc"], s["we"], s["ldw"] = _weights(c, g)
        s["bias"] = _randn(g, L, Nw) if c["bias"] else None
        s["res"] = _randn(g, R, N, dtype=dt) if c["residual"] else None
        s["out"] = torch.zeros(R, N, device=dev, dtype=dt)
        s["pre"] = torch.zeros(R, Nw, device=dev, dtype=dt) if op == "matmul" and _keeps(c) else None
        if op == "matmul_grad":
            s["dout"] = _randn(g, R, N, dtype=dt).masked_fill_(~real[:, None], float("nan"))
            s["pre"] = _randn(g, R, Nw, dtype=dt).masked_fill_(~real[:, None], float("nan")) if c["act"] != "none" else None
            s["dx"] = torch.zeros(R, K, device=dev, dtype=dt)
            s["dw"] = torch.zeros(L, Nw, K, device=dev, dtype=dt)
            s["db"] = torch.zeros(L, Nw, device=dev)
        if own:
            s["st"] = torch.zeros(1, dtype=torch.int32, device=dev)
            if op == "matmul_grad":
                import combine_fp8_quant_gb300 as mp
                s["ws"] = mp.GradWorkspace(R, L, Nw, dt, dev)
    else:
        T, H, dt = c["T"], c["H"], DT[c["dtype"]]
        s["x"] = _randn(g, T, H, dtype=dt, gain=2.0)  # the residual stream (after the sum, for the gradient)
        s["y"] = _randn(g, T, H, dtype=dt, gain=0.5) if c["post"] else None
        s["wpost"] = 1.0 + _randn(g, H, gain=0.2) if c["post"] else None
        s["wpre"] = 1.0 + _randn(g, H, gain=0.2) if c["pre"] else None
        s["gate"] = None
        if c["post"] and c["gate"] != "none":
            s["gate"] = torch.sigmoid(_randn(g, H if c["gate"] == "channel" else T))
        if op == "norm_grad":
            s["dxo"] = _randn(g, T, H, dtype=dt)
            s["dh"] = _randn(g, T, H, dtype=dt) if c["pre"] else None
            f = s["x"].float()
            s["rx"] = torch.rsqrt((f * f).mean(1) + EPS) if c["pre"] else None
            f = s["y"].float() if c["post"] else None
            s["ry"] = torch.rsqrt((f * f).mean(1) + EPS) if c["post"] else None
            if own:
                import combine_fp8_quant_gb300 as mp
                s["ws"] = mp.NormWorkspace(T, H, dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import combine_fp8_quant_gb300 as mp
        return {"permute": _own_permute, "sort_grad": _own_sort_grad, "matmul": _own_matmul,
                "matmul_grad": _own_matmul_grad, "norm": _own_norm, "norm_grad": _own_norm_grad}[op](mp, s, s["case"])
    return {"permute": _permute, "sort_grad": _sort_grad, "matmul": _matmul, "matmul_grad": _matmul_grad,
            "norm": _norm, "norm_grad": _norm_grad}[op](s, s["case"])


def _own_permute(mp, s, c):
    o = mp.permute(s["x"], s["ids"], s["w"], c["E"], c["L"], block_e=c["block"], workspace=s["ws"], status=s["st"],
                   out=s["xs"], row_weights=s["rw"])
    return {k: o[k] for k in ("xs", "row_weights", "m_indices", "src2dst", "counts", "starts", "psum", "total")}


def _own_sort_grad(mp, s, c):
    o = mp.combine_grad(s["dout"], s["y"], s["s2d"], s["w"], status=s["st"], dy=s["dy"])
    dx = mp.permute_grad(s["dxs"], s["s2d"], status=s["st"])
    return {"dy": o["dy"], "dw": o["dweights"], "dx": dx}


def _own_matmul(mp, s, c):
    out = mp.expert_matmul(s["x"], s["wt"], s["starts"], s["psum"], bias=s["bias"], act=c["act"], gated=c["gated"],
                           residual=s["res"], x_scales=s.get("xsc"), ld_xs=s.get("ldx", 0), w_scales=s["wsc"],
                           ld_ws=s["ldw"], out=s["out"], pre=s["pre"], status=s["st"])
    return {"out": out, "pre": s["pre"]}


def _own_matmul_grad(mp, s, c):
    o = mp.expert_matmul_grad(s["dout"], s["x"], s["wt"], s["starts"], s["psum"], pre=s["pre"], act=c["act"],
                              gated=c["gated"], dx=s["dx"], dw=s["dw"], dbias=s["db"] if c["bias"] else None,
                              workspace=s["ws"], status=s["st"])
    return {"dx": o["dx"], "dw": o["dw"], "db": o["dbias"]}


def _own_norm(mp, s, c):
    o = mp.block_norm(s["x"], s["y"], w_post=s["wpost"], gate=s["gate"], scale=c["scale"], w_pre=s["wpre"], eps=EPS)
    return {"x": o["x"] if c["post"] else None, "h": o["h"]}


def _own_norm_grad(mp, s, c):
    o = mp.block_norm_grad(s["dxo"], s["dh"], s["x"], s["y"], w_post=s["wpost"], gate=s["gate"], scale=c["scale"],
                           w_pre=s["wpre"], rstd_pre=s["rx"], rstd_post=s["ry"], workspace=s["ws"])
    return {k: o[k] for k in ("dx", "dy", "dw_pre", "dw_post", "dgate")}


def _permute(s, c):
    counts, starts, psum, total, row = _layout(s["ids"], c["L"], c["block"])
    R, T, k = s["R"], c["T"], c["topk"]
    flat = row.reshape(-1)
    dst = torch.where(flat >= 0, flat, torch.full_like(flat, R))
    src = torch.arange(T, device=flat.device).repeat_interleave(k)
    xs = torch.zeros(R + 1, c["H"], device=flat.device, dtype=s["x"].dtype)
    xs[dst] = s["x"][src]
    rw = torch.zeros(R + 1, device=flat.device)
    rw[dst] = s["w"].reshape(-1)
    mi = torch.full((R + 1,), -1, dtype=torch.int32, device=flat.device)
    mi[dst] = s["ids"].reshape(-1)
    i32 = torch.int32
    return {"xs": xs[:R], "row_weights": rw[:R], "m_indices": mi[:R], "src2dst": row.to(i32), "counts": counts.to(i32),
            "starts": starts.to(i32), "psum": psum.to(i32), "total": total.to(i32)[None]}


def _sort_grad(s, c):
    R, k = s["R"], c["topk"]
    row = s["s2d"].to(torch.int64)
    kept = row >= 0
    at = row.clamp_min(0)
    g = s["dout"].float()
    dy = torch.zeros(R + 1, c["H"], device=g.device)
    dw = torch.zeros_like(s["w"])
    dx = torch.zeros_like(g)
    for j in range(k):
        m = kept[:, j, None]
        dy[torch.where(kept[:, j], at[:, j], torch.full_like(at[:, j], R))] = s["w"][:, j, None] * g
        dw[:, j] = torch.where(m, s["y"][at[:, j]].float() * g, torch.zeros_like(g)).sum(1)
        dx = dx + torch.where(m, s["dxs"][at[:, j]].float(), torch.zeros_like(g))
    return {"dy": dy[:R].to(s["y"].dtype), "dw": dw, "dx": dx.to(s["y"].dtype)}


def _act(name, v):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    return v


def _dact(name, v):
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "relu":
        return torch.where(v > 0, torch.ones_like(v), torch.zeros_like(v))
    return torch.ones_like(v)


def _wide(q, e, dt):
    """Values of e4m3 codes with an exponent per 128 elements."""
    v = q.to(dt).reshape(*q.shape[:-1], q.shape[-1] // 128, 128)
    return (v * torch.exp2(e.to(dt))[..., None]).reshape(q.shape)


def _matmul(s, c, dt=torch.float32):
    out = torch.zeros_like(s["out"], dtype=dt)
    pre = torch.zeros_like(s["pre"], dtype=dt) if s["pre"] is not None else None
    N = c["N"]
    for e, (lo, hi) in enumerate(s["seg"]):
        if hi <= lo:
            continue
        if c["dtype"] == "e4m3":
            p = _wide(s["x"][lo:hi], s["xe"][lo:hi], dt) @ _wide(s["wt"][e], s["we"][e], dt).t()
        else:
            p = s["x"][lo:hi].to(dt) @ s["wt"][e].to(dt).t()
        if s["bias"] is not None:
            p = p + s["bias"][e].to(dt)
        if pre is not None:
            pre[lo:hi] = p
        v = _act(c["act"], p[:, :N]) * p[:, N:] if c["gated"] else _act(c["act"], p)
        out[lo:hi] = v + s["res"][lo:hi].to(dt) if s["res"] is not None else v
    if dt == torch.float64:
        return {"out": out, "pre": pre}
    return {"out": out.to(s["out"].dtype), "pre": None if pre is None else pre.to(s["out"].dtype)}


def _matmul_grad(s, c):
    N = c["N"]
    dx = torch.zeros(s["x"].shape, device="cuda")
    dw = torch.zeros(s["wt"].shape, device="cuda")
    db = torch.zeros(s["db"].shape, device="cuda")
    for e, (lo, hi) in enumerate(s["seg"]):
        if hi <= lo:
            continue
        g = s["dout"][lo:hi].float()
        if c["act"] != "none" or c["gated"]:
            p = s["pre"][lo:hi].float()
            if c["gated"]:
                g = torch.cat([g * p[:, N:] * _dact(c["act"], p[:, :N]), g * _act(c["act"], p[:, :N])], dim=1)
            else:
                g = g * _dact(c["act"], p)
        dx[lo:hi] = g @ s["wt"][e].float()
        dw[e] = g.t() @ s["x"][lo:hi].float()
        db[e] = g.sum(0)
    dt = s["x"].dtype
    return {"dx": dx.to(dt), "dw": dw.to(dt), "db": db if c["bias"] else None}


def _norm(s, c):
    x = s["x"].float()
    h = None
    if c["post"]:
        y = s["y"].float()
        n = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["wpost"]
        if s["gate"] is not None:
            n = n * (s["gate"][:, None] if c["gate"] == "token" else s["gate"])
        x = x + c["scale"] * n
    if c["pre"]:
        h = (x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["wpre"]).to(s["x"].dtype)
    return {"x": x.to(s["x"].dtype) if c["post"] else None, "h": h}


def _norm_grad(s, c):
    dt = s["x"].dtype
    g = s["dxo"].float()
    dwpre = dwpost = dgate = dy = None
    if c["pre"]:
        xh = s["x"].float() * s["rx"][:, None]
        dh = s["dh"].float()
        t = dh * s["wpre"]
        g = g + s["rx"][:, None] * (t - xh * (t * xh).mean(1, keepdim=True))
        dwpre = (dh * xh).sum(0)
    if c["post"]:
        yh = s["y"].float() * s["ry"][:, None]
        u = c["scale"] * g
        if s["gate"] is not None:
            un = u * yh * s["wpost"]
            dgate = un.sum(1) if c["gate"] == "token" else un.sum(0)
            u = u * (s["gate"][:, None] if c["gate"] == "token" else s["gate"])
        dwpost = (u * yh).sum(0)
        t = u * s["wpost"]
        dy = (s["ry"][:, None] * (t - yh * (t * yh).mean(1, keepdim=True))).to(dt)
    return {"dx": g.to(dt), "dy": dy, "dw_pre": dwpre, "dw_post": dwpost, "dgate": dgate}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s, op = prepare(c, seed), c["op"]
    if op == "permute":
        return _exact_permute(s, c)
    if op == "sort_grad":
        return _exact_sort_grad(s, c)
    if op == "matmul":
        return _exact_matmul(s, c)
    if op == "matmul_grad":
        return _exact_matmul_grad(s, c)
    return _exact_norm(s, c) if op == "norm" else _exact_norm_grad(s, c)


def _exact_permute(s, c):
    """Expert by expert on the host: the slots of an expert in ascending order fill its segment."""
    ids = s["ids"].cpu().numpy()
    flat, k, b, R, L = ids.reshape(-1), c["topk"], c["block"], s["R"], c["L"]
    row = np.full(flat.size, -1, np.int32)
    token, mi = np.full(R, -1, np.int64), np.full(R, -1, np.int32)
    counts, starts = np.zeros(L, np.int32), np.zeros(L, np.int32)
    at = 0
    for e in range(L):
        slots = np.nonzero(flat == e)[0]
        starts[e], counts[e] = at, slots.size
        row[slots] = at + np.arange(slots.size)
        token[at:at + slots.size] = slots // k
        mi[at:at + slots.size] = e
        at += -(-slots.size // b) * b
    dev = s["x"].device
    live = torch.from_numpy(token >= 0).to(dev)
    xs = s["x"].double()[torch.from_numpy(np.maximum(token, 0)).to(dev)] * live[:, None]
    w = s["w"].double().cpu().numpy().reshape(-1)
    rw = np.zeros(R)
    rw[row[row >= 0]] = w[row >= 0]
    to = lambda a: torch.from_numpy(a).to(dev)
    return {"xs": xs, "row_weights": to(rw), "m_indices": to(mi), "src2dst": to(row.reshape(ids.shape)), "counts": to(counts),
            "starts": to(starts), "psum": to(starts + counts), "total": to(np.array([at], np.int32))}


def _exact_sort_grad(s, c):
    """Row by row of the sorted side: each kept row knows its slot."""
    R, T, k, H = s["R"], c["T"], c["topk"], c["H"]
    row = s["s2d"].reshape(-1).to(torch.int64)
    slots = torch.nonzero(row >= 0)[:, 0]
    token = slots // k
    dy = torch.zeros(R, H, device="cuda", dtype=torch.float64)
    dw = torch.zeros(T * k, device="cuda", dtype=torch.float64)
    dx = torch.zeros(T, H, device="cuda", dtype=torch.float64)
    w = s["w"].reshape(-1).double()
    for p in range(0, slots.numel(), 8192):
        sl, tk = slots[p:p + 8192], token[p:p + 8192]
        g = s["dout"][tk].double()
        dy[row[sl]] = g * w[sl, None]
        dw[sl] = torch.einsum("ij,ij->i", g, s["y"][row[sl]].double())
        dx.index_add_(0, tk, s["dxs"][row[sl]].double())
    return {"dy": dy, "dw": dw.reshape(T, k), "dx": dx}


def _phi(name, v):
    """(activation, derivative) in 64 bits."""
    if name == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * (1 - p)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-v / math.sqrt(2.0))
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return v.clamp_min(0), (v > 0).double()
    return v, torch.ones_like(v)


def _values64(s, key, ekey, sl, c):
    v = s[key][sl].double()
    if c["dtype"] == "e4m3":
        v = v * torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), s[ekey][sl].double()).repeat_interleave(128, -1)
    return v


def _exact_matmul(s, c):
    N, out = c["N"], torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
    pre = torch.zeros(s["pre"].shape, device="cuda", dtype=torch.float64) if s["pre"] is not None else None
    for e, (lo, hi) in enumerate(s["seg"]):
        if hi > lo:
            p = torch.einsum("rk,nk->rn", _values64(s, "x", "xe", slice(lo, hi), c), _values64(s, "wt", "we", e, c))
            p += s["bias"][e].double() if c["bias"] else 0.0
            if pre is not None:
                pre[lo:hi] = p
            a = _phi(c["act"], p[:, :N])[0]
            out[lo:hi] = a * p[:, N:] if c["gated"] else a
            if c["residual"]:
                out[lo:hi] += s["res"][lo:hi].double()
    return {"out": out, "pre": pre}


def _exact_matmul_grad(s, c):
    N, f64 = c["N"], torch.float64
    dx = torch.zeros(s["dx"].shape, device="cuda", dtype=f64)
    dw = torch.zeros(s["dw"].shape, device="cuda", dtype=f64)
    db = torch.zeros(s["db"].shape, device="cuda", dtype=f64)
    for e, (lo, hi) in enumerate(s["seg"]):
        if hi <= lo:
            continue
        g = s["dout"][lo:hi].double()
        if s["pre"] is not None:
            p = s["pre"][lo:hi].double()
            a, d = _phi(c["act"], p[:, :N])
            g = torch.cat([g * d * p[:, N:], g * a], 1) if c["gated"] else g * d
        torch.matmul(g, s["wt"][e].double(), out=dx[lo:hi])
        torch.matmul(g.t(), s["x"][lo:hi].double(), out=dw[e])
        db[e] = g.sum(0)
    return {"dx": dx, "dw": dw, "db": db if c["bias"] else None}


def _exact_norm(s, c):
    x, h, H = s["x"].double(), None, c["H"]
    if c["post"]:
        y = s["y"].double()
        n = y / torch.sqrt(torch.einsum("th,th->t", y, y) / H + EPS)[:, None]
        gate = 1.0 if s["gate"] is None else (s["gate"].double()[:, None] if c["gate"] == "token" else s["gate"].double())
        x = x + c["scale"] * gate * s["wpost"].double() * n
    if c["pre"]:
        h = x / torch.sqrt(torch.einsum("th,th->t", x, x) / H + EPS)[:, None] * s["wpre"].double()
    return {"x": x if c["post"] else None, "h": h}


def _exact_norm_grad(s, c):
    """The same reciprocal roots as the call is given, so only the gradient's own arithmetic counts."""
    H, g = c["H"], s["dxo"].double()
    out = {"dx": None, "dy": None, "dw_pre": None, "dw_post": None, "dgate": None}
    if c["pre"]:
        r = s["rx"].double()
        x, dh, w = s["x"].double(), s["dh"].double(), s["wpre"].double()
        dot = torch.einsum("th,h,th->t", dh, w, x)
        g = g + r[:, None] * dh * w - x * (r ** 3 * dot / H)[:, None]
        out["dw_pre"] = torch.einsum("th,th,t->h", dh, x, r)
    out["dx"] = g
    if c["post"]:
        r, y, w = s["ry"].double(), s["y"].double(), s["wpost"].double()
        u = c["scale"] * g
        if s["gate"] is not None:
            n = y * r[:, None] * w
            out["dgate"] = torch.einsum("th,th->t" if c["gate"] == "token" else "th,th->h", u, n)
            u = u * (s["gate"].double()[:, None] if c["gate"] == "token" else s["gate"].double())
        out["dw_post"] = torch.einsum("th,th,t->h", u, y, r)
        dot = torch.einsum("th,h,th->t", u, w, y)
        out["dy"] = r[:, None] * u * w - y * (r ** 3 * dot / H)[:, None]
    return out
