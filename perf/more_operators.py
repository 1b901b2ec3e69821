"""Cases of the router's operators and of the four-bit rows and weights: what each reads and computes, in plain torch and
through the package.

  route         the experts of each token and their weights, from the router's logits
  balance       the balance and z losses of a batch, with the slots and probabilities of each expert
  route_grad    the gradient of the logits through the weights and both losses
  quant         rows to four bits and back: quant_fp4, dequant_fp4
  experts       tokens sorted by expert in four bits, and the experts' product: dispatch_fp4, expert_matmul_fp4
  product       expert_matmul_fp4 alone, on rows that are in four bits already

With ``own`` false, ``run`` computes an operator from elementary torch operations; with ``own`` true it makes the package's
calls. Both take the same state. Scale layout of the four-bit rows: byte b of piece c of row r, at [c, r, b], is the scale of
group 16 c + b of the row.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the eight codes; the fourth bit is the sign


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step: launch latency is all there is
        dict(name="route_one_token", op="route", T=1, E=256, K=8, dtype="fp32", score="sigmoid", bias=True, renorm=True, scale=2.5),
        # the router of a prefill batch, with the load-balancing bias
        dict(name="route_prefill", op="route", T=16384, E=256, K=8, dtype="fp32", score="sigmoid", bias=True, renorm=True, scale=2.5),
        # 16-bit logits of an odd batch over an odd number of experts, probabilities as they are
        dict(name="route_odd", op="route", T=4099, E=77, K=6, dtype="bf16", score="softmax", bias=False, renorm=False, scale=1.0),
        # the losses of one training batch, all tokens one group
        dict(name="balance_batch", op="balance", T=8192, E=64, K=6, dtype="bf16", score="softmax", groups=1),
        # sequence-wise losses: 61 ragged sequences in a padded batch
        dict(name="balance_sequences", op="balance", T=65536, E=256, K=8, dtype="fp32", score="sigmoid", groups=61),
        # gradients of the same two
        dict(name="route_grad_batch", op="route_grad", T=8192, E=64, K=6, dtype="bf16", score="softmax", groups=1, renorm=True,
             scale=1.0),
        dict(name="route_grad_sequences", op="route_grad", T=65536, E=256, K=8, dtype="fp32", score="sigmoid", groups=61, renorm=True,
             scale=2.5),
        # the activations between two products of a decode batch, padding rows among them
        dict(name="quant_segments", op="quant", R=1111, H=2048, dtype="bf16", fmt="nv", tscale=True, padded=True),
        # the rows of a prefill batch, a power-of-two scale for each 32 elements
        dict(name="quant_prefill", op="quant", R=16384, H=7168, dtype="bf16", fmt="mx", tscale=False, padded=False),
        # a decode batch on one of eight ranks: 32 of 256 experts are local, a few rows each; weights are all the traffic
        dict(name="experts_decode", op="experts", T=128, E=256, L=32, topk=8, block=128, K=7168, N=2048, act="silu", gated=True,
             dtype="bf16", fmt="nv"),
        # a prefill batch over 64 experts: the tensor cores count
        dict(name="experts_prefill", op="experts", T=4096, E=64, L=64, topk=8, block=128, K=7168, N=2048, act="silu", gated=True,
             dtype="bf16", fmt="nv"),
        # one token through a dense output projection with bias and residual
        dict(name="product_one_token", op="product", R=1, K=2048, N=7168, act="none", gated=False, bias=True, residual=True,
             fmt="e8m0"),
    ]


def _spread(rng, lo, hi, step=1):
    """A size in [lo, hi], spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(max(round(v / step) * step, lo), hi))


def draw(rng):
    while True:
        op = rng.choice(["route", "balance", "route_grad", "quant", "experts", "experts", "product"])
        fmt = rng.choice(["nv", "nv", "mx", "e8m0"])
        if op in ("route", "balance", "route_grad"):
            E = rng.choice([rng.choice([8, 64, 128, 256]), _spread(rng, 2, 1024)])
            c = dict(op=op, T=_spread(rng, 1, 65536), E=E, K=min(E, rng.randint(1, 10)), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                     score=rng.choice(["softmax", "sigmoid"]))
            if op != "balance":
                c.update(renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
            if op == "route":
                c.update(bias=rng.random() < 0.5)
            else:
                c.update(groups=min(c["T"], rng.choice([1, 1, _spread(rng, 2, 200)])))
        elif op == "quant":
            c = dict(op=op, R=_spread(rng, 1, 32768), H=_spread(rng, 64, 7168, 64), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     fmt=fmt, tscale=fmt == "nv" and rng.random() < 0.7, padded=rng.random() < 0.4)
        elif op == "experts":
            E = rng.choice([_spread(rng, 2, 64), _spread(rng, 8, 256)])
            gated = rng.random() < 0.6
            c = dict(op=op, T=_spread(rng, 1, 8192), E=E, L=rng.choice([E, max(1, E // 8)]), topk=min(E, rng.choice([1, 2, 6, 8])),
                     block=rng.choice([1, 16, 128]), K=_spread(rng, 64, 7168, 64), N=_spread(rng, 64, 2048 if gated else 7168, 16),
                     act=rng.choice(["silu", "gelu"] if gated else ["none", "relu"]), gated=gated, dtype=rng.choice(["bf16", "bf16", "fp16"]),
                     fmt=fmt)
        else:
            gated = rng.random() < 0.3
            c = dict(op=op, R=_spread(rng, 1, 8192), K=_spread(rng, 64, 7168, 64), N=_spread(rng, 64, 2048 if gated else 7168, 16),
                     act="silu" if gated else "none", gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5, fmt=fmt)
        w = work(c)
        if w["flops"] <= 1.92e12 and w["bytes"] <= 1.1e9:
            return c


def _elem(c):
    return {"bf16": 2, "fp16": 2, "fp32": 4}[c["dtype"]]


def _group(fmt):
    return 16 if fmt == "nv" else 32


def work(c):
    op = c["op"]
    if op == "route":
        return {"bytes": c["T"] * (c["E"] * _elem(c) + 8 * c["K"]), "flops": 4 * c["T"] * c["E"]}
    if op == "balance":
        return {"bytes": c["T"] * (c["E"] * _elem(c) + 4 * c["K"]) + 8 * c["groups"] * c["E"], "flops": 6 * c["T"] * c["E"]}
    if op == "route_grad":
        return {"bytes": c["T"] * (2 * c["E"] * _elem(c) + 8 * c["K"]) + 4 * c["groups"] * c["E"], "flops": 12 * c["T"] * c["E"]}
    if op == "quant":  # there and back: the rows in, their values out, the codes and scales written and read
        return {"bytes": int(c["R"] * c["H"] * (2 * _elem(c) + 2 * (0.5 + 1 / _group(c["fmt"])))), "flops": 4 * c["R"] * c["H"]}
    per = 0.5 + 1 / _group(c["fmt"])
    K, Nw = c["K"], c["N"] * (2 if c["gated"] else 1)
    if op == "product":
        return {"bytes": int(Nw * K * per + c["R"] * (K * per + 2 * c["N"] * (2 if c["residual"] else 1))), "flops": 2 * c["R"] * Nw * K}
    A = max(1.0, c["T"] * c["topk"] * c["L"] / c["E"])
    active = c["L"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** c["T"]) if c["topk"] < c["E"] else c["L"]
    return {"bytes": int(max(1.0, active) * Nw * K * per + c["T"] * K * _elem(c) + 2 * A * K * per + 2 * A * c["N"]), "flops": int(2 * A * Nw * K)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, gain=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * gain).to(dtype)


def _choice(T, E, k, g):
    """k distinct experts for each token, by noise on a mild popularity."""
    pop = -0.5 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    u = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-20, 1.0 - 1e-7)
    return (pop - torch.log(-torch.log(u))).topk(k, dim=1).indices.to(torch.int32).contiguous()


def _bound(A, L, b):
    n = min(A, L)
    return b * (n + (A - n) // b)


def _groups(c, g):
    """Token ranges of the groups: a padded batch of ragged sequences, begin [Q] and end [Q]."""
    Q, T = c["groups"], c["T"]
    if Q == 1:
        return None, None
    room = T // Q
    n = (torch.rand(Q, device="cuda", generator=g).square() * (room + 1)).to(torch.int32).clamp_(max=room)
    begin = torch.arange(Q, device="cuda", dtype=torch.int32) * room
    return begin, begin + n


def _weights4(c, g, L):
    """The experts' weights in four bits, made expert by expert: codes, scales, tensor scales."""
    K, Nw = c["K"], c["N"] * (2 if c["gated"] else 1)
    C = -(-K // _group(c["fmt"]) // 16)
    w = torch.empty(L, Nw, K // 2, device="cuda", dtype=torch.uint8)
    sc = torch.empty(C, L * Nw, 16, device="cuda", dtype=torch.uint8)
    ts = torch.ones(L, device="cuda")
    for e in range(L):
        v = _randn(g, Nw, K, gain=K ** -0.5)
        if c["fmt"] == "nv":
            ts[e] = v.abs().amax() / (6 * 448)
        w[e], sc[:, e * Nw:(e + 1) * Nw] = _to4(v, c["fmt"], ts[e])
    return w, sc, ts if c["fmt"] == "nv" else None


def _rows(g, R, H, dtype):
    """Activations: normal, one element in a hundred 50 times as large."""
    x = torch.randn(R, H, device="cuda", generator=g)
    return torch.where(torch.rand(R, H, device="cuda", generator=g) < 0.01, x * 50, x).to(dtype)


def prepare(c, seed):
    g, op, dev = _gen(seed), c["op"], "cuda"
    s = {"case": dict(c)}
    if op in ("route", "balance", "route_grad"):
        T, E, K = c["T"], c["E"], c["K"]
        s["logits"] = _randn(g, T, E, dtype=DT[c["dtype"]], gain=1.5)
        if op == "route":
            s["bias"] = _randn(g, E, gain=0.1) if c["bias"] else None
        else:
            s["ids"] = _choice(T, E, K, g)
            s["begin"], s["end"] = _groups(c, g)
        if op == "route_grad":
            s["dw"] = _randn(g, T, K, gain=0.1)
            s["dloss"] = torch.tensor([0.01, 0.001], device=dev) * (1 + torch.rand(2, device=dev, generator=g))
            s["counts"] = _counts(s, c)[0].to(torch.int32)
    elif op == "quant":
        R, H, dt = c["R"], c["H"], DT[c["dtype"]]
        s["x"] = _rows(g, R, H, dt)
        s["ts"] = (s["x"].abs().amax().float() / (6 * 448))[None].contiguous() if c["tscale"] else None
        s["expert"] = None
        if c["padded"]:  # the expert of every row, -1 on the padding of segments
            s["expert"] = torch.where(torch.rand(R, device=dev, generator=g) < 0.8, 1, -1).to(torch.int32)
        s["out"] = torch.zeros(R, H, device=dev, dtype=dt)
    elif op == "experts":
        T, L, K = c["T"], c["L"], c["K"]
        s["x"] = _rows(g, T, K, DT[c["dtype"]])
        s["ids"] = _choice(T, c["E"], c["topk"], g)
        s["w"] = torch.softmax(_randn(g, T, c["topk"]), dim=1).contiguous()
        s["ts"] = (s["x"].abs().amax().float() / (6 * 448))[None].contiguous() if c["fmt"] == "nv" else None
        s["wt"], s["wsc"], s["wts"] = _weights4(c, g, L)
        s["R"] = R = max(1, _bound(T * c["topk"], L, c["block"]))
        s["most"] = int(_layout(s["ids"], L, c["block"])[0].max())  # the largest expert's rows, as the host plans them
        s["out"] = torch.zeros(R, c["N"], device=dev, dtype=torch.bfloat16)
    else:
        R, K, Nw = c["R"], c["K"], c["N"] * (2 if c["gated"] else 1)
        x = _rows(g, R, K, torch.float32)
        s["ts"] = (x.abs().amax() / (6 * 448))[None].contiguous() if c["fmt"] == "nv" else None
        s["xq"], s["xsc"] = _to4(x, c["fmt"], s["ts"])
        s["wt"], s["wsc"], s["wts"] = _weights4(c, g, 1)
        s["bias"] = _randn(g, 1, Nw) if c["bias"] else None
        s["res"] = _randn(g, R, c["N"], dtype=torch.bfloat16) if c["residual"] else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import combine_fp8_quant_gb300 as mp
        return {"route": _own_route, "balance": _own_balance, "route_grad": _own_route_grad, "quant": _own_quant,
                "experts": _own_experts, "product": _own_product}[op](mp, s, s["case"])
    return {"route": _route, "balance": _balance, "route_grad": _route_grad, "quant": _quant, "experts": _experts,
            "product": _product}[op](s, s["case"])


def _own_route(mp, s, c):
    o = mp.route(s["logits"], c["K"], bias=s["bias"], score=c["score"], renorm=c["renorm"], scale=c["scale"])
    return {"ids": o["topk_ids"], "w": o["topk_weights"]}


def _own_balance(mp, s, c):
    o = mp.balance_loss(s["logits"], s["ids"], seq_begin=s["begin"], seq_end=s["end"], score=c["score"])
    return {"loss": o["loss"], "counts": o["counts"], "prob_sums": o["prob_sums"]}


def _own_route_grad(mp, s, c):
    return mp.route_grad(s["logits"], s["ids"], dweights=s["dw"], dloss=s["dloss"], counts=s["counts"], seq_begin=s["begin"],
                         seq_end=s["end"], score=c["score"], renorm=c["renorm"], scale=c["scale"])


def _own_quant(mp, s, c):
    q = mp.quant_fp4(s["x"], fmt=c["fmt"], tensor_scale=s["ts"], m_indices=s["expert"])
    return mp.dequant_fp4(q["xq"], q["scales"], fmt=c["fmt"], tensor_scale=s["ts"], m_indices=s["expert"], out=s["out"])


def _own_experts(mp, s, c):
    d = mp.dispatch_fp4(s["x"], s["ids"], s["w"], c["E"], c["L"], block_e=c["block"], fmt=c["fmt"], tensor_scale=s["ts"])
    out = mp.expert_matmul_fp4(d["xq"], s["wt"], d["scales"], s["wsc"], fmt=c["fmt"], starts=d["starts"], psum=d["psum"],
                               x_tscale=s["ts"], w_tscale=s["wts"], act=c["act"], gated=c["gated"], out=s["out"][:d["bound"]],
                               status=d["status"])
    return {"out": out, **{k: d[k] for k in ("m_indices", "src2dst", "counts", "starts", "psum", "total")}}


def _own_product(mp, s, c):
    return mp.expert_matmul_fp4(s["xq"], s["wt"], s["xsc"], s["wsc"], fmt=c["fmt"], x_tscale=s["ts"], w_tscale=s["wts"],
                                bias=s["bias"], act=c["act"], gated=c["gated"], residual=s["res"])


def _route(s, c):
    """The choice in 64 bits (a key next to another must not be rounded onto it), the weights in 32."""
    f = s["logits"].float()
    key = f
    if s["bias"] is not None:
        d = s["logits"].double()
        e = torch.exp(d - d.amax(1, keepdim=True))
        key = (e / e.sum(1, keepdim=True) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-d))) + s["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    if c["score"] == "softmax":
        e = torch.exp(f - f.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-f))
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": w * c["scale"]}


def _member(s, c):
    """[T] the group of each token (groups: none), and [Q] tokens of each."""
    Q, T = c["groups"], c["T"]
    if s["begin"] is None:
        return torch.zeros(T, dtype=torch.int64, device="cuda"), torch.full((1,), float(T), device="cuda")
    t = torch.arange(T, device="cuda")[:, None]
    inside = (t >= s["begin"]) & (t < s["end"])
    q = torch.where(inside.any(1), inside.to(torch.int32).argmax(1), Q)
    return q, (s["end"] - s["begin"]).float()


def _counts(s, c):
    Q, E, K = c["groups"], c["E"], c["K"]
    q, n = _member(s, c)
    at = (q[:, None] * E + s["ids"].to(torch.int64)).reshape(-1)
    counts = torch.zeros((Q + 1) * E, dtype=torch.int64, device="cuda").scatter_add_(0, at, torch.ones_like(at)).reshape(Q + 1, E)[:Q]
    return counts, q, n


def _probs(s, c):
    """(p, logsumexp, softmax, sigmoid) of every token in 32 bits."""
    f = s["logits"].float()
    m = f.amax(1, keepdim=True)
    e = torch.exp(f - m)
    z = e.sum(1, keepdim=True)
    soft, lse = e / z, m[:, 0] + torch.log(z[:, 0])
    if c["score"] == "softmax":
        return soft, lse, soft, None
    sg = 1.0 / (1.0 + torch.exp(-f))
    return sg / sg.sum(1, keepdim=True), lse, soft, sg


def _balance(s, c):
    Q, E, K = c["groups"], c["E"], c["K"]
    counts, q, n = _counts(s, c)
    p, lse, _, _ = _probs(s, c)
    of = torch.zeros(Q + 1, c["T"], device="cuda").scatter_(0, q[None], torch.ones(1, c["T"], device="cuda"))[:Q]  # [Q, T]
    P = of @ p
    some = (n > 0).float()
    per = (counts.float() * P).sum(1) * E / (K * torch.clamp(n, min=1.0) ** 2)
    balance = per.sum() / torch.clamp(some.sum(), min=1.0)
    z = (torch.where(q < Q, lse * lse, torch.zeros_like(lse))).double().sum().float() / torch.clamp(n.sum(), min=1.0)
    return {"loss": torch.stack([balance, z]), "counts": counts.to(torch.int32), "prob_sums": P}


def _route_grad(s, c):
    Q, E, K = c["groups"], c["E"], c["K"]
    q, n = _member(s, c)
    p, lse, soft, sg = _probs(s, c)
    live = (q < Q).float()[:, None]
    pad = torch.cat([s["counts"].float(), torch.zeros(1, E, device="cuda")])
    n1 = torch.cat([n, n.new_ones(1)])
    share = s["dloss"][0] * E / (K * torch.clamp((n > 0).float().sum(), min=1.0))
    gr = share * pad[q] / (n1[q] ** 2)[:, None]
    d = p * (gr - (p * gr).sum(1, keepdim=True))
    if sg is not None:
        d = d * (1.0 - sg)
    d = d + s["dloss"][1] * 2.0 / torch.clamp(n.sum(), min=1.0) * lse[:, None] * soft
    d = d * live
    ids, dw = s["ids"].to(torch.int64), s["dw"]
    base = sg if sg is not None else soft
    chosen = torch.gather(base, 1, ids)
    if c["renorm"]:
        u = chosen / chosen.sum(1, keepdim=True)
        dk = c["scale"] * u * (dw - (u * dw).sum(1, keepdim=True))
        if sg is not None:
            dk = dk * (1.0 - chosen)
    elif sg is not None:
        dk = c["scale"] * dw * chosen * (1.0 - chosen)
    else:
        dk = c["scale"] * dw * chosen
        d = d - c["scale"] * soft * (dw * chosen).sum(1, keepdim=True)
    return (d + torch.zeros_like(d).scatter_add_(1, ids, dk)).to(s["logits"].dtype)


def _pow2(e):
    """2^e in 32 bits for e in [-127, 127], from the bits: a value on a border must not move."""
    return torch.where(e > -127, (e.to(torch.int32) + 127) << 23, 1 << 22).view(torch.float32)


def _to4(x, fmt, ts):
    """Rows to four bits: codes [R, H / 2], the even element in the low half of its byte, and scales [C, R, 16]."""
    R, H = x.shape
    g = _group(fmt)
    v = x.float().reshape(R, H // g, g)
    amax = v.abs().amax(2)
    if fmt == "nv":
        t = 1.0 if ts is None else ts
        b = (amax / (6.0 * t)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = (b.float() * t)[:, :, None]
        a = torch.where(d > 0, v / d, torch.zeros_like(v))
        byte = b.view(torch.uint8)
    else:
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 3 + (m > 0.75).to(e.dtype) if fmt == "e8m0" else e - 3, -127).clamp(-127, 127)
        a = v * _pow2(-e)[:, :, None]
        byte = (e + 127).to(torch.uint8)
    mag = a.abs()
    code = ((mag > 0.25).to(torch.uint8) + (mag >= 0.75).to(torch.uint8) + (mag > 1.25).to(torch.uint8) + (mag >= 1.75).to(torch.uint8)
            + (mag > 2.5).to(torch.uint8) + (mag >= 3.5).to(torch.uint8) + (mag > 5.0).to(torch.uint8) + 8 * (a < 0).to(torch.uint8))
    code = code.reshape(R, H // 2, 2)
    G = H // g
    C = -(-G // 16)
    sc = torch.zeros(R, C * 16, dtype=torch.uint8, device=x.device)
    sc[:, :G] = byte
    return code[:, :, 0] | (code[:, :, 1] << 4), sc.reshape(R, C, 16).transpose(0, 1).contiguous()


def _from4(q, sc, fmt, ts):
    """Values [R, H] of codes [R, H / 2] and scales [C, R, 16], with one tensor scale or one for each row."""
    R, H = q.shape[0], q.shape[1] * 2
    g = _group(fmt)
    one = torch.tensor(CODES + tuple(-v for v in CODES), device=q.device)
    byte = torch.arange(256, device=q.device)
    v = torch.stack([one[byte & 15], one[byte >> 4]], 1)[q.to(torch.int32)].reshape(R, H // g, g)
    b = sc.transpose(0, 1).reshape(R, -1)[:, :H // g].contiguous()
    if fmt == "nv":
        d = b.view(torch.float8_e4m3fn).float()
        if ts is not None:
            d = d * ts.reshape(-1, 1)
    else:
        d = _pow2(b.to(torch.int32) - 127)
    return (v * d[:, :, None]).reshape(R, H)


def _quant(s, c):
    q, sc = _to4(s["x"], c["fmt"], s["ts"])
    v = _from4(q, sc, c["fmt"], s["ts"]).to(s["x"].dtype)
    return v if s["expert"] is None else torch.where(s["expert"][:, None] >= 0, v, torch.zeros_like(v))


def _layout(ids, L, b):
    """counts, starts, psum [L] and total of the compact layout, and the row of every slot (-1 when not local)."""
    flat = ids.reshape(-1).to(torch.int64)
    local = (flat >= 0) & (flat < L)
    key = torch.where(local, flat, torch.full_like(flat, L))
    counts = torch.zeros(L + 1, dtype=torch.int64, device=flat.device).scatter_add_(0, key, torch.ones_like(key))[:L]
    aligned = (counts + b - 1) // b * b
    starts = torch.cumsum(aligned, 0) - aligned
    order = torch.sort(key, stable=True).indices
    first = torch.cat([torch.cumsum(counts, 0) - counts, counts.sum()[None]])
    starts1 = torch.cat([starts, torch.zeros_like(starts[:1])])
    skey = key[order]
    rank = torch.arange(flat.numel(), device=flat.device) - first[skey]
    row = torch.empty_like(flat)
    row[order] = torch.where(skey < L, starts1[skey] + rank, torch.full_like(skey, -1))
    return counts, starts, starts + counts, aligned.sum(), row.reshape(ids.shape)


def _act(name, v):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    return v


def _experts(s, c):
    L, N, K, R, most = c["L"], c["N"], c["K"], s["R"], max(1, s["most"])
    Nw = 2 * N if c["gated"] else N
    counts, starts, psum, total, row = _layout(s["ids"], L, c["block"])
    i32, dev = torch.int32, s["x"].device
    mi = torch.full((R + 1,), -1, dtype=i32, device=dev)
    flat, kept = row.reshape(-1), row.reshape(-1) >= 0
    dst = torch.where(kept, flat, torch.full_like(flat, R))
    mi[dst] = torch.where(kept, s["ids"].reshape(-1), torch.full_like(s["ids"].reshape(-1), -1))
    token = torch.zeros(R + 1, dtype=torch.int64, device=dev)
    token[dst] = torch.arange(c["T"], device=dev).repeat_interleave(c["topk"])
    x = _from4(*_to4(s["x"], c["fmt"], s["ts"]), c["fmt"], s["ts"])
    w = _from4(s["wt"].reshape(L * Nw, K // 2), s["wsc"], c["fmt"],
               None if s["wts"] is None else s["wts"].repeat_interleave(Nw)).reshape(L, Nw, K)
    j = torch.arange(most, device=dev)
    slab = starts[:, None] + j                                     # row of slab row (e, j)
    real = j < counts[:, None]
    p = torch.bmm(x[token[torch.where(real, slab, torch.full_like(slab, R))]], w.transpose(1, 2))
    v = _act(c["act"], p[:, :, :N]) * p[:, :, N:] if c["gated"] else _act(c["act"], p)
    out = torch.zeros(R + 1, N, device=dev)
    out[torch.where(real, slab, torch.full_like(slab, R))] = v
    b = _bound(c["T"] * c["topk"], L, c["block"])
    return {"out": out[:b].to(torch.bfloat16), "m_indices": mi[:b], "src2dst": row.to(i32), "counts": counts.to(i32),
            "starts": starts.to(i32), "psum": psum.to(i32), "total": total.to(i32)[None]}


def _product(s, c):
    N = c["N"]
    p = _from4(s["xq"], s["xsc"], c["fmt"], s["ts"]) @ _from4(s["wt"][0], s["wsc"], c["fmt"], s["wts"]).t()
    if s["bias"] is not None:
        p = p + s["bias"]
    v = _act(c["act"], p[:, :N]) * p[:, N:] if c["gated"] else _act(c["act"], p)
    return (v + s["res"].float() if s["res"] is not None else v).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s, op = prepare(c, seed), c["op"]
    if op == "route":
        return _exact_route(s, c)
    if op in ("balance", "route_grad"):
        return _exact_losses(s, c)
    if op == "quant":
        v = _exact_round(s["x"], c["fmt"], s["ts"])
        return v if s["expert"] is None else v * (s["expert"] >= 0)[:, None]
    return _exact_experts(s, c) if op == "experts" else _exact_product(s, c)


def _exact_route(s, c):
    """Each token's experts one after the other: the largest key left, the lowest index among equals."""
    l = s["logits"].double()
    sc = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    key = l.clone() if s["bias"] is None else sc + s["bias"].double()
    ids = torch.empty(c["T"], c["K"], dtype=torch.int64, device=l.device)
    index = torch.arange(c["E"], device=l.device)
    for k in range(c["K"]):
        best = key.max(1, keepdim=True).values
        ids[:, k] = torch.where(key == best, index, c["E"]).min(1).values
        key.scatter_(1, ids[:, k:k + 1], -math.inf)
    w = sc.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": c["scale"] * w}


def _exact_losses(s, c):
    """Group by group, the gradient by torch's own differentiation."""
    E, K, T = c["E"], c["K"], c["T"]
    l = s["logits"].double().requires_grad_(c["op"] == "route_grad")
    spans = [(0, T)] if s["begin"] is None else list(zip(s["begin"].tolist(), s["end"].tolist()))
    sg = torch.sigmoid(l)
    p = torch.softmax(l, 1) if c["score"] == "softmax" else sg / sg.sum(1, keepdim=True)
    lse = torch.logsumexp(l, 1)
    balance, z, Q, N = 0.0, 0.0, sum(b > a for a, b in spans), sum(b - a for a, b in spans)
    counts, sums = [], []
    for a, b in spans:
        n = torch.bincount(s["ids"][a:b].reshape(-1).to(torch.int64), minlength=E)
        counts.append(n)
        sums.append(p[a:b].sum(0))
        if b > a:
            balance = balance + (n.double() * sums[-1]).sum() * E / (K * (b - a) ** 2) / Q
            z = z + (lse[a:b] ** 2).sum() / N
    if c["op"] == "balance":
        loss = torch.stack([torch.as_tensor(v, dtype=torch.float64, device=l.device) for v in (balance, z)])
        return {"loss": loss, "counts": torch.stack(counts).to(torch.int32), "prob_sums": torch.stack(sums)}
    w = (p if c["score"] == "softmax" else sg).gather(1, s["ids"].to(torch.int64))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    total = c["scale"] * (w * s["dw"].double()).sum() + s["dloss"][0].double() * balance + s["dloss"][1].double() * z
    total.backward()
    return l.grad


def _nearest(v, table):
    """Index of the nearest of an ascending table of non-negative values, ties to the even index."""
    hi = torch.searchsorted(table, v).clamp_(1, table.numel() - 1)
    down, up = v - table[hi - 1], table[hi] - v
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def _exact_round(x, fmt, ts):
    """Rows rounded to four bits by the definition: nearest codes by search, 32-bit steps where it names them."""
    codes = torch.tensor(CODES, dtype=torch.float64, device=x.device)
    g = _group(fmt)
    v = x.double().reshape(x.shape[0], -1, g)
    amax = v.abs().amax(2)
    f32 = lambda t: t.float().double()
    two = lambda e: ((e.to(torch.int64) + 1023) << 52).view(torch.float64)
    if fmt == "nv":
        t = torch.ones((), dtype=torch.float64, device=x.device) if ts is None else ts.double()
        small = [m * 2.0 ** -9 for m in range(8)]
        e4m3 = torch.tensor(small + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119], dtype=torch.float64, device=x.device)
        b = e4m3[_nearest(f32(amax / f32(6.0 * t)).clamp(max=448.0), e4m3)]
        d = f32(b * t)
    else:
        e = (amax.clamp(min=2.0 ** -149).view(torch.int64) >> 52) - 1025  # floor(log2), exactly, less 2
        if fmt == "e8m0":
            e = torch.where(6.0 * two(e) >= amax, e, e + 1)
        d = two(e.clamp(-127, 127))
    r = f32(v / torch.where(d > 0, d, 1.0)[:, :, None])
    q = codes[_nearest(r.abs().clamp(max=6.0), codes)] * torch.sign(r)
    return (q * d[:, :, None]).reshape(x.shape)


def _wide(q, sc, fmt, ts):
    """Values in 64 bits of four-bit rows, decoded from the bits of codes and scales."""
    g = _group(fmt)
    n = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1).to(torch.int64)
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e.double() - 1.0)) * (1.0 - 2.0 * (n >> 3).double())
    b = sc.permute(1, 0, 2).reshape(q.shape[0], -1)[:, :v.shape[1] // g].to(torch.int64)
    if fmt == "nv":
        e, m = b >> 3, (b & 7).double()
        d = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
        d = d if ts is None else d * ts.double().reshape(-1, 1)
    else:
        d = torch.pow(2.0, b.double() - 127.0)
    return v * d.repeat_interleave(g, 1)


def _phi(c, p):
    N = c["N"]
    a = p[:, :N] if c["gated"] else p
    a = {"silu": lambda t: t * torch.sigmoid(t), "gelu": lambda t: t * 0.5 * torch.erfc(-t / math.sqrt(2.0)),
         "relu": lambda t: t.clamp_min(0), "none": lambda t: t}[c["act"]](a)
    return a * p[:, N:] if c["gated"] else a


def _exact_experts(s, c):
    """Expert by expert: its slots in ascending order fill its segment."""
    ids = s["ids"].cpu().numpy()
    flat, k, b, L, N, K = ids.reshape(-1), c["topk"], c["block"], c["L"], c["N"], c["K"]
    R, Nw = _bound(c["T"] * k, c["L"], b), N * (2 if c["gated"] else 1)
    row, mi = np.full(flat.size, -1, np.int32), np.full(R, -1, np.int32)
    counts, starts = np.zeros(L, np.int32), np.zeros(L, np.int32)
    out = torch.zeros(R, N, device="cuda", dtype=torch.float64)
    x = _exact_round(s["x"], c["fmt"], s["ts"])
    at = 0
    for e in range(L):
        slots = np.nonzero(flat == e)[0]
        n = slots.size
        starts[e], counts[e] = at, n
        row[slots] = at + np.arange(n)
        mi[at:at + n] = e
        if n:
            w = _wide(s["wt"][e], s["wsc"][:, e * Nw:(e + 1) * Nw], c["fmt"], None if s["wts"] is None else s["wts"][e:e + 1])
            out[at:at + n] = _phi(c, torch.einsum("rk,nk->rn", x[torch.from_numpy(slots // k).cuda()], w))
        at += -(-n // b) * b
    to = lambda a: torch.from_numpy(a).cuda()
    return {"out": out, "m_indices": to(mi), "src2dst": to(row.reshape(ids.shape)), "counts": to(counts), "starts": to(starts),
            "psum": to(starts + counts), "total": to(np.array([at], np.int32))}


def _exact_product(s, c):
    p = torch.einsum("rk,nk->rn", _wide(s["xq"], s["xsc"], c["fmt"], s["ts"]), _wide(s["wt"][0], s["wsc"], c["fmt"], s["wts"]))
    v = _phi(c, p + s["bias"].double() if c["bias"] else p)
    return v + s["res"].double() if c["residual"] else v
