"""One MoE block through the library's calls, for serving and for training.

    h  = rms(x) * w_in                        block_norm
    route h to top-k experts                  (torch: logits) route
    serving    rows in e4m3                   dispatch_compact
               silu(gate) * up, in e4m3       expert_matmul, quant_group
               down projection                expert_matmul
      or       rows in four bits              dispatch_fp4
               silu(gate) * up, in four bits  expert_matmul_fp4, quant_fp4
               down projection                expert_matmul_fp4
    training   rows in bf16                   permute
               silu(gate) * up, P kept        expert_matmul
               down projection                expert_matmul
    y  = sum_k w_k * expert output            combine
    x' = x + scale * gate * rms(y) * w_out    block_norm

and for training the router's balance and z losses (balance_loss) and the backward
pass through the same steps, written out call by call: block_norm_grad,
combine_grad, expert_matmul_grad twice, permute_grad, route_grad (through the
top-k weights and both losses) and block_norm_grad again.

Run it on a GB300:  python examples/moe_block.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_fp8_quant_gb300 as mp  # noqa: E402

BLOCK_E = 128


@dataclass
class Weights:
    """The block's parameters: norms and gate in float32, the rest in bfloat16."""
    w_in: torch.Tensor      # [H] norm before the block
    w_out: torch.Tensor     # [H] norm after it
    gate: torch.Tensor      # [H] gate on the block's output
    router: torch.Tensor    # [E, H]
    up: torch.Tensor        # [E, 2F, H]: gate rows, then up rows
    up_bias: torch.Tensor   # [E, 2F] float32
    down: torch.Tensor      # [E, H, F]
    scale: float = 1.0


def make_weights(E, H, F, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=device, generator=g)
    bf = lambda t: t.to(torch.bfloat16)
    return Weights(w_in=1 + 0.1 * r(H), w_out=1 + 0.1 * r(H), gate=torch.sigmoid(r(H)), router=bf(r(E, H) * H ** -0.5),
                   up=bf(r(E, 2 * F, H) * H ** -0.5), up_bias=0.1 * r(E, 2 * F), down=bf(r(E, H, F) * F ** -0.5), scale=0.5)


def router_logits(h, router):
    return h.float() @ router.float().t()


def route(h, router, top_k):
    """Top-k experts of each token and the softmax over their logits."""
    r = mp.route(router_logits(h, router), top_k)
    return r["topk_ids"], r["topk_weights"]


class Serving:
    """The block with its expert weights laid out once in e4m3."""

    def __init__(self, w: Weights):
        self.w = w
        E, F2, H = w.up.shape
        up = mp.quant_group(w.up.view(E * F2, H))
        down = mp.quant_group(w.down.view(E * H, F2 // 2))
        self.up, self.up_sc, self.up_ld = up["xq"].view(E, F2, H), up["scales"], up["ld_s"]
        self.down, self.down_sc, self.down_ld = down["xq"].view(E, H, F2 // 2), down["scales"], down["ld_s"]

    def __call__(self, x, top_k):
        w, E = self.w, self.up.shape[0]
        h = mp.block_norm(x, w_pre=w.w_in)["h"]
        ids, tw = route(h, w.router, top_k)
        d = mp.dispatch_compact(h, ids, tw, E, E, block_e=BLOCK_E)
        seg = dict(starts=d["starts"], psum=d["psum"], status=d["status"])
        a = mp.expert_matmul(d["xq"], self.up, bias=w.up_bias, act="silu", gated=True, x_scales=d["scales"],
                             ld_xs=d["ld_s"], w_scales=self.up_sc, ld_ws=self.up_ld, **seg)
        q = mp.quant_group(a)
        y = mp.expert_matmul(q["xq"], self.down, x_scales=q["scales"], ld_xs=q["ld_s"], w_scales=self.down_sc,
                             ld_ws=self.down_ld, **seg)
        out = mp.combine(y, d["src2dst"], tw, status=d["status"])
        return mp.block_norm(x, out, w_post=w.w_out, gate=w.gate, gate_mode="channel", scale=w.scale)["x"]


class Serving4:
    """The block with its expert weights laid out once in four bits: e2m1 with a float8
    scale for each 16 elements and a float32 scale for each expert."""

    def __init__(self, w: Weights):
        self.w = w

        def lay_out(t):
            L, N, K = t.shape
            ts = (t.abs().amax((1, 2)).float() / (6 * 448)).contiguous()
            q = mp.quant_fp4(t.view(L * N, K), tensor_scale=ts)
            return q["xq"].view(L, N, K // 2), q["scales"], ts

        self.up, self.up_sc, self.up_ts = lay_out(w.up)
        self.down, self.down_sc, self.down_ts = lay_out(w.down)

    def __call__(self, x, top_k):
        w, E = self.w, self.up.shape[0]
        h = mp.block_norm(x, w_pre=w.w_in)["h"]
        ids, tw = route(h, w.router, top_k)
        d = mp.dispatch_fp4(h, ids, tw, E, E, block_e=BLOCK_E)
        seg = dict(starts=d["starts"], psum=d["psum"], status=d["status"])
        a = mp.expert_matmul_fp4(d["xq"], self.up, d["scales"], self.up_sc, w_tscale=self.up_ts, bias=w.up_bias,
                                 act="silu", gated=True, **seg)
        q = mp.quant_fp4(a, m_indices=d["m_indices"])
        y = mp.expert_matmul_fp4(q["xq"], self.down, q["scales"], self.down_sc, w_tscale=self.down_ts, **seg)
        out = mp.combine(y, d["src2dst"], tw, status=d["status"])
        return mp.block_norm(x, out, w_post=w.w_out, gate=w.gate, gate_mode="channel", scale=w.scale)["x"]


def forward(x, w: Weights, top_k, coef=None):
    """The training forward pass: (x', what the backward pass needs). coef: float32 [2],
    what the balance and the z loss count for in the training loss; the losses
    themselves are in saved["loss"]."""
    E = w.up.shape[0]
    pre_norm = mp.block_norm(x, w_pre=w.w_in, save_rstd=True)
    h = pre_norm["h"]
    logits = router_logits(h, w.router)
    r = mp.route(logits, top_k)
    ids, tw = r["topk_ids"], r["topk_weights"]
    balance = mp.balance_loss(logits, ids) if coef is not None else dict(loss=None, counts=None)
    p = mp.permute(h, ids, tw, E, E, block_e=BLOCK_E)
    seg = dict(starts=p["starts"], psum=p["psum"], status=p["status"])
    P = torch.empty(p["bound"], w.up.shape[1], dtype=x.dtype, device=x.device)
    a = mp.expert_matmul(p["xs"], w.up, bias=w.up_bias, act="silu", gated=True, pre=P, **seg)
    y = mp.expert_matmul(a, w.down, **seg)
    out = mp.combine(y, p["src2dst"], tw, status=p["status"])
    post = mp.block_norm(x, out, w_post=w.w_out, gate=w.gate, gate_mode="channel", scale=w.scale, save_rstd=True)
    saved = dict(x=x, h=h, logits=logits, ids=ids, tw=tw, coef=coef, loss=balance["loss"], counts=balance["counts"],
                 xs=p["xs"], P=P, a=a, y=y, out=out, seg=seg, src2dst=p["src2dst"],
                 x_out=post["x"], rstd_in=pre_norm["rstd_pre"], rstd_out=post["rstd_post"])
    return post["x"], saved


def backward(dx_out, s, w: Weights):
    """Gradients of every parameter and of x for the gradient of x'."""
    post = mp.block_norm_grad(dx_out, None, s["x_out"], s["out"], w_post=w.w_out, gate=w.gate,
                              gate_mode="channel", scale=w.scale, rstd_post=s["rstd_out"])
    st = s["seg"]["status"]
    c = mp.combine_grad(post["dy"], s["y"], s["src2dst"], s["tw"], status=st)
    down = mp.expert_matmul_grad(c["dy"], s["a"], w.down, need=("dx", "dw"), **s["seg"])
    up = mp.expert_matmul_grad(down["dx"], s["xs"], w.up, pre=s["P"], act="silu", gated=True,
                               need=("dx", "dw", "dbias"), **s["seg"])
    dh = mp.permute_grad(up["dx"], s["src2dst"], status=st)
    # the router: through the softmax of the chosen logits and through its losses
    dlogits = mp.route_grad(s["logits"], s["ids"], dweights=c["dweights"], dloss=s["coef"], counts=s["counts"])
    drouter = dlogits.t() @ s["h"].float()
    dh = (dh.float() + dlogits @ w.router.float()).to(dh.dtype)
    pre = mp.block_norm_grad(post["dx"], dh, s["x"], w_pre=w.w_in, rstd_pre=s["rstd_in"])
    return dict(x=pre["dx"], w_in=pre["dw_pre"], w_out=post["dw_post"], gate=post["dgate"], router=drouter,
                up=up["dw"], up_bias=up["dbias"], down=down["dw"])


def main():
    T, H, F, E, top_k = 512, 2048, 1024, 16, 4
    w = make_weights(E, H, F)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    served, served4 = Serving(w)(x, top_k), Serving4(w)(x, top_k)
    out, saved = forward(x, w, top_k, coef=torch.tensor([0.01, 0.001], device="cuda"))
    grads = backward(torch.ones_like(out), saved, w)
    code = mp.moe_status_sync(saved["seg"]["status"])
    diff, diff4 = ((t.float() - out.float()).norm() / out.float().norm() for t in (served, served4))
    print(f"status {code}; e4m3 and four-bit against bf16 block output: relative difference {diff:.4f}, {diff4:.4f}")
    print(f"balance loss {saved['loss'][0]:.4f}, z loss {saved['loss'][1]:.4f}")
    for k, g in grads.items():
        print(f"  d{k:8s} {str(tuple(g.shape)):18s} norm {g.float().norm():.4f}")


if __name__ == "__main__":
    main()
