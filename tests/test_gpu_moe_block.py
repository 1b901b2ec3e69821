"""The example's MoE block end to end: the training pass and all its gradients
against torch's autograd on the formulas in 64 bits, and the e4m3 serving pass
against the same block. The bounds are on norms: a chain of about ten roundings
to bf16 (2^-8 each, independent) keeps relative norms below 10 * 2^-8; e4m3
rounds rows, activations and both weights to 2^-4 at most, and errors of sums
average, so 4 * 2^-4 bounds the block's update."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block(dev):
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["moe_block"] = m
    spec.loader.exec_module(m)
    return m


NAMES = ("w_in", "w_out", "gate", "router", "up", "up_bias", "down")


def reference(x, w, ids, dout):
    """The block in 64 bits with the given routing: (x', gradients by torch)."""
    leaves = {k: getattr(w, k).double().requires_grad_() for k in NAMES}
    leaves["x"] = x.double().requires_grad_()
    v = leaves
    rms = lambda t: t * torch.rsqrt((t * t).mean(1, keepdim=True) + 1e-6)
    h = rms(v["x"]) * v["w_in"]
    tw = torch.softmax((h @ v["router"].t()).gather(1, ids.long()), 1)
    y = torch.zeros_like(h)
    F = w.down.shape[2]
    for e in range(w.up.shape[0]):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            P = h[t] @ v["up"][e].t() + v["up_bias"][e]
            a = torch.nn.functional.silu(P[:, :F]) * P[:, F:]
            y = y.index_add(0, t, tw[t, k, None] * (a @ v["down"][e].t()))
    out = v["x"] + w.scale * v["gate"] * rms(y) * v["w_out"]
    out.backward(dout.double())
    return out.detach(), {k: t.grad for k, t in leaves.items()}


@pytest.mark.parametrize("T,H,F,E,k", [(1, 128, 64, 4, 2), (37, 256, 128, 8, 3), (300, 512, 256, 6, 2)])
def test_training_step(dev, block, T, H, F, E, k):
    w = block.make_weights(E, H, F, seed=T)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    dout = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    out, saved = block.forward(x, w, k)
    g = block.backward(dout, saved, w)
    assert dev.moe_status_sync(saved["seg"]["status"]) == dev.MOE_OK
    want, gw = reference(x, w, saved["ids"], dout)
    assert (out.double() - want).norm() <= 10 * 2.0 ** -8 * want.norm()
    for name, ref in gw.items():
        assert (g[name].double() - ref).norm() <= 10 * 2.0 ** -8 * ref.norm(), name


@pytest.mark.parametrize("T,k", [(1, 2), (64, 3)])
def test_serving_pass(dev, block, T, k):
    H, F, E = 512, 256, 8
    w = block.make_weights(E, H, F, seed=3)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()
    out = block.Serving(w)(x, k)
    ids, _ = block.route(dev.block_norm(x, w_pre=w.w_in)["h"], w.router, k)
    want, _ = reference(x, w, ids, torch.zeros_like(x))
    assert (out.double() - want).norm() <= 4 * 2.0 ** -4 * (want - x.double()).norm()
