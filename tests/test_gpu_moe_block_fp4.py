"""The example's block with its router's losses and in four bits: gradients against
torch's autograd on the formulas in 64 bits, and the four-bit serving pass against
the same block.

Bounds on norms. Training: a chain of about ten roundings to bf16 (2^-8 each,
independent), as for the block without the losses. Four bits: with a group's largest
element at 6, half a step of e2m1 is 1 at most and the steps' errors are below 2 / sqrt(12) on
average, against an rms of about 6 / 1.8 in a group of 16 normal values: 2^-2.5 of a
tensor's norm. Rows, activations and both weights are rounded so, and errors of sums
average: 4 * 2^-2.5 bounds the block's update."""
import pytest
import torch

from test_gpu_moe_block import block, reference  # noqa: F401  (block is a fixture)

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


@pytest.mark.parametrize("T,H,F,E,k", [(1, 128, 64, 4, 2), (37, 256, 128, 8, 3), (300, 512, 256, 6, 2)])
def test_training_step_with_the_routers_losses(dev, block, T, H, F, E, k):  # noqa: F811
    w = block.make_weights(E, H, F, seed=T)
    x = torch.randn(T, H, device="cuda", generator=gen(1)).bfloat16()
    dout = torch.randn(T, H, device="cuda", generator=gen(2)).bfloat16()
    coef = torch.tensor([20.0, 3.0], device="cuda")  # (large, so that the losses' part counts)
    out, saved = block.forward(x, w, k, coef=coef)
    g = block.backward(dout, saved, w)
    assert dev.moe_status_sync(saved["seg"]["status"]) == dev.MOE_OK
    want, gw = reference(x, w, saved["ids"], dout)
    # the losses' own gradients of the router and of what it reads
    v = {n: t.double().requires_grad_() for n, t in (("x", x), ("w_in", w.w_in), ("router", w.router))}
    rms = v["x"] * torch.rsqrt((v["x"] * v["x"]).mean(1, keepdim=True) + 1e-6)
    logits = (rms * v["w_in"]) @ v["router"].t()
    counts = torch.bincount(saved["ids"].reshape(-1).long(), minlength=E).double()
    balance = E / (k * T * T) * (counts * torch.softmax(logits, 1).sum(0)).sum()
    z = (torch.logsumexp(logits, 1) ** 2).mean()
    for got, loss in zip(saved["loss"].tolist(), (balance.item(), z.item())):
        assert abs(got - loss) <= 10 * 2.0 ** -8 * loss
    (coef[0].double() * balance + coef[1].double() * z).backward()
    assert (out.double() - want).norm() <= 10 * 2.0 ** -8 * want.norm()
    for name, ref in gw.items():
        ref = ref + v[name].grad if name in v else ref
        assert (g[name].double() - ref).norm() <= 10 * 2.0 ** -8 * ref.norm(), name


@pytest.mark.parametrize("T,k", [(1, 2), (64, 3), (700, 4)])
def test_serving_pass_in_four_bits(dev, block, T, k):  # noqa: F811
    H, F, E = 512, 256, 8
    w = block.make_weights(E, H, F, seed=3)
    x = torch.randn(T, H, device="cuda", generator=gen(4)).bfloat16()
    out = block.Serving4(w)(x, k)
    ids, _ = block.route(dev.block_norm(x, w_pre=w.w_in)["h"], w.router, k)
    want, _ = reference(x, w, ids, torch.zeros_like(x))
    assert torch.isfinite(out).all()
    assert (out.double() - want).norm() <= 4 * 2.0 ** -2.5 * (want - x.double()).norm()
    assert torch.equal(out, block.Serving4(w)(x, k))
