"""Host-side checks of the router's calls (no GPU work): every argument error is
refused before any launch. Pointers are fake and never dereferenced."""
import pytest
import torch

FAKE = 1 << 20
BF, FH, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


class _Stream:
    cuda_stream = 0


S = _Stream()


@pytest.fixture(scope="module")
def mp():
    from combine_fp8_quant_gb300 import build
    build.build()
    import combine_fp8_quant_gb300 as m
    m.load()
    return m


def call(mp, name, args, over):
    a = dict(args)
    assert set(over) <= set(a), over
    a.update(over)
    return getattr(mp, name)(*a.values(), stream=S)


ROUTE = dict(logits=FAKE, ldl=256, dtype=F32, T=64, d_num_tokens=None, E=256, K=8, score="softmax", bias=None, renorm=True,
             scale=1.0, topk_ids=FAKE, topk_weights=FAKE, d_status=None)
LOGITS = [dict(dtype=E4), dict(T=-1), dict(T=(1 << 30) + 1), dict(E=0), dict(E=1025, ldl=1025), dict(K=0), dict(K=33), dict(E=7, K=8), dict(ldl=255),
          dict(logits=None), dict(logits=FAKE + 2), dict(dtype=BF, logits=FAKE + 1), dict(d_num_tokens=FAKE + 2),
          dict(d_status=FAKE + 1)]


@pytest.mark.parametrize("over", LOGITS + [
    dict(topk_ids=None), dict(topk_weights=None), dict(topk_ids=FAKE + 2), dict(topk_weights=FAKE + 1), dict(bias=FAKE + 2),
])
def test_route_refuses(mp, over):
    assert call(mp, "moe_route", ROUTE, over) == mp.MOE_ERR_INVALID_ARG


def test_nothing_to_route(mp):
    assert call(mp, "moe_route", ROUTE, dict(T=0, logits=None, topk_ids=None, topk_weights=None)) == mp.MOE_OK
    assert call(mp, "moe_route_grad", GRAD, dict(T=0, logits=None, dlogits=None)) == mp.MOE_OK


BALANCE = dict(logits=FAKE, ldl=256, dtype=F32, T=64, d_num_tokens=None, E=256, topk_ids=FAKE, K=8, score="sigmoid", seq_begin=None,
               seq_end=None, Q=1, loss=FAKE, counts=FAKE, prob_sums=FAKE, workspace=FAKE, workspace_bytes=1 << 24, d_status=None)
GROUPS = [dict(Q=0), dict(Q=2), dict(Q=4097, seq_begin=FAKE, seq_end=FAKE), dict(seq_begin=FAKE), dict(seq_end=FAKE),
          dict(Q=2, seq_begin=FAKE + 1, seq_end=FAKE)]


@pytest.mark.parametrize("over", LOGITS + GROUPS + [
    dict(topk_ids=None), dict(loss=None), dict(counts=None), dict(prob_sums=None), dict(loss=FAKE + 2), dict(counts=FAKE + 1),
    dict(prob_sums=FAKE + 2), dict(workspace=None), dict(workspace=FAKE + 4), dict(workspace_bytes=1000),
])
def test_balance_loss_refuses(mp, over):
    assert call(mp, "moe_balance_loss", BALANCE, over) == mp.MOE_ERR_INVALID_ARG


GRAD = dict(logits=FAKE, ldl=256, dtype=F32, T=64, d_num_tokens=None, E=256, topk_ids=FAKE, K=8, score="softmax", renorm=True,
            scale=1.0, dweights=FAKE, dloss=FAKE, counts=FAKE, seq_begin=None, seq_end=None, Q=1, dlogits=FAKE, ldd=256, d_status=None)


@pytest.mark.parametrize("over", LOGITS + GROUPS + [
    dict(dweights=None, dloss=None), dict(counts=None), dict(topk_ids=None), dict(dlogits=None), dict(dlogits=FAKE + 2), dict(ldd=255),
    dict(dweights=FAKE + 2), dict(dloss=FAKE + 1), dict(counts=FAKE + 2), dict(topk_ids=FAKE + 2),
])
def test_route_grad_refuses(mp, over):
    assert call(mp, "moe_route_grad", GRAD, over) == mp.MOE_ERR_INVALID_ARG


def test_balance_workspace(mp):
    one = mp.moe_balance_loss_workspace_bytes(256, 1)
    assert 0 < one <= mp.moe_balance_loss_workspace_bytes(256, 64)
    assert [mp.moe_balance_loss_workspace_bytes(*v) for v in ((0, 1), (1025, 1), (8, 0), (8, 4097))] == [0] * 4


def test_binding_refuses(mp):
    """Shapes and types that the binding turns away itself, and tensors that are not on the device."""
    x, ids, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in (lambda: mp.route(x.double(), 2), lambda: mp.route(x[0], 2), lambda: mp.route(x.t(), 2),
                lambda: mp.route(x, 2, score="tanh"), lambda: mp.route(x, 2, bias=torch.zeros(15)), lambda: mp.route(x, 2),
                lambda: mp.balance_loss(x, ids.long()), lambda: mp.balance_loss(x, ids, seq_begin=ids[0]),
                lambda: mp.balance_loss(x, ids, ids[0], ids[0].long()), lambda: mp.balance_loss(x, ids),
                lambda: mp.route_grad(x, ids), lambda: mp.route_grad(x, ids, dloss=torch.zeros(2)),
                lambda: mp.route_grad(x, ids, dweights=w[:3]), lambda: mp.route_grad(x, ids, dweights=w, out=x.half()),
                lambda: mp.route_grad(x, ids, dweights=w)):
        with pytest.raises((ValueError, AssertionError, RuntimeError)):
            bad()


def test_status_clear_refuses(mp):
    assert mp.moe_status_clear(None, stream=S) == mp.MOE_ERR_INVALID_ARG
    assert mp.moe_status_clear(FAKE + 2, stream=S) == mp.MOE_ERR_INVALID_ARG
