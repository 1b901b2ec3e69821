"""Host-side checks of the four-bit calls (no GPU work): every argument error is
refused before any launch. Pointers are fake and never dereferenced."""
import pytest
import torch

FAKE = 1 << 20
ODD = FAKE + 8
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


QUANT = dict(x=FAKE, ldx=512, dtype=BF, R=128, H=512, fmt="nv", tensor_scale=None, n_scales=1, d_num_live=None, m_indices=None,
             masked_m=None, cap=0, xq=FAKE, scales=FAKE, ld_s=128, d_status=None)
ROWS = [dict(dtype=E4), dict(R=-1), dict(R=1 << 31, ld_s=1 << 31), dict(H=0), dict(H=480), dict(H=-64), dict(x=None), dict(x=ODD), dict(ldx=511),
        dict(ldx=516), dict(dtype=F32, ldx=514), dict(xq=None), dict(xq=ODD), dict(scales=None), dict(scales=ODD), dict(ld_s=127),
        dict(tensor_scale=FAKE, n_scales=0), dict(tensor_scale=FAKE, n_scales=3), dict(tensor_scale=FAKE + 2),
        dict(tensor_scale=FAKE, fmt="mx"), dict(d_num_live=FAKE, m_indices=FAKE), dict(m_indices=FAKE, masked_m=FAKE, cap=64),
        dict(masked_m=FAKE), dict(masked_m=FAKE, cap=100), dict(m_indices=FAKE + 1), dict(d_status=FAKE + 2)]


@pytest.mark.parametrize("over", ROWS)
def test_quant_refuses(mp, over):
    assert call(mp, "moe_quant_fp4", QUANT, over) == mp.MOE_ERR_INVALID_ARG


DEQUANT = dict(xq=FAKE, scales=FAKE, ld_s=128, R=128, H=512, fmt="nv", tensor_scale=None, n_scales=1, d_num_live=None, m_indices=None,
               masked_m=None, cap=0, x=FAKE, ldx=512, dtype=BF, d_status=None)


@pytest.mark.parametrize("over", ROWS)
def test_dequant_refuses(mp, over):
    assert call(mp, "moe_dequant_fp4", DEQUANT, over) == mp.MOE_ERR_INVALID_ARG


DISPATCH = dict(x=FAKE, ldx=1024, dtype=BF, T=64, d_num_tokens=None, H=1024, topk_ids=FAKE, topk_weights=FAKE, K=8, E=256, L=32,
                block_e=128, fmt="nv", tensor_scale=None, xq=FAKE, scales=FAKE, ld_s=1 << 20, m_indices=FAKE, bound=1 << 20,
                src2dst=FAKE, counts=FAKE, starts=FAKE, psum=FAKE, total=FAKE, row_weights=None, workspace=FAKE,
                workspace_bytes=1 << 20, d_status=FAKE)


@pytest.mark.parametrize("over", [
    dict(dtype=E4), dict(H=1040, ldx=1040), dict(H=0), dict(H=32832, ldx=32832), dict(ldx=1000), dict(ldx=1028), dict(x=ODD), dict(x=None),
    dict(xq=ODD), dict(xq=None), dict(scales=None), dict(scales=ODD), dict(ld_s=(1 << 20) - 1), dict(K=0), dict(K=33), dict(L=0),
    dict(L=1025, E=2000), dict(E=31), dict(block_e=0), dict(T=-1), dict(T=1 << 18), dict(bound=100), dict(bound=1 << 31, ld_s=1 << 31),
    dict(topk_ids=None), dict(src2dst=None), dict(m_indices=None), dict(counts=None), dict(starts=None), dict(psum=None),
    dict(total=None), dict(row_weights=FAKE, topk_weights=None), dict(workspace=None), dict(workspace=ODD),
    dict(workspace_bytes=64), dict(fmt="e8m0", tensor_scale=FAKE), dict(tensor_scale=FAKE + 1),
])
def test_dispatch_refuses(mp, over):
    assert call(mp, "moe_dispatch_fp4", DISPATCH, over) == mp.MOE_ERR_INVALID_ARG


MATMUL = dict(x=FAKE, ldx=256, x_scales=FAKE, ld_xs=1024, x_tscale=None, R=1024, K=512, w=FAKE, w_scales=FAKE, ld_ws=2048,
              w_tscale=None, fmt="nv", L=4, N=256, gated=True, act="silu", bias=None, seg_begin=FAKE, seg_end=FAKE, cap=0,
              residual=None, ld_res=0, out=FAKE, ldo=256, out_dtype=BF, d_status=FAKE)


@pytest.mark.parametrize("over", [
    dict(out_dtype=F32), dict(out_dtype=E4), dict(R=-1), dict(R=1 << 31), dict(L=0), dict(L=1025), dict(K=0), dict(K=544), dict(N=0), dict(N=248),
    dict(gated=False, N=252), dict(N=1 << 29), dict(seg_begin=None), dict(seg_end=None), dict(seg_begin=None, seg_end=None), dict(cap=256),
    dict(seg_begin=None, cap=100), dict(cap=-1), dict(x=None), dict(x=ODD), dict(ldx=255), dict(ldx=264), dict(w=None), dict(w=ODD),
    dict(x_scales=None), dict(x_scales=ODD), dict(ld_xs=1023), dict(w_scales=None), dict(w_scales=ODD), dict(ld_ws=2047),
    dict(out=None), dict(ldo=200), dict(out=FAKE + 1), dict(residual=FAKE, ld_res=100), dict(residual=FAKE + 1, ld_res=256),
    dict(bias=FAKE + 2), dict(fmt="mx", x_tscale=FAKE), dict(fmt="e8m0", w_tscale=FAKE), dict(x_tscale=FAKE + 2), dict(w_tscale=FAKE + 1),
])
def test_expert_matmul_refuses(mp, over):
    assert call(mp, "moe_expert_matmul_fp4", MATMUL, over) == mp.MOE_ERR_INVALID_ARG


def test_nothing_to_do(mp):
    none = dict(R=0, x=None, xq=None, scales=None, ld_s=0)
    assert call(mp, "moe_quant_fp4", QUANT, none) == mp.MOE_OK
    assert call(mp, "moe_dequant_fp4", DEQUANT, none) == mp.MOE_OK
    assert call(mp, "moe_expert_matmul_fp4", MATMUL, dict(R=0, x=None, x_scales=None, out=None)) == mp.MOE_OK


def test_scale_bytes(mp):
    assert mp.moe_fp4_scale_bytes(100, 7168, "nv") == 28 * 100 * 16 and mp.moe_fp4_scale_bytes(100, 7168, "mx") == 14 * 100 * 16
    assert mp.moe_fp4_scale_bytes(3, 64, "e8m0") == 48 and mp.moe_fp4_scale_bytes(3, 320, "nv") == 96
    assert mp.moe_fp4_scale_bytes(3, 100, "nv") == 0 and mp.moe_fp4_scale_bytes(-1, 64, "nv") == 0


def test_binding_refuses(mp):
    """Shapes and types that the binding turns away itself, and tensors that are not on the device."""
    x, q, sc = torch.zeros(8, 128), torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(1, 8, 16, dtype=torch.uint8)
    w, ids, tw = torch.zeros(2, 16, 64, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.int32), torch.zeros(8, 2)
    one, seg = torch.ones(1), torch.zeros(2, dtype=torch.int32)
    wsc = torch.zeros(1, 32, 16, dtype=torch.uint8)
    for bad in (lambda: mp.quant_fp4(x.double()), lambda: mp.quant_fp4(x, fmt="fp4"), lambda: mp.quant_fp4(x, fmt="mx", tensor_scale=one),
                lambda: mp.quant_fp4(x, num_live=seg[:1], m_indices=torch.zeros(8, dtype=torch.int32)), lambda: mp.quant_fp4(x.t()),
                lambda: mp.quant_fp4(x, m_indices=seg), lambda: mp.quant_fp4(x, masked_m=torch.zeros(3, dtype=torch.int32)),
                lambda: mp.quant_fp4(x), lambda: mp.dequant_fp4(q.float(), sc), lambda: mp.dequant_fp4(q, sc[:, :7]),
                lambda: mp.dequant_fp4(q, sc.int()), lambda: mp.dequant_fp4(q, sc, out=x[:, :64]), lambda: mp.dequant_fp4(q, sc, dtype=torch.int8),
                lambda: mp.dequant_fp4(q, sc), lambda: mp.dispatch_fp4(x, ids.long(), tw, 2, 2), lambda: mp.dispatch_fp4(x, ids, tw, 2, 2, fmt="x"),
                lambda: mp.dispatch_fp4(x, ids, tw, 2, 2), lambda: mp.expert_matmul_fp4(q, w.float(), sc, wsc, starts=seg, psum=seg),
                lambda: mp.expert_matmul_fp4(q, w, sc, wsc[:, :31], starts=seg, psum=seg), lambda: mp.expert_matmul_fp4(q, w, sc, wsc),
                lambda: mp.expert_matmul_fp4(q, w, sc, wsc, starts=seg, psum=seg, w_tscale=one),
                lambda: mp.expert_matmul_fp4(q, w, sc, wsc, starts=seg, psum=seg, act="tanh"),
                lambda: mp.expert_matmul_fp4(q, w, sc, wsc, starts=seg, psum=seg, out_dtype=torch.float32),
                lambda: mp.expert_matmul_fp4(q, w, sc, wsc, starts=seg, psum=seg)):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
