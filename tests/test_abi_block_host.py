"""Host-side checks of the calls around the dispatch (no GPU work): every
argument error is refused before any launch. Pointers are fake and never
dereferenced."""
import pytest
import torch

FAKE = 1 << 20
ODD = FAKE + 4
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


PERMUTE = dict(x=FAKE, ldx=1024, dtype=BF, T=64, d_num_tokens=None, H=1024, topk_ids=FAKE, topk_weights=FAKE, K=8, E=256,
               L=32, block_e=128, xs=FAKE, m_indices=FAKE, bound=1 << 20, src2dst=FAKE, counts=FAKE, starts=FAKE, psum=FAKE,
               total=FAKE, row_weights=None, workspace=FAKE, workspace_bytes=1 << 20, d_status=FAKE)


@pytest.mark.parametrize("over", [
    dict(dtype=E4), dict(H=1020), dict(H=0), dict(H=32776, ldx=32776), dict(dtype=F32, H=1022), dict(ldx=1000), dict(ldx=1028),
    dict(x=ODD), dict(x=None), dict(xs=ODD), dict(xs=None), dict(K=0), dict(K=33), dict(L=0), dict(L=1025, E=2000), dict(E=31),
    dict(block_e=0), dict(T=-1), dict(T=1 << 18), dict(bound=100), dict(bound=1 << 31), dict(topk_ids=None),
    dict(src2dst=None), dict(m_indices=None), dict(counts=None), dict(starts=None), dict(psum=None), dict(total=None),
    dict(row_weights=FAKE, topk_weights=None), dict(workspace=None), dict(workspace=ODD), dict(workspace_bytes=64),
])
def test_permute_refuses(mp, over):
    assert call(mp, "moe_permute", PERMUTE, over) == mp.MOE_ERR_INVALID_ARG


COMBINE = dict(y=FAKE, ldy=1024, dtype=FH, R=100, src2dst=FAKE, w=FAKE, T=8, d_num_tokens=None, K=8, H=1024, out=FAKE,
               d_status=FAKE)


@pytest.mark.parametrize("over", [
    dict(dtype=E4), dict(H=1020), dict(ldy=1000), dict(ldy=1028), dict(y=ODD), dict(y=None), dict(K=0), dict(K=33), dict(T=-1),
    dict(R=-1), dict(src2dst=None), dict(out=None), dict(out=ODD),
])
def test_combine_refuses(mp, over):
    assert call(mp, "moe_combine_ex", COMBINE, over) == mp.MOE_ERR_INVALID_ARG


COMBINE_GRAD = dict(dout=FAKE, ldd=1024, y=FAKE, ldy=1024, dtype=BF, R=100, src2dst=FAKE, w=FAKE, T=8, d_num_tokens=None, K=8,
                    H=1024, dy=FAKE, lddy=1024, dw=FAKE, d_status=FAKE)


@pytest.mark.parametrize("over", [
    dict(dtype=E4), dict(H=1020), dict(ldd=1000), dict(ldy=1028), dict(lddy=1004), dict(dout=None), dict(dout=ODD), dict(y=None),
    dict(dy=ODD), dict(dy=None, dw=None), dict(K=33), dict(T=-1), dict(R=-1), dict(src2dst=None),
])
def test_combine_grad_refuses(mp, over):
    assert call(mp, "moe_combine_grad", COMBINE_GRAD, over) == mp.MOE_ERR_INVALID_ARG


NORM = dict(x=FAKE, ldx=1024, y=FAKE, ldy=1024, dtype=BF, T=8, H=1024, w_post=FAKE, gate=FAKE, gate_mode="channel", scale=1.0,
            w_pre=FAKE, eps=1e-6, x_out=FAKE, h=FAKE, rstd_post=None, rstd_pre=None)


@pytest.mark.parametrize("over", [
    dict(dtype=E4), dict(T=-1), dict(H=1020), dict(H=0), dict(H=16392, ldx=16392, ldy=16392), dict(dtype=F32, H=8196, ldx=8196),
    dict(x=None), dict(x=ODD), dict(ldx=1000), dict(ldy=1004), dict(y=ODD), dict(y=None), dict(y=None, gate_mode="none"),
    dict(y=None, w_post=None, gate_mode="none", w_pre=None), dict(gate=None), dict(gate=ODD), dict(w_post=ODD), dict(w_pre=ODD),
    dict(x_out=None), dict(h=None), dict(eps=-1.0), dict(eps=float("nan")),
])
def test_block_norm_refuses(mp, over):
    assert call(mp, "moe_block_norm", NORM, over) == mp.MOE_ERR_INVALID_ARG


NORM_GRAD = dict(dx_out=FAKE, ld_dxo=1024, dh=FAKE, ld_dh=1024, x_out=FAKE, ldx=1024, y=FAKE, ldy=1024, dtype=BF, T=8, H=1024,
                 w_post=FAKE, gate=FAKE, gate_mode="channel", scale=1.0, w_pre=FAKE, rstd_post=FAKE, rstd_pre=FAKE, dx=FAKE,
                 dy=FAKE, dw_post=FAKE, dgate=FAKE, dw_pre=FAKE, workspace=FAKE, workspace_bytes=1 << 24)


@pytest.mark.parametrize("over", [
    dict(dtype=E4), dict(H=1020), dict(T=-1), dict(dx_out=ODD), dict(ld_dxo=1000), dict(dh=None), dict(ld_dh=1004), dict(x_out=None),
    dict(y=ODD), dict(y=None), dict(rstd_post=None), dict(rstd_pre=None), dict(dx=None), dict(dy=None), dict(dw_post=None),
    dict(dw_pre=None), dict(dgate=None), dict(gate_mode="token", dgate=None), dict(workspace=None), dict(workspace_bytes=100),
    dict(gate=None),
])
def test_block_norm_grad_refuses(mp, over):
    assert call(mp, "moe_block_norm_grad", NORM_GRAD, over) == mp.MOE_ERR_INVALID_ARG


MATMUL = dict(x=FAKE, ldx=512, dtype=BF, x_scales=None, ld_xs=0, R=1024, K=512, w=FAKE, w_scales=None, ld_ws=0, L=4, N=256,
              gated=True, act="silu", bias=None, seg_begin=FAKE, seg_end=FAKE, cap=0, residual=None, ld_res=0, out=FAKE, ldo=256,
              out_dtype=BF, pre=None, ld_pre=0, d_status=FAKE)
E4M3 = dict(dtype=E4, x_scales=FAKE, ld_xs=1024, w_scales=FAKE, ld_ws=2048)


@pytest.mark.parametrize("over", [
    dict(dtype=F32), dict(out_dtype=FH), dict(out_dtype=F32), dict(R=-1), dict(R=1 << 31), dict(L=0), dict(L=1025), dict(K=0),
    dict(K=508), dict(N=0), dict(N=248), dict(gated=False, N=252), dict(N=1 << 29), dict(seg_begin=None), dict(seg_end=None),
    dict(seg_begin=None, seg_end=None), dict(cap=256), dict(seg_begin=None, cap=100), dict(cap=-1), dict(x=None), dict(x=ODD),
    dict(ldx=500), dict(ldx=516), dict(w=None), dict(w=ODD), dict(out=None), dict(ldo=200), dict(residual=FAKE, ld_res=100),
    dict(pre=FAKE, ld_pre=256), dict(out=FAKE + 1), dict(residual=FAKE + 1, ld_res=256), dict(pre=FAKE + 1, ld_pre=512),
    dict(bias=FAKE + 2),
    dict(E4M3, K=576, ldx=576), dict(E4M3, x_scales=None), dict(E4M3, w_scales=None), dict(E4M3, ld_xs=1000), dict(E4M3, ld_xs=1026),
    dict(E4M3, ld_ws=2044), dict(E4M3, ld_ws=2050), dict(E4M3, pre=FAKE, ld_pre=512), dict(E4M3, out_dtype=F32), dict(E4M3, ldx=520),
])
def test_expert_matmul_refuses(mp, over):
    assert call(mp, "moe_expert_matmul", MATMUL, over) == mp.MOE_ERR_INVALID_ARG


GRAD = dict(dout=FAKE, ldd=256, x=FAKE, ldx=512, dtype=BF, R=1024, K=512, w=FAKE, L=4, N=256, gated=True, act="silu", pre=FAKE,
            ld_pre=512, seg_begin=FAKE, seg_end=FAKE, cap=0, dx=FAKE, ld_dx=512, dw=FAKE, dw_dtype=BF, dbias=FAKE, workspace=FAKE,
            workspace_bytes=1 << 30, d_status=FAKE)


@pytest.mark.parametrize("over", [
    dict(dtype=E4), dict(dtype=F32), dict(R=-1), dict(L=0), dict(K=508), dict(N=250), dict(dx=None, dw=None, dbias=None),
    dict(dw_dtype=FH), dict(dw_dtype=E4), dict(dout=None), dict(dout=ODD), dict(ldd=200), dict(ldd=260), dict(pre=None),
    dict(ld_pre=256), dict(x=None), dict(ldx=500), dict(w=None), dict(ld_dx=500), dict(workspace=None), dict(workspace_bytes=1000),
    dict(seg_begin=None), dict(cap=256), dict(dx=FAKE + 1), dict(dw=FAKE + 1), dict(dw=FAKE + 2, dw_dtype=F32), dict(dbias=FAKE + 2),
])
def test_expert_matmul_grad_refuses(mp, over):
    assert call(mp, "moe_expert_matmul_grad", GRAD, over) == mp.MOE_ERR_INVALID_ARG


def test_workspace_sizes(mp):
    assert mp.moe_block_norm_workspace_bytes(0, 64) == 2 * 64 * 4
    assert mp.moe_block_norm_workspace_bytes(100000, 64) == mp.moe_block_norm_workspace_bytes(304, 64)
    assert mp.moe_block_norm_workspace_bytes(-1, 64) == 0
    assert mp.moe_expert_matmul_grad_workspace_bytes(0, 4, 64) == 0
    assert mp.moe_expert_matmul_grad_workspace_bytes(1000, 4, 64) >= 1000 * 64 * 2
    assert mp.moe_expert_matmul_grad_workspace_bytes(-1, 4, 64) == 0


def test_the_binding_refuses(mp):
    """Wrong shapes, types, strides and devices raise before the library is called."""
    x, w = torch.zeros(8, 64, dtype=BF), torch.zeros(2, 32, 64, dtype=BF)
    seg = torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: mp.expert_matmul(x, w),                                            # two experts, no segments
        lambda: mp.expert_matmul(x, w, seg),                                       # starts without psum
        lambda: mp.expert_matmul(x, w, seg, seg, masked_m=seg),
        lambda: mp.expert_matmul(x, w, seg.long(), seg.long()),
        lambda: mp.expert_matmul(x, w, seg, seg, act="tanh"),
        lambda: mp.expert_matmul(x, w.half(), seg, seg),
        lambda: mp.expert_matmul(x.float(), w.float(), seg, seg),
        lambda: mp.expert_matmul(x.to(torch.int8), w.to(torch.int8), seg, seg),
        lambda: mp.expert_matmul(x[:, :32], w, seg, seg),
        lambda: mp.expert_matmul(x.t(), w, seg, seg),
        lambda: mp.expert_matmul(x, w, seg, seg, bias=torch.zeros(2, 31)),
        lambda: mp.expert_matmul(x, w, seg, seg, out=torch.zeros(8, 31, dtype=BF)),
        lambda: mp.expert_matmul(x, w, masked_m=seg),                              # slabs are 3-D
        lambda: mp.expert_matmul(x.to(E4), w.to(E4), seg, seg),                    # no scales
        lambda: mp.expert_matmul(x, w, seg, seg),                                  # all well, but on the CPU
        lambda: mp.expert_matmul_grad(x[:, :32], x, w, seg, seg, act="silu"),      # no pre
        lambda: mp.expert_matmul_grad(x, x, w, seg, seg),                          # dout is [8, 32]
        lambda: mp.permute(x.to(E4), seg.view(2, 1), torch.zeros(2, 1), 4, 4),
        lambda: mp.permute(x, torch.zeros(8, 2), torch.zeros(8, 2), 4, 4),
        lambda: mp.combine_grad(x, x[:4].float(), seg.view(2, 1)),
        lambda: mp.permute_grad(x.t(), seg.view(2, 1)),
        lambda: mp.block_norm(x, x[:4]),
        lambda: mp.block_norm(x, x, gate=torch.zeros(5)),
        lambda: mp.block_norm(x, x, w_post=torch.zeros(64, dtype=BF)),
        lambda: mp.block_norm(x, w_pre=torch.zeros(64)),                           # all well, but on the CPU
        lambda: mp.block_norm_grad(x, x, x[:, :32], w_pre=torch.zeros(32)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")


def test_a_gate_that_fits_both_kinds_is_named(mp):
    x, g = torch.zeros(8, 8), torch.ones(8)
    for call in (lambda **k: mp.block_norm(x, x, gate=g, **k), lambda **k: mp.block_norm_grad(x, None, x, x, gate=g, **k)):
        with pytest.raises(ValueError, match="gate_mode"):
            call()
        with pytest.raises(ValueError, match="gate_mode"):
            call(gate_mode="row")
    kind = mp.moeperm._gate_mode
    assert kind(g, 8, 8, "token") == "token" and kind(g, 8, 8, "channel") == "channel"
    assert kind(g[None], 8, 8) == "channel" and kind(g[:, None], 8, 8) == "token"
    assert kind(g, 8, 16) == "token" and kind(g, 16, 8) == "channel" and kind(None, 8, 8) == "none"
    for args in ((g, 8, 16, "channel"), (g, 16, 8, "token"), (g[None], 8, 8, "token"), (g, 4, 16)):
        with pytest.raises(ValueError):
            kind(*args)


def test_combine_refuses_what_does_not_fit(mp):
    """The output is written in y's type: any other type, shape or layout would be written past or misread."""
    T, K, R, H = 4, 2, 6, 64
    y, row, w = torch.zeros(R, H), torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)
    bad = [
        ("out", dict(out=torch.zeros(T, H, dtype=BF))),                       # half of what fp32 rows need
        ("out", dict(y=y.half(), out=torch.zeros(T, H, dtype=BF))),
        ("out", dict(y=y.half(), out=torch.zeros(T, H, dtype=torch.int16))),
        ("out", dict(out=torch.zeros(T - 1, H))),
        ("out", dict(out=torch.zeros(H, T))),
        ("out", dict(out=torch.zeros(T * H))),
        ("out", dict(out=torch.zeros(T, 2 * H)[:, :H])),
        ("y", dict(y=y.double())),
        ("y", dict(y=torch.zeros(R, H, dtype=torch.int32))),
        ("y", dict(y=y.to(E4))),
        ("y", dict(y=torch.zeros(H, R).t())),
        ("y", dict(y=torch.zeros(R, 1, H))),
        ("src2dst", dict(src2dst=row.long())),
        ("src2dst", dict(src2dst=torch.zeros(K, T, dtype=torch.int32).t())),
        ("weights", dict(weights=w.double())),
        ("weights", dict(weights=w[:, :1])),
        ("weights", dict(weights=w[:-1])),
        ("weights", dict(weights=torch.zeros(K, T).t())),
    ]
    for what, over in bad:
        with pytest.raises(ValueError, match=f"moeperm: (the rows of )?{what} must"):
            mp.combine(**dict(dict(y=y, src2dst=row, weights=w), **over))
    fits = [dict(), dict(y=y.to(BF)), dict(y=y.to(BF), out=torch.zeros(T + 3, H, dtype=BF)), dict(weights=torch.zeros(T + 1, K)),
            dict(y=torch.zeros(R, H, dtype=torch.int16)), dict(y=y.to(BF), out=torch.zeros(T, H, dtype=torch.int16))]
    for over in fits:  # all well, but on the CPU
        with pytest.raises(ValueError, match="must be on a CUDA device"):
            mp.combine(**dict(dict(y=y, src2dst=row, weights=w), **over))


def test_expert_matmul_refuses_scales_that_do_not_hold_the_rows(mp):
    """Packed words of every row and group: fewer would be read past their end, other formats misread."""
    L, N, K, R, cap = 2, 32, 640, 10, 8  # five groups: two words a row
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    x, w, seg = torch.zeros(R, K, dtype=torch.uint8), torch.zeros(L, N, K, dtype=torch.uint8), i32(L)
    args = dict(x=x, w=w, starts=seg, psum=seg, x_scales=i32(1, 2, 12), ld_xs=12, w_scales=i32(2, 64), ld_ws=64)
    slabs = dict(x=torch.zeros(L, cap, K, dtype=torch.uint8), starts=None, psum=None, masked_m=seg, x_scales=i32(L, 2, cap),
                 ld_xs=cap)
    bad = [
        ("x_scales", dict(x_scales=i32(1, 1, 12))),                         # one word a row
        ("x_scales", dict(x_scales=i32(1, 2, 12)[:, :, :8].contiguous())),  # eight rows
        ("x_scales", dict(ld_xs=16)),
        ("x_scales", dict(x_scales=torch.zeros(R, 5, dtype=torch.uint8), ld_xs=12)),
        ("x_scales", dict(x_scales=torch.zeros(R, 5), ld_xs=12)),
        ("x_scales", dict(x_scales=i32(12, 2).t())),                        # a word's rows are not neighbours
        ("w_scales", dict(w_scales=i32(1, 64))),
        ("w_scales", dict(w_scales=i32(2, 32), ld_ws=64)),
        ("w_scales", dict(w_scales=torch.zeros(64, 5, dtype=torch.uint8))),
        ("x_scales", dict(slabs, x_scales=i32(1, 2, cap))),                 # one expert's block
        ("x_scales", dict(slabs, x_scales=i32(L, 1, cap))),
    ]
    for what, over in bad:
        with pytest.raises(ValueError, match=f"moeperm: {what} must"):
            mp.expert_matmul(**dict(args, **over))
    fits = [dict(), slabs, dict(x_scales=i32(2, 12)[:, :R]), dict(x_scales=i32(30)), dict(x_scales=i32(4, 12))]
    for over in fits:  # all well, but on the CPU
        with pytest.raises(ValueError, match="must be on a CUDA device"):
            mp.expert_matmul(**dict(args, **over))


@pytest.mark.parametrize("over", [
    dict(T=0, gate=None), dict(T=0, gate=ODD), dict(T=0, y=None, gate=None), dict(T=0, w_post=ODD), dict(T=0, w_pre=ODD),
    dict(T=0, gate=FAKE + 2, gate_mode="channel"), dict(gate=FAKE + 2, gate_mode="token"),
])
def test_block_norms_refuse_a_gate_that_is_read_without_tokens(mp, over):
    """The gradient launches for T = 0 too (its sums are zeros) and reads a gate per channel."""
    for name, args in (("moe_block_norm", NORM), ("moe_block_norm_grad", NORM_GRAD)):
        assert call(mp, name, args, over) == mp.MOE_ERR_INVALID_ARG, name


@pytest.mark.parametrize("L,Nw", [(1, 64), (4, 200), (16, 2816), (64, 2816), (1000, 16)])
def test_a_gradient_workspace_serves_fewer_rows(mp, L, Nw):
    """Sized for the largest batch, it is enough for every smaller one, on both sides of 128 rows an expert."""
    edges = {0, 1, 63, 64, 65, 8000, 12000, 100_000, 1_000_000}
    for m in (1, 32, 64, 127, 128, 129, 255, 256, 257, 1024, 8192):
        edges |= {m * L - 1, m * L, m * L + 1}
    sizes = [mp.moe_expert_matmul_grad_workspace_bytes(R, L, Nw) for R in sorted(edges)]
    assert sizes == sorted(sizes)


WORDS = {  # 32-bit vectors of each call
    "moe_permute": (PERMUTE, "d_num_tokens topk_ids topk_weights m_indices src2dst counts starts psum total row_weights d_status"),
    "moe_combine_ex": (COMBINE, "src2dst w d_num_tokens d_status"),
    "moe_combine_grad": (COMBINE_GRAD, "src2dst w d_num_tokens dw d_status"),
    "moe_block_norm": (NORM, "rstd_post rstd_pre"),
    "moe_block_norm_grad": (NORM_GRAD, "rstd_post rstd_pre dw_post dgate dw_pre"),
    "moe_expert_matmul": (MATMUL, "seg_begin seg_end d_status bias"),
    "moe_expert_matmul_grad": (GRAD, "seg_begin seg_end d_status dbias"),
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, (_, args) in WORDS.items() for a in args.split()])
def test_vectors_of_words_start_at_a_word(mp, name, arg):
    """Kernels read and write them an element at a time, which faults at any other address."""
    assert call(mp, name, WORDS[name][0], {arg: FAKE + 2}) == mp.MOE_ERR_INVALID_ARG
