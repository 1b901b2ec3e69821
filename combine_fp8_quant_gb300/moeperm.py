"""Python binding of libmoeperm (include/moeperm.h).

Thin marshalling only: every function here passes device pointers, sizes and
the current CUDA stream of torch to the C ABI of the same name. All arithmetic
of the path runs in the library's sm_103a kernels; there is no CPU fallback.
If the shared library is missing or cannot be loaded, loading raises.

Two layers:
  * ``moe_*`` / ``fp8_requant_per_tensor``: one-to-one with the C calls, taking
    torch tensors (or None) and returning the status code.
  * ``dispatch_compact`` / ``dispatch_masked`` / ``quant_group`` / ``combine`` /
    ``expand_to_slab`` / ``expand_from_slab`` / ``requant``: allocate the output
    tensors with torch (device memory is PyTorch's job) and call the C ABI.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoeperm.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_OVERFLOW = 0, 1, 2
MOE_ERR_LIVE_OVERFLOW, MOE_ERR_BAD_LAYOUT, MOE_ERR_CUDA, MOE_ERR_TIMEOUT = 3, 4, 5, 6
STATUS_OVERFLOW, STATUS_LIVE_OVERFLOW, STATUS_BAD_LAYOUT, STATUS_TIMEOUT = 1, 2, 4, 8
FMT = {"u8": 0, "packed": 1, "f32pow2": 2, "f32": 3, "mx": 4}

ELEM = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
GATE = {"none": 0, "channel": 1, "token": 2}
SCORE = {"softmax": 0, "sigmoid": 1}
FP4 = {"e8m0": 0, "mx": 1, "nv": 2}

_lock = threading.Lock()
_lib = None


class MoePermError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = _lib.moe_status_string(code).decode() if _lib is not None else str(code)
        super().__init__(f"{where}: {msg} (status {code})")


def load(path: str | None = None):
    """Load libmoeperm.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"libmoeperm.so not found at {p}: build it first (python -c "
                "'import __graft_entry__ as g; g.build()'). There is no CPU fallback.")
        lib = C.CDLL(p)
        _declare(lib)
        _lib = lib
        return lib


def _declare(L):
    vp, i32, i64, sz, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.c_float
    sig = {
        "moe_compact_bound": (i64, [i64, i32, i32]),
        "moe_should_use_masked": (i32, [i32, i32]),
        "moe_scale_bytes": (sz, [i32, i64, i32, i32]),
        "moe_workspace_bytes": (sz, [i32, i32, i32]),
        "moe_dispatch_compact": (i32, [vp, i64, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                       vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "moe_dispatch_masked": (i32, [vp, i64, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                      vp, vp, i64, vp, vp, vp, vp, i32, vp, sz, vp, vp]),
        "moe_dispatch_compact_noalloc": (i32, [vp, i64, i32, vp, i32, vp, vp, i32, i32, i32, i32,
                                               i32, i32, vp, vp, i64, vp, i64, vp, vp, vp, vp, vp,
                                               vp, vp, vp]),
        "moe_quant_group": (i32, [vp, i64, i32, vp, i32, i32, i32, vp, vp, i64, vp, vp]),
        "moe_combine": (i32, [vp, i64, i64, vp, vp, i32, vp, i32, i32, vp, vp, vp]),
        "moe_expand_to_slab": (i32, [vp, i32, i32, i64, vp, i64, vp, i32, i32, i32, i32, i32, vp,
                                     vp, i64, vp, vp, vp]),
        "moe_expand_from_slab": (i32, [vp, i32, i32, vp, i64, vp, i32, i32, i32, i32, i32, vp, vp,
                                       i64, vp, i64, vp, vp, vp]),
        "fp8_requant_per_tensor": (i32, [vp, i64, vp, i32, i32, vp, vp, vp]),
        "fp8_requant_per_tensor_ex": (i32, [vp, i64, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]),
        "moe_permute": (i32, [vp, i64, i32, i32, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, i64,
                              vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "moe_combine_ex": (i32, [vp, i64, i32, i64, vp, vp, i32, vp, i32, i32, vp, vp, vp]),
        "moe_combine_grad": (i32, [vp, i64, vp, i64, i32, i64, vp, vp, i32, vp, i32, i32, vp, i64,
                                   vp, vp, vp]),
        "moe_block_norm": (i32, [vp, i64, vp, i64, i32, i32, i32, vp, vp, i32, f32, vp, f32, vp, vp,
                                 vp, vp, vp]),
        "moe_block_norm_workspace_bytes": (sz, [i32, i32]),
        "moe_block_norm_grad": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32, vp, vp, i32,
                                      f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_expert_matmul": (i32, [vp, i64, i32, vp, i64, i64, i32, vp, vp, i64, i32, i32, i32, i32,
                                    vp, vp, vp, i32, vp, i64, vp, i64, i32, vp, i64, vp, vp]),
        "moe_expert_matmul_grad_workspace_bytes": (sz, [i64, i32, i32]),
        "moe_expert_matmul_grad": (i32, [vp, i64, vp, i64, i32, i64, i32, vp, i32, i32, i32, i32, vp,
                                         i64, vp, vp, i32, vp, i64, vp, i32, vp, vp, sz, vp, vp]),
        "moe_fp4_scale_bytes": (sz, [i64, i32, i32]),
        "moe_quant_fp4": (i32, [vp, i64, i32, i64, i32, i32, vp, i32, vp, vp, vp, i32, vp, vp, i64, vp, vp]),
        "moe_dequant_fp4": (i32, [vp, vp, i64, i64, i32, i32, vp, i32, vp, vp, vp, i32, vp, i64, i32, vp, vp]),
        "moe_dispatch_fp4": (i32, [vp, i64, i32, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, i64,
                                   vp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "moe_expert_matmul_fp4": (i32, [vp, i64, vp, i64, vp, i64, i32, vp, vp, i64, vp, i32, i32, i32, i32, i32,
                                        vp, vp, vp, i32, vp, i64, vp, i64, i32, vp, vp]),
        "moe_route": (i32, [vp, i64, i32, i32, vp, i32, i32, i32, vp, i32, f32, vp, vp, vp, vp]),
        "moe_balance_loss_workspace_bytes": (sz, [i32, i32]),
        "moe_balance_loss": (i32, [vp, i64, i32, i32, vp, i32, vp, i32, i32, vp, vp, i32, vp, vp, vp, vp,
                                   sz, vp, vp]),
        "moe_route_grad": (i32, [vp, i64, i32, i32, vp, i32, vp, i32, i32, i32, f32, vp, vp, vp, vp, vp,
                                 i32, vp, i64, vp, vp]),
        "moe_status_sync": (i32, [vp, vp]),
        "moe_status_clear": (i32, [vp, vp]),
        "moe_status_string": (C.c_char_p, [i32]),
        "moe_version": (C.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args


def lib():
    return _lib if _lib is not None else load()


def _ptr(t):
    """Device address of a CUDA tensor (or a raw integer address, or None).
    A CPU tensor is rejected here: its host address would reach a kernel.
    Plain integers go to ctypes as they are (a void* argument accepts them)."""
    if t is None:
        return None
    if type(t) is int:
        return t
    if not t.is_cuda:
        raise ValueError(f"moeperm: tensor on {t.device}, but every tensor argument must be on "
                         "a CUDA device")
    return t.data_ptr()


def _off_device(t):
    raise ValueError(f"moeperm: tensor on {t.device}, but every tensor argument must be on a CUDA "
                     "device")


def _ptrs(*tensors):
    """_ptr of several tensors (or None) at once: the helpers below go straight to
    the library with these, which saves a small call a few microseconds."""
    return [None if t is None else t.data_ptr() if t.is_cuda else _off_device(t) for t in tensors]


def _elsewhere(t, cur):
    if not t.is_cuda:
        _off_device(t)
    raise ValueError(f"moeperm: tensor on {t.device}, but the current device is cuda:{cur}")


def _on_current(*tensors):
    """_ptrs of tensors that all have to be on the current device, whose stream the call uses."""
    cur = _cur_device() if _cur_device is not None else torch.cuda.current_device()
    return [None if t is None else t.data_ptr() if t.get_device() == cur else _elsewhere(t, cur) for t in tensors]


def _status(status, needed, dev):
    """The caller's status word, or a new one where the call can meet an error in its data
    (cleared by the library: a fill by torch takes 10 us of the host)."""
    if status is not None or not needed:
        return status
    st = torch.empty(1, dtype=torch.int32, device=dev)
    _check(lib().moe_status_clear(*_on_current(st), _stream()), "moe_status_clear")
    return st


def _words(dev, *sizes):
    """int32 vectors of these sizes from one allocation."""
    return torch.unsafe_split_with_sizes(torch.empty(sum(sizes), dtype=torch.int32, device=dev), sizes)


# The current stream's raw handle without building a torch Stream object (the
# public call costs microseconds per launch on small problems); the public
# call is the fallback where these functions are absent.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _cur_device is not None:
        return _raw_stream(_cur_device())
    return torch.cuda.current_stream().cuda_stream


def _check(code: int, where: str):
    if code != MOE_OK:
        raise MoePermError(code, where)


# ---------------------------------------------------------------------------
# One-to-one C calls
# ---------------------------------------------------------------------------

def moe_compact_bound(A: int, L: int, block_e: int) -> int:
    return int(lib().moe_compact_bound(A, L, block_e))


def moe_should_use_masked(E: int, L: int) -> bool:
    return bool(lib().moe_should_use_masked(E, L))


def moe_scale_bytes(fmt: str, rows: int, H: int, g: int) -> int:
    return int(lib().moe_scale_bytes(FMT[fmt], rows, H, g))


def moe_workspace_bytes(T: int, K: int, L: int) -> int:
    return int(lib().moe_workspace_bytes(T, K, L))


def moe_dispatch_compact(x, ldx, T, d_num_tokens, H, topk_ids, topk_weights, K, E, L, block_e,
                         g, fmt, xq, scales, ld_s, m_indices, bound, src2dst, counts, starts,
                         psum, total, row_weights, workspace, workspace_bytes, d_status,
                         stream=None) -> int:
    return int(lib().moe_dispatch_compact(
        _ptr(x), ldx, T, _ptr(d_num_tokens), H, _ptr(topk_ids), _ptr(topk_weights), K, E, L,
        block_e, g, FMT[fmt], _ptr(xq), _ptr(scales), ld_s, _ptr(m_indices), bound,
        _ptr(src2dst), _ptr(counts), _ptr(starts), _ptr(psum), _ptr(total), _ptr(row_weights),
        _ptr(workspace), workspace_bytes, _ptr(d_status), _stream(stream)))


def moe_dispatch_compact_noalloc(x, ldx, T, d_num_tokens, H, topk_ids, topk_weights, K, E, L,
                                 block_e, g, fmt, xq, scales, ld_s, m_indices, bound, src2dst,
                                 counts, starts, psum, total, row_weights, d_status,
                                 stream=None) -> int:
    """moe_dispatch_compact for callers that cannot allocate device memory: the
    scratch is a static device array inside the library (see the C header)."""
    return int(lib().moe_dispatch_compact_noalloc(
        _ptr(x), ldx, T, _ptr(d_num_tokens), H, _ptr(topk_ids), _ptr(topk_weights), K, E, L,
        block_e, g, FMT[fmt], _ptr(xq), _ptr(scales), ld_s, _ptr(m_indices), bound,
        _ptr(src2dst), _ptr(counts), _ptr(starts), _ptr(psum), _ptr(total), _ptr(row_weights),
        _ptr(d_status), _stream(stream)))


def moe_dispatch_masked(x, ldx, T, d_num_tokens, H, topk_ids, topk_weights, K, E, L, cap, g,
                        fmt, xq, scales, ld_s, masked_m, src2dst, row_weights, psum, psum_align,
                        workspace, workspace_bytes, d_status, stream=None) -> int:
    return int(lib().moe_dispatch_masked(
        _ptr(x), ldx, T, _ptr(d_num_tokens), H, _ptr(topk_ids), _ptr(topk_weights), K, E, L,
        cap, g, FMT[fmt], _ptr(xq), _ptr(scales), ld_s, _ptr(masked_m), _ptr(src2dst),
        _ptr(row_weights), _ptr(psum), psum_align, _ptr(workspace), workspace_bytes,
        _ptr(d_status), _stream(stream)))


def moe_quant_group(x, ldx, T_cap, d_num_live, H, g, fmt, xq, scales, ld_s, d_status,
                    stream=None) -> int:
    return int(lib().moe_quant_group(_ptr(x), ldx, T_cap, _ptr(d_num_live), H, g, FMT[fmt],
                                      _ptr(xq), _ptr(scales), ld_s, _ptr(d_status),
                                      _stream(stream)))


def moe_combine(y, ldy, R, src2dst, w, T, d_num_tokens, K, H, out, d_status, stream=None) -> int:
    return int(lib().moe_combine(_ptr(y), ldy, R, _ptr(src2dst), _ptr(w), T, _ptr(d_num_tokens),
                                 K, H, _ptr(out), _ptr(d_status), _stream(stream)))


def moe_expand_to_slab(exp, elem_bytes, H, R, exp_scales, ld_es, psum, L, align, cap, fmt, g,
                       slab, slab_scales, ld_ss, masked_m, d_status, stream=None) -> int:
    return int(lib().moe_expand_to_slab(
        _ptr(exp), elem_bytes, H, R, _ptr(exp_scales), ld_es, _ptr(psum), L, align, cap,
        FMT[fmt], g, _ptr(slab), _ptr(slab_scales), ld_ss, _ptr(masked_m), _ptr(d_status),
        _stream(stream)))


def moe_expand_from_slab(slab, elem_bytes, H, slab_scales, ld_ss, psum, L, align, cap, fmt, g,
                         row_weights, exp, R, exp_scales, ld_es, m_indices, d_status,
                         stream=None) -> int:
    return int(lib().moe_expand_from_slab(
        _ptr(slab), elem_bytes, H, _ptr(slab_scales), ld_ss, _ptr(psum), L, align, cap,
        FMT[fmt], g, _ptr(row_weights), _ptr(exp), R, _ptr(exp_scales), ld_es, _ptr(m_indices),
        _ptr(d_status), _stream(stream)))


def fp8_requant_per_tensor(q, ldq, s_tok, T, H, q_out, d_scale_out, stream=None) -> int:
    return int(lib().fp8_requant_per_tensor(_ptr(q), ldq, _ptr(s_tok), T, H, _ptr(q_out),
                                            _ptr(d_scale_out), _stream(stream)))


TOKSCALE = {"f32": 0, "ue8m0": 1}
REQUANT_MODE = {"max_scale": 0, "amax": 1}


def fp8_requant_per_tensor_ex(q, ldq, s_tok, s_fmt, T, H, mode, q_out, d_scale_out, workspace,
                              workspace_bytes, stream=None) -> int:
    return int(lib().fp8_requant_per_tensor_ex(
        _ptr(q), ldq, _ptr(s_tok), TOKSCALE[s_fmt], T, H, REQUANT_MODE[mode], _ptr(q_out),
        _ptr(d_scale_out), _ptr(workspace), workspace_bytes, _stream(stream)))


def moe_permute(x, ldx, dtype, T, d_num_tokens, H, topk_ids, topk_weights, K, E, L, block_e, xs,
                m_indices, bound, src2dst, counts, starts, psum, total, row_weights, workspace,
                workspace_bytes, d_status, stream=None) -> int:
    return int(lib().moe_permute(
        _ptr(x), ldx, ELEM[dtype], T, _ptr(d_num_tokens), H, _ptr(topk_ids), _ptr(topk_weights), K,
        E, L, block_e, _ptr(xs), _ptr(m_indices), bound, _ptr(src2dst), _ptr(counts), _ptr(starts),
        _ptr(psum), _ptr(total), _ptr(row_weights), _ptr(workspace), workspace_bytes,
        _ptr(d_status), _stream(stream)))


def moe_combine_ex(y, ldy, dtype, R, src2dst, w, T, d_num_tokens, K, H, out, d_status,
                   stream=None) -> int:
    return int(lib().moe_combine_ex(_ptr(y), ldy, ELEM[dtype], R, _ptr(src2dst), _ptr(w), T,
                                    _ptr(d_num_tokens), K, H, _ptr(out), _ptr(d_status),
                                    _stream(stream)))


def moe_combine_grad(dout, ldd, y, ldy, dtype, R, src2dst, w, T, d_num_tokens, K, H, dy, lddy, dw,
                     d_status, stream=None) -> int:
    return int(lib().moe_combine_grad(_ptr(dout), ldd, _ptr(y), ldy, ELEM[dtype], R,
                                      _ptr(src2dst), _ptr(w), T, _ptr(d_num_tokens), K, H,
                                      _ptr(dy), lddy, _ptr(dw), _ptr(d_status), _stream(stream)))


def moe_block_norm(x, ldx, y, ldy, dtype, T, H, w_post, gate, gate_mode, scale, w_pre, eps, x_out,
                   h, rstd_post, rstd_pre, stream=None) -> int:
    return int(lib().moe_block_norm(_ptr(x), ldx, _ptr(y), ldy, ELEM[dtype], T, H, _ptr(w_post),
                                    _ptr(gate), GATE[gate_mode], scale, _ptr(w_pre), eps,
                                    _ptr(x_out), _ptr(h), _ptr(rstd_post), _ptr(rstd_pre),
                                    _stream(stream)))


def moe_block_norm_workspace_bytes(T: int, H: int) -> int:
    return int(lib().moe_block_norm_workspace_bytes(T, H))


def moe_block_norm_grad(dx_out, ld_dxo, dh, ld_dh, x_out, ldx, y, ldy, dtype, T, H, w_post, gate,
                        gate_mode, scale, w_pre, rstd_post, rstd_pre, dx, dy, dw_post, dgate,
                        dw_pre, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().moe_block_norm_grad(
        _ptr(dx_out), ld_dxo, _ptr(dh), ld_dh, _ptr(x_out), ldx, _ptr(y), ldy, ELEM[dtype], T, H,
        _ptr(w_post), _ptr(gate), GATE[gate_mode], scale, _ptr(w_pre), _ptr(rstd_post),
        _ptr(rstd_pre), _ptr(dx), _ptr(dy), _ptr(dw_post), _ptr(dgate), _ptr(dw_pre),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def moe_expert_matmul(x, ldx, dtype, x_scales, ld_xs, R, K, w, w_scales, ld_ws, L, N, gated, act,
                      bias, seg_begin, seg_end, cap, residual, ld_res, out, ldo, out_dtype, pre,
                      ld_pre, d_status, stream=None) -> int:
    return int(lib().moe_expert_matmul(
        _ptr(x), ldx, ELEM[dtype], _ptr(x_scales), ld_xs, R, K, _ptr(w), _ptr(w_scales), ld_ws, L, N,
        int(gated), ACT[act], _ptr(bias), _ptr(seg_begin), _ptr(seg_end), cap, _ptr(residual),
        ld_res, _ptr(out), ldo, ELEM[out_dtype], _ptr(pre), ld_pre, _ptr(d_status),
        _stream(stream)))


def moe_expert_matmul_grad_workspace_bytes(R: int, L: int, Nw: int) -> int:
    return int(lib().moe_expert_matmul_grad_workspace_bytes(R, L, Nw))


def moe_expert_matmul_grad(dout, ldd, x, ldx, dtype, R, K, w, L, N, gated, act, pre, ld_pre,
                           seg_begin, seg_end, cap, dx, ld_dx, dw, dw_dtype, dbias, workspace,
                           workspace_bytes, d_status, stream=None) -> int:
    return int(lib().moe_expert_matmul_grad(
        _ptr(dout), ldd, _ptr(x), ldx, ELEM[dtype], R, K, _ptr(w), L, N, int(gated), ACT[act],
        _ptr(pre), ld_pre, _ptr(seg_begin), _ptr(seg_end), cap, _ptr(dx), ld_dx, _ptr(dw),
        ELEM[dw_dtype], _ptr(dbias), _ptr(workspace), workspace_bytes, _ptr(d_status),
        _stream(stream)))


def moe_fp4_scale_bytes(ld: int, H: int, fmt: str) -> int:
    return int(lib().moe_fp4_scale_bytes(ld, H, FP4[fmt]))


def moe_quant_fp4(x, ldx, dtype, R, H, fmt, tensor_scale, n_scales, d_num_live, m_indices, masked_m, cap, xq,
                  scales, ld_s, d_status, stream=None) -> int:
    return int(lib().moe_quant_fp4(
        _ptr(x), ldx, ELEM[dtype], R, H, FP4[fmt], _ptr(tensor_scale), n_scales, _ptr(d_num_live),
        _ptr(m_indices), _ptr(masked_m), cap, _ptr(xq), _ptr(scales), ld_s, _ptr(d_status), _stream(stream)))


def moe_dequant_fp4(xq, scales, ld_s, R, H, fmt, tensor_scale, n_scales, d_num_live, m_indices, masked_m, cap,
                    x, ldx, dtype, d_status, stream=None) -> int:
    return int(lib().moe_dequant_fp4(
        _ptr(xq), _ptr(scales), ld_s, R, H, FP4[fmt], _ptr(tensor_scale), n_scales, _ptr(d_num_live),
        _ptr(m_indices), _ptr(masked_m), cap, _ptr(x), ldx, ELEM[dtype], _ptr(d_status), _stream(stream)))


def moe_dispatch_fp4(x, ldx, dtype, T, d_num_tokens, H, topk_ids, topk_weights, K, E, L, block_e, fmt,
                     tensor_scale, xq, scales, ld_s, m_indices, bound, src2dst, counts, starts, psum, total,
                     row_weights, workspace, workspace_bytes, d_status, stream=None) -> int:
    return int(lib().moe_dispatch_fp4(
        _ptr(x), ldx, ELEM[dtype], T, _ptr(d_num_tokens), H, _ptr(topk_ids), _ptr(topk_weights), K, E, L,
        block_e, FP4[fmt], _ptr(tensor_scale), _ptr(xq), _ptr(scales), ld_s, _ptr(m_indices), bound,
        _ptr(src2dst), _ptr(counts), _ptr(starts), _ptr(psum), _ptr(total), _ptr(row_weights),
        _ptr(workspace), workspace_bytes, _ptr(d_status), _stream(stream)))


def moe_expert_matmul_fp4(x, ldx, x_scales, ld_xs, x_tscale, R, K, w, w_scales, ld_ws, w_tscale, fmt, L, N,
                          gated, act, bias, seg_begin, seg_end, cap, residual, ld_res, out, ldo, out_dtype,
                          d_status, stream=None) -> int:
    return int(lib().moe_expert_matmul_fp4(
        _ptr(x), ldx, _ptr(x_scales), ld_xs, _ptr(x_tscale), R, K, _ptr(w), _ptr(w_scales), ld_ws,
        _ptr(w_tscale), FP4[fmt], L, N, int(gated), ACT[act], _ptr(bias), _ptr(seg_begin), _ptr(seg_end), cap,
        _ptr(residual), ld_res, _ptr(out), ldo, ELEM[out_dtype], _ptr(d_status), _stream(stream)))


def moe_route(logits, ldl, dtype, T, d_num_tokens, E, K, score, bias, renorm, scale, topk_ids,
              topk_weights, d_status, stream=None) -> int:
    return int(lib().moe_route(_ptr(logits), ldl, ELEM[dtype], T, _ptr(d_num_tokens), E, K, SCORE[score],
                               _ptr(bias), int(renorm), scale, _ptr(topk_ids), _ptr(topk_weights),
                               _ptr(d_status), _stream(stream)))


def moe_balance_loss_workspace_bytes(E: int, Q: int) -> int:
    return int(lib().moe_balance_loss_workspace_bytes(E, Q))


def moe_balance_loss(logits, ldl, dtype, T, d_num_tokens, E, topk_ids, K, score, seq_begin, seq_end, Q,
                     loss, counts, prob_sums, workspace, workspace_bytes, d_status, stream=None) -> int:
    return int(lib().moe_balance_loss(
        _ptr(logits), ldl, ELEM[dtype], T, _ptr(d_num_tokens), E, _ptr(topk_ids), K, SCORE[score],
        _ptr(seq_begin), _ptr(seq_end), Q, _ptr(loss), _ptr(counts), _ptr(prob_sums), _ptr(workspace),
        workspace_bytes, _ptr(d_status), _stream(stream)))


def moe_route_grad(logits, ldl, dtype, T, d_num_tokens, E, topk_ids, K, score, renorm, scale, dweights,
                   dloss, counts, seq_begin, seq_end, Q, dlogits, ldd, d_status, stream=None) -> int:
    return int(lib().moe_route_grad(
        _ptr(logits), ldl, ELEM[dtype], T, _ptr(d_num_tokens), E, _ptr(topk_ids), K, SCORE[score],
        int(renorm), scale, _ptr(dweights), _ptr(dloss), _ptr(counts), _ptr(seq_begin), _ptr(seq_end), Q,
        _ptr(dlogits), ldd, _ptr(d_status), _stream(stream)))


def moe_status_sync(d_status, stream=None) -> int:
    return int(lib().moe_status_sync(_ptr(d_status), _stream(stream)))


def moe_status_clear(d_status, stream=None) -> int:
    return int(lib().moe_status_clear(_ptr(d_status), _stream(stream)))


def moe_version() -> str:
    return lib().moe_version().decode()


# ---------------------------------------------------------------------------
# Allocating helpers (torch owns the memory)
# ---------------------------------------------------------------------------

def scale_tensor(fmt: str, rows: int, H: int, g: int, device, blocks: int = 1, ld: int | None = None):
    """Allocate a scale tensor in `fmt`: u8 -> uint8 [rows, G]; f32pow2 -> float32
    [rows, G]; packed -> int32 [blocks, G4, ld] (ld = rows per block rounded up
    to 4). Returns (tensor, ld)."""
    G = H // g
    if fmt in ("u8", "mx"):
        ld = G if ld is None else ld
        return torch.empty((rows, ld), dtype=torch.uint8, device=device), ld
    if fmt in ("f32pow2", "f32"):
        ld = G if ld is None else ld
        return torch.empty((rows, ld), dtype=torch.float32, device=device), ld
    rpb = rows // blocks
    ld = (rpb + 3) // 4 * 4 if ld is None else ld
    return torch.empty((blocks, (G + 3) // 4, ld), dtype=torch.int32, device=device), ld


class Workspace:
    """Dispatch workspace, reusable across calls on one stream. Every dispatch
    writes the chunk table before reading it, so no initialisation is needed
    (no fill kernel per allocation)."""

    def __init__(self, T: int, K: int, L: int, device):
        self.nbytes = moe_workspace_bytes(T, K, L)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)

    def fits(self, T, K, L):
        return moe_workspace_bytes(T, K, L) <= self.nbytes


def dispatch_compact(x, topk_ids, topk_weights, num_experts, num_local_experts, block_e=128,
                     group_size=128, scale_fmt="packed", num_tokens=None, workspace=None,
                     status=None, row_weights=True):
    """Quantise + scatter into the compact layout. Returns a dict of tensors."""
    T, H = x.shape
    K = topk_ids.shape[1]
    L = num_local_experts
    dev = x.device
    bound = moe_compact_bound(T * K, L, block_e)
    xq = torch.empty((bound, H), dtype=torch.uint8, device=dev)
    sc, ld = scale_tensor(scale_fmt, bound, H, group_size, dev)
    out = dict(
        xq=xq, scales=sc, ld_s=ld, bound=bound,
        m_indices=torch.empty(bound, dtype=torch.int32, device=dev),
        src2dst=torch.empty((T, K), dtype=torch.int32, device=dev),
        counts=torch.empty(L, dtype=torch.int32, device=dev),
        starts=torch.empty(L, dtype=torch.int32, device=dev),
        psum=torch.empty(L, dtype=torch.int32, device=dev),
        total=torch.empty(1, dtype=torch.int32, device=dev),
        row_weights=torch.empty(bound, dtype=torch.float32, device=dev) if row_weights else None,
    )
    ws = workspace if workspace is not None else Workspace(T, K, L, dev)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    code = moe_dispatch_compact(
        x, x.stride(0), T, num_tokens, H, topk_ids, topk_weights, K, num_experts, L, block_e,
        group_size, scale_fmt, xq, sc, ld, out["m_indices"], bound, out["src2dst"],
        out["counts"], out["starts"], out["psum"], out["total"], out["row_weights"], ws.buf,
        ws.nbytes, st)
    _check(code, "moe_dispatch_compact")
    out["status"] = st
    return out


def dispatch_masked(x, topk_ids, topk_weights, num_experts, num_local_experts, cap,
                    group_size=128, scale_fmt="packed", num_tokens=None, workspace=None,
                    status=None, row_weights=True, psum_align=128):
    """Quantise + scatter into per-expert slabs [L, cap, H]. Returns a dict,
    including psum [L], the expanded layout of the slab rows aligned to
    psum_align (None: not computed), and expand_rows, the static row count of
    that layout."""
    T, H = x.shape
    K = topk_ids.shape[1]
    L = num_local_experts
    dev = x.device
    xq = torch.empty((L, cap, H), dtype=torch.uint8, device=dev)
    sc, ld = scale_tensor(scale_fmt, L * cap, H, group_size, dev, blocks=L)
    out = dict(
        xq=xq, scales=sc, ld_s=ld,
        masked_m=torch.empty(L, dtype=torch.int32, device=dev),
        src2dst=torch.empty((T, K), dtype=torch.int32, device=dev),
        row_weights=torch.empty(L * cap, dtype=torch.float32, device=dev) if row_weights else None,
        psum=torch.empty(L, dtype=torch.int32, device=dev) if psum_align else None,
        expand_rows=moe_compact_bound(T * K, L, psum_align) if psum_align else 0,
    )
    ws = workspace if workspace is not None else Workspace(T, K, L, dev)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    code = moe_dispatch_masked(
        x, x.stride(0), T, num_tokens, H, topk_ids, topk_weights, K, num_experts, L, cap,
        group_size, scale_fmt, xq, sc, ld, out["masked_m"], out["src2dst"], out["row_weights"],
        out["psum"], psum_align or 1, ws.buf, ws.nbytes, st)
    _check(code, "moe_dispatch_masked")
    out["status"] = st
    return out


def quant_group(x, group_size=128, scale_fmt="packed", num_live=None, status=None):
    """Quantise rows [0, num_live) of x (all rows when num_live is None)."""
    T_cap, H = x.shape
    dev = x.device
    xq = torch.empty((T_cap, H), dtype=torch.uint8, device=dev)
    sc, ld = scale_tensor(scale_fmt, T_cap, H, group_size, dev)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    _check(moe_quant_group(x, x.stride(0), T_cap, num_live, H, group_size, scale_fmt, xq, sc, ld,
                           st), "moe_quant_group")
    return dict(xq=xq, scales=sc, ld_s=ld, status=st)


def _like(t, shape, dtype, dev, name):
    """The caller's output tensor, checked, or a new one. Outputs are dense."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"moeperm: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t


def _rows(t, name, shape=None, dtype=None):
    """Row stride of a 2-D tensor whose rows are dense; checks shape and dtype when given."""
    own = t.shape
    if len(own) != 2 or (shape is not None and own != shape) or (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"moeperm: {name} must be 2-D{'' if shape is None else f' of shape {tuple(shape)}'}"
                         f"{'' if dtype is None else f' and {dtype}'}, not {t.dtype} of shape {tuple(own)}")
    rows, width = own
    ld, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"moeperm: the rows of {name} must be dense")
    return ld if rows > 1 or ld >= width else width


def _vec(t, n, name, dtype=torch.float32):
    """A dense vector argument of n elements (or None)."""
    if t is not None and (t.dtype is not dtype or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"moeperm: {name} must be a contiguous {dtype} tensor of {n} elements")
    return t


def _elem(t, allowed, name):
    if t.dtype not in allowed:
        raise ValueError(f"moeperm: {name} must be one of {[str(d) for d in allowed]}, not {t.dtype}")
    return t.dtype


FLOATS = (torch.bfloat16, torch.float16, torch.float32)
E4M3_BYTES = (torch.uint8, torch.float8_e4m3fn)
BF16_BITS = (torch.int16, torch.uint16)


def combine(y, src2dst, weights=None, num_tokens=None, status=None, out=None):
    """out[t] = sum_k w[t,k] * y[src2dst[t,k]] in fp32, rounded once to y's type
    (bfloat16, float16 or float32; 16-bit integers are taken for bfloat16 bits).
    `out` may have more than T rows; the first T are written."""
    ldy = _rows(y, "y")
    T, K = src2dst.shape
    R, H = y.shape
    dev = y.device
    dtype = torch.bfloat16 if y.dtype in BF16_BITS else _elem(y, FLOATS, "y")
    _vec(src2dst, T * K, "src2dst", torch.int32)
    if weights is not None and (weights.dtype is not torch.float32 or weights.numel() < T * K
                                or not weights.is_contiguous()):
        raise ValueError(f"moeperm: weights must be a contiguous float32 tensor of {T * K} elements")
    if out is None:
        out = torch.empty((T, H), dtype=dtype, device=dev)
    elif ((out.dtype is not dtype and not (dtype is torch.bfloat16 and out.dtype in BF16_BITS))
          or out.dim() != 2 or out.shape[0] < T or out.shape[1] != H or not out.is_contiguous()):
        raise ValueError(f"moeperm: out must be a contiguous {dtype} tensor of shape [{T}, {H}], not "
                         f"{out.dtype} of shape {tuple(out.shape)}")
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    if dtype is torch.bfloat16:
        _check(moe_combine(y, ldy, R, src2dst, weights, T, num_tokens, K, H, out, st), "moe_combine")
    else:
        _check(moe_combine_ex(y, ldy, dtype, R, src2dst, weights, T, num_tokens, K, H, out, st),
               "moe_combine_ex")
    return out


def permute(x, topk_ids, topk_weights, num_experts, num_local_experts, block_e=128,
            num_tokens=None, workspace=None, status=None, row_weights=True, out=None):
    """Copy every token's row to the rows of its kept slots in the compact layout,
    unquantised: out[src2dst[t,k]] = x[t] (bfloat16, float16 or float32; padding
    rows of `out` are not written). row_weights: True, False or the [bound]
    float32 tensor to fill. Returns a dict: xs and the layout tensors of
    dispatch_compact."""
    dtype = _elem(x, FLOATS, "x")
    ldx = _rows(x, "x")
    T, H = x.shape
    K, L, dev = topk_ids.shape[1], num_local_experts, x.device
    _vec(topk_ids, T * K, "topk_ids", torch.int32)
    _vec(topk_weights, T * K, "topk_weights")
    bound = moe_compact_bound(T * K, L, block_e)
    if row_weights is True:
        row_weights = torch.empty(bound, dtype=torch.float32, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    o = dict(xs=_like(out, (bound, H), dtype, dev, "out"), bound=bound,
             m_indices=torch.empty(bound, **i32), src2dst=torch.empty((T, K), **i32),
             counts=torch.empty(L, **i32), starts=torch.empty(L, **i32), psum=torch.empty(L, **i32),
             total=torch.empty(1, **i32),
             row_weights=None if row_weights is False else _vec(row_weights, bound, "row_weights"))
    ws = workspace if workspace is not None else Workspace(T, K, L, dev)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    px, pn, pi, pw, *po, pws, pst = _ptrs(x, num_tokens, topk_ids, topk_weights, o["xs"],
                                          o["m_indices"], o["src2dst"], o["counts"], o["starts"],
                                          o["psum"], o["total"], o["row_weights"], ws.buf, st)
    _check(lib().moe_permute(px, ldx, ELEM[dtype], T, pn, H, pi, pw, K, num_experts, L, block_e,
                             po[0], po[1], bound, *po[2:], pws, ws.nbytes, pst, _stream()),
           "moe_permute")
    o["status"] = st
    return o


def permute_grad(dxs, src2dst, num_tokens=None, status=None, out=None):
    """Gradient of permute: dx[t] = sum over kept k of dxs[src2dst[t,k]]."""
    dtype = _elem(dxs, FLOATS, "dxs")
    ld = _rows(dxs, "dxs")
    T, K = src2dst.shape
    R, H = dxs.shape
    _vec(src2dst, T * K, "src2dst", torch.int32)
    out = _like(out, (T, H), dtype, dxs.device, "out")
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dxs.device)
    pd, ps, pn, po, pst = _ptrs(dxs, src2dst, num_tokens, out, st)
    _check(lib().moe_combine_ex(pd, ld, ELEM[dtype], R, ps, None, T, pn, K, H, po, pst, _stream()),
           "moe_combine_ex")
    return out


def combine_grad(dout, y, src2dst, weights=None, num_tokens=None, status=None, dy=None,
                 need_dy=True, need_dweights=True):
    """Gradients of combine(y, src2dst, weights) for the output gradient dout:
    dy[src2dst[t,k]] = w[t,k] * dout[t] (rows without a kept slot are not
    written) and dweights[t,k] = <dout[t], y[src2dst[t,k]]> in float32. Returns
    a dict (dy, dweights, status)."""
    dtype = _elem(dout, FLOATS, "dout")
    T, K = src2dst.shape
    R, H = y.shape
    ldd, ldy = _rows(dout, "dout", (T, H)), _rows(y, "y", None, dtype)
    _vec(src2dst, T * K, "src2dst", torch.int32)
    _vec(weights, T * K, "weights")
    dev = dout.device
    dy = _like(dy, (R, H), dtype, dev, "dy") if need_dy else None
    dw = torch.empty((T, K), dtype=torch.float32, device=dev) if need_dweights else None
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    pd, py, ps, pw, pn, pdy, pdw, pst = _ptrs(dout, y, src2dst, weights, num_tokens, dy, dw, st)
    _check(lib().moe_combine_grad(pd, ldd, py, ldy, ELEM[dtype], R, ps, pw, T, pn, K, H, pdy, H, pdw,
                                  pst, _stream()), "moe_combine_grad")
    return dict(dy=dy, dweights=dw, status=st)


def _segments(starts, psum, masked_m, L):
    """Checks where the experts' rows are: (seg_begin, seg_end)."""
    if masked_m is not None:
        if starts is not None or psum is not None:
            raise ValueError("moeperm: give starts and psum, or masked_m, not both")
        return None, _vec(masked_m, L, "masked_m", torch.int32)
    if (starts is None) != (psum is None) or (starts is None and L != 1):
        raise ValueError("moeperm: the experts' rows need starts and psum, or masked_m (a single "
                         "expert may have all rows)")
    return _vec(starts, L, "starts", torch.int32), _vec(psum, L, "psum", torch.int32)


def _expert_rows(t, masked, L, name):
    """Rows [R, width] of a compact tensor or of slabs [L, cap, width]: (2-D tensor, cap)."""
    if not masked:
        return t, 0
    if t.dim() != 3 or t.shape[0] != L or not t.is_contiguous():
        raise ValueError(f"moeperm: with masked_m, {name} must be contiguous slabs [{L}, cap, width]")
    return t.view(-1, t.shape[2]), t.shape[1]


def _expert_weights(w, gated):
    """[L, N (gated: 2N), K] from [.., .., K]: (L, N, K)."""
    if w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("moeperm: w must be contiguous, [L, N, K] or [N, K] (gated: 2N)")
    Nw, K = w.shape[-2:]
    if gated and Nw % 2:
        raise ValueError("moeperm: gated weights hold gate and up rows: [.., 2N, K]")
    return (w.shape[0] if w.dim() == 3 else 1), (Nw // 2 if gated else Nw), K


def _scale_words(t, rows, ld, words, name, blocks=1):
    """Packed scale words [blocks, words, ld] of `rows` rows in each block. Other scale
    formats have the same bytes in another order, or fewer: their types are refused."""
    need = (blocks * words - 1) * ld + rows
    if t.dtype not in (torch.int32, torch.uint32):
        raise ValueError(f"moeperm: {name} must be packed scale words (int32), not {t.dtype}")
    if t.numel() < need or not t.is_contiguous():  # a part of a larger buffer may hold them too
        held = t.untyped_storage().nbytes() // 4 - t.storage_offset()
        if held < need or (t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1):
            raise ValueError(f"moeperm: {name} must hold {blocks} x {words} x {ld} packed words of {rows} rows, "
                             f"not {tuple(t.shape)}")


def expert_matmul(x, w, starts=None, psum=None, bias=None, act="none", gated=False, residual=None,
                  masked_m=None, x_scales=None, ld_xs=0, w_scales=None, ld_ws=0, out=None, pre=None,
                  out_dtype=torch.bfloat16, status=None):
    """Every expert's product over its rows: P = x w_e^T + bias_e, out = act(P)
    [+ residual], or gated act(P[:, :N]) * P[:, N:] [+ residual].

    x [R, K] with the segments starts / psum of dispatch_compact or permute, or
    slabs [L, cap, K] with masked_m of dispatch_masked, or all rows of one
    expert. w [L, N, K] (gated [L, 2N, K]: gate rows, then up rows); bias
    [L, N or 2N] float32. bfloat16, float16, or e4m3 (uint8 or float8_e4m3fn)
    with the packed scales of the dispatch (x_scales, ld_xs) and of
    quant_group(w.view(-1, K)) (w_scales, ld_ws) and an output of out_dtype. act:
    none, relu, silu or gelu. `pre` receives P for expert_matmul_grad. Rows of
    no expert are not written. Returns out."""
    fp8 = x.dtype in E4M3_BYTES
    dtype = torch.float8_e4m3fn if fp8 else _elem(x, FLOATS[:2], "x")
    L, N, K = _expert_weights(w, gated)
    if w.dtype != dtype and not (fp8 and w.dtype in E4M3_BYTES):
        raise ValueError(f"moeperm: w must have the type of x ({dtype}), not {w.dtype}")
    if fp8 and (x_scales is None or w_scales is None):
        raise ValueError("moeperm: e4m3 rows and weights need x_scales and w_scales")
    if act not in ACT:
        raise ValueError(f"moeperm: act must be one of {sorted(ACT)}, not {act!r}")
    masked = masked_m is not None
    begin, end = _segments(starts, psum, masked_m, L)
    shape3 = x.shape
    x, cap = _expert_rows(x, masked, L, "x")
    ldx = _rows(x, "x", (x.shape[0], K))
    R = x.shape[0]
    Nw = 2 * N if gated else N
    if fp8:
        words = (K + 511) // 512
        _scale_words(w_scales, L * Nw, ld_ws, words, "w_scales")
        if R > 0:
            _scale_words(x_scales, cap if masked else R, ld_xs, words, "x_scales", L if masked else 1)
    odt = out_dtype if fp8 else dtype
    if odt not in (torch.bfloat16, torch.float16):
        raise ValueError(f"moeperm: out_dtype must be bfloat16 or float16, not {odt}")
    _vec(bias, L * Nw, "bias")
    full = (*shape3[:-1], N)
    if out is None:
        out = torch.empty(full, dtype=odt, device=x.device)
    elif tuple(out.shape) != full:
        raise ValueError(f"moeperm: out must have shape {full}")
    o2 = _expert_rows(out, masked, L, "out")[0]
    ldo = _rows(o2, "out", (R, N), odt)
    res, ld_res = None, 0
    if residual is not None:
        res = _expert_rows(residual, masked, L, "residual")[0]
        ld_res = _rows(res, "residual", (R, N), odt)
    p2, ld_pre = None, 0
    if pre is not None:
        p2 = _expert_rows(pre, masked, L, "pre")[0]
        ld_pre = _rows(p2, "pre", (R, Nw), dtype)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=x.device)
    px, pxs, pw, pws, pb, p0, p1, pr, po, pp, pst = _ptrs(x, x_scales, w, w_scales, bias, begin, end,
                                                          res, o2, p2, st)
    _check(lib().moe_expert_matmul(px, ldx, ELEM[dtype], pxs, ld_xs, R, K, pw, pws, ld_ws, L, N,
                                   1 if gated else 0, ACT[act], pb, p0, p1, cap, pr, ld_res, po, ldo,
                                   ELEM[odt], pp, ld_pre, pst, _stream()), "moe_expert_matmul")
    return out


class GradWorkspace:
    """Workspace of expert_matmul_grad for up to R rows, L experts and Nw weight rows
    per expert (gated: 2N), reusable across calls on one stream; needs no
    initialisation. Its size is the same for both types."""

    def __init__(self, R: int, L: int, Nw: int, dtype, device):
        _ = dtype  # 16 bits for both types: the argument changes nothing
        self.nbytes = moe_expert_matmul_grad_workspace_bytes(R, L, Nw)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def expert_matmul_grad(dout, x, w, starts=None, psum=None, pre=None, act="none", gated=False,
                       masked_m=None, need=("dx", "dw"), dx=None, dw=None, dbias=None,
                       dw_dtype=None, workspace=None, status=None):
    """Gradients of expert_matmul for the output gradient dout: those of dx, dw and
    dbias that `need` names or that a tensor is given for, from the kept `pre` (not
    needed without act and gate). dw [as w] in dw_dtype: w's type, or float32, which
    keeps the gradient of `pre` beyond its 16 bits too. dbias [L, N or 2N] float32;
    both are written in full, dx on the experts' rows. The residual's gradient is
    dout. Returns a dict (dx, dw, dbias, status)."""
    dtype = _elem(x, FLOATS[:2], "x")
    L, N, K = _expert_weights(w, gated)
    if w.dtype != dtype:
        raise ValueError(f"moeperm: w must have the type of x ({dtype}), not {w.dtype}")
    if act not in ACT:
        raise ValueError(f"moeperm: act must be one of {sorted(ACT)}, not {act!r}")
    masked = masked_m is not None
    begin, end = _segments(starts, psum, masked_m, L)
    dev, shape3 = x.device, x.shape
    x2, cap = _expert_rows(x, masked, L, "x")
    ldx = _rows(x2, "x", (x2.shape[0], K))
    R, Nw = x2.shape[0], (2 * N if gated else N)
    d2 = _expert_rows(dout, masked, L, "dout")[0]
    ldd = _rows(d2, "dout", (R, N), dtype)
    p2, ld_pre = None, 0
    if act != "none" or gated:
        if pre is None:
            raise ValueError("moeperm: the gradient through an activation needs pre")
        p2 = _expert_rows(pre, masked, L, "pre")[0]
        ld_pre = _rows(p2, "pre", (R, Nw), dtype)
    x_out, w_out, b_out = None, None, None
    dwt = dw.dtype if dw is not None else (dw_dtype or dtype)
    if "dx" in need or dx is not None:
        x_out = _like(dx, tuple(shape3), dtype, dev, "dx")
    if "dw" in need or dw is not None:
        w_out = _like(dw, tuple(w.shape), dwt, dev, "dw")
    if "dbias" in need or dbias is not None:
        b_out = _vec(dbias, L * Nw, "dbias")
        if b_out is None:
            b_out = torch.empty((L, Nw), dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else GradWorkspace(R, L, Nw, dtype, dev)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    _check(moe_expert_matmul_grad(d2, ldd, x2, ldx, dtype, R, K, w, L, N, gated, act, p2, ld_pre,
                                  begin, end, cap, x_out, K, w_out, dwt, b_out, ws.buf, ws.nbytes,
                                  st), "moe_expert_matmul_grad")
    return dict(dx=x_out, dw=w_out, dbias=b_out, status=st)


class NormWorkspace:
    """Workspace of block_norm_grad for up to T tokens of H elements, reusable
    across calls on one stream; needs no initialisation."""

    def __init__(self, T: int, H: int, device):
        self.nbytes = moe_block_norm_workspace_bytes(T, H)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def _gate_mode(gate, T, H, mode=None, name="gate"):
    """none / channel / token: [H] or [1, H] is per channel, [T] or [T, 1] per token. A
    1-D gate with T = H fits both: the caller has to name its mode, since a guess
    would change a gate's meaning with the number of tokens in a batch."""
    if mode not in (None, "channel", "token") and not (mode == "none" and gate is None):
        raise ValueError(f"moeperm: gate_mode must be 'channel' or 'token', not {mode!r}")
    if gate is None:
        return "none"
    shape = tuple(gate.shape)
    fits = [m for m, shapes in (("channel", ((H,), (1, H))), ("token", ((T,), (T, 1)))) if shape in shapes]
    if mode is not None:
        fits = [m for m in fits if m == mode]
    if not fits:
        want = {"channel": f"[{H}]", "token": f"[{T}]", None: f"[{H}] or [{T}]"}[mode]
        raise ValueError(f"moeperm: {name} must have shape {want}, not {shape}")
    if len(fits) > 1:
        raise ValueError(f"moeperm: {name} {shape} fits both a gate per channel and one per token: name gate_mode")
    _vec(gate, gate.numel(), name)
    return fits[0]


def block_norm(x, y=None, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-6,
               save_rstd=False, gate_mode=None):
    """The step between two blocks: x' = x + scale * gate * (rms(y) * w_post) and
    h = rms(x') * w_pre, rms(v) = v / sqrt(mean(v^2) + eps). y: the last block's
    output (None: x' = x); w_post None: y is added unnormalised; w_pre None: no
    h. gate [H] (per channel) or [T] (per token); gate_mode "channel" or "token"
    says which, and has to where T can equal H. Returns a dict: x (x'), h, and
    with save_rstd rstd_post and rstd_pre for block_norm_grad."""
    dtype = _elem(x, FLOATS, "x")
    ldx = _rows(x, "x")
    T, H = x.shape
    dev = x.device
    ldy = _rows(y, "y", (T, H), dtype) if y is not None else 0
    mode = _gate_mode(gate, T, H, gate_mode)
    _vec(w_post, H, "w_post")
    _vec(w_pre, H, "w_pre")
    xo = torch.empty((T, H), dtype=dtype, device=dev) if y is not None else None
    h = torch.empty((T, H), dtype=dtype, device=dev) if w_pre is not None else None
    r_post = r_pre = None
    if save_rstd:
        if w_post is not None:
            r_post = torch.empty(T, dtype=torch.float32, device=dev)
        if w_pre is not None:
            r_pre = torch.empty(T, dtype=torch.float32, device=dev)
    px, py, pw, pg, pp, po, ph, pr0, pr1 = _ptrs(x, y, w_post, gate, w_pre, xo, h, r_post, r_pre)
    _check(lib().moe_block_norm(px, ldx, py, ldy, ELEM[dtype], T, H, pw, pg, GATE[mode], scale, pp,
                                eps, po, ph, pr0, pr1, _stream()), "moe_block_norm")
    return dict(x=x if y is None else xo, h=h, rstd_post=r_post, rstd_pre=r_pre)


def block_norm_grad(dx_out, dh, x_out, y=None, w_post=None, gate=None, scale=1.0, w_pre=None,
                    rstd_pre=None, rstd_post=None, workspace=None, gate_mode=None):
    """Gradients of block_norm for dx_out (None: zeros) and dh. x_out is the stream
    after the sum (x itself without y), the rstds are the forward call's. Returns
    a dict: dx, dy, dw_post, dgate, dw_pre (None where there is none)."""
    dtype = _elem(x_out, FLOATS, "x_out")
    ldx = _rows(x_out, "x_out")
    T, H = x_out.shape
    dev = x_out.device
    ld = lambda t, name: _rows(t, name, (T, H), dtype) if t is not None else 0
    ldo, ldh, ldy = ld(dx_out, "dx_out"), ld(dh, "dh"), ld(y, "y")
    mode = _gate_mode(gate, T, H, gate_mode)
    _vec(w_post, H, "w_post")
    _vec(w_pre, H, "w_pre")
    _vec(rstd_pre, T, "rstd_pre")
    _vec(rstd_post, T, "rstd_post")
    f32 = dict(dtype=torch.float32, device=dev)
    o = dict(dx=torch.empty((T, H), dtype=dtype, device=dev),
             dy=torch.empty((T, H), dtype=dtype, device=dev) if y is not None else None,
             dw_post=torch.empty(H, **f32) if w_post is not None else None,
             dgate=torch.empty(gate.shape, **f32) if gate is not None else None,
             dw_pre=torch.empty(H, **f32) if w_pre is not None else None)
    ws = workspace if workspace is not None else NormWorkspace(T, H, dev)
    _check(moe_block_norm_grad(dx_out, ldo, dh, ldh, x_out, ldx, y, ldy, dtype, T, H, w_post, gate,
                               mode, scale, w_pre, rstd_post, rstd_pre, o["dx"], o["dy"],
                               o["dw_post"], o["dgate"], o["dw_pre"], ws.buf, ws.nbytes),
           "moe_block_norm_grad")
    return o


FP4_BYTES = (torch.uint8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ())


def _fp4(fmt):
    if fmt not in FP4:
        raise ValueError(f"moeperm: fmt must be one of {sorted(FP4)}, not {fmt!r}")
    return FP4[fmt]


def fp4_scale_tensor(rows: int, H: int, fmt: str, device, ld: int | None = None):
    """Allocate the scale bytes [pieces, ld, 16] of `rows` four-bit rows of H elements
    (ld: rows by default)."""
    _fp4(fmt)
    g = 16 if fmt == "nv" else 32
    return torch.empty(((H // g + 15) // 16, rows if ld is None else ld, 16), dtype=torch.uint8, device=device)


def _fp4_scales(t, rows, H, fmt, name):
    """The leading dimension of a scale tensor that holds `rows` rows of H elements."""
    pieces = (H // (16 if fmt == "nv" else 32) + 15) // 16
    s = t.shape
    if t.dtype is not torch.uint8 or len(s) != 3 or s[0] < pieces or s[1] < rows or s[2] != 16 or not t.is_contiguous():
        raise ValueError(f"moeperm: {name} must be contiguous uint8 scales [{pieces}, >= {rows}, 16] ({fmt}), not "
                         f"{t.dtype} of shape {tuple(s)}")
    return s[1]


def _tensor_scale(t, fmt, name, n=None):
    """Float32 scales of a tensor ("nv" only): how many."""
    if t is None:
        return 1
    if fmt != "nv":
        raise ValueError(f"moeperm: {name} belongs to the nv format, not to {fmt}")
    _vec(t, t.numel() if n is None else n, name)
    return t.numel()


def _fp4_rows(R, num_live, m_indices, masked_m):
    """The rows to work on, named in one way at most: cap."""
    if (num_live is not None) + (m_indices is not None) + (masked_m is not None) > 1:
        raise ValueError("moeperm: give one of num_live, m_indices and masked_m")
    if m_indices is not None:
        _vec(m_indices, R, "m_indices", torch.int32)
    if masked_m is None:
        _vec(num_live, 1, "num_live", torch.int32)
        return 0
    L = masked_m.numel()
    _vec(masked_m, L, "masked_m", torch.int32)
    if L < 1 or R % L:
        raise ValueError(f"moeperm: {R} rows are not slabs of {L} experts")
    return R // L


def quant_fp4(x, fmt="nv", tensor_scale=None, num_live=None, m_indices=None, masked_m=None, status=None):
    """Rows to four bits (e2m1): x [R, H] (slabs [L, cap, H] with masked_m) in bfloat16,
    float16 or float32, H a multiple of 64. fmt "nv": a float8 scale for each 16
    elements and tensor_scale, float32 [1] or one for each of n equal blocks of rows
    (amax / 2688 is a good one, 0 for zeros); "e8m0" and "mx": a power of two for each 32, the
    smallest that saturates nothing, or OCP MX's. Only the first num_live rows, those
    with m_indices >= 0 as a dispatch writes it, or the first masked_m of each slab,
    where one is given. Returns a dict: xq uint8 [.., H / 2], scales uint8
    [pieces, R, 16], ld_s, status."""
    dtype = _elem(x, FLOATS, "x")
    f = _fp4(fmt)
    lead = tuple(x.shape[:-1])
    if x.dim() == 3 and masked_m is not None:
        if not x.is_contiguous() or masked_m.numel() != x.shape[0]:
            raise ValueError("moeperm: with masked_m, x must be contiguous slabs [L, cap, H]")
        x = x.view(-1, x.shape[2])
    ldx = _rows(x, "x")
    R, H = x.shape
    cap = _fp4_rows(R, num_live, m_indices, masked_m)
    nts = _tensor_scale(tensor_scale, fmt, "tensor_scale")
    dev = x.device
    xq = torch.empty((*lead, H // 2), dtype=torch.uint8, device=dev)
    sc = fp4_scale_tensor(R, H, fmt, dev)
    st = _status(status, num_live is not None, dev)
    px, pt, pn, pi, pm, pq, ps, pst = _on_current(x, tensor_scale, num_live, m_indices, masked_m, xq, sc, st)
    _check(lib().moe_quant_fp4(px, ldx, ELEM[dtype], R, H, f, pt, nts, pn, pi, pm, cap, pq, ps, R, pst, _stream()),
           "moe_quant_fp4")
    return dict(xq=xq, scales=sc, ld_s=R, status=st)


def dequant_fp4(xq, scales, fmt="nv", tensor_scale=None, dtype=torch.bfloat16, num_live=None, m_indices=None,
                masked_m=None, status=None, out=None):
    """The values of four-bit rows xq [R, H / 2] (slabs [L, cap, H / 2] with masked_m) with
    their scales, in dtype or into `out`; rows as for quant_fp4, others are not
    written. status: the int32 word that a num_live above R is flagged in (quant_fp4's,
    say)."""
    f = _fp4(fmt)
    if xq.dtype not in FP4_BYTES:
        raise ValueError(f"moeperm: xq must be uint8 pairs of elements, not {xq.dtype}")
    lead, H = tuple(xq.shape[:-1]), xq.shape[-1] * 2
    if not xq.is_contiguous() or xq.dim() != (3 if xq.dim() == 3 and masked_m is not None else 2):
        raise ValueError("moeperm: xq must be contiguous [R, H / 2] (with masked_m also [L, cap, H / 2])")
    R = xq.numel() * 2 // H if H else 0
    cap = _fp4_rows(R, num_live, m_indices, masked_m)
    nts = _tensor_scale(tensor_scale, fmt, "tensor_scale")
    ld = _fp4_scales(scales, R, H, fmt, "scales")
    if out is None:
        out = torch.empty((*lead, H), dtype=dtype, device=xq.device)
    elif tuple(out.shape) != (*lead, H):
        raise ValueError(f"moeperm: out must have shape {(*lead, H)}")
    dtype = _elem(out, FLOATS, "out")
    o2 = out.view(R, H) if out.dim() == 3 else out
    ldx = _rows(o2, "out")
    pq, ps, pt, pn, pi, pm, po, pst = _on_current(xq, scales, tensor_scale, num_live, m_indices, masked_m, o2, status)
    _check(lib().moe_dequant_fp4(pq, ps, ld, R, H, f, pt, nts, pn, pi, pm, cap, po, ldx, ELEM[dtype], pst, _stream()),
           "moe_dequant_fp4")
    return out


def dispatch_fp4(x, topk_ids, topk_weights, num_experts, num_local_experts, block_e=128, fmt="nv",
                 tensor_scale=None, num_tokens=None, workspace=None, status=None, row_weights=True):
    """Quantise to four bits and scatter into the compact layout: xq [bound, H / 2] and
    scales [pieces, bound, 16] as quant_fp4 makes them, and the layout tensors of
    dispatch_compact. x in bfloat16, float16 or float32. Returns a dict."""
    dtype = _elem(x, FLOATS, "x")
    f = _fp4(fmt)
    ldx = _rows(x, "x")
    T, H = x.shape
    K, L, dev = topk_ids.shape[1], num_local_experts, x.device
    _vec(topk_ids, T * K, "topk_ids", torch.int32)
    _vec(topk_weights, T * K, "topk_weights")
    _tensor_scale(tensor_scale, fmt, "tensor_scale", 1)
    bound = moe_compact_bound(T * K, L, block_e)
    # one allocation for the small outputs, and for the workspace (first, so aligned) and the
    # status word where the caller gives none: each costs the host as much as a short kernel
    ws_words = 0 if workspace is not None else (moe_workspace_bytes(T, K, L) + 15) // 16 * 4
    ws, m_indices, s2d, counts, starts, psum, total, rw, st = _words(
        dev, ws_words, bound, T * K, L, L, L, 1, bound if row_weights else 0, int(status is None))
    if workspace is not None:
        ws, ws_bytes = workspace.buf, workspace.nbytes
    else:
        ws_bytes = ws_words * 4
    if status is not None:
        st = status
    else:
        _check(lib().moe_status_clear(*_on_current(st), _stream()), "moe_status_clear")
    o = dict(xq=torch.empty((bound, H // 2), dtype=torch.uint8, device=dev),
             scales=fp4_scale_tensor(bound, H, fmt, dev), ld_s=bound, bound=bound, m_indices=m_indices,
             src2dst=s2d.view(T, K), counts=counts, starts=starts, psum=psum, total=total,
             row_weights=rw.view(torch.float32) if row_weights else None)
    px, pn, pi, pw, pt, *po, pws, pst = _on_current(
        x, num_tokens, topk_ids, topk_weights, tensor_scale, o["xq"], o["scales"], o["m_indices"], o["src2dst"],
        o["counts"], o["starts"], o["psum"], o["total"], o["row_weights"], ws, st)
    _check(lib().moe_dispatch_fp4(px, ldx, ELEM[dtype], T, pn, H, pi, pw, K, num_experts, L, block_e, f, pt, po[0],
                                  po[1], bound, po[2], bound, *po[3:], pws, ws_bytes, pst, _stream()),
           "moe_dispatch_fp4")
    o["status"] = st
    return o


def expert_matmul_fp4(x, w, x_scales, w_scales, fmt="nv", starts=None, psum=None, x_tscale=None, w_tscale=None,
                      bias=None, act="none", gated=False, residual=None, masked_m=None, out=None,
                      out_dtype=torch.bfloat16, status=None):
    """expert_matmul with four-bit rows and weights of one format, as quant_fp4 and
    dispatch_fp4 make them: x uint8 [R, K / 2] (slabs [L, cap, K / 2] with masked_m),
    w uint8 [L, N, K / 2] (gated [L, 2N, K / 2]) with the scales of w.view(-1, K / 2),
    x_tscale float32 [1] and w_tscale [L] ("nv" only). The rest as in expert_matmul, the
    output in out_dtype (bfloat16 or float16). Returns out."""
    f = _fp4(fmt)
    if x.dtype not in FP4_BYTES or w.dtype not in FP4_BYTES:
        raise ValueError(f"moeperm: x and w must be uint8 pairs of four-bit elements, not {x.dtype} and {w.dtype}")
    L, N, K2 = _expert_weights(w, gated)
    if act not in ACT:
        raise ValueError(f"moeperm: act must be one of {sorted(ACT)}, not {act!r}")
    if out_dtype not in FLOATS[:2]:
        raise ValueError(f"moeperm: out_dtype must be bfloat16 or float16, not {out_dtype}")
    masked = masked_m is not None
    begin = end = None
    if L != 1 or masked or starts is not None or psum is not None:
        begin, end = _segments(starts, psum, masked_m, L)
    full = (*x.shape[:-1], N)
    x, cap = _expert_rows(x, masked, L, "x")
    R, Nw = x.shape[0], (2 * N if gated else N)
    ldx = _rows(x, "x", (R, K2))
    ld_xs = _fp4_scales(x_scales, R, 2 * K2, fmt, "x_scales")
    ld_ws = _fp4_scales(w_scales, L * Nw, 2 * K2, fmt, "w_scales")
    if x_tscale is not None:
        _tensor_scale(x_tscale, fmt, "x_tscale", 1)
    if w_tscale is not None:
        _tensor_scale(w_tscale, fmt, "w_tscale", L)
    if bias is not None:
        _vec(bias, L * Nw, "bias")
    if out is None:
        out, odt, o2, ldo = torch.empty(full, dtype=out_dtype, device=x.device), out_dtype, None, N
    else:
        if tuple(out.shape) != full:
            raise ValueError(f"moeperm: out must have shape {full}")
        odt = _elem(out, FLOATS[:2], "out")
        o2 = _expert_rows(out, masked, L, "out")[0]
        ldo = _rows(o2, "out", (R, N), odt)
    res, ld_res = None, 0
    if residual is not None:
        res = _expert_rows(residual, masked, L, "residual")[0]
        ld_res = _rows(res, "residual", (R, N), odt)
    px, pxs, pxt, pw, pws, pwt, pb, p0, p1, pr, po, pst = _on_current(
        x, x_scales, x_tscale, w, w_scales, w_tscale, bias, begin, end, res, out if o2 is None else o2, status)
    _check(lib().moe_expert_matmul_fp4(px, ldx, pxs, ld_xs, pxt, R, 2 * K2, pw, pws, ld_ws, pwt, f, L, N,
                                       1 if gated else 0, ACT[act], pb, p0, p1, cap, pr, ld_res, po, ldo, ELEM[odt],
                                       pst, _stream()), "moe_expert_matmul_fp4")
    return out


def _score(score):
    if score not in SCORE:
        raise ValueError(f"moeperm: score must be one of {sorted(SCORE)}, not {score!r}")
    return SCORE[score]


def _logits(t):
    """Shape, row stride and element type of logits."""
    code = ELEM.get(t.dtype, 3)
    if code > 2 or t.dim() != 2:
        _elem(t, FLOATS, "logits")
    ld = _rows(t, "logits")
    T, E = t.shape
    return T, E, ld, code


def _groups(seq_begin, seq_end):
    """Groups of tokens: how many."""
    if seq_begin is None and seq_end is None:
        return 1
    if seq_begin is None or seq_end is None:
        raise ValueError("moeperm: groups of tokens need seq_begin and seq_end")
    Q = seq_begin.numel()
    _vec(seq_begin, Q, "seq_begin", torch.int32)
    _vec(seq_end, Q, "seq_end", torch.int32)
    return Q


def route(logits, top_k, bias=None, score="softmax", renorm=True, scale=1.0, num_tokens=None, status=None):
    """The experts of each token and their weights from the router's logits [T, E]
    (bfloat16, float16 or float32): the top_k largest logits or, with a bias [E]
    float32 for the choice alone, scores plus bias; lowest index first among equals.
    score "softmax" or "sigmoid"; renorm: weights sum to scale, else they are scale
    times the scores. Experts masked by -inf are never chosen: where too few are left
    the id is -1 (which the dispatches drop) and the weight 0. Returns a dict:
    topk_ids [T, top_k] int32, topk_weights [T, top_k] float32, status."""
    T, E, ldl, code = _logits(logits)
    if bias is not None:
        _vec(bias, E, "bias")
    dev = logits.device
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    st = _status(status, num_tokens is not None, dev)
    pl, pn, pb, pi, pw, pst = _on_current(logits, num_tokens, bias, ids, w, st)
    _check(lib().moe_route(pl, ldl, code, T, pn, E, top_k, _score(score), pb, 1 if renorm else 0, scale, pi, pw,
                           pst, _stream()), "moe_route")
    return dict(topk_ids=ids, topk_weights=w, status=st)


class BalanceWorkspace:
    """Workspace of balance_loss for E experts and up to Q groups, for any number of
    tokens, reusable across calls on one stream; needs no initialisation."""

    def __init__(self, E: int, Q: int, device):
        self.nbytes = moe_balance_loss_workspace_bytes(E, Q)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)


def balance_loss(logits, topk_ids, seq_begin=None, seq_end=None, score="softmax", num_tokens=None,
                 workspace=None, status=None):
    """The router's losses over groups of tokens [seq_begin[q], seq_end[q]) (None: all
    tokens one group; groups one after the other, rows between them belong to none).
    Returns a dict: loss [2] float32, the balance loss (mean over the groups of
    E / (K n^2) sum_e counts * prob_sums, 1 for even use) and the z loss (mean over
    the tokens of logsumexp(logits)^2); counts [Q, E] int32, the slots of each expert;
    prob_sums [Q, E] float32; status."""
    T, E, ldl, code = _logits(logits)
    K, Q, dev = topk_ids.shape[1], _groups(seq_begin, seq_end), logits.device
    _vec(topk_ids, T * K, "topk_ids", torch.int32)
    loss = torch.empty(2, dtype=torch.float32, device=dev)
    counts = torch.empty((Q, E), dtype=torch.int32, device=dev)
    sums = torch.empty((Q, E), dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else BalanceWorkspace(E, Q, dev)
    st = _status(status, num_tokens is not None or seq_begin is not None, dev)
    pl, pn, pi, pb, pe, po, pc, ps, pw, pst = _on_current(logits, num_tokens, topk_ids, seq_begin, seq_end, loss, counts,
                                                          sums, ws.buf, st)
    _check(lib().moe_balance_loss(pl, ldl, code, T, pn, E, pi, K, _score(score), pb, pe, Q, po, pc, ps, pw,
                                  ws.nbytes, pst, _stream()), "moe_balance_loss")
    return dict(loss=loss, counts=counts, prob_sums=sums, status=st)


def route_grad(logits, topk_ids, dweights=None, dloss=None, counts=None, seq_begin=None, seq_end=None,
               score="softmax", renorm=True, scale=1.0, num_tokens=None, status=None, out=None):
    """Gradient of the logits through the weights of route (dweights [T, K]) and through
    both losses of balance_loss (dloss [2], with its counts and groups), in logits'
    type; 0 for tokens that are not live. score, renorm and scale as in the forward
    calls. status: the int32 word that groups out of order and a num_tokens above T
    are flagged in (balance_loss's, which meets the same)."""
    T, E, ldl, code = _logits(logits)
    K, Q, dev = topk_ids.shape[1], _groups(seq_begin, seq_end), logits.device
    _vec(topk_ids, T * K, "topk_ids", torch.int32)
    _vec(dweights, T * K, "dweights")
    _vec(dloss, 2, "dloss")
    _vec(counts, Q * E, "counts", torch.int32)
    if dweights is None and dloss is None:
        raise ValueError("moeperm: route_grad needs dweights, dloss or both")
    if dloss is not None and counts is None:
        raise ValueError("moeperm: the gradient of the balance loss needs its counts")
    out = _like(out, (T, E), logits.dtype, dev, "out")
    pl, pn, pi, pw, pd, pc, pb, pe, po, pst = _on_current(logits, num_tokens, topk_ids, dweights, dloss, counts,
                                                          seq_begin, seq_end, out, status)
    _check(lib().moe_route_grad(pl, ldl, code, T, pn, E, pi, K, _score(score), 1 if renorm else 0, scale, pw,
                                pd, pc, pb, pe, Q, po, E, pst, _stream()), "moe_route_grad")
    return out


def expand_to_slab(exp, psum, num_local_experts, cap, align=128, exp_scales=None, ld_es=0,
                   scale_fmt="packed", group_size=128, status=None):
    """Expanded rows (e4m3 as uint8 / float8, or bfloat16 [R, H]) with segment
    ends psum [L] -> per-expert slabs [L, cap, H]; the scales follow when
    exp_scales is given. Returns a dict (slab, scales, ld_s, masked_m, status)."""
    R, H = exp.shape
    L = num_local_experts
    dev = exp.device
    slab = torch.empty((L, cap, H), dtype=exp.dtype, device=dev)
    ssc, ld_ss = (scale_tensor(scale_fmt, L * cap, H, group_size, dev, blocks=L)
                  if exp_scales is not None else (None, 0))
    masked_m = torch.empty(L, dtype=torch.int32, device=dev)
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    _check(moe_expand_to_slab(exp, exp.element_size(), H, R, exp_scales, ld_es, psum, L, align,
                              cap, scale_fmt, group_size, slab, ssc, ld_ss, masked_m, st),
           "moe_expand_to_slab")
    return dict(slab=slab, scales=ssc, ld_s=ld_ss, masked_m=masked_m, status=st)


def expand_from_slab(slab, psum, num_rows, align=128, slab_scales=None, ld_ss=0,
                     scale_fmt="packed", group_size=128, row_weights=None, status=None,
                     m_indices=True):
    """Per-expert slabs [L, cap, H] -> expanded rows [num_rows, H] at the
    segment ends psum [L]; bfloat16 rows are scaled by row_weights when given.
    Returns a dict (exp, scales, ld_s, m_indices, status)."""
    L, cap, H = slab.shape
    dev = slab.device
    exp = torch.empty((num_rows, H), dtype=slab.dtype, device=dev)
    esc, ld_es = (scale_tensor(scale_fmt, num_rows, H, group_size, dev)
                  if slab_scales is not None else (None, 0))
    mi = torch.empty(num_rows, dtype=torch.int32, device=dev) if m_indices else None
    st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    _check(moe_expand_from_slab(slab, slab.element_size(), H, slab_scales, ld_ss, psum, L, align,
                                cap, scale_fmt, group_size, row_weights, exp, num_rows, esc,
                                ld_es, mi, st), "moe_expand_from_slab")
    return dict(exp=exp, scales=esc, ld_s=ld_es, m_indices=mi, status=st)


def requant(q, s_tok, s_fmt="f32", mode="max_scale"):
    """Per-token -> per-tensor e4m3 requant. s_tok: fp32 [T] ("f32") or e8m0
    bytes [T] ("ue8m0"); mode "max_scale" (S = max s) or "amax" (S = max of
    s * row amax / 448). Returns (q_out uint8 [T,H], S [1] f32)."""
    T, H = q.shape
    q_out = torch.empty((T, H), dtype=torch.uint8, device=q.device)
    S = torch.empty(1, dtype=torch.float32, device=q.device)
    if s_fmt == "f32" and mode == "max_scale":
        _check(fp8_requant_per_tensor(q, q.stride(0), s_tok, T, H, q_out, S),
               "fp8_requant_per_tensor")
    else:
        ws = torch.empty(max(T, 1), dtype=torch.float32, device=q.device)
        _check(fp8_requant_per_tensor_ex(q, q.stride(0), s_tok, s_fmt, T, H, mode, q_out, S, ws,
                                         ws.numel() * 4), "fp8_requant_per_tensor_ex")
    return q_out, S
