"""Thin Python binding of the POET-X C ABI (``include/poetx.h``).

Argument marshalling only: every function forwards torch tensors' device pointers, sizes
and the current CUDA stream to the function of the same name in ``libpoetx.so`` and raises
``PoetxError`` on a non-OK status.  No computation happens here, and there is no fallback:
if the library is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading
from array import array
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpoetx.so")

F32, BF16, I8 = 0, 1, 2
FAST, MEM = 0, 1
SILU, GELU = 0, 1
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8}
_TORCH_DT = {F32: torch.float32, BF16: torch.bfloat16, I8: torch.int8}

_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_ll = ctypes.c_longlong


class PoetxError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg}")
        self.status = status


class LayerDesc(ctypes.Structure):
    """Mirror of ``poetx_layer``."""
    _fields_ = [("m", _i), ("n", _i), ("b", _i), ("order", _i), ("act", _i), ("wdt", _i),
                ("variant", _i), ("perm_m", _vp), ("perm_n", _vp), ("Wp", _vp),
                ("w_scale", _vp), ("q_R", _vp), ("q_P", _vp)]


class AdamDesc(ctypes.Structure):
    """Mirror of ``poetx_adam``."""
    _fields_ = [("lr", _f), ("beta1", _f), ("beta2", _f), ("eps", _f), ("weight_decay", _f),
                ("step", _i)]


class RopeDesc(ctypes.Structure):
    """Mirror of ``poetx_rope``."""
    _fields_ = [("head_dim", _i), ("rot_dim", _i), ("interleaved", _i), ("axes", _i), ("norm", _i),
                ("eps", _f), ("inv_freq", _vp), ("axis", _vp)]


class HeadsDesc(ctypes.Structure):
    """Mirror of ``poetx_heads``."""
    _fields_ = [("heads", _i), ("x", _vp), ("x_pitch", _ll), ("gamma", _vp), ("dy", _vp),
                ("dy_pitch", _ll), ("y", _vp), ("y_pitch", _ll), ("dgamma", _vp)]


_SIGS = {
    "poetx_status_str": (ctypes.c_char_p, [_i]),
    "poetx_get_device_error": (_i, [_vp]),
    "poetx_selftest_timeout": (_i, [ctypes.c_uint, _vp]),
    "poetx_set_gemm_engine": (_i, [_i]),
    "poetx_set_fusion": (_i, [_i]),
    "poetx_set_overlap": (_i, [_i]),
    "poetx_launch_count": (ctypes.c_ulonglong, []),
    "poetx_timeout_site": (_i, []),
    "poetx_profile_enable": (_i, [_i]),
    "poetx_set_trace_buffer": (_i, [_vp, _sz]),
    "poetx_profile_collect": (_i, [ctypes.POINTER(_i), ctypes.POINTER(_f), _i]),
    "poetx_stage_name": (ctypes.c_char_p, [_i]),
    "poetx_cnp_workspace_bytes": (_sz, [_i, _i, _i]),
    "poetx_cnp_fwd": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "poetx_cnp_bwd": (_i, [_vp, _vp, _i, _i, _i, _i, _vp, _i, _vp, _sz, _vp]),
    "poetx_cnp_fwd_noalloc": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "poetx_triu_unpack": (_i, [_vp, _i, _i, _vp, _vp]),
    "poetx_triu_grad_pack": (_i, [_vp, _i, _i, _vp, _i, _vp]),
    "poetx_perm_gather": (_i, [_i, _vp, _i, _i, _vp, _vp, _vp]),
    "poetx_perm_scatter": (_i, [_i, _vp, _i, _i, _vp, _vp, _vp]),
    "poetx_merge_perm": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "poetx_merge_perm_padded": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "poetx_quantize_rows_int8": (_i, [_vp, _i, _i, _vp, _vp, _vp]),
    "poetx_blockdiag_mm": (_i, [_i, _vp, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp]),
    "poetx_blockdiag_wgrad": (_i, [_i, _vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "poetx_wprime_gemm": (_i, [_i, _i, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp]),
    "poetx_layer_workspace_bytes": (_sz, [ctypes.POINTER(LayerDesc), _i, _i]),
    "poetx_layer_saved_bytes": (_sz, [ctypes.POINTER(LayerDesc), _i]),
    "poetx_layer_cuda_core_steps": (_i, [ctypes.POINTER(LayerDesc), _i]),
    "poetx_layer_fwd": (_i, [ctypes.POINTER(LayerDesc), _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "poetx_layer_bwd": (_i, [ctypes.POINTER(LayerDesc), _vp, _vp, _i, _vp, _vp, _vp, _vp, _i,
                             _vp, _sz, _vp]),
    "poetx_layer_step_host_bytes": (_sz, [ctypes.POINTER(LayerDesc), _i]),
    "poetx_layer_step_host": (_i, [ctypes.POINTER(LayerDesc), _vp, _vp, _i, _vp, _vp, _vp, _vp,
                                   _vp, _sz, _vp]),
    "poetx_merge_reinit_workspace_bytes": (_sz, [ctypes.POINTER(LayerDesc)]),
    "poetx_merge_reinit": (_i, [ctypes.POINTER(LayerDesc), _vp, _vp, _sz, _vp]),
    "poetx_adam_triu": (_i, [_vp, _vp, _vp, _vp, ctypes.c_longlong, ctypes.POINTER(AdamDesc),
                             _vp]),
    "poetx_layer_bwd_adam": (_i, [ctypes.POINTER(LayerDesc), _vp, _vp, _i, _vp, _vp, _vp, _vp,
                                  _i, ctypes.POINTER(AdamDesc), _vp, _vp, _vp, _vp, _vp, _sz,
                                  _vp]),
    "poetx_group_saved_bytes": (_sz, [ctypes.POINTER(LayerDesc), _i, _i]),
    "poetx_group_workspace_bytes": (_sz, [ctypes.POINTER(LayerDesc), _i, _i]),
    "poetx_group_cnp_fwd": (_i, [ctypes.POINTER(LayerDesc), _i, _i, _vp, _vp]),
    "poetx_group_layer_fwd": (_i, [ctypes.POINTER(LayerDesc), _i, _i, _vp, _i, _vp, _vp, _vp, _sz,
                                   _vp]),
    "poetx_group_layer_bwd": (_i, [ctypes.POINTER(LayerDesc), _i, _i, _vp, _vp, _i, _vp, _vp, _vp,
                                   _sz, _vp]),
    "poetx_group_cnp_bwd": (_i, [ctypes.POINTER(LayerDesc), _i, _i, _vp,
                                 ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p),
                                 _i, _vp, _sz, _vp]),
    "poetx_group_step_host_bytes": (_sz, [ctypes.POINTER(LayerDesc), _i, _i]),
    "poetx_group_step_host": (_i, [ctypes.POINTER(LayerDesc), _i] +
                              [ctypes.POINTER(ctypes.c_void_p)] * 2 + [_i] +
                              [ctypes.POINTER(ctypes.c_void_p)] * 4 + [_vp, _sz, _vp]),
    "poetx_layernorm_fwd": (_i, [_i, _vp, _i, _i, _vp, _vp, _f, _vp, _vp, _vp, _vp]),
    "poetx_layernorm_bwd_workspace_bytes": (_sz, [_i, _i, _i]),
    "poetx_layernorm_bwd": (_i, [_i, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz,
                                 _vp]),
    "poetx_head_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "poetx_head_ce": (_i, [_i, _vp, _i, _i, _vp, _i, _vp, _f, _vp, _vp, _vp, _vp, _vp, _i, _vp,
                           _sz, _vp]),
    "poetx_head_distill": (_i, [_i, _vp, _i, _i, _vp, _i, _vp, _vp, _i, _f, _vp, _vp, _vp, _vp,
                                _vp, _i, _vp, _sz, _vp]),
    "poetx_glu_fwd": (_i, [_i, _i, _vp, _vp, _i, _i, _ll, _vp, _vp]),
    "poetx_glu_bwd": (_i, [_i, _i, _vp, _vp, _vp, _i, _i, _ll, _vp, _vp, _ll, _vp]),
    "poetx_ffn_fwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "poetx_ffn_fwd": (_i, [_i, _i, _vp, _i, _i, _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "poetx_ffn_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "poetx_ffn_bwd": (_i, [_i, _i, _vp, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "poetx_qk_rope_fwd": (_i, [ctypes.POINTER(RopeDesc), _i, _vp, _i, ctypes.POINTER(HeadsDesc),
                               ctypes.POINTER(HeadsDesc), _vp]),
    "poetx_qk_rope_bwd_workspace_bytes": (_sz, [ctypes.POINTER(RopeDesc)]),
    "poetx_qk_rope_bwd": (_i, [ctypes.POINTER(RopeDesc), _i, _vp, _i, ctypes.POINTER(HeadsDesc),
                               ctypes.POINTER(HeadsDesc), _i, _vp, _sz, _vp]),
    "poetx_grad_norm_workspace_bytes": (_sz, [_i]),
    "poetx_grad_norm": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "poetx_grad_clip": (_i, [_vp, _vp, _vp, _i, _f, _vp, _vp]),
    "poetx_adam_group": (_i, [_vp, _vp, _vp, _vp, _vp, _i, ctypes.POINTER(AdamDesc), _f, _vp, _vp]),
}

_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load ``libpoetx.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("poetx: tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("poetx: tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, st: int):
    if st != 0:
        raise PoetxError(fn, st, lib().poetx_status_str(st).decode())


def status_str(st: int) -> str:
    return lib().poetx_status_str(st).decode()


def poetx_get_device_error(stream=None) -> int:
    return lib().poetx_get_device_error(_stream(stream))


def poetx_selftest_timeout(timeout_us: int, stream=None):
    _check("poetx_selftest_timeout", lib().poetx_selftest_timeout(timeout_us, _stream(stream)))


def poetx_set_gemm_engine(engine: int):
    _check("poetx_set_gemm_engine", lib().poetx_set_gemm_engine(engine))


def poetx_set_fusion(on):
    """True / False: every fused kernel on / off; an int: the library's bit mask (bit 0 the
    W' contraction with the block product after it, bit 1 the backward block product with
    its weight gradient)."""
    mask = (3 if on else 0) if isinstance(on, bool) else int(on)
    _check("poetx_set_fusion", lib().poetx_set_fusion(mask))


def poetx_set_overlap(on: bool):
    _check("poetx_set_overlap", lib().poetx_set_overlap(1 if on else 0))


def poetx_launch_count() -> int:
    return lib().poetx_launch_count()


def poetx_profile_enable(on: bool):
    _check("poetx_profile_enable", lib().poetx_profile_enable(int(bool(on))))


def poetx_set_trace_buffer(buf=None):
    _check("poetx_set_trace_buffer",
           lib().poetx_set_trace_buffer(_p(buf), 0 if buf is None else buf.numel() * buf.element_size()))


def poetx_profile_collect(cap: int = 4096):
    """[(stage name, milliseconds)] for every launch timed since the last collect."""
    st = (_i * cap)()
    ms = (_f * cap)()
    n = lib().poetx_profile_collect(st, ms, cap)
    return [(lib().poetx_stage_name(st[k]).decode(), float(ms[k])) for k in range(n)]


def dtype_code(t: torch.Tensor) -> int:
    return _DT[t.dtype]


# ---------------------------------------------------------------- CNP
def poetx_cnp_workspace_bytes(nblk: int, b: int, phase: int) -> int:
    return lib().poetx_cnp_workspace_bytes(nblk, b, phase)


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def poetx_cnp_fwd(q, b, G_f32=None, G_bf16=None, Gt_bf16=None, ws=None, order=3, stream=None):
    nblk = q.shape[0]
    if ws is None:
        ws = workspace(poetx_cnp_workspace_bytes(nblk, b, 0), q.device)
    _check("poetx_cnp_fwd", lib().poetx_cnp_fwd(_p(q), nblk, b, order, _p(G_f32), _p(G_bf16),
                                                _p(Gt_bf16), _p(ws), ws.numel(),
                                                _stream(stream)))


CNP_NOALLOC_MAX_ELEMS = 2 * 1024 * 1024


def poetx_cnp_fwd_noalloc(q, b, G_f32=None, G_bf16=None, Gt_bf16=None, order=3, stream=None):
    """poetx_cnp_fwd without a workspace: its scratch is a fixed array inside the library
    (for callers that cannot allocate device memory; see include/poetx.h)."""
    _check("poetx_cnp_fwd_noalloc", lib().poetx_cnp_fwd_noalloc(_p(q), q.shape[0], b, order,
                                                                _p(G_f32), _p(G_bf16),
                                                                _p(Gt_bf16), _stream(stream)))


def poetx_cnp_bwd(q, dG, b, dq, accumulate=False, ws=None, order=3, stream=None):
    nblk = q.shape[0]
    splits = dG.shape[0] if dG.dim() == 4 else 1
    if ws is None:
        ws = workspace(poetx_cnp_workspace_bytes(nblk, b, 1), q.device)
    _check("poetx_cnp_bwd", lib().poetx_cnp_bwd(_p(q), _p(dG), splits, nblk, b, order, _p(dq),
                                                int(bool(accumulate)), _p(ws), ws.numel(),
                                                _stream(stream)))


def poetx_triu_unpack(q, b, Q, stream=None):
    _check("poetx_triu_unpack", lib().poetx_triu_unpack(_p(q), q.shape[0], b, _p(Q),
                                                        _stream(stream)))


def poetx_triu_grad_pack(Qbar, dq, accumulate=False, stream=None):
    nblk, b, _ = Qbar.shape
    _check("poetx_triu_grad_pack", lib().poetx_triu_grad_pack(_p(Qbar), nblk, b, _p(dq),
                                                              int(bool(accumulate)),
                                                              _stream(stream)))


# ---------------------------------------------------------------- permutations
def poetx_perm_gather(X, perm, Y, stream=None):
    N, D = X.shape
    _check("poetx_perm_gather", lib().poetx_perm_gather(dtype_code(X), _p(X), N, D, _p(perm),
                                                        _p(Y), _stream(stream)))


def poetx_perm_scatter(X, perm, Y, stream=None):
    N, D = X.shape
    _check("poetx_perm_scatter", lib().poetx_perm_scatter(dtype_code(X), _p(X), N, D, _p(perm),
                                                          _p(Y), _stream(stream)))


def poetx_merge_perm(W0, perm_n, perm_m, Wp, scale=None, scale_p=None, stream=None):
    n, m = W0.shape
    _check("poetx_merge_perm", lib().poetx_merge_perm(_p(W0), _p(scale), dtype_code(W0), n, m,
                                                      _p(perm_n), _p(perm_m), _p(Wp), _p(scale_p),
                                                      _stream(stream)))


def poetx_merge_perm_padded(W0, perm_n, perm_m, Wp, scale=None, scale_p=None, stream=None):
    """Wp [n_pad, m_pad] (its shape gives the padding) <- the merge of W0 [n, m], zero
    elsewhere; scale_p [n_pad] likewise for int8."""
    n, m = W0.shape
    n_pad, m_pad = Wp.shape
    _check("poetx_merge_perm_padded", lib().poetx_merge_perm_padded(
        _p(W0), _p(scale), dtype_code(W0), n, m, n_pad, m_pad, _p(perm_n), _p(perm_m), _p(Wp),
        _p(scale_p), _stream(stream)))


def poetx_quantize_rows_int8(W, Wq, scale, stream=None):
    n, m = W.shape
    _check("poetx_quantize_rows_int8", lib().poetx_quantize_rows_int8(_p(W), n, m, _p(Wq),
                                                                      _p(scale), _stream(stream)))


# ---------------------------------------------------------------- products
def poetx_blockdiag_mm(X, G, Y, trans=False, col_scale=None, out_perm=None, stream=None):
    N = X.shape[0]
    nblk, b, _ = G.shape
    _check("poetx_blockdiag_mm", lib().poetx_blockdiag_mm(dtype_code(X), _p(X), N, nblk, b, _p(G),
                                                          int(bool(trans)), _p(col_scale),
                                                          _p(out_perm), _p(Y), _stream(stream)))


def poetx_blockdiag_wgrad(X, dY, b, dG, stream=None):
    N, D = X.shape
    splits = dG.shape[0]
    _check("poetx_blockdiag_wgrad", lib().poetx_blockdiag_wgrad(dtype_code(X), _p(X), _p(dY), N,
                                                                D // b, b, splits, _p(dG),
                                                                _stream(stream)))


def poetx_wprime_gemm(A, W, C, trans=False, w_scale=None, stream=None):
    N = A.shape[0]
    n, m = W.shape
    _check("poetx_wprime_gemm", lib().poetx_wprime_gemm(dtype_code(A), dtype_code(W), _p(A), N, m,
                                                        n, _p(W), _p(w_scale), int(bool(trans)),
                                                        _p(C), _stream(stream)))


# ---------------------------------------------------------------- the layer
def make_layer(m, n, b, act, wdt, variant, perm_m, perm_n, Wp, q_R, q_P, w_scale=None,
               order=3) -> LayerDesc:
    """Build a ``poetx_layer`` descriptor; the tensors must outlive its use."""
    return LayerDesc(m, n, b, order, act, wdt, variant, _p(perm_m), _p(perm_n), _p(Wp),
                     _p(w_scale), _p(q_R), _p(q_P))


def poetx_layer_workspace_bytes(L: LayerDesc, N: int, phase: int) -> int:
    return lib().poetx_layer_workspace_bytes(ctypes.byref(L), N, phase)


def poetx_layer_cuda_core_steps(L: LayerDesc, N: int) -> int:
    """Bit mask of the layer's products on the CUDA cores (bit 0 CNP, bit 1 block-diagonal
    products, bit 2 W' contraction); 0: all on the tensor cores; -1: invalid descriptor."""
    return lib().poetx_layer_cuda_core_steps(ctypes.byref(L), N)


def poetx_layer_saved_bytes(L: LayerDesc, N: int) -> int:
    return lib().poetx_layer_saved_bytes(ctypes.byref(L), N)


def poetx_layer_fwd(L: LayerDesc, x, y, saved, ws, stream=None):
    N = x.shape[0]
    _check("poetx_layer_fwd", lib().poetx_layer_fwd(ctypes.byref(L), _p(x), N, _p(y), _p(saved),
                                                    _p(ws), ws.numel(), _stream(stream)))


def poetx_layer_bwd(L: LayerDesc, x, dy, saved, dx, dq_R, dq_P, ws, accumulate=False,
                    stream=None):
    N = x.shape[0]
    _check("poetx_layer_bwd", lib().poetx_layer_bwd(ctypes.byref(L), _p(x), _p(dy), N, _p(saved),
                                                    _p(dx), _p(dq_R), _p(dq_P),
                                                    int(bool(accumulate)), _p(ws), ws.numel(),
                                                    _stream(stream)))


def poetx_layer_step_host_bytes(L: LayerDesc, N: int) -> int:
    return lib().poetx_layer_step_host_bytes(ctypes.byref(L), N)


def poetx_layer_step_host(L: LayerDesc, x, dy, y, dx, dq_R, dq_P, dev, stream=None):
    """Forward + backward with host (CPU, preferably pinned) tensors x, dy in and y, dx,
    dq_R, dq_P out; dev: device scratch of poetx_layer_step_host_bytes(L, N) bytes.  The
    outputs are valid once `stream` has been synchronised."""
    for t in (x, dy, y, dx, dq_R, dq_P):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("poetx_layer_step_host takes contiguous host tensors")
    N = x.shape[0]
    h = lambda t: ctypes.c_void_p(t.data_ptr())
    _check("poetx_layer_step_host", lib().poetx_layer_step_host(
        ctypes.byref(L), h(x), h(dy), N, h(y), h(dx), h(dq_R), h(dq_P), _p(dev),
        dev.numel() * dev.element_size(), _stream(stream)))


def poetx_merge_reinit_workspace_bytes(L: LayerDesc) -> int:
    return lib().poetx_merge_reinit_workspace_bytes(ctypes.byref(L))


def poetx_merge_reinit(L: LayerDesc, W0_new, ws, stream=None):
    """W0_new [n, m] fp32 <- the layer's current map as a plain weight (q reset is the
    caller's)."""
    _check("poetx_merge_reinit", lib().poetx_merge_reinit(ctypes.byref(L), _p(W0_new), _p(ws),
                                                          ws.numel(), _stream(stream)))


def poetx_adam_triu(q, dq, m, v, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                    eps: float = 1e-8, weight_decay: float = 0.0, stream=None):
    """In-place Adam step on the packed triangles q (m, v: state, zero at step 1)."""
    hp = AdamDesc(lr, beta1, beta2, eps, weight_decay, step)
    _check("poetx_adam_triu", lib().poetx_adam_triu(_p(q), _p(dq), _p(m), _p(v), q.numel(),
                                                    ctypes.byref(hp), _stream(stream)))


def poetx_timeout_site() -> int:
    """Site id of the first expired bounded wait reported by the last poetx_get_device_error
    (file id x 10000 + source line), 0 if none."""
    return lib().poetx_timeout_site()


def poetx_layer_bwd_adam(L: LayerDesc, x, dy, saved, dx, dq_R, dq_P, ws, m_R, v_R, m_P, v_P,
                         step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                         eps: float = 1e-8, weight_decay: float = 0.0, accumulate=False,
                         stream=None):
    """poetx_layer_bwd, then Adam on the layer's q_R and q_P in place (fused into the
    gradient pack)."""
    hp = AdamDesc(lr, beta1, beta2, eps, weight_decay, step)
    N = x.shape[0]
    _check("poetx_layer_bwd_adam", lib().poetx_layer_bwd_adam(
        ctypes.byref(L), _p(x), _p(dy), N, _p(saved), _p(dx), _p(dq_R), _p(dq_P),
        int(bool(accumulate)), ctypes.byref(hp), _p(m_R), _p(v_R), _p(m_P), _p(v_P), _p(ws),
        ws.numel(), _stream(stream)))


# ---------------------------------------------------------------- layer groups
GROUP_MAX_LAYERS = 16


def make_group(layers):
    """A ctypes array of ``poetx_layer`` descriptors (the group); the tensors the descriptors
    point to must outlive its use."""
    arr = (LayerDesc * len(layers))(*layers)
    return arr


def poetx_group_saved_bytes(G, N: int) -> int:
    return lib().poetx_group_saved_bytes(G, len(G), N)


def poetx_group_workspace_bytes(G, N: int) -> int:
    return lib().poetx_group_workspace_bytes(G, len(G), N)


def poetx_group_cnp_fwd(G, N: int, saved, stream=None):
    _check("poetx_group_cnp_fwd", lib().poetx_group_cnp_fwd(G, len(G), N, _p(saved),
                                                            _stream(stream)))


def poetx_group_layer_fwd(G, i: int, x, y, saved, ws, stream=None):
    N = x.shape[0]
    _check("poetx_group_layer_fwd", lib().poetx_group_layer_fwd(
        G, len(G), i, _p(x), N, _p(y), _p(saved), _p(ws), ws.numel(), _stream(stream)))


def poetx_group_layer_bwd(G, i: int, x, dy, saved, dx, ws, stream=None):
    N = x.shape[0]
    _check("poetx_group_layer_bwd", lib().poetx_group_layer_bwd(
        G, len(G), i, _p(x), _p(dy), N, _p(saved), _p(dx), _p(ws), ws.numel(),
        _stream(stream)))


def poetx_group_cnp_bwd(G, N: int, saved, dq_R, dq_P, ws, accumulate=False, stream=None):
    """dq_R, dq_P: one fp32 tensor per layer of the group."""
    if len(dq_R) != len(G) or len(dq_P) != len(G):
        raise ValueError("poetx_group_cnp_bwd: one dq_R and one dq_P per layer")
    pr = (ctypes.c_void_p * len(G))(*[t.data_ptr() for t in dq_R])
    pp = (ctypes.c_void_p * len(G))(*[t.data_ptr() for t in dq_P])
    for t in list(dq_R) + list(dq_P):
        _p(t)
    _check("poetx_group_cnp_bwd", lib().poetx_group_cnp_bwd(
        G, len(G), N, _p(saved), pr, pp, int(bool(accumulate)), _p(ws), ws.numel(),
        _stream(stream)))


def poetx_group_step_host_bytes(G, N: int) -> int:
    return lib().poetx_group_step_host_bytes(G, len(G), N)


def poetx_group_step_host(G, xs, dys, ys, dxs, dq_R, dq_P, dev, stream=None):
    """One training step of the group with host (CPU, preferably pinned) tensors: xs, dys in,
    ys, dxs, dq_R, dq_P out (one per layer); dev: device scratch of
    poetx_group_step_host_bytes(G, N) bytes.  The outputs are valid once `stream` has been
    synchronised."""
    k = len(G)
    lists = (xs, dys, ys, dxs, dq_R, dq_P)
    if any(len(t) != k for t in lists):
        raise ValueError("poetx_group_step_host: one tensor per layer in every list")
    for ts in lists:
        for t in ts:
            if t.is_cuda or not t.is_contiguous():
                raise ValueError("poetx_group_step_host takes contiguous host tensors")
    N = xs[0].shape[0]
    arr = lambda ts: (ctypes.c_void_p * k)(*[t.data_ptr() for t in ts])
    _check("poetx_group_step_host", lib().poetx_group_step_host(
        G, k, arr(xs), arr(dys), N, arr(ys), arr(dxs), arr(dq_R), arr(dq_P), _p(dev),
        dev.numel() * dev.element_size(), _stream(stream)))


# ---------------------------------------------------------------- layer norm
def _want(fn: str, what: str, t, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype is not dtype):
        raise ValueError(f"{fn}: {what} must be {tuple(shape)} of {dtype}, "
                         f"got {tuple(t.shape)} of {t.dtype}")


def _here(t):
    """Refuses a tensor that does not live on the current device, whose stream and limits a call takes."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("poetx: tensors must live on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError("poetx: tensors must live on the current device")


def _addr(t):
    """A tensor's device address as an integer (None: None)."""
    if t is None:
        return None
    _here(t)
    if not t.is_contiguous():
        raise ValueError("poetx: tensors must be contiguous")
    return t.data_ptr()


def _raw_stream(stream, t):
    """The stream's handle (None: the current one of t's device, without building its object)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream.cuda_stream


_kept = threading.local()
_KEPT_BYTES = 64 << 20


def _scratch(nbytes: int, t, stream, handle: int):
    """Scratch for one call on the device of t.  On the default stream, where a thread's calls follow
    one another, the thread keeps one buffer of up to 64 MB (allocating and freeing one costs more
    host time than a small call's launches); elsewhere it comes from the allocator pool of the stream
    that will use it."""
    if stream is None:
        if handle == 0 and nbytes <= _KEPT_BYTES:
            kept, dev = _kept.__dict__, t.get_device()
            ws = kept.get(dev)
            if ws is None or ws.numel() < nbytes:
                ws = kept[dev] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8,
                                             device=t.device)
            return ws
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=t.device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=t.device)


def poetx_layernorm_fwd(x, y, gamma=None, beta=None, mean=None, rstd=None, eps=1e-5, stream=None):
    """y = layer norm of the rows of x [N, D] (bf16 or fp32); gamma, beta [D] fp32; mean, rstd [N]
    fp32 outputs, kept for the backward."""
    fn, f32 = "poetx_layernorm_fwd", torch.float32
    N, D = x.shape
    _want(fn, "y", y, x.shape, x.dtype)
    _want(fn, "gamma", gamma, (D,), f32)
    _want(fn, "beta", beta, (D,), f32)
    _want(fn, "mean", mean, (N,), f32)
    _want(fn, "rstd", rstd, (N,), f32)
    st = lib().poetx_layernorm_fwd(_DT[x.dtype], _addr(x), N, D, _addr(gamma), _addr(beta), eps,
                                   _addr(y), _addr(mean), _addr(rstd), _raw_stream(stream, x))
    if st:
        _check(fn, st)


def poetx_layernorm_bwd_workspace_bytes(dt: int, N: int, D: int) -> int:
    return lib().poetx_layernorm_bwd_workspace_bytes(dt, N, D)


def poetx_layernorm_bwd(x, dy, mean, rstd, dx, gamma=None, dgamma=None, dbeta=None,
                        accumulate=False, ws=None, stream=None):
    """dx [N, D] and (where given) dgamma, dbeta [D] fp32 from dy and the forward's x, mean and
    rstd."""
    fn, f32 = "poetx_layernorm_bwd", torch.float32
    N, D = x.shape
    _want(fn, "dy", dy, x.shape, x.dtype)
    _want(fn, "dx", dx, x.shape, x.dtype)
    _want(fn, "gamma", gamma, (D,), f32)
    _want(fn, "dgamma", dgamma, (D,), f32)
    _want(fn, "dbeta", dbeta, (D,), f32)
    _want(fn, "mean", mean, (N,), f32)
    _want(fn, "rstd", rstd, (N,), f32)
    dt, L, px = _DT[x.dtype], lib(), _addr(x)
    handle = _raw_stream(stream, x)
    if ws is None:
        ws = _scratch(L.poetx_layernorm_bwd_workspace_bytes(dt, N, D), x, stream, handle)
    st = L.poetx_layernorm_bwd(dt, px, _addr(dy), N, D, _addr(gamma), _addr(mean), _addr(rstd),
                               _addr(dx), _addr(dgamma), _addr(dbeta), 1 if accumulate else 0,
                               _addr(ws), ws.numel(), handle)
    if st:
        _check(fn, st)


# ---------------------------------------------------------------- the linear head's loss
def poetx_head_workspace_bytes(dt: int, N: int, D: int, V: int, K: int = 1, want_dx: bool = True,
                               want_dW: bool = True) -> int:
    return lib().poetx_head_workspace_bytes(dt, N, D, V, K, int(want_dx), int(want_dW))


def _head(fn, call, x, W, K, target, logit, loss, dloss, dx, dW, lse, ws, stream, option, accumulate):
    """Checks and marshals what both head losses share (logit: None for labels; option: the call's
    own argument before dloss)."""
    f32 = torch.float32
    (N, D), V = x.shape, W.shape[0]
    _want(fn, "W", W, (V, D), x.dtype)
    _want(fn, "dx", dx, x.shape, x.dtype)
    _want(fn, "dW", dW, (V, D), x.dtype)
    _want(fn, "loss", loss, (N,), f32)
    _want(fn, "lse", lse, (N,), f32)
    _want(fn, "dloss", dloss, (N,), f32)
    dt, px = _DT[x.dtype], _addr(x)
    targets = (_addr(target),) if logit is None else (_addr(target), _addr(logit), K)
    handle = _raw_stream(stream, x)
    if ws is None:
        ws = _scratch(lib().poetx_head_workspace_bytes(dt, N, D, V, K, dx is not None,
                                                       dW is not None), x, stream, handle)
    st = call(dt, px, N, D, _addr(W), V, *targets, option, _addr(dloss), _addr(loss), _addr(lse),
              _addr(dx), _addr(dW), 1 if accumulate else 0, _addr(ws), ws.numel(), handle)
    if st:
        _check(fn, st)


def poetx_head_ce(x, W, target, loss, dloss=None, dx=None, dW=None, lse=None, z_loss=0.0,
                  accumulate=False, ws=None, stream=None):
    """loss [N] fp32 of the softmax cross entropy of x W^T against target [N] int32 (negative:
    ignored), and with dloss [N] fp32 (the upstream gradients) dx and / or dW."""
    fn = "poetx_head_ce"
    _want(fn, "target", target, (x.shape[0],), torch.int32)
    _head(fn, lib().poetx_head_ce, x, W, 1, target, None, loss, dloss, dx, dW, lse, ws, stream,
          z_loss, accumulate)


def poetx_head_distill(x, W, t_index, t_logit, loss, dloss=None, dx=None, dW=None, lse=None,
                       temperature=1.0, accumulate=False, ws=None, stream=None):
    """loss [N] fp32 of T^2 KL(teacher || student) from the teacher's top logits t_logit [N, K]
    fp32 at the entries t_index [N, K] int32 (negative: absent), and with dloss the gradients."""
    fn = "poetx_head_distill"
    shape = (x.shape[0], t_index.shape[-1])
    _want(fn, "t_index", t_index, shape, torch.int32)
    _want(fn, "t_logit", t_logit, shape, torch.float32)
    _head(fn, lib().poetx_head_distill, x, W, shape[1], t_index, t_logit, loss, dloss, dx, dW, lse,
          ws, stream, temperature, accumulate)


# ---------------------------------------------------------------- the gated feed-forward block
def _dtype(fn: str, t) -> int:
    """The code of t's type."""
    dt = _DT.get(t.dtype)
    if dt is None or dt == I8:
        raise ValueError(f"{fn}: bf16 or fp32, got {t.dtype}")
    return dt


def _rows(fn: str, what: str, t, width: int):
    """(address, elements from row to row) of t [N, ...] whose rows of `width` elements are each
    contiguous."""
    _here(t)
    if t.is_contiguous():
        return t.data_ptr(), width
    at = width
    for size, stride in zip(t.shape[1:], t.stride()[1:]):
        at //= size if size else 1
        if size > 1 and stride != at:
            raise ValueError(f"{fn}: the rows of {what} must be contiguous")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else width


def poetx_glu_fwd(g, u, h, act=SILU, stream=None):
    """h [N, F] = a(g) u (bf16 or fp32); g and u [N, F] may be the halves of one [N, 2 F] tensor, or
    any two with the same distance from row to row."""
    fn = "poetx_glu_fwd"
    N, F = g.shape
    _want(fn, "u", u, g.shape, g.dtype)
    _want(fn, "h", h, g.shape, g.dtype)
    dt = _dtype(fn, g)
    (pg, pitch), (pu, pitch_u) = _rows(fn, "g", g, F), _rows(fn, "u", u, F)
    if pitch != pitch_u:
        raise ValueError(f"{fn}: g and u must have the same distance from row to row")
    st = lib().poetx_glu_fwd(dt, act, pg, pu, N, F, pitch, _addr(h), _raw_stream(stream, g))
    if st:
        _check(fn, st)


def poetx_glu_bwd(g, u, dh, dg, du, act=SILU, stream=None):
    """dg = dh u a'(g) and du = dh a(g); dg and du have the same distance from row to row, and may be g
    and u themselves."""
    fn = "poetx_glu_bwd"
    N, F = g.shape
    for what, t in (("u", u), ("dh", dh), ("dg", dg), ("du", du)):
        _want(fn, what, t, g.shape, g.dtype)
    dt = _dtype(fn, g)
    (pg, pitch), (pu, pitch_u) = _rows(fn, "g", g, F), _rows(fn, "u", u, F)
    (pdg, d_pitch), (pdu, d_pitch_u) = _rows(fn, "dg", dg, F), _rows(fn, "du", du, F)
    if pitch != pitch_u or d_pitch != d_pitch_u:
        raise ValueError(f"{fn}: g and u (dg and du) must have the same distance from row to row")
    st = lib().poetx_glu_bwd(dt, act, pg, pu, _addr(dh), N, F, pitch, pdg, pdu, d_pitch,
                             _raw_stream(stream, g))
    if st:
        _check(fn, st)


def poetx_ffn_fwd_workspace_bytes(dt: int, N: int, D: int, F: int) -> int:
    return lib().poetx_ffn_fwd_workspace_bytes(dt, N, D, F)


def poetx_ffn_fwd(x, W, h, z=None, act=SILU, ws=None, stream=None):
    """h [N, F] = a(x Wg^T) (x Wu^T) with W [2 F, D] = Wg's rows, then Wu's (bf16 or fp32); z [N, 2 F]
    (optional): the projections, for the backward."""
    fn = "poetx_ffn_fwd"
    (N, D), F = x.shape, W.shape[0] // 2
    _want(fn, "W", W, (2 * F, D), x.dtype)
    _want(fn, "h", h, (N, F), x.dtype)
    _want(fn, "z", z, (N, 2 * F), x.dtype)
    dt, L, px = _dtype(fn, x), lib(), _addr(x)
    handle = _raw_stream(stream, x)
    if ws is None and dt == F32:
        ws = _scratch(L.poetx_ffn_fwd_workspace_bytes(dt, N, D, F), x, stream, handle)
    st = L.poetx_ffn_fwd(dt, act, px, N, D, _addr(W), F, _addr(h), _addr(z), _addr(ws),
                         0 if ws is None else ws.numel(), handle)
    if st:
        _check(fn, st)


def poetx_ffn_bwd_workspace_bytes(dt: int, N: int, D: int, F: int, have_z: bool = True,
                                  want_dx: bool = True, want_dW: bool = True) -> int:
    return lib().poetx_ffn_bwd_workspace_bytes(dt, N, D, F, int(have_z), int(want_dx), int(want_dW))


def poetx_ffn_bwd(x, W, dh, z=None, dx=None, dW=None, act=SILU, accumulate=False, ws=None,
                  stream=None):
    """dx [N, D] and / or dW [2 F, D] from dh [N, F]; z: the forward's projections, or None (they are
    computed again)."""
    fn = "poetx_ffn_bwd"
    (N, D), F = x.shape, W.shape[0] // 2
    _want(fn, "W", W, (2 * F, D), x.dtype)
    _want(fn, "dh", dh, (N, F), x.dtype)
    _want(fn, "z", z, (N, 2 * F), x.dtype)
    _want(fn, "dx", dx, x.shape, x.dtype)
    _want(fn, "dW", dW, (2 * F, D), x.dtype)
    dt, L, px = _dtype(fn, x), lib(), _addr(x)
    handle = _raw_stream(stream, x)
    if ws is None:
        ws = _scratch(L.poetx_ffn_bwd_workspace_bytes(dt, N, D, F, z is not None, dx is not None,
                                                      dW is not None), x, stream, handle)
    st = L.poetx_ffn_bwd(dt, act, px, N, D, _addr(W), F, _addr(z), _addr(dh), _addr(dx), _addr(dW),
                         1 if accumulate else 0, _addr(ws), ws.numel(), handle)
    if st:
        _check(fn, st)


# ---------------------------------------------------------------- queries and keys
def _rope(fn, x, pos, inv_freq, rot_dim, axis, interleaved, norm, eps):
    """The checked descriptor and type of a call on x [N, heads, head_dim]."""
    N, _, dh = x.shape
    half = (dh if rot_dim is None else rot_dim) // 2
    axes = pos.shape[0] if pos.dim() == 2 else 1
    _want(fn, "pos", pos, (axes, N) if pos.dim() == 2 else (N,), torch.int32)
    _want(fn, "inv_freq", inv_freq, (half,), torch.float32)
    _want(fn, "axis", axis, (half,), torch.int32)
    return _dtype(fn, x), RopeDesc(dh, dh if rot_dim is None else rot_dim, 1 if interleaved else 0,
                                   axes, 1 if norm else 0, eps, _addr(inv_freq), _addr(axis))


def _heads(fn, what, x, gamma, y, like, dy=None, dgamma=None):
    """The descriptor of one side (None: x is None)."""
    if x is None:
        return None
    shape, dtype = x.shape, x.dtype
    N, H, dh = shape
    if x is not like and (N, dh, dtype) != (like.shape[0], like.shape[2], like.dtype):
        raise ValueError(f"{fn}: queries and keys must have the same tokens, head width and type")
    _want(fn, what + "'s output", y, shape, dtype)
    if gamma is not None:
        _want(fn, "gamma_" + what, gamma, (dh,), torch.float32)
        gamma = _addr(gamma)
    px, pitch = _rows(fn, what, x, H * dh)
    py, y_pitch = _rows(fn, what + "'s output", y, H * dh)
    if dy is None:
        return HeadsDesc(H, px, pitch, gamma, None, 0, py, y_pitch, None)
    _want(fn, "d" + what, dy, shape, dtype)
    _want(fn, "dgamma_" + what, dgamma, (dh,), torch.float32)
    return HeadsDesc(H, px, pitch, gamma, *_rows(fn, "d" + what, dy, H * dh), py, y_pitch,
                     _addr(dgamma))


def poetx_qk_rope_fwd(q, k, pos, inv_freq, q_out, k_out, rot_dim=None, axis=None, interleaved=False,
                      norm=True, gamma_q=None, gamma_k=None, eps=1e-6, stream=None):
    """q_out [N, Hq, dh], k_out [N, Hk, dh] = queries and keys with each head normalised (norm) and
    rotated by the angles pos * inv_freq.  pos [N] or [axes, N] int32; inv_freq [rot_dim / 2] fp32; axis
    [rot_dim / 2] int32 (which positions each pair takes).  Tokens may be any distance apart, so that
    q and k can lie in one row with the values; k may be None; an output may be its input."""
    fn = "poetx_qk_rope_fwd"
    dt, r = _rope(fn, q, pos, inv_freq, rot_dim, axis, interleaved, norm, eps)
    sq = _heads(fn, "q", q, gamma_q, q_out, q)
    sk = _heads(fn, "k", k, gamma_k, k_out, q)
    st = lib().poetx_qk_rope_fwd(r, dt, _addr(pos), q.shape[0], sq, sk, _raw_stream(stream, q))
    if st:
        _check(fn, st)


def poetx_qk_rope_bwd_workspace_bytes(r: RopeDesc) -> int:
    return lib().poetx_qk_rope_bwd_workspace_bytes(ctypes.byref(r))


def poetx_qk_rope_bwd(q, k, dq, dk, pos, inv_freq, dq_in, dk_in, rot_dim=None, axis=None,
                      interleaved=False, norm=True, gamma_q=None, gamma_k=None, dgamma_q=None,
                      dgamma_k=None, eps=1e-6, accumulate=False, ws=None, stream=None):
    """dq_in, dk_in (the gradients of the forward's q and k) and, with norm and where given, dgamma_q,
    dgamma_k [dh] fp32, from dq, dk (those of its outputs)."""
    fn = "poetx_qk_rope_bwd"
    dt, r = _rope(fn, q, pos, inv_freq, rot_dim, axis, interleaved, norm, eps)
    sq = _heads(fn, "q", q, gamma_q, dq_in, q, dq, dgamma_q)
    sk = _heads(fn, "k", k, gamma_k, dk_in, q, dk, dgamma_k)
    handle, L = _raw_stream(stream, q), lib()
    if ws is None and norm and (dgamma_q is not None or dgamma_k is not None):
        ws = _scratch(L.poetx_qk_rope_bwd_workspace_bytes(r), q, stream, handle)
    st = L.poetx_qk_rope_bwd(r, dt, _addr(pos), q.shape[0], sq, sk, 1 if accumulate else 0, _addr(ws),
                             0 if ws is None else ws.numel(), handle)
    if st:
        _check(fn, st)


# ---------------------------------------------------------------- many tensors
_GRAD_TYPES = {torch.float32, torch.bfloat16}
_FP32 = {torch.float32}
_dtype_of = operator.attrgetter("dtype")


def _arrays(fn, what, ts, types):
    """(the tensors' addresses as an array for the library, the set of their types).  Maps: with hundreds of
    tensors the host's work is as long as the kernels'."""
    found = set(map(_dtype_of, ts))
    if found - types or not all(map(torch.Tensor.is_contiguous, ts)) or \
            set(map(torch.Tensor.get_device, ts)) - {torch._C._cuda_getDevice()}:
        raise ValueError(f"{fn}: {what} must be contiguous tensors on the current CUDA device, of "
                         f"{' or '.join(map(str, types))}")
    return array("Q", map(torch.Tensor.data_ptr, ts)), found


def _at(a):
    return a.buffer_info()[0]


def _distinct(fn, what, p, counts):
    """Refuses tensors that are written and named twice: two blocks would do so at once."""
    if len(set(p)) == len(p):
        return
    some = [a for a, n in zip(p, counts) if n]
    if len(set(some)) != len(some):
        raise ValueError(f"{fn}: a tensor is among {what} twice")


def _gradients(fn, grads):
    if not isinstance(grads, (list, tuple)):
        grads = list(grads)  # (gone through several times)
    p, found = _arrays(fn, "gradients", grads, _GRAD_TYPES)
    if len(found) == 1:
        codes = array("i", [_DT[found.pop()]]) * len(grads)
    else:
        codes = array("i", [_DT[t.dtype] for t in grads])
    return p, codes, array("q", map(torch.Tensor.numel, grads))


def poetx_grad_norm_workspace_bytes(n: int) -> int:
    return lib().poetx_grad_norm_workspace_bytes(n)


def poetx_grad_norm(grads, norm, ws=None, stream=None):
    """norm [1] fp32 = the 2-norm over all elements of the tensors in the list grads (fp32 or bf16,
    mixed)."""
    fn = "poetx_grad_norm"
    _want(fn, "norm", norm, (1,), torch.float32)
    pn = _addr(norm)
    p, dts, counts = _gradients(fn, grads)
    handle = _raw_stream(stream, norm)
    if ws is None:
        ws = _scratch(lib().poetx_grad_norm_workspace_bytes(len(p)), norm, stream, handle)
    st = lib().poetx_grad_norm(_at(p), _at(dts), _at(counts), len(p), pn, _addr(ws), ws.numel(), handle)
    if st:
        _check(fn, st)


def poetx_grad_clip(grads, norm, max_norm: float, stream=None):
    """Every tensor of the list times min(1, max_norm / (norm + 1e-6)), in place; norm [1] as
    poetx_grad_norm leaves it.  The tensors must not overlap (one that is listed twice is refused)."""
    fn = "poetx_grad_clip"
    _want(fn, "norm", norm, (1,), torch.float32)
    pn = _addr(norm)
    p, dts, counts = _gradients(fn, grads)
    _distinct(fn, "the gradients", p, counts)
    st = lib().poetx_grad_clip(_at(p), _at(dts), _at(counts), len(p), max_norm, pn,
                               _raw_stream(stream, norm))
    if st:
        _check(fn, st)


def poetx_adam_group(q, dq, m, v, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                     eps: float = 1e-8, weight_decay: float = 0.0, norm=None,
                     max_norm: float = float("inf"), stream=None):
    """poetx_adam_triu on lists of fp32 tensors at once; with norm [1] every gradient is multiplied by
    min(1, max_norm / (norm + 1e-6)) as it is read (dq is not written).  The tensors of q, m and v must not
    overlap (one that is listed twice is refused)."""
    fn = "poetx_adam_group"
    n = len(q)
    if len(dq) != n or len(m) != n or len(v) != n:
        raise ValueError(f"{fn}: one dq, m and v per q")
    count = array("q", map(torch.Tensor.numel, q))
    arrays = []
    for what, ts in (("q", q), ("dq", dq), ("m", m), ("v", v)):
        if ts is not q and array("q", map(torch.Tensor.numel, ts)) != count:
            raise ValueError(f"{fn}: dq, m and v must have the sizes of q")
        arrays.append(_arrays(fn, what, ts, _FP32)[0])
        if what != "dq":
            _distinct(fn, what, arrays[-1], count)
    _want(fn, "norm", norm, (1,), torch.float32)
    hp = AdamDesc(lr, beta1, beta2, eps, weight_decay, step)
    handle = _stream(stream) if n == 0 else _raw_stream(stream, q[0])
    st = lib().poetx_adam_group(*map(_at, arrays), _at(count), n, hp, max_norm, _addr(norm), handle)
    if st:
        _check(fn, st)
