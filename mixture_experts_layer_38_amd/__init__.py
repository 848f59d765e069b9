"""MI355X (gfx950) MoE layer forward pass: Python binding of libmoe.so.

The functions below carry the names of the C ABI in include/moe.h and do
argument marshalling only: every step of the layer runs in the HIP kernels of
libmoe.so.  Tensors are torch tensors on the GPU (torch supplies device memory
and the stream); optional arguments may be None.  The binding raises MoEError
for any non-OK status, and raises at import of the library when libmoe.so has
not been built (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os

from .configs import CONFIGS, MoEConfig

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
MOE_FLAG_BIAS_SELECT_ONLY, MOE_FLAG_COMBINE_MEAN = 1, 2

KERNEL_IDS = {
    "router": 0, "dispatch_count": 1, "dispatch_scan": 2, "dispatch_scatter": 3,
    "dispatch_gather": 4, "ffn_gate_up": 5, "ffn_down": 6, "combine": 7, "aux_loss": 8,
    "bias_update": 9, "ffn_plan": 10, "router_losses": 11, "ffn": 12, "ffn_train": 13,
    "ffn_backward": 14, "combine_backward": 15, "route_backward": 16, "quantize": 17, "ffn_i8": 18,
}


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib().moe_status_string(status).decode() if status >= 0 else "?"
        super().__init__(f"{where}: status {status} ({msg})")


class MoEProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class MoEDebugOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "logits", "probs", "prob_sum", "topk_ids", "topk_w", "counts", "kept", "offsets",
        "assign_row", "row_assign", "z_loss", "aux_topk")]


class MoEI8Weights(ctypes.Structure):
    """The experts' 8-bit weights (device pointers); build one with i8_weights()."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("w1", "w3", "w2", "s1", "s3", "s2")]


_LIB = None


def _lib():
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m mixture_experts_layer_38_amd.build` (no fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    P = ctypes.POINTER(MoEProblem)
    sigs = {
        "moe_route_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_dispatch_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_expert_ffn_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_router_losses_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_combine_concat_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_forward_chunked_workspace_size": [P, ctypes.c_int32, ctypes.POINTER(sz)],
        "moe_forward_chunked": [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp,
                                ctypes.POINTER(MoEDebugOut), vp, sz, vp],
        "moe_router_losses": [P, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_combine_concat": [P, vp, vp, vp, vp, vp, sz, vp],
        "moe_route": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_dispatch": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_expert_ffn": [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_combine": [P, vp, vp, vp, vp, vp],
        "moe_forward": [P, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(MoEDebugOut), vp, sz, vp],
        "moe_forward_noalloc": [P, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(MoEDebugOut), vp],
        "moe_aux_loss": [P, vp, vp, vp, vp],
        "moe_bias_update": [P, vp, f32, vp, vp],
        "moe_expert_ffn_train_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_expert_ffn_train": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_expert_ffn_backward_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_expert_ffn_backward": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_combine_backward": [P, vp, vp, vp, vp, vp, vp, vp],
        "moe_route_backward_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_route_backward": [P, vp, vp, vp, vp, vp, vp, vp, vp, f32, f32, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_quantize_rows": [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp],
        "moe_expert_ffn_i8_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_expert_ffn_i8": [P, vp, vp, ctypes.POINTER(MoEI8Weights), vp, vp, vp, sz, vp],
        "moe_forward_i8_workspace_size": [P, ctypes.POINTER(sz)],
        "moe_forward_i8": [P, vp, vp, ctypes.POINTER(MoEI8Weights), vp, vp, ctypes.POINTER(MoEDebugOut), vp, sz,
                           vp],
        "moe_set_kernel_timer": [i32, vp, vp, i32, ctypes.POINTER(i32)],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_version.restype = ctypes.c_char_p
    lib.moe_kernel_name.argtypes = [ctypes.c_int]
    lib.moe_kernel_name.restype = ctypes.c_char_p
    _LIB = lib
    return lib


def load():
    """Load libmoe.so (raises when it is missing)."""
    return _lib()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # current_stream() builds an object (2.5 us)
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _check(status: int, where: str):
    if status != 0:
        raise MoEError(status, where)


def problem(T: int, d_model: int, n_experts: int, top_k: int, d_ff: int, dtype: str = "bf16",
            capacity: int = -1, flags: int = 0) -> MoEProblem:
    code = {"f32": MOE_DTYPE_F32, "bf16": MOE_DTYPE_BF16}[dtype]
    return MoEProblem(T, d_model, n_experts, top_k, d_ff, code, capacity, flags)


def problem_of(cfg: MoEConfig, T: int | None = None) -> MoEProblem:
    return problem(cfg.T if T is None else T, cfg.d, cfg.E, cfg.K, cfg.F, cfg.dtype, cfg.capacity)


def _size(fn, p: MoEProblem) -> int:
    out = ctypes.c_size_t(0)
    _check(fn(ctypes.byref(p), ctypes.byref(out)), fn.__name__)
    return out.value


def moe_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_workspace_size, p)


def moe_route_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_route_workspace_size, p)


def moe_dispatch_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_dispatch_workspace_size, p)


def moe_expert_ffn_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_expert_ffn_workspace_size, p)


def moe_router_losses_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_router_losses_workspace_size, p)


def moe_route(p, x, w_router, logit_bias, logits, probs, prob_sum, topk_ids, topk_w,
              ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib().moe_route(ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(logit_bias),
                            _ptr(logits), _ptr(probs), _ptr(prob_sum), _ptr(topk_ids),
                            _ptr(topk_w), _ptr(ws), ws_bytes, _stream(stream)), "moe_route")


def moe_dispatch(p, topk_ids, x, counts, kept, offsets, assign_row, row_assign, x_perm, ws,
                 stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib().moe_dispatch(ctypes.byref(p), _ptr(topk_ids), _ptr(x), _ptr(counts), _ptr(kept),
                               _ptr(offsets), _ptr(assign_row), _ptr(row_assign), _ptr(x_perm),
                               _ptr(ws), ws_bytes, _stream(stream)), "moe_dispatch")


def moe_expert_ffn(p, x_perm, offsets, w1, w3, w2, act, h, ws, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib().moe_expert_ffn(ctypes.byref(p), _ptr(x_perm), _ptr(offsets), _ptr(w1), _ptr(w3),
                                 _ptr(w2), _ptr(act), _ptr(h), _ptr(ws), ws_bytes,
                                 _stream(stream)), "moe_expert_ffn")


def moe_combine(p, h, assign_row, topk_w, y, stream=None):
    _check(_lib().moe_combine(ctypes.byref(p), _ptr(h), _ptr(assign_row), _ptr(topk_w), _ptr(y),
                              _stream(stream)), "moe_combine")


def moe_forward(p, x, w_router, w1, w3, w2, logit_bias, y, ws, dbg: dict | None = None,
                stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    d = None
    if dbg:
        d = MoEDebugOut(**{k: _ptr(v) for k, v in dbg.items()})
    _check(_lib().moe_forward(ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(w1), _ptr(w3),
                              _ptr(w2), _ptr(logit_bias), _ptr(y),
                              ctypes.byref(d) if d is not None else None, _ptr(ws), ws_bytes,
                              _stream(stream)), "moe_forward")


MOE_NOALLOC_WS_BYTES = 32 << 20


def moe_forward_noalloc(p, x, w_router, w1, w3, w2, logit_bias, y, dbg: dict | None = None, stream=None):
    """The layer on the library's static per-GPU workspace (no allocation)."""
    d = None
    if dbg:
        d = MoEDebugOut(**{k: _ptr(v) for k, v in dbg.items()})
    _check(_lib().moe_forward_noalloc(ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(w1), _ptr(w3),
                                      _ptr(w2), _ptr(logit_bias), _ptr(y),
                                      ctypes.byref(d) if d is not None else None, _stream(stream)),
           "moe_forward_noalloc")


def moe_forward_chunked_workspace_size(p: MoEProblem, chunk_tokens: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib().moe_forward_chunked_workspace_size(ctypes.byref(p), chunk_tokens, ctypes.byref(out)),
           "moe_forward_chunked_workspace_size")
    return out.value


def moe_forward_chunked(p, chunk_tokens: int, x, w_router, w1, w3, w2, logit_bias, y, ws,
                        dbg: dict | None = None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    d = None
    if dbg:
        d = MoEDebugOut(**{k: _ptr(v) for k, v in dbg.items()})
    _check(_lib().moe_forward_chunked(ctypes.byref(p), chunk_tokens, _ptr(x), _ptr(w_router), _ptr(w1),
                                      _ptr(w3), _ptr(w2), _ptr(logit_bias), _ptr(y),
                                      ctypes.byref(d) if d is not None else None, _ptr(ws), ws_bytes,
                                      _stream(stream)), "moe_forward_chunked")


def moe_aux_loss(p, counts, prob_sum, aux, stream=None):
    _check(_lib().moe_aux_loss(ctypes.byref(p), _ptr(counts), _ptr(prob_sum), _ptr(aux),
                               _stream(stream)), "moe_aux_loss")


def moe_combine_concat_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_combine_concat_workspace_size, p)


def moe_combine_concat(p, h, assign_row, w_cat, y, ws, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib().moe_combine_concat(ctypes.byref(p), _ptr(h), _ptr(assign_row), _ptr(w_cat), _ptr(y),
                                     _ptr(ws), ws_bytes, _stream(stream)), "moe_combine_concat")


def moe_router_losses(p, logits, logit_bias, topk_ids, counts, z_loss, aux_topk, ws, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib().moe_router_losses(ctypes.byref(p), _ptr(logits), _ptr(logit_bias), _ptr(topk_ids),
                                    _ptr(counts), _ptr(z_loss), _ptr(aux_topk), _ptr(ws), ws_bytes,
                                    _stream(stream)), "moe_router_losses")


def moe_bias_update(p, counts, alpha: float, bias, stream=None):
    _check(_lib().moe_bias_update(ctypes.byref(p), _ptr(counts), ctypes.c_float(alpha), _ptr(bias),
                                  _stream(stream)), "moe_bias_update")


# ---- training and 8-bit experts ----------------------------------------------
# These bindings check their tensors before the call: contiguous, on the
# current GPU, of the expected type, and large enough for the problem.

def _tensors(where: str, **args):
    """args: name -> (tensor, torch dtype or None for the workspace, elements).
    None and raw device pointers pass unchecked."""
    import torch
    dev = torch.cuda.current_device()
    for name, (t, dtype, numel) in args.items():
        if t is None or isinstance(t, int):
            continue
        if t.get_device() != dev:  # -1 for host tensors
            raise ValueError(f"{where}: {name} is on {t.device}, the current device is cuda:{dev}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} is not contiguous")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{where}: {name} is {t.dtype}, expected {dtype}")
        if t.numel() < numel:
            raise ValueError(f"{where}: {name} has {t.numel()} elements, {numel} are needed")


def _dtype(p: MoEProblem):
    import torch
    return torch.bfloat16 if p.dtype == MOE_DTYPE_BF16 else torch.float32


def _ws_bytes(ws) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def moe_expert_ffn_train_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_expert_ffn_train_workspace_size, p)


def moe_expert_ffn_train(p, x_perm, offsets, w1, w3, w2, gate, up, h, ws, stream=None):
    """moe_expert_ffn that keeps the gate and up projections for moe_expert_ffn_backward."""
    import torch
    n, wd, dt = p.T * p.top_k, p.n_experts * p.d_ff * p.d_model, _dtype(p)
    _tensors("moe_expert_ffn_train", x_perm=(x_perm, dt, n * p.d_model), offsets=(offsets, torch.int32, p.n_experts + 1),
             w1=(w1, dt, wd), w3=(w3, dt, wd), w2=(w2, dt, wd), gate=(gate, dt, n * p.d_ff),
             up=(up, dt, n * p.d_ff), h=(h, dt, n * p.d_model), ws=(ws, None, 0))
    _check(_lib().moe_expert_ffn_train(ctypes.byref(p), _ptr(x_perm), _ptr(offsets), _ptr(w1), _ptr(w3), _ptr(w2),
                                       _ptr(gate), _ptr(up), _ptr(h), _ptr(ws), _ws_bytes(ws), _stream(stream)),
           "moe_expert_ffn_train")


def moe_expert_ffn_backward_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_expert_ffn_backward_workspace_size, p)


def moe_expert_ffn_backward(p, x_perm, offsets, w1, w3, w2, gate, up, dh, dx_perm, dw1, dw3, dw2, ws, stream=None):
    """Gradients of the expert FFN; dx_perm, or dw1, dw3 and dw2 together, may be None."""
    import torch
    n, wd, dt = p.T * p.top_k, p.n_experts * p.d_ff * p.d_model, _dtype(p)
    nd, nf = n * p.d_model, n * p.d_ff
    _tensors("moe_expert_ffn_backward", x_perm=(x_perm, dt, nd), offsets=(offsets, torch.int32, p.n_experts + 1),
             w1=(w1, dt, wd), w3=(w3, dt, wd), w2=(w2, dt, wd), gate=(gate, dt, nf), up=(up, dt, nf),
             dh=(dh, dt, nd), dx_perm=(dx_perm, dt, nd), dw1=(dw1, dt, wd), dw3=(dw3, dt, wd), dw2=(dw2, dt, wd),
             ws=(ws, None, 0))
    _check(_lib().moe_expert_ffn_backward(ctypes.byref(p), _ptr(x_perm), _ptr(offsets), _ptr(w1), _ptr(w3), _ptr(w2),
                                          _ptr(gate), _ptr(up), _ptr(dh), _ptr(dx_perm), _ptr(dw1), _ptr(dw3),
                                          _ptr(dw2), _ptr(ws), _ws_bytes(ws), _stream(stream)),
           "moe_expert_ffn_backward")


def moe_combine_backward(p, dy, h, assign_row, topk_w, dh, dtopk_w, stream=None):
    """Gradients of the weighted combine; h and dtopk_w may be None together."""
    import torch
    n, dt = p.T * p.top_k, _dtype(p)
    _tensors("moe_combine_backward", dy=(dy, dt, p.T * p.d_model), h=(h, dt, n * p.d_model),
             assign_row=(assign_row, torch.int32, n), topk_w=(topk_w, torch.float32, n),
             dh=(dh, dt, n * p.d_model), dtopk_w=(dtopk_w, torch.float32, n))
    _check(_lib().moe_combine_backward(ctypes.byref(p), _ptr(dy), _ptr(h), _ptr(assign_row), _ptr(topk_w), _ptr(dh),
                                       _ptr(dtopk_w), _stream(stream)), "moe_combine_backward")


def moe_route_backward_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_route_backward_workspace_size, p)


def moe_route_backward(p, x, w_router, logit_bias, logits, topk_ids, topk_w, dtopk_w, counts, d_aux: float,
                       d_z: float, dx_perm, assign_row, dlogits, dx, dw_router, ws=None, stream=None):
    """Gradients of routing (scores, layer input, router weight) and of the dispatch's gather."""
    import torch
    n, dt = p.T * p.top_k, _dtype(p)
    f32, i32 = torch.float32, torch.int32
    _tensors("moe_route_backward", x=(x, dt, p.T * p.d_model), w_router=(w_router, dt, p.d_model * p.n_experts),
             logit_bias=(logit_bias, f32, p.n_experts), logits=(logits, f32, p.T * p.n_experts),
             topk_ids=(topk_ids, i32, n), topk_w=(topk_w, f32, n), dtopk_w=(dtopk_w, f32, n),
             counts=(counts, i32, p.n_experts), dx_perm=(dx_perm, dt, n * p.d_model), assign_row=(assign_row, i32, n),
             dlogits=(dlogits, f32, p.T * p.n_experts), dx=(dx, dt, p.T * p.d_model),
             dw_router=(dw_router, dt, p.d_model * p.n_experts), ws=(ws, None, 0))
    _check(_lib().moe_route_backward(ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(logits),
                                     _ptr(topk_ids), _ptr(topk_w), _ptr(dtopk_w), _ptr(counts),
                                     ctypes.c_float(d_aux), ctypes.c_float(d_z), _ptr(dx_perm), _ptr(assign_row),
                                     _ptr(dlogits), _ptr(dx), _ptr(dw_router), _ptr(ws), _ws_bytes(ws),
                                     _stream(stream)), "moe_route_backward")


def moe_quantize_rows(x, q, scale, stream=None):
    """Per row of x [..., cols] (f32 or bf16): q int8 of x's shape, scale f32 of its leading shape."""
    import torch
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"moe_quantize_rows: x is {x.dtype}, expected float32 or bfloat16")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    _tensors("moe_quantize_rows", x=(x, None, 0), q=(q, torch.int8, x.numel()), scale=(scale, torch.float32, rows))
    code = MOE_DTYPE_BF16 if x.dtype == torch.bfloat16 else MOE_DTYPE_F32
    _check(_lib().moe_quantize_rows(rows, cols, code, _ptr(x), _ptr(q), _ptr(scale), _stream(stream)),
           "moe_quantize_rows")


def i8_weights(w1, s1, w3, s3, w2, s2) -> MoEI8Weights:
    """8-bit expert weights and their scales (moe_quantize_rows of the [E, F, d], [E, F, d] and
    [E, d, F] weights).  The structure keeps the tensors alive."""
    import torch
    _tensors("i8_weights", w1=(w1, torch.int8, 0), w3=(w3, torch.int8, 0), w2=(w2, torch.int8, 0),
             s1=(s1, torch.float32, 0), s3=(s3, torch.float32, 0), s2=(s2, torch.float32, 0))
    w = MoEI8Weights(_ptr(w1), _ptr(w3), _ptr(w2), _ptr(s1), _ptr(s3), _ptr(s2))
    w.tensors = {"w1": w1, "s1": s1, "w3": w3, "s3": s3, "w2": w2, "s2": s2}
    return w


def _i8_sizes(where: str, p: MoEProblem, w: MoEI8Weights):
    import torch
    e, wd = p.n_experts, p.n_experts * p.d_ff * p.d_model
    need = {"w1": wd, "w3": wd, "w2": wd, "s1": e * p.d_ff, "s3": e * p.d_ff, "s2": e * p.d_model}
    _tensors(where, **{k: (t, None, need[k]) for k, t in getattr(w, "tensors", {}).items()})


def moe_expert_ffn_i8_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_expert_ffn_i8_workspace_size, p)


def moe_expert_ffn_i8(p, x_perm, offsets, weights: MoEI8Weights, act, h, ws, stream=None):
    """moe_expert_ffn on 8-bit weights."""
    import torch
    n, dt = p.T * p.top_k, torch.bfloat16
    _tensors("moe_expert_ffn_i8", x_perm=(x_perm, dt, n * p.d_model), offsets=(offsets, torch.int32, p.n_experts + 1),
             act=(act, dt, n * p.d_ff), h=(h, dt, n * p.d_model), ws=(ws, None, 0))
    _i8_sizes("moe_expert_ffn_i8", p, weights)
    _check(_lib().moe_expert_ffn_i8(ctypes.byref(p), _ptr(x_perm), _ptr(offsets), ctypes.byref(weights), _ptr(act),
                                    _ptr(h), _ptr(ws), _ws_bytes(ws), _stream(stream)), "moe_expert_ffn_i8")


def moe_forward_i8_workspace_size(p: MoEProblem) -> int:
    return _size(_lib().moe_forward_i8_workspace_size, p)


def moe_forward_i8(p, x, w_router, weights: MoEI8Weights, logit_bias, y, ws, dbg: dict | None = None, stream=None):
    """moe_forward on 8-bit expert weights."""
    import torch
    dt = torch.bfloat16
    _tensors("moe_forward_i8", x=(x, dt, p.T * p.d_model), w_router=(w_router, dt, p.d_model * p.n_experts),
             logit_bias=(logit_bias, torch.float32, p.n_experts), y=(y, dt, p.T * p.d_model), ws=(ws, None, 0))
    _i8_sizes("moe_forward_i8", p, weights)
    d = MoEDebugOut(**{k: _ptr(v) for k, v in dbg.items()}) if dbg else None
    _check(_lib().moe_forward_i8(ctypes.byref(p), _ptr(x), _ptr(w_router), ctypes.byref(weights), _ptr(logit_bias),
                                 _ptr(y), ctypes.byref(d) if d is not None else None, _ptr(ws), _ws_bytes(ws),
                                 _stream(stream)), "moe_forward_i8")


def moe_set_kernel_timer(kernel: str | int, start_events, stop_events):
    """Bracket the next len(start_events) launches of `kernel` with the given
    torch.cuda.Event pairs (recorded on the kernel's own stream)."""
    kid = KERNEL_IDS[kernel] if isinstance(kernel, str) else kernel
    n = len(start_events)
    if n == 0:
        _check(_lib().moe_set_kernel_timer(kid, None, None, 0, None), "moe_set_kernel_timer")
        return None
    arr_t = ctypes.c_void_p * n
    starts = arr_t(*[e.cuda_event for e in start_events])
    stops = arr_t(*[e.cuda_event for e in stop_events])
    _check(_lib().moe_set_kernel_timer(kid, starts, stops, n, None), "moe_set_kernel_timer")
    return (starts, stops)  # caller keeps these alive while the hook is set


def moe_kernel_timer_count(kernel: str | int) -> int:
    kid = KERNEL_IDS[kernel] if isinstance(kernel, str) else kernel
    out = ctypes.c_int(0)
    _check(_lib().moe_set_kernel_timer(kid, None, None, -1, ctypes.byref(out)), "moe_set_kernel_timer")
    return out.value


__all__ = [
    "CONFIGS", "MoEConfig", "MoEError", "MoEProblem", "MoEDebugOut", "load", "problem", "problem_of",
    "moe_workspace_size", "moe_route_workspace_size", "moe_dispatch_workspace_size",
    "moe_expert_ffn_workspace_size", "moe_route", "moe_dispatch", "moe_expert_ffn", "moe_combine",
    "moe_forward", "moe_forward_chunked", "moe_forward_chunked_workspace_size", "moe_aux_loss", "moe_bias_update", "moe_router_losses",
    "moe_combine_concat", "moe_combine_concat_workspace_size",
    "moe_router_losses_workspace_size", "moe_set_kernel_timer",
    "moe_kernel_timer_count",
    "moe_expert_ffn_train", "moe_expert_ffn_train_workspace_size", "moe_expert_ffn_backward",
    "moe_expert_ffn_backward_workspace_size", "moe_combine_backward", "moe_route_backward",
    "moe_route_backward_workspace_size", "moe_quantize_rows", "MoEI8Weights", "i8_weights",
    "moe_expert_ffn_i8", "moe_expert_ffn_i8_workspace_size", "moe_forward_i8",
    "moe_forward_i8_workspace_size",
]
