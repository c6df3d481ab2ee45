"""Python binding of the C ABI in include/moe.h and moe_rows.h (argument marshalling only).

Every step of the layer runs in the CUDA kernels of libmoe_b200.so; this
module only turns torch tensors into device pointers and checks status
codes (through ctypes; the row and 8-bit integer calls through the compiled
module _rows_binding).  There is no fallback: if the library is missing, importing the
functions raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_SHAPE = 2
MOE_ERR_WORKSPACE_TOO_SMALL = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_TIMEOUT = 5
MOE_ERR_DEVICE_BOUNDS = 6

MOE_FLAG_ROUTER_CUDA_CORE = 1
MOE_FLAG_ROUTER_TENSOR = 2
MOE_FLAG_DOWN_F16 = 4
MOE_FLAG_GEMM_SINGLE_CTA = 8
MOE_FLAG_GEMM_PAIR = 16
MOE_FLAG_BIAS_SELECTION_ONLY = 32
MOE_FLAG_FP8_EXPERTS = 64
MOE_FLAG_COMBINE_REDUCE = 128
MOE_FLAG_FUSED_EXPERTS = 256

# Every symbol the header declares (checked by the CPU tests).
EXPORTED = ["moe_workspace_size", "moe_workspace_size_upto", "moe_route_workspace_size",
            "moe_route", "moe_permute", "moe_forward",
            "moe_read_device_status", "moe_selftest_bounded_wait", "moe_status_string",
            "moe_last_launch_count", "moe_profile_next_forward", "moe_prepare_down_f16",
            "moe_logits_offset", "moe_permute_static", "moe_route_masked",
            "moe_forward_masked", "moe_prepare_fp8", "moe_forward_fp8"]
# Those of include/moe_rows.h.
ROWS_EXPORTED = ["moe_sort_workspace_size", "moe_sort", "moe_dispatch",
                 "moe_dispatch_backward", "moe_combine", "moe_combine_backward",
                 "moe_route_backward", "moe_quantize_int8", "moe_dispatch_int8",
                 "moe_matmul_int8"]

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F16 = 1
MOE_DTYPE_F32 = 2

MOE_INT8_SWIGLU = 1

# Flags that choose what MoeLayer(int8=True) does not have.
INT8_REFUSED_FLAGS = (MOE_FLAG_GEMM_SINGLE_CTA | MOE_FLAG_GEMM_PAIR | MOE_FLAG_FP8_EXPERTS |
                      MOE_FLAG_COMBINE_REDUCE | MOE_FLAG_FUSED_EXPERTS)

# Expert id of a (token, slot) pair that is not routed (a padding token).
MOE_NOT_ROUTED = -1


class MoeError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class moe_dims_t(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("T", ctypes.c_int32),
                ("d_model", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("num_experts_per_tok", ctypes.c_int32), ("moe_intermediate_size", ctypes.c_int32),
                ("shared_intermediate_size", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float), ("norm_topk_prob", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class moe_weights_t(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("ws_gate", ctypes.c_void_p),
                ("ws_up", ctypes.c_void_p), ("ws_down", ctypes.c_void_p),
                ("w_down_f16", ctypes.c_void_p), ("ws_down_f16", ctypes.c_void_p)]


class moe_fp8_weights_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
                 "ws_gate", "ws_up", "ws_down", "ss_gate", "ss_up", "ss_down")]


class moe_routing_t(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("perm", ctypes.c_void_p)]


class moe_int8_matmul_t(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("M", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("G", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("a", ctypes.c_void_p), ("a_stride", ctypes.c_int64),
                ("a_scale", ctypes.c_void_p), ("b", ctypes.c_void_p), ("b_stride", ctypes.c_int64),
                ("b_scale", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64)]


_LIB = None


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} "
                               "(run python -m sparse_moe_layer_select_b200.build)")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        D = ctypes.POINTER(moe_dims_t)
        L.moe_workspace_size.restype = ctypes.c_size_t
        L.moe_workspace_size.argtypes = [D]
        L.moe_workspace_size_upto.restype = ctypes.c_size_t
        L.moe_workspace_size_upto.argtypes = [D]
        L.moe_route_workspace_size.restype = ctypes.c_size_t
        L.moe_route_workspace_size.argtypes = [D]
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [D, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_permute.restype = ctypes.c_int
        L.moe_permute.argtypes = [D, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_forward.restype = ctypes.c_int
        L.moe_forward.argtypes = [D, ctypes.POINTER(moe_weights_t), P, P,
                                  ctypes.POINTER(moe_routing_t), P, ctypes.c_size_t, P]
        L.moe_prepare_fp8.restype = ctypes.c_int
        L.moe_prepare_fp8.argtypes = [D, ctypes.POINTER(moe_weights_t),
                                      ctypes.POINTER(moe_fp8_weights_t), P, ctypes.c_size_t, P]
        L.moe_forward_fp8.restype = ctypes.c_int
        L.moe_forward_fp8.argtypes = [D, ctypes.POINTER(moe_weights_t),
                                      ctypes.POINTER(moe_fp8_weights_t), P, P,
                                      ctypes.POINTER(moe_routing_t), P, ctypes.c_size_t, P]
        L.moe_route_masked.restype = ctypes.c_int
        L.moe_route_masked.argtypes = [D, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_forward_masked.restype = ctypes.c_int
        L.moe_forward_masked.argtypes = [D, ctypes.POINTER(moe_weights_t), P, P, P,
                                         ctypes.POINTER(moe_routing_t), P, ctypes.c_size_t, P]
        L.moe_read_device_status.restype = ctypes.c_int
        L.moe_read_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
        L.moe_selftest_bounded_wait.restype = ctypes.c_int
        L.moe_selftest_bounded_wait.argtypes = [P, ctypes.c_size_t, ctypes.c_uint32, P]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_last_launch_count.restype = ctypes.c_int32
        L.moe_last_launch_count.argtypes = []
        L.moe_prepare_down_f16.restype = ctypes.c_int
        L.moe_prepare_down_f16.argtypes = [D, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_permute_static.restype = ctypes.c_int
        L.moe_permute_static.argtypes = [D, P, P, P, P, P]
        L.moe_logits_offset.restype = ctypes.c_size_t
        L.moe_logits_offset.argtypes = [D]
        L.moe_profile_next_forward.restype = ctypes.c_int
        L.moe_profile_next_forward.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32]
        L.moe_sort_workspace_size.restype = ctypes.c_size_t
        L.moe_sort_workspace_size.argtypes = [D]
        _LIB = L
    return _LIB


def status_string(code: int) -> str:
    return lib().moe_status_string(code).decode()


def make_dims(T, d_model, num_experts, num_experts_per_tok, moe_intermediate_size,
              shared_intermediate_size, routed_scaling_factor=2.5, norm_topk_prob=1, flags=0):
    return moe_dims_t(ctypes.sizeof(moe_dims_t), T, d_model, num_experts, num_experts_per_tok,
                      moe_intermediate_size, shared_intermediate_size, routed_scaling_factor,
                      norm_topk_prob, flags)


def dims_for(w, T=None, flags=0, norm_topk_prob=1):
    """moe_dims_t of an inputs.Workload (optionally with another token count)."""
    return make_dims(w.T if T is None else T, w.d_model, w.E, w.k, w.F, w.Fs,
                     w.routed_scaling_factor, norm_topk_prob, flags)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, where):
    if code != MOE_OK:
        raise MoeError(code, where)


def workspace_size(dims) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(dims)))


def workspace_size_upto(dims) -> int:
    """The same for every batch of up to dims.T tokens (a smaller batch can need more)."""
    return int(lib().moe_workspace_size_upto(ctypes.byref(dims)))


def route_workspace_size(dims) -> int:
    """What the router alone needs, for every batch of up to dims.T tokens."""
    return int(lib().moe_route_workspace_size(ctypes.byref(dims)))


def _workspace(n, name, device):
    import torch
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, name)
    return torch.empty(n, dtype=torch.uint8, device=device)


def alloc_workspace(dims, device="cuda", upto=False):
    """A workspace for these dims, or (upto) for every batch of up to dims.T tokens."""
    if upto:
        return _workspace(workspace_size_upto(dims), "moe_workspace_size_upto", device)
    return _workspace(workspace_size(dims), "moe_workspace_size", device)


def alloc_route_workspace(dims, device="cuda"):
    """A workspace for moe_route alone, for every batch of up to dims.T tokens."""
    return _workspace(route_workspace_size(dims), "moe_route_workspace_size", device)


def route(dims, x, w_router, bias, topk_idx, topk_w, ws, stream=None, token_mask=None):
    """moe_route, or moe_route_masked when a [T] uint8 token_mask (0 = padding) is given."""
    if token_mask is None:
        _check(lib().moe_route(ctypes.byref(dims), _p(x), _p(w_router), _p(bias), _p(topk_idx),
                               _p(topk_w), _p(ws), ws.numel(), _stream(stream)), "moe_route")
    else:
        _check(lib().moe_route_masked(ctypes.byref(dims), _p(x), _p(w_router), _p(bias),
                                      _p(token_mask), _p(topk_idx), _p(topk_w), _p(ws),
                                      ws.numel(), _stream(stream)), "moe_route_masked")


def permute(dims, topk_idx, counts, offsets, perm, ws, x=None, x_perm=None, stream=None):
    _check(lib().moe_permute(ctypes.byref(dims), _p(topk_idx), _p(counts), _p(offsets), _p(perm),
                             _p(x), _p(x_perm), _p(ws), ws.numel(), _stream(stream)),
           "moe_permute")


def weights_struct(W):
    return moe_weights_t(*[None if W.get(k) is None else W[k].data_ptr() for k in
                           ("w_router", "router_bias", "w_gate", "w_up", "w_down", "ws_gate",
                            "ws_up", "ws_down", "w_down_f16", "ws_down_f16")])


def prepare_down_f16(dims, W, stream=None):
    """fp16 copies of the down projections (moe_prepare_down_f16); adds them to W and
    returns the device status of the conversion."""
    import torch
    W["w_down_f16"] = torch.empty(W["w_down"].shape, dtype=torch.float16, device=W["w_down"].device)
    if W.get("ws_down") is not None:
        W["ws_down_f16"] = torch.empty(W["ws_down"].shape, dtype=torch.float16,
                                       device=W["ws_down"].device)
    hdr = torch.zeros(256, dtype=torch.uint8, device=W["w_down"].device)
    _check(lib().moe_prepare_down_f16(ctypes.byref(dims), _p(W["w_down"]), _p(W.get("ws_down")),
                                      _p(W["w_down_f16"]), _p(W.get("ws_down_f16")), _p(hdr), 256,
                                      _stream(stream)), "moe_prepare_down_f16")
    return read_device_status(hdr, stream)


FP8_FIELDS = ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
              "ws_gate", "ws_up", "ws_down", "ss_gate", "ss_up", "ss_down")


def prepare_fp8(dims, W, stream=None):
    """FP8 copies of the expert weights (moe_prepare_fp8): returns a dict of device tensors
    (e4m3 codes as uint8, float32 row scales) and the device status."""
    import torch
    dev = W["w_gate"].device
    E, F, d = W["w_gate"].shape
    Q = {"w_gate": torch.empty((E, F, d), dtype=torch.uint8, device=dev),
         "w_up": torch.empty((E, F, d), dtype=torch.uint8, device=dev),
         "w_down": torch.empty((E, d, F), dtype=torch.uint8, device=dev),
         "s_gate": torch.empty(E * F, dtype=torch.float32, device=dev),
         "s_up": torch.empty(E * F, dtype=torch.float32, device=dev),
         "s_down": torch.empty(E * d, dtype=torch.float32, device=dev)}
    if W.get("ws_gate") is not None:
        Fs = W["ws_gate"].shape[0]
        Q.update(ws_gate=torch.empty((Fs, d), dtype=torch.uint8, device=dev),
                 ws_up=torch.empty((Fs, d), dtype=torch.uint8, device=dev),
                 ws_down=torch.empty((d, Fs), dtype=torch.uint8, device=dev),
                 ss_gate=torch.empty(Fs, dtype=torch.float32, device=dev),
                 ss_up=torch.empty(Fs, dtype=torch.float32, device=dev),
                 ss_down=torch.empty(d, dtype=torch.float32, device=dev))
    hdr = torch.zeros(256, dtype=torch.uint8, device=dev)
    _check(lib().moe_prepare_fp8(ctypes.byref(dims), ctypes.byref(weights_struct(W)),
                                 ctypes.byref(fp8_struct(Q)), _p(hdr), 256, _stream(stream)),
           "moe_prepare_fp8")
    return Q, read_device_status(hdr, stream)


def fp8_struct(Q):
    return moe_fp8_weights_t(*[None if Q.get(k) is None else Q[k].data_ptr() for k in FP8_FIELDS])


def forward_fp8(dims, weights, fp8, x, y, routing, ws, stream=None):
    """moe_forward_fp8 (dims.flags must include MOE_FLAG_FP8_EXPERTS)."""
    ws_s = weights if isinstance(weights, moe_weights_t) else weights_struct(weights)
    q_s = fp8 if isinstance(fp8, moe_fp8_weights_t) else fp8_struct(fp8)
    r_s = routing if isinstance(routing, moe_routing_t) else routing_struct(routing)
    _check(lib().moe_forward_fp8(ctypes.byref(dims), ctypes.byref(ws_s), ctypes.byref(q_s), _p(x),
                                 _p(y), ctypes.byref(r_s), _p(ws), ws.numel(), _stream(stream)),
           "moe_forward_fp8")


def logits_offset(dims) -> int:
    return int(lib().moe_logits_offset(ctypes.byref(dims)))


def routing_struct(R):
    return moe_routing_t(*[R[k].data_ptr() for k in ("topk_idx", "topk_w", "counts", "offsets",
                                                     "perm")])


def forward(dims, weights, x, y, routing, ws, stream=None, token_mask=None):
    """moe_forward on torch tensors; weights/routing are dicts of tensors (or prebuilt structs).
    With a [T] uint8 token_mask (0 = padding token) it calls moe_forward_masked."""
    ws_s = weights if isinstance(weights, moe_weights_t) else weights_struct(weights)
    r_s = routing if isinstance(routing, moe_routing_t) else routing_struct(routing)
    if token_mask is None:
        _check(lib().moe_forward(ctypes.byref(dims), ctypes.byref(ws_s), _p(x), _p(y),
                                 ctypes.byref(r_s), _p(ws), ws.numel(), _stream(stream)),
               "moe_forward")
    else:
        _check(lib().moe_forward_masked(ctypes.byref(dims), ctypes.byref(ws_s), _p(x),
                                        _p(token_mask), _p(y), ctypes.byref(r_s), _p(ws),
                                        ws.numel(), _stream(stream)), "moe_forward_masked")


def alloc_routing(dims, device="cuda"):
    import torch
    T, k, E = dims.T, dims.num_experts_per_tok, dims.num_experts
    return {"topk_idx": torch.empty((T, k), dtype=torch.int32, device=device),
            "topk_w": torch.empty((T, k), dtype=torch.float32, device=device),
            "counts": torch.empty(E, dtype=torch.int32, device=device),
            "offsets": torch.empty(E + 1, dtype=torch.int32, device=device),
            "perm": torch.empty(T * k, dtype=torch.int32, device=device)}


def read_device_status(ws, stream=None):
    site = ctypes.c_int32(0)
    code = lib().moe_read_device_status(_p(ws), _stream(stream), ctypes.byref(site))
    return int(code), int(site.value)


def selftest_bounded_wait(ws, limit_us, stream=None):
    _check(lib().moe_selftest_bounded_wait(_p(ws), ws.numel(), limit_us, _stream(stream)),
           "moe_selftest_bounded_wait")


def profile_next_forward(events):
    """Arm per-kernel event recording for the next forward call (torch.cuda.Event list)."""
    if events is None:
        _check(lib().moe_profile_next_forward(None, 0), "moe_profile_next_forward")
        return
    import torch
    for e in events:  # torch creates the CUDA event handle on first record
        if e.cuda_event == 0:
            e.record(torch.cuda.current_stream())
    if any(e.cuda_event == 0 for e in events):
        raise RuntimeError("profile_next_forward: CUDA events were not created")
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    profile_next_forward._keep = arr
    _check(lib().moe_profile_next_forward(arr, len(events)), "moe_profile_next_forward")


# Stage names of the kernel-marker intervals recorded by moe_forward, in order.
FORWARD_STAGES = ("router", "index", "gemm1_swiglu", "gemm2_down_scale", "combine")


def last_launch_count() -> int:
    return int(lib().moe_last_launch_count())


# ---------------------------------------------------------------- rows and 8-bit products
# Types, sizes and strides are taken from the tensors (and checked) by the compiled module
# _rows_binding: at decode sizes these calls take less time on the device than that takes in
# Python.  An argument that does not fit raises MoeError(MOE_ERR_INVALID_ARG) before anything is
# launched; every tensor has to be on the current device.

_ROWS = None


def _rows():
    """The compiled binding (raises if it has not been built)."""
    global _ROWS
    if _ROWS is None:
        lib()
        try:
            from . import _rows_binding
        except ImportError as e:
            raise RuntimeError("binding not built (run python -m "
                               f"sparse_moe_layer_select_b200.build): {e}") from e
        _ROWS = _rows_binding
    return _ROWS


def _raise(code, where):
    if isinstance(code, str):  # an argument that does not fit
        raise MoeError(MOE_ERR_INVALID_ARG, f"{where} ({code})")
    raise MoeError(code, where)


def sort_workspace_size(dims) -> int:
    return int(lib().moe_sort_workspace_size(ctypes.byref(dims)))


def alloc_sort_workspace(dims, device="cuda"):
    """Workspace of moe_sort (and a cleared status header for the calls that follow it)."""
    import torch
    n = sort_workspace_size(dims)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_sort_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_sort(dims, device="cuda"):
    """Outputs of moe_sort: counts [E], offsets [E + 1], perm [T * k], inv [T, k]."""
    import torch
    T, k, E = dims.T, dims.num_experts_per_tok, dims.num_experts
    new = lambda *s: torch.empty(s, dtype=torch.int32, device=device)  # noqa: E731
    return {"counts": new(E), "offsets": new(E + 1), "perm": new(T * k), "inv": new(T, k)}


def sort(dims, topk_idx, out, ws, x=None, x_perm=None, stream=None):
    """moe_sort into the buffers of alloc_sort; with x [T, d] and x_perm [T * k, d], the rows
    are copied to expert order too."""
    code = (_ROWS or _rows()).sort(dims, topk_idx, out["counts"], out["offsets"], out["perm"],
                                   out["inv"], ws, x, x_perm, stream)
    if code != MOE_OK:
        _raise(code, "moe_sort")


def dispatch(dims, x, inv, x_perm, ws=None, stream=None):
    """moe_dispatch: x_perm[inv[t, j]] = x[t]."""
    code = (_ROWS or _rows()).dispatch(dims, x, inv, x_perm, ws, stream)
    if code != MOE_OK:
        _raise(code, "moe_dispatch")


def dispatch_backward(dims, d_x_perm, inv, d_x, ws=None, add=None, stream=None):
    """moe_dispatch_backward: d_x[t] = sum_j d_x_perm[inv[t, j]] (+ add[t])."""
    code = (_ROWS or _rows()).dispatch_backward(dims, d_x_perm, inv, d_x, ws, add, stream)
    if code != MOE_OK:
        _raise(code, "moe_dispatch_backward")


def combine(dims, o, inv, topk_w, y, ws=None, shared=None, stream=None):
    """moe_combine: y[t] = routed_scaling_factor sum_j topk_w[t, j] o[inv[t, j]] (+ shared[t])."""
    code = (_ROWS or _rows()).combine(dims, o, inv, topk_w, y, ws, shared, stream)
    if code != MOE_OK:
        _raise(code, "moe_combine")


def combine_backward(dims, d_y, o, inv, topk_w, d_o, d_topk_w, ws=None, stream=None):
    """moe_combine_backward: the gradients of combine's o (d_o may be o) and topk_w."""
    code = (_ROWS or _rows()).combine_backward(dims, d_y, o, inv, topk_w, d_o, d_topk_w, ws, stream)
    if code != MOE_OK:
        _raise(code, "moe_combine_backward")


def route_backward(dims, logits, topk_idx, d_topk_w, d_logits, ws=None, stream=None):
    """moe_route_backward: the gradient of the router's logits [T, E] from that of its weights."""
    code = (_ROWS or _rows()).route_backward(dims, logits, topk_idx, d_topk_w, d_logits, ws, stream)
    if code != MOE_OK:
        _raise(code, "moe_route_backward")


def alloc_codes(rows, cols, device="cuda"):
    """Codes [rows, cols] and scales [rows]; rows start a multiple of 16 bytes apart."""
    import torch
    pitch = (cols + 15) // 16 * 16
    return (torch.empty((rows, pitch), dtype=torch.int8, device=device)[:, :cols],
            torch.empty(rows, dtype=torch.float32, device=device))


def quantize_int8(x, codes, scales, n_rows=None, stream=None):
    """moe_quantize_int8: int8 codes and fp32 scales of the rows of x (of its first n_rows[0],
    a device int32, if given)."""
    code = (_ROWS or _rows()).quantize_int8(x, codes, scales, n_rows, stream)
    if code != MOE_OK:
        _raise(code, "moe_quantize_int8")


def dispatch_int8(dims, x, inv, codes, scales, ws=None, stream=None):
    """moe_dispatch_int8: each token's row quantized and stored to its slots' expert-order rows."""
    code = (_ROWS or _rows()).dispatch_int8(dims, x, inv, codes, scales, ws, stream)
    if code != MOE_OK:
        _raise(code, "moe_dispatch_int8")


def matmul_int8(a, a_scale, b, b_scale, out, ws, offsets=None, swiglu=False, stream=None):
    """moe_matmul_int8: out[r, c] = (a[r] . b[g, c]) a_scale[r] b_scale[g, c].

    a [M, K] and b [N, K] (or [G, N, K] with offsets [G + 1], the first row of each group) are
    int8; swiglu: b has 2 N rows per group (gate, then up) and out = silu(gate) * up."""
    code = (_ROWS or _rows()).matmul_int8(a, a_scale, b, b_scale, out, ws, offsets, swiglu, stream)
    if code != MOE_OK:
        _raise(code, "moe_matmul_int8")


def prepare_int8(W, stream=None):
    """int8 copies of the expert weights (a model-load step): gate and up rows of each expert in
    one matrix, as moe_matmul_int8's SwiGLU form takes them.  Returns a dict of codes and scales:
    gate_up [E, 2F, d], down [E, d, F] and, with a shared expert, s_gate_up [2Fs, d] and
    s_down [d, Fs]; "<name>_scale" has one fp32 scale per row.

    A weight row that holds an infinity or NaN has no scale, and every output of its channel
    would be NaN: MoeError(MOE_ERR_DEVICE_BOUNDS).  Waits for the stream."""
    import torch

    def rows(w):
        q, s = alloc_codes(w.shape[0], w.shape[1], w.device)
        quantize_int8(w, q, s, stream=stream)
        return q, s

    E, F, d = W["w_gate"].shape
    dev = W["w_gate"].device
    Q = {"gate_up": torch.empty((E, 2 * F, d), dtype=torch.int8, device=dev),
         "gate_up_scale": torch.empty((E, 2 * F), dtype=torch.float32, device=dev)}
    for e in range(E):  # one expert at a time: no second copy of the weights is held
        for i, name in enumerate(("w_gate", "w_up")):
            quantize_int8(W[name][e], Q["gate_up"][e, i * F:(i + 1) * F],
                          Q["gate_up_scale"][e, i * F:(i + 1) * F], stream=stream)
    q, s = rows(W["w_down"].view(E * d, F))
    Q["down"], Q["down_scale"] = q.view(E, d, F), s.view(E, d)
    if W.get("ws_gate") is not None:
        Fs = W["ws_gate"].shape[0]
        Q["s_gate_up"] = torch.empty((2 * Fs, d), dtype=torch.int8, device=dev)
        Q["s_gate_up_scale"] = torch.empty(2 * Fs, dtype=torch.float32, device=dev)
        for i, name in enumerate(("ws_gate", "ws_up")):
            quantize_int8(W[name], Q["s_gate_up"][i * Fs:(i + 1) * Fs],
                          Q["s_gate_up_scale"][i * Fs:(i + 1) * Fs], stream=stream)
        Q["s_down"], Q["s_down_scale"] = rows(W["ws_down"])
    if stream is not None:
        torch.cuda.ExternalStream(stream.cuda_stream, device=dev).synchronize()
    bad = [n for n, t in Q.items() if n.endswith("_scale") and bool(torch.isnan(t).any())]
    if bad:
        raise MoeError(MOE_ERR_DEVICE_BOUNDS,
                       f"prepare_int8 (weight rows with an infinity or NaN: {', '.join(bad)})")
    return Q


class MoeLayer:
    """A layer instance: device weights, routing buffers and workspace, reused across calls.

    fp8 or int8 (one of the two) make 8-bit copies of the expert weights.  fp8 runs
    moe_forward_fp8; int8 runs the row and 8-bit integer calls one after another, and keeps
    the copies instead of the weights (a token mask is taken; flags of the 16-bit experts'
    engines and combine raise ValueError)."""

    def __init__(self, weights: dict, d_model, num_experts, num_experts_per_tok,
                 moe_intermediate_size, shared_intermediate_size, routed_scaling_factor=2.5,
                 max_tokens=1, flags=0, device="cuda", prepare=True, fp8=False, int8=False):
        if fp8 and int8:
            raise ValueError("fp8 or int8 experts, not both")
        if int8 and flags & INT8_REFUSED_FLAGS:
            raise ValueError("the int8 layer has one combine and its own choice of products: "
                             f"flags {flags & INT8_REFUSED_FLAGS} have no meaning there")
        self.W = dict(weights)
        self.cfg = dict(d_model=d_model, num_experts=num_experts,
                        num_experts_per_tok=num_experts_per_tok,
                        moe_intermediate_size=moe_intermediate_size,
                        shared_intermediate_size=shared_intermediate_size,
                        routed_scaling_factor=routed_scaling_factor, flags=flags)
        self.device = device
        self.fp8 = None
        self.int8 = None
        if int8:  # one-time int8 copies of the expert weights (model-load step)
            if workspace_size(self.dims(1)) == 0:
                raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_workspace_size")
            self.int8 = prepare_int8(self.W)
            self.W = {n: self.W.get(n) for n in ("w_router", "router_bias")}
        elif fp8:  # one-time FP8 copies of the expert weights (model-load step)
            self.cfg["flags"] |= MOE_FLAG_FP8_EXPERTS
            self.fp8, (code, site) = prepare_fp8(self.dims(1), self.W)
            if code != MOE_OK:
                raise MoeError(code, f"moe_prepare_fp8 (site {site})")
            self._q_struct = fp8_struct(self.fp8)
        elif prepare:  # one-time fp16 copy of the down projections (model-load step)
            self.cfg["flags"] |= MOE_FLAG_DOWN_F16
            code, site = prepare_down_f16(self.dims(1), self.W)
            if code != MOE_OK:
                raise MoeError(code, f"moe_prepare_down_f16 (site {site})")
        self._ws_struct = weights_struct(self.W)
        self._reserve(max_tokens)

    def dims(self, T):
        c = self.cfg
        return make_dims(T, c["d_model"], c["num_experts"], c["num_experts_per_tok"],
                         c["moe_intermediate_size"], c["shared_intermediate_size"],
                         c["routed_scaling_factor"], 1, c["flags"])

    def _reserve(self, T):
        self.max_tokens = T
        d = self.dims(T)
        if self.int8 is not None:  # self.ws is the router's
            self.ws = alloc_route_workspace(d, self.device)
        else:
            self.ws = alloc_workspace(d, self.device, upto=True)
        self.ws[:256].zero_()  # the status that device_status() reads before a first forward
        self.routing = alloc_routing(d, self.device)
        self._r_struct = routing_struct(self.routing)
        if self.int8 is not None:
            import torch
            c, n = self.cfg, T * d.num_experts_per_tok
            new = lambda *s, dtype: torch.empty(s, dtype=dtype, device=self.device)  # noqa: E731
            self.routing["inv"] = new(T, d.num_experts_per_tok, dtype=torch.int32)
            # a workspace of its own: moe_sort clears the status word, which the router's call
            # may have set in self.ws
            self._sort_ws = alloc_sort_workspace(d, self.device)

            def buffers(rows, F):
                # the activation stays in fp32 up to its codes: rounded to fp16 first, codes near
                # a border would move.  The experts' outputs are rounded to fp16, as the 16-bit
                # layer's are (2^-11 of each at most, an eighth of the sum's own rounding to
                # bf16): half the bytes for the product to write and the combine to read
                b = {"h": new(rows, F, dtype=torch.float32),
                     "o": new(rows, c["d_model"], dtype=torch.float16)}
                b["xq"], b["xs"] = alloc_codes(rows, c["d_model"], self.device)
                b["hq"], b["hs"] = alloc_codes(rows, F, self.device)
                return b
            self._routed = buffers(n, c["moe_intermediate_size"])
            self._shared = (buffers(T, c["shared_intermediate_size"])
                            if c["shared_intermediate_size"] else None)

    def _forward_int8(self, d, x, y, stream, token_mask):
        T, k, E = d.T, d.num_experts_per_tok, d.num_experts
        Q, R, n = self.int8, self.routing, T * d.num_experts_per_tok
        out = {"counts": R["counts"], "offsets": R["offsets"], "perm": R["perm"][:n],
               "inv": R["inv"][:T]}
        idx, w = R["topk_idx"].view(-1)[:n].view(T, k), R["topk_w"].view(-1)[:n].view(T, k)
        route(d, x, self.W["w_router"], self.W.get("router_bias"), idx, w, self.ws, stream,
              token_mask)
        sort(d, idx, out, self._sort_ws, stream=stream)
        b = {name: t[:n] for name, t in self._routed.items()}
        dispatch_int8(d, x, out["inv"], b["xq"], b["xs"], self.ws, stream)
        matmul_int8(b["xq"], b["xs"], Q["gate_up"], Q["gate_up_scale"], b["h"], self.ws,
                    R["offsets"], True, stream)
        quantize_int8(b["h"], b["hq"], b["hs"], R["offsets"][E:], stream)
        matmul_int8(b["hq"], b["hs"], Q["down"], Q["down_scale"], b["o"], self.ws, R["offsets"],
                    False, stream)
        shared = None
        if self._shared is not None:
            s = {name: t[:T] for name, t in self._shared.items()}
            quantize_int8(x, s["xq"], s["xs"], stream=stream)
            matmul_int8(s["xq"], s["xs"], Q["s_gate_up"], Q["s_gate_up_scale"], s["h"], self.ws,
                        None, True, stream)
            quantize_int8(s["h"], s["hq"], s["hs"], stream=stream)
            matmul_int8(s["hq"], s["hs"], Q["s_down"], Q["s_down_scale"], s["o"], self.ws,
                        stream=stream)
            shared = s["o"]
        combine(d, b["o"], out["inv"], w, y, self.ws, shared, stream)

    def device_status(self, stream=None):
        """(code, site) of the first device-side error of the last forward that had tokens
        (synchronises)."""
        status = read_device_status(self.ws, stream)
        if status[0] == MOE_OK and self.int8 is not None:
            status = read_device_status(self._sort_ws, stream)
        return status

    def forward(self, x, y=None, stream=None, token_mask=None):
        import torch
        T = x.shape[0]
        if T > self.max_tokens:
            self._reserve(T)
        if y is None:
            y = torch.empty_like(x)
        if self.fp8 is not None and token_mask is not None:
            raise ValueError("the FP8-expert forward takes no token mask")
        if T == 0:  # (an empty tensor has no address to pass on)
            return y
        d = self.dims(T)
        if self.int8 is not None:
            self._forward_int8(d, x, y, stream, token_mask)
        elif self.fp8 is not None:
            forward_fp8(d, self._ws_struct, self._q_struct, x, y, self._r_struct, self.ws, stream)
        else:
            forward(d, self._ws_struct, x, y, self._r_struct, self.ws, stream,
                    token_mask=token_mask)
        return y
