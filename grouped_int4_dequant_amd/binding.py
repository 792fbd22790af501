"""ctypes binding of libmoe_int4.so (the C ABI in include/moe_int4.h).

Argument marshalling only: every step of the layer runs in the HIP kernels of
the library. PyTorch supplies device memory and the current HIP stream. The
module raises when the library is missing; there is no fallback path.

Tensor formats:
  bf16 values       torch.bfloat16 tensors (passed as uint16 bit patterns)
  packed int4 codes torch.int32 tensors holding the uint32 words
  logits, y         torch.float32
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_int4.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP = 0, -1, -2, -3, -4

_P = ctypes.c_void_p
_I32 = ctypes.c_int32


class MoeLayerT(ctypes.Structure):
    _fields_ = [("d", _I32), ("f", _I32), ("E", _I32), ("k", _I32), ("f_sh", _I32),
                ("gu_q", _P), ("gu_s", _P), ("gu_b", _P),
                ("dn_q", _P), ("dn_s", _P), ("dn_b", _P),
                ("sh_gu_q", _P), ("sh_gu_s", _P), ("sh_gu_b", _P),
                ("sh_dn_q", _P), ("sh_dn_s", _P), ("sh_dn_b", _P),
                ("prep", _P)]


class MoeRoutingT(ctypes.Structure):
    _fields_ = [("topk_ids", _P), ("topk_w", _P), ("counts", _P), ("offsets", _P),
                ("sorted_pair", _P), ("sorted_token", _P), ("pair_pos", _P),
                ("block_map", _P), ("num_blocks", _P)]


class MoeWorkspaceLayoutT(ctypes.Structure):
    _fields_ = [("decode_form", _I32), ("x16", ctypes.c_int64), ("h", ctypes.c_int64),
                ("h_sh", ctypes.c_int64), ("o", ctypes.c_int64), ("o_sh", ctypes.c_int64),
                ("dec_h", ctypes.c_int64)]


class MoeLayer16T(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("d", _I32), ("f", _I32), ("E", _I32), ("k", _I32), ("f_sh", _I32),
                ("gu", _P), ("dn", _P), ("sh_gu", _P), ("sh_dn", _P)]


_lib = None


def load() -> ctypes.CDLL:
    """Load the HIP library (once). Raises FileNotFoundError when it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FileNotFoundError(
                f"{LIB_PATH} is missing: build it with grouped_int4_dequant_amd/build.py")
        lib = ctypes.CDLL(LIB_PATH)
        lib.moe_max_blocks.argtypes = [_I32, _I32, _I32]
        lib.moe_max_blocks.restype = _I32
        lib.moe_workspace_bytes.argtypes = [_I32, ctypes.POINTER(MoeLayerT)]
        lib.moe_workspace_bytes.restype = ctypes.c_size_t
        lib.moe_workspace_layout.argtypes = [_I32, ctypes.POINTER(MoeLayerT), ctypes.POINTER(MoeWorkspaceLayoutT)]
        lib.moe_workspace_layout.restype = ctypes.c_int
        lib.moe_route_workspace_bytes.argtypes = [_I32, _I32]
        lib.moe_route_workspace_bytes.restype = ctypes.c_size_t
        lib.moe_route.argtypes = [_P, _I32, _I32, _I32, ctypes.POINTER(MoeRoutingT), _P,
                                  ctypes.c_size_t, _P]
        lib.moe_route.restype = ctypes.c_int
        lib.moe_grouped_gemm_int4.argtypes = [_P, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _I32,
                                              _P, _I32, _P]
        lib.moe_grouped_gemm_int4.restype = ctypes.c_int
        lib.moe_layer_forward.argtypes = [ctypes.POINTER(MoeLayerT), _P, _P, _I32, _P,
                                          ctypes.POINTER(MoeRoutingT), _P, ctypes.c_size_t, _P]
        lib.moe_layer_forward.restype = ctypes.c_int
        lib.moe_prefill_chunked.argtypes = [ctypes.POINTER(MoeLayerT), _P, _P, _I32, _I32, _P, _P,
                                            ctypes.c_size_t, _P]
        lib.moe_layer_forward_ablation.argtypes = [ctypes.POINTER(MoeLayerT), _P, _P, _I32, _P,
                                                   ctypes.POINTER(MoeRoutingT), _P, ctypes.c_size_t, _P,
                                                   _I32]
        lib.moe_layer_forward_ablation.restype = ctypes.c_int
        lib.moe_layer_forward_noalloc.argtypes = [ctypes.POINTER(MoeLayerT), _P, _P, _I32, _P,
                                                  ctypes.POINTER(MoeRoutingT), _P]
        lib.moe_layer_forward_noalloc.restype = ctypes.c_int
        lib.moe_layer_forward_checked.argtypes = [ctypes.POINTER(MoeLayerT), _P, _P, _I32, _P,
                                                  ctypes.POINTER(MoeRoutingT), _P, ctypes.c_size_t, _P, _P]
        lib.moe_layer_forward_checked.restype = ctypes.c_int
        lib.moe_router_topk.argtypes = [_P, _I32, _I32, _P, _I32, _I32, _P, _P, _P, _P]
        lib.moe_router_topk.restype = ctypes.c_int
        lib.moe_layer_forward_router.argtypes = [ctypes.POINTER(MoeLayerT), _P, _P, _I32, _P,
                                                 ctypes.POINTER(MoeRoutingT), _P, ctypes.c_size_t, _P]
        lib.moe_layer_forward_router.restype = ctypes.c_int
        lib.moe_layer_graph_create.argtypes = [ctypes.POINTER(MoeLayerT), _P, _P, _I32, _P, _P, ctypes.c_size_t,
                                               _I32, _I32, _P, ctypes.POINTER(_P)]
        lib.moe_layer_graph_create.restype = ctypes.c_int
        lib.moe_layer_graph_launch.argtypes = [_P, _P]
        lib.moe_layer_graph_launch.restype = ctypes.c_int
        lib.moe_layer_graph_destroy.argtypes = [_P]
        lib.moe_layer_graph_destroy.restype = ctypes.c_int
        lib.moe_router_logits.argtypes = [_P, _I32, _I32, _P, _I32, _P, _P]
        lib.moe_router_logits.restype = ctypes.c_int
        lib.moe_ablation_workspace_bytes.argtypes = [_I32, ctypes.POINTER(MoeLayerT), _I32]
        lib.moe_ablation_workspace_bytes.restype = ctypes.c_size_t
        lib.moe_prefill_chunked.restype = ctypes.c_int
        lib.moe_prepared_bytes.argtypes = [ctypes.POINTER(MoeLayerT)]
        lib.moe_prepared_bytes.restype = ctypes.c_size_t
        lib.moe_prepare_weights.argtypes = [ctypes.POINTER(MoeLayerT), _P, ctypes.c_size_t, _P]
        lib.moe_prepare_weights.restype = ctypes.c_int
        I, L = _I32, ctypes.c_int64
        lib.moe_grouped_gemm.argtypes = [I, _P, L, I, _P, _P, I, I, I, I, _P, _P, I, L, _P]
        lib.moe_grouped_gemm_dgrad.argtypes = [I, _P, L, _P, I, I, I, I, _P, _P, I, L, _P]
        lib.moe_grouped_gemm_wgrad.argtypes = [I, _P, L, _P, L, I, _P, _P, I, I, I, I, _P, I, I, _P]
        lib.moe_combine.argtypes = [I, _P, L, I, _P, _P, I, I, I, _P, I, L, _P, I, L, _P]
        lib.moe_combine_backward.argtypes = [I, _P, L, _P, L, I, _P, _P, I, I, I, _P, L, _P, _P]
        lib.moe_adapter_plan.argtypes = [_P, I, I, _P, _P, _P]
        lib.moe_adapter_forward.argtypes = [I, _P, L, I, I, I, I, I, _P, _P, _P, _P, _P, _P, L, _P, I, L, _P]
        lib.moe_adapter_backward.argtypes = [I, _P, L, _P, L, I, I, I, I, I, _P, _P, _P, _P, _P, _P, L, _P, I, L,
                                             _P, _P, I, I, _P, ctypes.c_size_t, _P]
        for name in ("moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_combine",
                     "moe_combine_backward", "moe_adapter_plan", "moe_adapter_forward", "moe_adapter_backward"):
            getattr(lib, name).restype = ctypes.c_int
        lib.moe_adapter_backward_workspace_bytes.argtypes = [I, I]
        lib.moe_adapter_backward_workspace_bytes.restype = ctypes.c_size_t
        F, Z = ctypes.c_float, ctypes.c_size_t
        lib.moe_linear.argtypes = [I, _P, L, I, I, I, _P, _P, I, I, _P, L, _P, L, _P, I, L, _P]
        lib.moe_linear_backward.argtypes = [I, _P, L, _P, L, I, I, I, _P, _P, L, I, _P, I, L, _P, _P, I, I, _P, Z, _P]
        lib.moe_residual_norm.argtypes = [I, _P, L, _P, L, I, I, I, _P, _P, I, _P, I, F, F, _P, L, _P, L, _P]
        lib.moe_residual_norm_backward.argtypes = [I, _P, L, _P, L, _P, L, _P, L, I, I, I, _P, _P, I, _P, I, F, F, _P, L, _P, L,
                                                   _P, _P, _P, I, I, _P, Z, _P]
        lib.moe_few_tokens_layer.argtypes = [ctypes.POINTER(MoeLayer16T), _P, L, _P, I, _P, L, _P, I, L, _P, _P, _P, Z, _P]
        lib.moe_few_tokens_workspace_bytes.argtypes = [ctypes.POINTER(MoeLayer16T), I]
        lib.moe_few_tokens_workspace_bytes.restype = Z
        for name in ("moe_linear", "moe_linear_backward", "moe_residual_norm", "moe_residual_norm_backward", "moe_few_tokens_layer"):
            getattr(lib, name).restype = ctypes.c_int
        lib.moe_linear_backward_workspace_bytes.argtypes = [I, I, I, I]
        lib.moe_linear_backward_workspace_bytes.restype = Z
        lib.moe_residual_norm_backward_workspace_bytes.argtypes = [I, I, I]
        lib.moe_residual_norm_backward_workspace_bytes.restype = Z
        lib.moe_status_string.argtypes = [ctypes.c_int]
        lib.moe_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != MOE_OK:
        raise ValueError(f"{what}: {status_string(status)} (status {status})")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


class Layer:
    """Device weights of one MoE layer plus the moe_layer_t that points at them."""

    KEYS = ("gu_q", "gu_s", "gu_b", "dn_q", "dn_s", "dn_b",
            "sh_gu_q", "sh_gu_s", "sh_gu_b", "sh_dn_q", "sh_dn_s", "sh_dn_b")

    def __init__(self, d: int, f: int, E: int, k: int, f_sh: int, tensors: Dict[str, torch.Tensor],
                 prepare: bool = True):
        self.d, self.f, self.E, self.k, self.f_sh = d, f, E, k, f_sh
        self.tensors = dict(tensors)
        shapes = {"gu_q": (E, 2 * f, d // 8), "gu_s": (E, 2 * f, d // 64), "gu_b": (E, 2 * f, d // 64),
                  "dn_q": (E, d, f // 8), "dn_s": (E, d, f // 64), "dn_b": (E, d, f // 64),
                  "sh_gu_q": (2 * f_sh, d // 8), "sh_gu_s": (2 * f_sh, d // 64),
                  "sh_gu_b": (2 * f_sh, d // 64), "sh_dn_q": (d, f_sh // 8),
                  "sh_dn_s": (d, f_sh // 64), "sh_dn_b": (d, f_sh // 64)}
        ptrs = {}
        for key in self.KEYS:
            if key.startswith("sh_") and f_sh == 0:
                ptrs[key] = None
                continue
            t = self.tensors[key]
            _need(t, key, torch.int32 if key.endswith("_q") else torch.bfloat16, shapes[key])
            ptrs[key] = t.data_ptr()
        self.c = MoeLayerT(d, f, E, k, f_sh, *[ptrs[k_] for k_ in self.KEYS], None)
        self.prep = None
        if prepare:
            self.prepare()

    def prepare(self, stream=None) -> bool:
        """moe_prepare_weights into a new device buffer, then point c.prep at
        it. Returns False (and leaves c.prep null) when the layer's shape has
        no prepared form (d, f or f_sh not a multiple of 128)."""
        lib = load()
        n = int(lib.moe_prepared_bytes(ctypes.byref(self.c)))
        if n == 0:
            return False
        dev = self.tensors["gu_q"].device
        buf = torch.empty(n + 256, dtype=torch.uint8, device=dev)
        ptr = (buf.data_ptr() + 255) // 256 * 256
        _check(lib.moe_prepare_weights(ctypes.byref(self.c), ptr, n, _stream(stream)), "moe_prepare_weights")
        self.prep, self.c.prep = buf, ptr
        return True

    @classmethod
    def from_numpy(cls, d, f, E, k, f_sh, arrays, device="cuda", prepare: bool = True):
        """Upload generator arrays (uint32 codes, uint16 bf16 bits) to the GPU
        (and, with prepare, build the prepared copy the prefill GEMMs read)."""
        import numpy as np
        ts = {}
        for key, a in arrays.items():
            if key.endswith("_q"):
                ts[key] = torch.from_numpy(np.ascontiguousarray(a).view(np.int32)).to(device)
            else:
                ts[key] = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(device)
        return cls(d, f, E, k, f_sh, ts, prepare=prepare)


def max_blocks(T: int, E: int, k: int) -> int:
    return int(load().moe_max_blocks(T, E, k))


def prepared_bytes(layer: Layer) -> int:
    return int(load().moe_prepared_bytes(ctypes.byref(layer.c)))


def workspace_bytes(T: int, layer: Layer) -> int:
    return int(load().moe_workspace_bytes(T, ctypes.byref(layer.c)))


def workspace_layout(T: int, layer: Layer) -> Dict[str, int]:
    """moe_workspace_layout: byte offsets of the fp16 intermediates a
    moe_layer_forward call of T tokens keeps in its workspace (-1: absent)."""
    out = MoeWorkspaceLayoutT()
    _check(load().moe_workspace_layout(T, ctypes.byref(layer.c), ctypes.byref(out)), "moe_workspace_layout")
    return {name: int(getattr(out, name)) for name, _ in MoeWorkspaceLayoutT._fields_}


def route_workspace_bytes(T: int, E: int) -> int:
    return int(load().moe_route_workspace_bytes(T, E))


def alloc_routing(T: int, E: int, k: int, device="cuda") -> Dict[str, torch.Tensor]:
    mb = max_blocks(T, E, k)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(topk_ids=torch.empty((T, k), **i32),
                topk_w=torch.empty((T, k), dtype=torch.float32, device=device),
                counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                sorted_pair=torch.empty(T * k, **i32), sorted_token=torch.empty(T * k, **i32),
                pair_pos=torch.empty(T * k, **i32), block_map=torch.empty((mb, 3), **i32),
                num_blocks=torch.empty(1, **i32))


def _routing_struct(r: Dict[str, torch.Tensor]) -> MoeRoutingT:
    for key, t in r.items():
        _need(t, key, torch.float32 if key == "topk_w" else torch.int32)
    return MoeRoutingT(*[r[k].data_ptr() for k in ("topk_ids", "topk_w", "counts", "offsets",
                                                   "sorted_pair", "sorted_token", "pair_pos",
                                                   "block_map", "num_blocks")])


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Workspace buffer (torch's caching allocator returns 256-byte aligned storage)."""
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def route(logits: torch.Tensor, k: int, out: Optional[Dict[str, torch.Tensor]] = None,
          ws: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """moe_route: GPU top-k, gates, histogram, scan, stable scatter and block map."""
    T, E = logits.shape
    _need(logits, "logits", torch.float32)
    out = alloc_routing(T, E, k, logits.device) if out is None else out
    need = route_workspace_bytes(T, E)
    ws = alloc_workspace(need, logits.device) if ws is None else ws
    rs = _routing_struct(out)
    _check(load().moe_route(logits.data_ptr(), T, E, k, ctypes.byref(rs), ws.data_ptr(),
                            ws.numel(), _stream(stream)), "moe_route")
    return out


def grouped_gemm_int4(A: torch.Tensor, a_row: Optional[torch.Tensor], N: int, K: int,
                      Wq: torch.Tensor, Ws: torch.Tensor, Wb: torch.Tensor,
                      block_map: torch.Tensor, num_blocks: torch.Tensor, C: torch.Tensor,
                      stream=None) -> torch.Tensor:
    """moe_grouped_gemm_int4: C[p] = A[row(p)] @ W_e(p)^T for the rows of every block."""
    _need(A, "A", torch.bfloat16)
    _need(Wq, "Wq", torch.int32)
    _need(Ws, "Ws", torch.bfloat16)
    _need(Wb, "Wb", torch.bfloat16)
    _need(block_map, "block_map", torch.int32)
    _need(num_blocks, "num_blocks", torch.int32)
    _need(C, "C", torch.float32)
    if a_row is not None:
        _need(a_row, "a_row", torch.int32)
    _check(load().moe_grouped_gemm_int4(A.data_ptr(), A.shape[-1], _ptr(a_row), N, K,
                                        Wq.data_ptr(), Ws.data_ptr(), Wb.data_ptr(),
                                        block_map.data_ptr(), num_blocks.data_ptr(),
                                        block_map.shape[0], C.data_ptr(), C.shape[-1],
                                        _stream(stream)), "moe_grouped_gemm_int4")
    return C


def layer_forward(layer: Layer, x: torch.Tensor, logits: torch.Tensor,
                  y: Optional[torch.Tensor] = None,
                  routing: Optional[Dict[str, torch.Tensor]] = None,
                  ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_layer_forward: the whole layer for T tokens into fp32 y."""
    T = x.shape[0]
    _need(x, "x", torch.bfloat16, (T, layer.d))
    _need(logits, "logits", torch.float32, (T, layer.E))
    y = torch.empty((T, layer.d), dtype=torch.float32, device=x.device) if y is None else y
    _need(y, "y", torch.float32, (T, layer.d))
    ws = alloc_workspace(workspace_bytes(T, layer), x.device) if ws is None else ws
    rs = _routing_struct(routing) if routing is not None else None
    _check(load().moe_layer_forward(ctypes.byref(layer.c), x.data_ptr(), logits.data_ptr(), T,
                                    y.data_ptr(), ctypes.byref(rs) if rs is not None else None,
                                    ws.data_ptr(), ws.numel(), _stream(stream)),
           "moe_layer_forward")
    return y


OVERFLOW_X, OVERFLOW_H, OVERFLOW_O = 1, 2, 4


def layer_forward_checked(layer: Layer, x: torch.Tensor, logits: torch.Tensor, overflow: torch.Tensor,
                          y: Optional[torch.Tensor] = None,
                          routing: Optional[Dict[str, torch.Tensor]] = None,
                          ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_layer_forward_checked: the layer, ORing OVERFLOW_* bits into the
    int32 device tensor `overflow` (one element, set by the caller) when a
    value kept in fp16 leaves fp16's finite range."""
    T = x.shape[0]
    _need(x, "x", torch.bfloat16, (T, layer.d))
    _need(logits, "logits", torch.float32, (T, layer.E))
    _need(overflow, "overflow", torch.int32, (1,))
    y = torch.empty((T, layer.d), dtype=torch.float32, device=x.device) if y is None else y
    _need(y, "y", torch.float32, (T, layer.d))
    ws = alloc_workspace(workspace_bytes(T, layer), x.device) if ws is None else ws
    rs = _routing_struct(routing) if routing is not None else None
    _check(load().moe_layer_forward_checked(ctypes.byref(layer.c), x.data_ptr(), logits.data_ptr(), T,
                                            y.data_ptr(), ctypes.byref(rs) if rs is not None else None,
                                            ws.data_ptr(), ws.numel(), _stream(stream), overflow.data_ptr()),
           "moe_layer_forward_checked")
    return y


def layer_forward_noalloc(layer: Layer, x: torch.Tensor, logits: torch.Tensor,
                          y: Optional[torch.Tensor] = None,
                          routing: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> torch.Tensor:
    """moe_layer_forward_noalloc: the layer with the library's static per-GPU
    scratch array as its workspace (no device allocation in the call)."""
    T = x.shape[0]
    _need(x, "x", torch.bfloat16, (T, layer.d))
    _need(logits, "logits", torch.float32, (T, layer.E))
    y = torch.empty((T, layer.d), dtype=torch.float32, device=x.device) if y is None else y
    _need(y, "y", torch.float32, (T, layer.d))
    rs = _routing_struct(routing) if routing is not None else None
    _check(load().moe_layer_forward_noalloc(ctypes.byref(layer.c), x.data_ptr(), logits.data_ptr(), T,
                                            y.data_ptr(), ctypes.byref(rs) if rs is not None else None,
                                            _stream(stream)), "moe_layer_forward_noalloc")
    return y


def router_logits(x: torch.Tensor, w_r: torch.Tensor, logits: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """moe_router_logits: logits fp32 [T][E] = x W_r^T from bf16 x [T][d] and
    bf16 W_r [E][d]."""
    T, d = x.shape
    E = w_r.shape[0]
    _need(x, "x", torch.bfloat16, (T, d))
    _need(w_r, "w_r", torch.bfloat16, (E, d))
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device) if logits is None else logits
    _need(logits, "logits", torch.float32, (T, E))
    _check(load().moe_router_logits(x.data_ptr(), T, d, w_r.data_ptr(), E, logits.data_ptr(), _stream(stream)),
           "moe_router_logits")
    return logits


def router_topk(x: torch.Tensor, w_r: torch.Tensor, k: int, logits: Optional[torch.Tensor] = None,
                stream=None):
    """moe_router_topk: (topk_ids int32 [T][k], topk_w fp32 [T][k]) from bf16
    x [T][d] and bf16 W_r [E][d]; the fp32 logits [T][E] go to `logits`
    (allocated when not given)."""
    T, d = x.shape
    E = w_r.shape[0]
    _need(x, "x", torch.bfloat16, (T, d))
    _need(w_r, "w_r", torch.bfloat16, (E, d))
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device) if logits is None else logits
    _need(logits, "logits", torch.float32, (T, E))
    ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    _check(load().moe_router_topk(x.data_ptr(), T, d, w_r.data_ptr(), E, k, _ptr(logits), ids.data_ptr(),
                                  w.data_ptr(), _stream(stream)), "moe_router_topk")
    return ids, w


def layer_forward_router(layer: Layer, x: torch.Tensor, w_r: torch.Tensor,
                         y: Optional[torch.Tensor] = None,
                         routing: Optional[Dict[str, torch.Tensor]] = None,
                         ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_layer_forward_router: the whole layer from bf16 router weights
    W_r [E][d] instead of logits."""
    T = x.shape[0]
    _need(x, "x", torch.bfloat16, (T, layer.d))
    _need(w_r, "w_r", torch.bfloat16, (layer.E, layer.d))
    y = torch.empty((T, layer.d), dtype=torch.float32, device=x.device) if y is None else y
    _need(y, "y", torch.float32, (T, layer.d))
    ws = alloc_workspace(workspace_bytes(T, layer), x.device) if ws is None else ws
    rs = _routing_struct(routing) if routing is not None else None
    _check(load().moe_layer_forward_router(ctypes.byref(layer.c), x.data_ptr(), w_r.data_ptr(), T, y.data_ptr(),
                                           ctypes.byref(rs) if rs is not None else None, ws.data_ptr(),
                                           ws.numel(), _stream(stream)), "moe_layer_forward_router")
    return y


GRAPH_CONCURRENT = 1


class LayerGraph:
    """moe_layer_graph_create/_launch/_destroy: the layer captured once into a
    HIP graph bound to x, logits, y and a workspace; launch() recomputes y
    from their current contents. concurrent=True runs the shared expert on a
    branch beside the routing (shared_unit_rows rows per item; 0: 96)."""

    def __init__(self, layer: Layer, x: torch.Tensor, logits: torch.Tensor, y: torch.Tensor,
                 ws: Optional[torch.Tensor] = None, concurrent: bool = True, shared_unit_rows: int = 0):
        T = x.shape[0]
        _need(x, "x", torch.bfloat16, (T, layer.d))
        _need(logits, "logits", torch.float32, (T, layer.E))
        _need(y, "y", torch.float32, (T, layer.d))
        ws = alloc_workspace(workspace_bytes(T, layer), x.device) if ws is None else ws
        self._keep = (layer, x, logits, y, ws)  # the graph holds their addresses
        cap = torch.cuda.Stream(device=x.device)
        cap.wait_stream(torch.cuda.current_stream(x.device))
        h = ctypes.c_void_p()
        _check(load().moe_layer_graph_create(ctypes.byref(layer.c), x.data_ptr(), logits.data_ptr(), T,
                                             y.data_ptr(), ws.data_ptr(), ws.numel(),
                                             GRAPH_CONCURRENT if concurrent else 0, shared_unit_rows,
                                             cap.cuda_stream, ctypes.byref(h)), "moe_layer_graph_create")
        self._h = h.value

    def launch(self, stream=None):
        _check(load().moe_layer_graph_launch(self._h, _stream(stream)), "moe_layer_graph_launch")

    def close(self):
        if self._h:
            _check(load().moe_layer_graph_destroy(self._h), "moe_layer_graph_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


ABLATIONS = {"none": 0, "tile16": 1, "host_routing": 2, "unfused": 3}


def ablation_workspace_bytes(T: int, layer: Layer, variant: str) -> int:
    n = load().moe_ablation_workspace_bytes(T, ctypes.byref(layer.c), ABLATIONS[variant])
    if n == 0:
        raise ValueError("invalid layer, token count or ablation")
    return n


def layer_forward_ablation(layer: Layer, x: torch.Tensor, logits: torch.Tensor, variant: str,
                           y: Optional[torch.Tensor] = None,
                           routing: Optional[Dict[str, torch.Tensor]] = None,
                           ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_layer_forward_ablation: the prefill sequence with one of the pages'
    ablations ("none", "tile16", "host_routing", "unfused"); measurement only."""
    T = x.shape[0]
    _need(x, "x", torch.bfloat16, (T, layer.d))
    _need(logits, "logits", torch.float32, (T, layer.E))
    y = torch.empty((T, layer.d), dtype=torch.float32, device=x.device) if y is None else y
    _need(y, "y", torch.float32, (T, layer.d))
    ws = alloc_workspace(ablation_workspace_bytes(T, layer, variant), x.device) if ws is None else ws
    rs = _routing_struct(routing) if routing is not None else None
    _check(load().moe_layer_forward_ablation(ctypes.byref(layer.c), x.data_ptr(), logits.data_ptr(), T,
                                             y.data_ptr(), ctypes.byref(rs) if rs is not None else None,
                                             ws.data_ptr(), ws.numel(), _stream(stream), ABLATIONS[variant]),
           "moe_layer_forward_ablation")
    return y


def prefill_chunked(layer: Layer, x: torch.Tensor, logits: torch.Tensor, chunk: int = 2048,
                    y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """moe_prefill_chunked: the layer over bounded chunks with one reused workspace."""
    T = x.shape[0]
    _need(x, "x", torch.bfloat16, (T, layer.d))
    _need(logits, "logits", torch.float32, (T, layer.E))
    y = torch.empty((T, layer.d), dtype=torch.float32, device=x.device) if y is None else y
    _need(y, "y", torch.float32, (T, layer.d))
    ws = alloc_workspace(workspace_bytes(min(chunk, max(T, 1)), layer), x.device) if ws is None else ws
    _check(load().moe_prefill_chunked(ctypes.byref(layer.c), x.data_ptr(), logits.data_ptr(), T,
                                      chunk, y.data_ptr(), ws.data_ptr(), ws.numel(),
                                      _stream(stream)), "moe_prefill_chunked")
    return y


# ---------------------------------------------------------- 16-bit operators
# Tensors are bf16 or fp16 (one type per call), results of that type or fp32.
# Activations and results may be row-strided views (their columns contiguous);
# a call runs on the tensors' device, on `stream` or that device's current
# stream, and what it allocates belongs to that stream. The calls are not recorded
# for autograd: results carry no gradient function, whatever requires_grad says,
# and the gradients are the calls named for them.
_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _current_stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same handle without a Stream object: 0.1 against 1.9 us
    def _current_stream(device: torch.device) -> int:  # noqa: F811
        return torch._C._cuda_getCurrentRawStream(device.index)


_current_device = torch.cuda.current_device
if hasattr(torch._C, "_cuda_getDevice"):  # the same without a check whether torch has set up the GPU, which the tensors show: 0.1 against 0.3 us
    _current_device = torch._C._cuda_getDevice


class _Call:
    """One call: its device and stream, and the checks of its tensors."""

    __slots__ = ("lead", "dtype", "device", "index", "code", "stream", "given")

    def __init__(self, lead: torch.Tensor, name: str, stream):
        if not isinstance(lead, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        self.lead = lead
        self.dtype = lead.dtype
        if self.dtype is not torch.bfloat16 and self.dtype is not torch.float16:
            raise TypeError(f"{name} must be bfloat16 or float16, got {lead.dtype}")
        if not lead.is_cuda:
            raise ValueError(f"{name} must be on the GPU")
        self.device = lead.device
        self.index = self.device.index
        self.code = 0 if self.dtype is torch.bfloat16 else 1
        self.given = stream
        if stream is None:
            self.stream = _current_stream(self.device)
        elif stream.device != self.device:
            raise ValueError(f"stream must be of {lead.device}, got {stream.device}")
        else:
            self.stream = stream.cuda_stream

    def need(self, t, name, dtype, shape):
        """A contiguous tensor of the call's device."""
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == self.index and t.is_contiguous()):
            _need(t, name, dtype, shape)
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        return t

    def rows(self, t, name, shape, other=None):
        """A matrix of the call's type (or of `other`) with contiguous columns and a row stride of at least its width."""
        if isinstance(t, torch.Tensor) and t.dtype is self.dtype and t.shape == shape and t.get_device() == self.index and t.is_contiguous():
            return t
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not self.dtype and (other is None or t.dtype is not other):
            raise TypeError(f"{name} must be {self.dtype}{'' if other is None else f' or {other}'}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        if not t.is_contiguous() and ((shape[1] > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) < shape[1])):
            raise ValueError(f"{name} must have contiguous columns and rows that do not overlap")
        return t

    def ld(self, t, name, shape, other=None):
        """Row stride of a matrix as `rows` takes it; at least its width (that of a single row may be anything)."""
        if (isinstance(t, torch.Tensor) and (t.dtype is self.dtype or t.dtype is other) and t.shape == shape and t.get_device() == self.index
                and t.is_contiguous()):
            return shape[1]
        return max(self.rows(t, name, shape, other).stride(0), shape[1])

    def vector(self, t, name, shape):
        """A contiguous tensor of the call's type or fp32."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not self.dtype and t.dtype is not torch.float32:
            raise TypeError(f"{name} must be {self.dtype} or float32, got {t.dtype}")
        return self.need(t, name, t.dtype, shape)

    def result(self, t, name, shape, dtype):
        """The given result matrix, or a new one of `dtype` (None: the call's type)."""
        if t is not None:
            if dtype is not None and t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            return self.rows(t, name, shape, torch.float32)
        return self.new(shape, self._type(dtype, name))

    def whole(self, t, name, shape, dtype):
        """The given contiguous result, or a new one of `dtype` (None: the call's type)."""
        if t is None:
            return self.new(shape, self._type(dtype, name))
        if t.dtype not in (self.dtype, torch.float32) or (dtype is not None and t.dtype is not dtype):
            raise TypeError(f"{name} must be {dtype or self.dtype}, got {t.dtype}")
        return self.need(t, name, t.dtype, shape)

    def _type(self, dtype, name):
        if dtype is None:
            return self.dtype
        if dtype is not self.dtype and dtype is not torch.float32:
            raise TypeError(f"{name} must be {self.dtype} or float32, not {dtype}")
        return dtype

    def new(self, shape, dtype):
        """A new tensor that belongs to the call's stream."""
        if self.given is None:
            return self.lead.new_empty(shape, dtype=dtype)  # (0.4 us less than torch.empty)
        with torch.cuda.stream(self.given):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, ws, need):
        """The given workspace, or a new one of `need` bytes that belongs to the call's stream."""
        if ws is None:
            return self.new(max(need, 1), torch.uint8)
        if ws.device != self.device:
            raise ValueError(f"ws must be on {self.device}, got {ws.device}")
        if not ws.is_contiguous():
            raise ValueError("ws must be contiguous")
        return ws

    def __call__(self, what, *args):
        f = getattr(_lib or load(), what)
        if _current_device() == self.index:
            status = f(*args, self.stream)
        else:
            with torch.cuda.device(self.device):
                status = f(*args, self.stream)
        if status != MOE_OK:
            _check(status, what)


def _ld(t: Optional[torch.Tensor], width: int) -> int:
    """Row stride of a checked matrix; at least its width (that of a single row may be anything)."""
    return 0 if t is None else max(t.stride(0), width)


def _sizes(*sizes: int):
    """Sizes cross the C interface in 32 bits, where ctypes would cut off larger ones."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"sizes from 2^31 on are not supported, got {max(sizes)}")


def _groups(c: _Call, offsets: torch.Tensor, G: int) -> torch.Tensor:
    return c.need(offsets, "offsets", torch.int32, (G + 1,))


def grouped_gemm(A: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, a_row: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """moe_grouped_gemm: C[p] = A[row(p)] @ W[e]^T for the sorted rows p of
    each group e (offsets[e] .. offsets[e+1]). A [rows][K], W [G][N][K], a_row
    int32 [P] (None: row(p) = p). Returns C [P][N]; rows behind the last group
    are not written."""
    c = _Call(A, "A", stream)
    if A.dim() != 2 or not isinstance(W, torch.Tensor) or W.dim() != 3:
        raise ValueError("A must be [rows][K] and W [G][N][K]")
    G, N, K = W.shape
    c.rows(A, "A", (A.shape[0], K))
    c.need(W, "W", c.dtype, (G, N, K))
    P = A.shape[0] if a_row is None else a_row.numel()
    _sizes(A.shape[0], G, P, N, K)
    if a_row is not None:
        c.need(a_row, "a_row", torch.int32, (P,))
    _groups(c, offsets, G)
    C = c.result(out, "out", (P, N), out_dtype)
    c("moe_grouped_gemm", c.code, A.data_ptr(), _ld(A, K), A.shape[0], _ptr(a_row), offsets.data_ptr(), G, P, N, K,
      W.data_ptr(), C.data_ptr(), _CODES[C.dtype], _ld(C, N))
    return C


def grouped_gemm_dgrad(dC: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                       out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """moe_grouped_gemm_dgrad: dA[p] = dC[p] @ W[e] for the sorted rows p of
    each group e. Returns dA [P][K], by sorted row."""
    c = _Call(dC, "dC", stream)
    if dC.dim() != 2 or not isinstance(W, torch.Tensor) or W.dim() != 3:
        raise ValueError("dC must be [P][N] and W [G][N][K]")
    G, N, K = W.shape
    P = dC.shape[0]
    _sizes(G, P, N, K)
    c.rows(dC, "dC", (P, N))
    c.need(W, "W", c.dtype, (G, N, K))
    _groups(c, offsets, G)
    dA = c.result(out, "out", (P, K), out_dtype)
    c("moe_grouped_gemm_dgrad", c.code, dC.data_ptr(), _ld(dC, N), offsets.data_ptr(), G, P, N, K, W.data_ptr(),
      dA.data_ptr(), _CODES[dA.dtype], _ld(dA, K))
    return dA


def grouped_gemm_wgrad(dC: torch.Tensor, A: torch.Tensor, offsets: torch.Tensor, a_row: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                       accumulate: bool = False, stream=None) -> torch.Tensor:
    """moe_grouped_gemm_wgrad: dW[e] = dC[rows of e]^T @ A[row(rows of e)].
    Returns dW [G][N][K]; with accumulate it is added to `out` (fp32)."""
    c = _Call(dC, "dC", stream)
    if dC.dim() != 2 or not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("dC must be [P][N] and A [rows][K]")
    if not isinstance(offsets, torch.Tensor) or offsets.numel() < 2:
        raise ValueError("offsets must hold the G + 1 group bounds")
    P, N = dC.shape
    K, G = A.shape[1], offsets.numel() - 1
    _sizes(A.shape[0], G, P, N, K)
    c.rows(dC, "dC", (P, N))
    c.rows(A, "A", (A.shape[0], K))
    if a_row is not None:
        c.need(a_row, "a_row", torch.int32, (P,))
    elif A.shape[0] != P:
        raise ValueError(f"A must have the {P} rows of dC when a_row is not given, got {A.shape[0]}")
    _groups(c, offsets, G)
    if accumulate and out is None:
        raise ValueError("accumulate needs the tensor to add to in `out`")
    dW = c.whole(out, "out", (G, N, K), out_dtype)
    c("moe_grouped_gemm_wgrad", c.code, dC.data_ptr(), _ld(dC, N), A.data_ptr(), _ld(A, K), A.shape[0], _ptr(a_row),
      offsets.data_ptr(), G, P, N, K, dW.data_ptr(), _CODES[dW.dtype], int(accumulate))
    return dW


def combine(o: torch.Tensor, pair_pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
            add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """moe_combine: y[t] = sum_j weights[t][j] * o[pair_pos[t][j]] + add[t].
    o [P][d], pair_pos int32 [T][k], weights fp32 [T][k] (None: ones), add
    [T][d] (None: none). Returns y [T][d]."""
    c = _Call(o, "o", stream)
    if o.dim() != 2 or not isinstance(pair_pos, torch.Tensor) or pair_pos.dim() != 2:
        raise ValueError("o must be [P][d] and pair_pos [T][k]")
    (P, d), (T, k) = o.shape, pair_pos.shape
    _sizes(P, d, T, k)
    c.rows(o, "o", (P, d))
    c.need(pair_pos, "pair_pos", torch.int32, (T, k))
    if weights is not None:
        c.need(weights, "weights", torch.float32, (T, k))
    if add is not None:
        c.rows(add, "add", (T, d), torch.float32)
    y = c.result(out, "out", (T, d), out_dtype)
    c("moe_combine", c.code, o.data_ptr(), _ld(o, d), P, pair_pos.data_ptr(), _ptr(weights), T, k, d, _ptr(add),
      c.code if add is None else _CODES[add.dtype], _ld(add, d), y.data_ptr(), _CODES[y.dtype], _ld(y, d))
    return y


def combine_backward(dy: torch.Tensor, o: torch.Tensor, pair_pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
                     d_o: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None, stream=None):
    """moe_combine_backward: (d_o [P][d], dw fp32 [T][k]) with d_o[pair_pos[t][j]]
    = weights[t][j] * dy[t] and dw[t][j] = <dy[t], o[pair_pos[t][j]]>. Rows of
    d_o that no pair names are not written. Both are formed; the C call takes NULL
    for the one that is not wanted."""
    c = _Call(dy, "dy", stream)
    if dy.dim() != 2 or not isinstance(o, torch.Tensor) or o.dim() != 2 or not isinstance(pair_pos, torch.Tensor) or pair_pos.dim() != 2:
        raise ValueError("dy must be [T][d], o [P][d] and pair_pos [T][k]")
    (P, d), (T, k) = o.shape, pair_pos.shape
    _sizes(P, d, T, k)
    c.rows(dy, "dy", (T, d))
    c.rows(o, "o", (P, d))
    c.need(pair_pos, "pair_pos", torch.int32, (T, k))
    if weights is not None:
        c.need(weights, "weights", torch.float32, (T, k))
    d_o = c.new((P, d), c.dtype) if d_o is None else c.rows(d_o, "d_o", (P, d))
    dw = c.new((T, k), torch.float32) if dw is None else c.need(dw, "dw", torch.float32, (T, k))
    c("moe_combine_backward", c.code, dy.data_ptr(), _ld(dy, d), o.data_ptr(), _ld(o, d), P, pair_pos.data_ptr(), _ptr(weights),
      T, k, d, d_o.data_ptr(), _ld(d_o, d), dw.data_ptr())
    return d_o, dw


def adapter_plan(row_adapter: torch.Tensor, n: int, stream=None):
    """moe_adapter_plan: (rows int32 [T], offsets int32 [n+1]), the batch's rows
    sorted by adapter (row_adapter int32 [T]; outside [0, n): no adapter, sorted
    behind the others). One plan serves every projection of the batch."""
    _need(row_adapter, "row_adapter", torch.int32, (row_adapter.numel(),))
    if n < 1:
        raise ValueError("n must be at least 1")
    dev, T = row_adapter.device, row_adapter.numel()
    _sizes(T, n)
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream must be of {dev}, got {stream.device}")
    with torch.cuda.stream(torch.cuda.current_stream(dev) if stream is None else stream):
        rows = torch.empty(T, dtype=torch.int32, device=dev)
        offsets = torch.empty(n + 1, dtype=torch.int32, device=dev)
        _check(load().moe_adapter_plan(row_adapter.data_ptr(), T, n, rows.data_ptr(), offsets.data_ptr(),
                                       torch.cuda.current_stream(dev).cuda_stream), "moe_adapter_plan")
    return rows, offsets


def _adapter_args(c: _Call, x, A, B, scale, plan):
    if x.dim() != 2 or not isinstance(A, torch.Tensor) or A.dim() != 3 or not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("x must be [T][K], A [n][r][K] and B [n][N][r]")
    (T, K), (n, r, _), N = x.shape, A.shape, B.shape[1]
    _sizes(T, K, n, r, N)
    c.rows(x, "x", (T, K))
    c.need(A, "A", c.dtype, (n, r, K))
    c.need(B, "B", c.dtype, (n, N, r))
    if scale is not None:
        c.need(scale, "scale", torch.float32, (n,))
    rows, offsets = plan
    c.need(rows, "rows", torch.int32, (T,))
    c.need(offsets, "offsets", torch.int32, (n + 1,))
    return T, K, N, r, n, rows, offsets


def adapter_forward(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: Optional[torch.Tensor], plan,
                    base: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """moe_adapter_forward: y[t] = base[t] + scale[a] * (x[t] @ A[a]^T) @ B[a]^T
    with a the adapter of row t; y[t] = base[t] for rows without one. x [T][K],
    A [n][r][K], B [n][N][r], scale fp32 [n] (None: ones), plan =
    adapter_plan(...), base [T][N] of y's type (None: zeros). out may be base
    itself (in place). Returns y [T][N]."""
    c = _Call(x, "x", stream)
    T, K, N, r, n, rows, offsets = _adapter_args(c, x, A, B, scale, plan)
    if base is not None:
        c.rows(base, "base", (T, N), torch.float32)
        out_dtype = base.dtype if out_dtype is None and out is None else out_dtype
    y = c.result(out, "out", (T, N), out_dtype)
    if base is not None and base.dtype != y.dtype:
        raise TypeError(f"base must be {y.dtype} like the result, got {base.dtype}")
    c("moe_adapter_forward", c.code, x.data_ptr(), _ld(x, K), T, K, N, r, n, A.data_ptr(), B.data_ptr(), _ptr(scale),
      rows.data_ptr(), offsets.data_ptr(), _ptr(base), _ld(base, N), y.data_ptr(), _CODES[y.dtype], _ld(y, N))
    return y


def adapter_backward_workspace_bytes(T: int, r: int) -> int:
    _sizes(T, r)
    return int(load().moe_adapter_backward_workspace_bytes(T, r))


def adapter_backward(dy: torch.Tensor, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: Optional[torch.Tensor],
                     plan, dx_base: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                     dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                     grad_dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                     ws: Optional[torch.Tensor] = None, stream=None):
    """moe_adapter_backward: (dx [T][K], dA [n][r][K], dB [n][N][r]) from dy
    [T][N]. dx_base [T][K] (None: zeros) is added to dx, which is of its type
    (else x's) and may be dx_base itself; dA and dB are of grad_dtype (None:
    x's type), and with accumulate are added to the given dA and dB (fp32). All three
    are formed; the C call takes NULL for those that are not wanted."""
    c = _Call(x, "x", stream)
    T, K, N, r, n, rows, offsets = _adapter_args(c, x, A, B, scale, plan)
    c.rows(dy, "dy", (T, N))
    if dx_base is not None:
        c.rows(dx_base, "dx_base", (T, K), torch.float32)
    dx = c.result(dx, "dx", (T, K), None if dx_base is None else dx_base.dtype)
    if accumulate and (dA is None or dB is None):
        raise ValueError("accumulate needs the tensors to add to in dA and dB")
    dA = c.whole(dA, "dA", (n, r, K), grad_dtype)
    dB = c.whole(dB, "dB", (n, N, r), dA.dtype)
    need = adapter_backward_workspace_bytes(T, r)
    ws = c.workspace(ws, need)
    c("moe_adapter_backward", c.code, dy.data_ptr(), _ld(dy, N), x.data_ptr(), _ld(x, K), T, K, N, r, n, A.data_ptr(),
      B.data_ptr(), _ptr(scale), rows.data_ptr(), offsets.data_ptr(), _ptr(dx_base), _ld(dx_base, K), dx.data_ptr(),
      _CODES[dx.dtype], _ld(dx, K), dA.data_ptr(), dB.data_ptr(), _CODES[dA.dtype], int(accumulate), ws.data_ptr(),
      ws.numel() * ws.element_size())
    return dx, dA, dB


# --------------------------------------------- the block around the experts
# As the operators above: tensors of one device, row-strided views, nothing recorded for autograd.
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5, "geglu": 6}


def _activation(act: str, N: int):
    """(code, columns of the result) of an activation of N columns."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    if act not in ("swiglu", "geglu"):
        return ACTIVATIONS[act], N
    if N % 2:
        raise ValueError(f"{act} needs an even number of columns, got {N}")
    return ACTIVATIONS[act], N // 2


def linear(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
           pre: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_linear: y = act(x @ W^T + bias) + residual. x [T][K], W [N][K], bias
    [N] of x's type or fp32, act a name of ACTIVATIONS ("swiglu" and "geglu":
    curve(z[:, :N/2]) * z[:, N/2:]), residual of y's type (may be `out` itself);
    pre [T][N] of x's type receives x @ W^T + bias for linear_backward.
    Returns y [T][N], or [T][N/2] if gated."""
    c = _Call(x, "x", stream)
    if x.dim() != 2 or not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("x must be [T][K] and W [N][K]")
    (T, K), N = x.shape, W.shape[0]
    _sizes(T, N, K)
    code, cols = _activation(act, N)
    ldx = c.ld(x, "x", (T, K))
    c.need(W, "W", c.dtype, (N, K))
    b = r = z = None
    b_code, ldr, ldz = c.code, 0, 0
    if bias is not None:
        b, b_code = c.vector(bias, "bias", (N,)).data_ptr(), _CODES[bias.dtype]
    if residual is not None:
        ldr = c.ld(residual, "residual", (T, cols), torch.float32)
        r = residual.data_ptr()
        out_dtype = residual.dtype if out_dtype is None and out is None else out_dtype
    if out is None:
        y, ldy = c.new((T, cols), c._type(out_dtype, "out")), cols
    else:
        y = c.result(out, "out", (T, cols), out_dtype)
        ldy = _ld(y, cols)
    if residual is not None and residual.dtype != y.dtype:
        raise TypeError(f"residual must be {y.dtype} like the result, got {residual.dtype}")
    if pre is not None:
        ldz = c.ld(pre, "pre", (T, N))
        z = pre.data_ptr()
    c("moe_linear", c.code, x.data_ptr(), ldx, T, N, K, W.data_ptr(), b, b_code, code, r, ldr, z, ldz, y.data_ptr(), _CODES[y.dtype], ldy)
    return y


_ROUND_DZ = 0x100


def linear_backward_workspace_bytes(T: int, N: int, K: int, act: str = "none", round_dz: bool = False) -> int:
    _sizes(T, N, K)
    return int(load().moe_linear_backward_workspace_bytes(T, N, K, _activation(act, N)[0] | (_ROUND_DZ if round_dz else 0)))


def linear_backward(dy: torch.Tensor, x: Optional[torch.Tensor], W: Optional[torch.Tensor], pre: Optional[torch.Tensor] = None,
                    act: str = "none", bias_grad: bool = False, dx: Union[torch.Tensor, bool, None] = None, dW: Union[torch.Tensor, bool, None] = None,
                    db: Optional[torch.Tensor] = None, grad_dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                    ws: Optional[torch.Tensor] = None, stream=None, round_dz: bool = False):
    """moe_linear_backward: (dx [T][K], dW [N][K], db [N] or None) from dy
    [T][columns of y] and pre [T][N], which linear wrote (not needed without
    activation). db is formed with bias_grad or where it is given; dW and db are of
    grad_dtype (None: x's type), and with accumulate are added to the given ones
    (fp32). dx=False or dW=False: that one is not formed, and W or x may be None;
    None stands in its place. round_dz: the gradient of `pre` is rounded to x's type
    before the products, in about half the time (MOE_ACT_ROUND_DZ)."""
    c = _Call(dy, "dy", stream)
    if (dy.dim() != 2 or (not isinstance(x, torch.Tensor) or x.dim() != 2) and not (x is None and dW is False and W is not None)
            or (not isinstance(W, torch.Tensor) or W.dim() != 2) and not (W is None and dx is False and x is not None)):
        raise ValueError("dy must be [T][columns], x [T][K] (None only with dW=False) and W [N][K] (None only with dx=False)")
    T, K = dy.shape[0], (x if W is None else W).shape[1]
    N = W.shape[0] if W is not None else 2 * dy.shape[1] if act in ("swiglu", "geglu") else dy.shape[1]
    _sizes(T, N, K)
    code, cols = _activation(act, N)
    lddy, ldx = c.ld(dy, "dy", (T, cols)), K
    if x is not None:
        ldx = c.ld(x, "x", (T, K))
    if W is not None:
        c.need(W, "W", c.dtype, (N, K))
    z, ldz = None, 0
    if code:
        if pre is None:
            raise ValueError(f"{act} needs pre, which linear wrote")
        ldz = c.ld(pre, "pre", (T, N))
        z = pre.data_ptr()
    bias_grad = bias_grad or db is not None
    if accumulate and (dW is None or (bias_grad and db is None)):
        raise ValueError("accumulate needs the tensors to add to in dW and db")
    if dx is False and dW is False and not bias_grad:
        raise ValueError("one of dx, dW and db must be wanted")
    dx = None if dx is False else c.result(dx, "dx", (T, K), None)
    dW = None if dW is False else c.whole(dW, "dW", (N, K), grad_dtype)
    db = c.whole(db, "db", (N,), grad_dtype if dW is None else dW.dtype) if bias_grad else None
    sums = dW if dW is not None else db
    if round_dz:
        code |= _ROUND_DZ
    ws = c.workspace(ws, int(load().moe_linear_backward_workspace_bytes(T, N, K, code)))
    c("moe_linear_backward", c.code, dy.data_ptr(), lddy, _ptr(x), ldx, T, N, K, _ptr(W), z, ldz, code, _ptr(dx),
      c.code if dx is None else _CODES[dx.dtype], _ld(dx, K), _ptr(dW), _ptr(db), c.code if sums is None else _CODES[sums.dtype], int(accumulate), ws.data_ptr(),
      ws.numel() * ws.element_size())
    return dx, dW, db


def _norm_args(c: _Call, T: int, d: int, w_o, gate, w_n):
    """(their type's code, rows of gate, three addresses) of w_o and w_n [d] and gate [gates][d] or [d], all of one type."""
    dtype, gates, g = None, 1, None
    if w_o is not None:
        dtype = c.vector(w_o, "w_o", (d,)).dtype
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a torch.Tensor")
        gates = 1 if gate.dim() == 1 else gate.shape[0]
        if gates < 1 or T % gates:
            raise ValueError(f"gate must have a number of rows that divides {T}, got {gates}")
        c.vector(gate, "gate", (d,) if gate.dim() == 1 else (gates, d))
        if dtype is not None and gate.dtype is not dtype:
            raise TypeError(f"gate must be {dtype} like the other weights, got {gate.dtype}")
        dtype, g = gate.dtype, gate.data_ptr()
    if w_n is not None:
        c.vector(w_n, "w_n", (d,))
        if dtype is not None and w_n.dtype is not dtype:
            raise TypeError(f"w_n must be {dtype} like the other weights, got {w_n.dtype}")
        dtype = w_n.dtype
    return (c.code if dtype is None else _CODES[dtype]), gates, (None if w_o is None else w_o.data_ptr()), g, (None if w_n is None else w_n.data_ptr())


def residual_norm(o: Optional[torch.Tensor], x: Optional[torch.Tensor], w_o: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, scale: float = 1.0, w_n: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  y: Optional[torch.Tensor] = None, n: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None, stream=None):
    """moe_residual_norm: (y, n) with y = scale * x + gate * norm(o) * w_o and
    n = norm(y) * w_n. o [T][d] (the block's output) or None (before the first
    block), x [T][d] (the residual stream, of o's type or fp32) or None, w_o None:
    o itself, gate [d] or [gates][d] (each row for T / gates consecutive rows)
    or None, w_n None: no norm behind (n is None). w_o, gate and w_n are of one
    type, o's or fp32. y is of x's type (without x: o's) and may be x itself; n
    is of o's type and may be o itself. Without o, y is formed only where it is
    given, and n is of `dtype` (None: x's, which then must not be fp32)."""
    lead, name = (o, "o") if o is not None else (x, "x")
    if lead is None:
        raise ValueError("o or x must be given")
    if o is None and isinstance(x, torch.Tensor) and x.dtype is torch.float32:
        if dtype is None:
            raise TypeError("n's type must be given in dtype where x is float32 and o is None")
        lead = torch.empty(0, dtype=dtype, device=x.device)
    c = _Call(lead, name, stream)
    if dtype is not None and dtype is not c.dtype:
        raise TypeError(f"dtype must be {c.dtype}, got {dtype}")
    first = o if o is not None else x
    if first.dim() != 2:
        raise ValueError(f"{name} must be [T][d]")
    T, d = first.shape
    shape = (T, d)
    _sizes(T, d)
    ldo = ldx = ldy = ldn = 0
    f32 = torch.float32
    stream_type = c.dtype
    if o is not None:
        ldo = c.ld(o, "o", shape)
    if x is not None:
        ldx = c.ld(x, "x", shape, f32)
        stream_type = x.dtype
    elif y is not None:
        stream_type = y.dtype
    wcode, gates, p_o, p_g, p_n = _norm_args(c, T, d, w_o, gate, w_n)
    if y is not None:
        ldy = c.ld(y, "y", shape, f32)
        if y.dtype is not stream_type:
            raise TypeError(f"y must be {stream_type} like x, got {y.dtype}")
    elif o is not None:
        y, ldy = c.new(shape, stream_type), d
    if w_n is None:
        if n is not None or y is None:
            raise ValueError("n needs w_n, and without o one of y and w_n must be given")
    elif n is None:
        n, ldn = c.new(shape, c.dtype), d
    else:
        ldn = c.ld(n, "n", shape)
    c("moe_residual_norm", c.code, None if o is None else o.data_ptr(), ldo, None if x is None else x.data_ptr(), ldx, _CODES[stream_type], T, d,
      p_o, p_g, gates, p_n, wcode, scale, eps, None if y is None else y.data_ptr(), ldy, None if n is None else n.data_ptr(), ldn)
    return y, n


def residual_norm_backward_workspace_bytes(T: int, d: int, gates: int = 1) -> int:
    _sizes(T, d, gates)
    return int(load().moe_residual_norm_backward_workspace_bytes(T, d, gates))


def residual_norm_backward(dy: Optional[torch.Tensor], dn: Optional[torch.Tensor], o: Optional[torch.Tensor], y: Optional[torch.Tensor],
                           w_o: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                           w_n: Optional[torch.Tensor] = None, eps: float = 1e-6, dx: Union[torch.Tensor, bool, None] = None,
                           d_o: Union[torch.Tensor, bool, None] = None, dw_o: Union[torch.Tensor, bool, None] = None,
                           dgate: Union[torch.Tensor, bool, None] = None, dw_n: Union[torch.Tensor, bool, None] = None, grad_dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                           ws: Optional[torch.Tensor] = None, stream=None):
    """moe_residual_norm_backward: (dx, d_o, dw_o, dgate, dw_n) from dy and dn,
    the gradients of residual_norm's y (None: zeros) and n (None: no norm behind;
    then w_n and y are not read). o, w_o, gate, scale, w_n and eps as there; y is
    what it wrote (or x, where it formed n alone with scale 1). Those of what the
    forward call did not have are None. dx is of dy's type (without it y's) and may be
    dy itself; dw_o, dgate and dw_n are of grad_dtype (None: the weights' type), and with
    accumulate are added to the given ones (fp32). Those given as False are not formed, and
    None stands in their places."""
    lead, name = next(((t, n) for t, n in ((o, "o"), (dn, "dn"), (dy, "dy")) if t is not None), (None, None))
    if lead is None:
        raise ValueError("dy or dn must be given")
    c = _Call(lead, name, stream)
    if lead.dim() != 2:
        raise ValueError(f"{name} must be [T][d]")
    T, d = lead.shape
    _sizes(T, d)
    if dn is None:
        if dy is None:
            raise ValueError("dy or dn must be given")
        y = w_n = None
    elif w_n is None or y is None:
        raise ValueError("dn needs w_n and y")
    shape, f32 = (T, d), torch.float32
    stream_type = (dy if dy is not None else y).dtype
    lddy = lddn = ldo = ldy = lddo = 0
    p_dy = p_dn = p_of = p_y = p_do = None
    if dy is not None:
        lddy, p_dy = c.ld(dy, "dy", shape, f32), dy.data_ptr()
    if dn is not None:
        lddn, p_dn = c.ld(dn, "dn", shape), dn.data_ptr()
        ldy, p_y = c.ld(y, "y", shape, f32), y.data_ptr()
        if y.dtype is not stream_type:
            raise TypeError(f"y must be {stream_type} like dy, got {y.dtype}")
    if o is None:
        w_o = gate = None
    else:
        ldo, p_of = c.ld(o, "o", shape), o.data_ptr()
    wcode, gates, p_o, p_g, p_n = _norm_args(c, T, d, w_o, gate, w_n)
    dx = None if dx is False else c.result(dx, "dx", shape, stream_type)
    if d_o is False:
        d_o = None
    elif o is not None:
        d_o = c.new(shape, c.dtype) if d_o is None else c.rows(d_o, "d_o", shape)
        lddo, p_do = _ld(d_o, d), d_o.data_ptr()
    elif d_o is not None:
        raise ValueError("d_o has nothing that it is the gradient of")
    grads, ptrs, gcode = [], [], c.code
    for w, g, what in ((w_o, dw_o, "dw_o"), (gate, dgate, "dgate"), (w_n, dw_n, "dw_n")):
        if w is None or g is False:
            if g is not None and g is not False:
                raise ValueError(f"{what} has nothing that it is the gradient of")
            grads.append(None)
            ptrs.append(None)
            continue
        if g is None and accumulate:
            raise ValueError(f"accumulate needs the tensor to add to in {what}")
        g = c.whole(g, what, w.shape, w.dtype if grad_dtype is None else grad_dtype)
        grads.append(g)
        ptrs.append(g.data_ptr())
        gcode = _CODES[g.dtype]
    if dx is None and d_o is None and not any(ptrs):
        raise ValueError("one of the gradients must be wanted")
    p_ws, ws_bytes = None, 0
    if any(ptrs):
        ws = c.workspace(ws, int(load().moe_residual_norm_backward_workspace_bytes(T, d, gates)))
        p_ws, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    c("moe_residual_norm_backward", c.code, p_dy, lddy, p_dn, lddn, p_of, ldo, p_y, ldy, _CODES[stream_type], T, d, p_o, p_g, gates, p_n, wcode, scale,
      eps, _ptr(dx), _ld(dx, d), p_do, lddo, *ptrs, gcode, int(accumulate), p_ws, ws_bytes)
    return (dx, d_o, *grads)


MAX_FEW_TOKENS, MAX_FEW_PAIRS = 64, 512


def few_tokens_workspace_bytes(T: int, dtype: torch.dtype, d: int, f: int, E: int, k: int, f_sh: int = 0) -> int:
    _sizes(T, d, f, E, k, f_sh)
    L = MoeLayer16T(_CODES[dtype], d, f, E, k, f_sh, None, None, None, None)
    return int(load().moe_few_tokens_workspace_bytes(ctypes.byref(L), T))


def few_tokens_layer(x: torch.Tensor, logits: torch.Tensor, gu: torch.Tensor, dn: torch.Tensor, k: int,
                     sh_gu: Optional[torch.Tensor] = None, sh_dn: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                     topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_few_tokens_layer: the whole layer with 16-bit weights for at most
    MAX_FEW_TOKENS tokens (and MAX_FEW_PAIRS picks), y = sum of the k picked
    experts' FFN weighted by their gates + the shared expert's + add. x [T][d],
    logits fp32 [T][E], gu [E][2f][d] (rows 0 .. f-1 the gate's), dn [E][d][f], sh_gu
    [2 f_sh][d] and sh_dn [d][f_sh] (None: no shared expert), add of y's type [T][d]
    (may be `out` itself). topk_ids int32 and topk_w fp32 [T][k] receive the picks
    and their gates where given. Returns y [T][d]."""
    c = _Call(x, "x", stream)
    if x.dim() != 2 or not isinstance(gu, torch.Tensor) or gu.dim() != 3 or not isinstance(dn, torch.Tensor) or dn.dim() != 3:
        raise ValueError("x must be [T][d], gu [E][2f][d] and dn [E][d][f]")
    (T, d), (E, _, f) = x.shape, dn.shape
    if (sh_gu is None) != (sh_dn is None):
        raise ValueError("sh_gu and sh_dn are given together")
    if sh_dn is not None and (not isinstance(sh_dn, torch.Tensor) or sh_dn.dim() != 2):
        raise ValueError("sh_gu must be [2 f_sh][d] and sh_dn [d][f_sh]")
    f_sh = 0 if sh_dn is None else sh_dn.shape[1]
    _sizes(T, d, f, E, k, f_sh)
    c.rows(x, "x", (T, d))
    c.need(logits, "logits", torch.float32, (T, E))
    c.need(gu, "gu", c.dtype, (E, 2 * f, d))
    c.need(dn, "dn", c.dtype, (E, d, f))
    if f_sh:
        c.need(sh_gu, "sh_gu", c.dtype, (2 * f_sh, d))
        c.need(sh_dn, "sh_dn", c.dtype, (d, f_sh))
    if add is not None:
        c.rows(add, "add", (T, d), torch.float32)
        out_dtype = add.dtype if out_dtype is None and out is None else out_dtype
    if topk_ids is not None:
        c.need(topk_ids, "topk_ids", torch.int32, (T, k))
    if topk_w is not None:
        c.need(topk_w, "topk_w", torch.float32, (T, k))
    y = c.result(out, "out", (T, d), out_dtype)
    if add is not None and add.dtype != y.dtype:
        raise TypeError(f"add must be {y.dtype} like the result, got {add.dtype}")
    L = MoeLayer16T(c.code, d, f, E, k, f_sh, gu.data_ptr(), dn.data_ptr(), _ptr(sh_gu), _ptr(sh_dn))
    ws = c.workspace(ws, int(load().moe_few_tokens_workspace_bytes(ctypes.byref(L), T)))
    c("moe_few_tokens_layer", ctypes.byref(L), x.data_ptr(), _ld(x, d), logits.data_ptr(), T, _ptr(add), _ld(add, d), y.data_ptr(),
      _CODES[y.dtype], _ld(y, d), _ptr(topk_ids), _ptr(topk_w), ws.data_ptr(), ws.numel() * ws.element_size())
    return y
