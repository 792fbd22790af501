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
from typing import Dict, Optional

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


class _Call:
    """One call: its device and stream, and the checks of its tensors."""

    __slots__ = ("dtype", "device", "index", "code", "stream", "given")

    def __init__(self, lead: torch.Tensor, name: str, stream):
        if not isinstance(lead, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
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
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.given):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def __call__(self, what, *args):
        f = getattr(_lib or load(), what)
        if torch.cuda.current_device() == self.index:
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
    if ws is None:
        ws = c.new(max(need, 1), torch.uint8)
    elif ws.device != c.device:
        raise ValueError(f"ws must be on {c.device}, got {ws.device}")
    elif not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    c("moe_adapter_backward", c.code, dy.data_ptr(), _ld(dy, N), x.data_ptr(), _ld(x, K), T, K, N, r, n, A.data_ptr(),
      B.data_ptr(), _ptr(scale), rows.data_ptr(), offsets.data_ptr(), _ptr(dx_base), _ld(dx_base, K), dx.data_ptr(),
      _CODES[dx.dtype], _ld(dx, K), dA.data_ptr(), dB.data_ptr(), _CODES[dA.dtype], int(accumulate), ws.data_ptr(),
      ws.numel() * ws.element_size())
    return dx, dA, dB
