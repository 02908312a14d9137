"""Thin Python binding of libcolimoe (include/coli_moe.h).

Every function here only marshals arguments to the C ABI function of the same
name; all computation on the device happens in the library's CUDA kernels.
Device buffers are torch CUDA tensors (PyTorch serves as the allocator and the
stream source); host buffers are numpy arrays.  Importing this package loads the
in-tree ``libcolimoe.so`` and raises if it is missing: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

__all__ = [
    "ColiError", "COLI_F32", "COLI_BF16", "COLI_PATH_AUTO", "COLI_PATH_GEMV",
    "COLI_PATH_GEMM", "COLI_PATH_FUSED", "COLI_PATH_TWOPASS", "lib", "EXPORTS",
    "coli_moe_last_error", "coli_moe_quantize", "coli_moe_expert_bytes",
    "coli_moe_pack_expert", "coli_moe_quantize_expert_device", "coli_moe_layer_create",
    "coli_moe_layer_destroy", "coli_moe_workspace_size", "coli_moe_route",
    "coli_moe_union", "coli_moe_forward", "coli_moe_forward_ex", "coli_moe_rmsnorm",
    "coli_moe_stack_workspace_size", "coli_moe_stack_forward", "coli_moe_dequant_debug",
    "coli_moe_forward_noalloc", "NOALLOC_SCRATCH_BYTES", "coli_moe_status", "Desc",
    "coli_moe_layer_set_topp", "coli_moe_layer_set_partition",
    "COLI_GATE_NONE", "COLI_GATE_CHANNEL", "COLI_GATE_TOKEN", "COLI_GATE_FULL", "NormDesc",
    "COLI_MXFP4", "COLI_NVFP4", "COLI_ACT_NONE", "COLI_ACT_SWIGLU",
    "coli_moe_sort_workspace_size", "coli_moe_sort", "coli_moe_dispatch",
    "coli_moe_dispatch_backward", "coli_moe_combine", "coli_moe_combine_backward",
    "coli_moe_block_norm", "coli_moe_block_norm_backward_workspace_size",
    "coli_moe_block_norm_backward", "coli_moe_fp4_bytes", "coli_moe_fp4_quantize",
    "coli_moe_fp4_product_workspace_size", "coli_moe_fp4_product",
    "coli_moe_fp4_product_status", "coli_moe_fp4_set_wait_test",
    "coli_moe_block_norm_set_wait_test",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcolimoe.so")

COLI_F32, COLI_BF16 = 0, 1
COLI_PATH_AUTO, COLI_PATH_GEMV, COLI_PATH_GEMM, COLI_PATH_FUSED, COLI_PATH_TWOPASS = 0, 1, 2, 3, 4
COLI_GATE_NONE, COLI_GATE_CHANNEL, COLI_GATE_TOKEN, COLI_GATE_FULL = 0, 1, 2, 3
COLI_MXFP4, COLI_NVFP4 = 0, 1
COLI_ACT_NONE, COLI_ACT_SWIGLU = 0, 1

# every symbol include/coli_moe.h declares
EXPORTS = (
    "coli_moe_last_error", "coli_moe_quantize", "coli_moe_expert_bytes",
    "coli_moe_pack_expert", "coli_moe_quantize_expert_device", "coli_moe_layer_create",
    "coli_moe_layer_destroy", "coli_moe_workspace_size", "coli_moe_route",
    "coli_moe_union", "coli_moe_forward", "coli_moe_forward_ex", "coli_moe_rmsnorm",
    "coli_moe_stack_workspace_size", "coli_moe_stack_forward", "coli_moe_dequant_debug",
    "coli_moe_forward_noalloc", "coli_moe_status", "coli_moe_host_workspace_size",
    "coli_moe_forward_host", "coli_moe_stack_host_workspace_size", "coli_moe_stack_forward_host",
    "coli_moe_quantize_expert_fp8_device", "coli_moe_quantize8", "coli_moe_expert_bytes8",
    "coli_moe_pack_expert8", "coli_moe_layer_set_topp", "coli_moe_layer_set_partition",
    "coli_moe_quantize_expert8_device", "coli_moe_layer_set_wait_test", "coli_moe_union_readback",
    "coli_moe_sort_workspace_size", "coli_moe_sort", "coli_moe_dispatch",
    "coli_moe_dispatch_backward", "coli_moe_combine", "coli_moe_combine_backward",
    "coli_moe_block_norm", "coli_moe_block_norm_backward_workspace_size",
    "coli_moe_block_norm_backward", "coli_moe_fp4_bytes", "coli_moe_fp4_quantize",
    "coli_moe_fp4_product_workspace_size", "coli_moe_fp4_product",
    "coli_moe_fp4_product_status", "coli_moe_fp4_set_wait_test",
    "coli_moe_block_norm_set_wait_test",
)


class ColiError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libcolimoe error {code}: {msg}")
        self.code = code


class Desc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("group", ctypes.c_int32), ("routed_scale", ctypes.c_float),
                ("norm_topk", ctypes.c_int32), ("router_w", ctypes.c_void_p),
                ("router_b", ctypes.c_void_p), ("experts", ctypes.c_void_p),
                ("bits", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    """coli_norm_desc; post_gain and pre_gain are device addresses or None."""
    _fields_ = [("H", ctypes.c_int32), ("xt", ctypes.c_int32), ("bt", ctypes.c_int32),
                ("post_norm", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("eps", ctypes.c_float),
                ("post_gain", ctypes.c_void_p), ("pre_gain", ctypes.c_void_p)]


from . import build as _build  # noqa: E402

if _build.stale():
    try:
        _build.build()
    except Exception as exc:  # no fallback: the CUDA library is the product
        raise ImportError(f"{LIB_PATH} is missing or stale and nvcc failed: {exc}") from exc

lib = ctypes.CDLL(LIB_PATH)

_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "coli_moe_last_error": ([], ctypes.c_char_p),
    "coli_moe_quantize": ([_P, _I64, _I64, _I32, _P, _P], ctypes.c_int),
    "coli_moe_expert_bytes": ([_I32, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_pack_expert": ([_I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "coli_moe_quantize_expert_device": ([_I32, _I32, _I32, _P, _P, _P, _P, _P], ctypes.c_int),
    "coli_moe_quantize_expert8_device": ([_I32, _I32, _I32, _P, _P, _P, _P, _P], ctypes.c_int),
    "coli_moe_quantize_expert_fp8_device": ([_I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P],
                                            ctypes.c_int),
    "coli_moe_quantize8": ([_P, _I64, _I64, _I32, _P, _P], ctypes.c_int),
    "coli_moe_expert_bytes8": ([_I32, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_pack_expert8": ([_I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "coli_moe_layer_create": ([ctypes.POINTER(Desc), ctypes.POINTER(_P)], ctypes.c_int),
    "coli_moe_layer_destroy": ([_P], ctypes.c_int),
    "coli_moe_layer_set_topp": ([_P, ctypes.c_float], ctypes.c_int),
    "coli_moe_layer_set_wait_test": ([_P, _I32], ctypes.c_int),
    "coli_moe_layer_set_partition": ([_P, _I32, _I32, _I32, _P], ctypes.c_int),
    "coli_moe_workspace_size": ([_P, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_route": ([_P, _P, ctypes.c_int, _I32, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "coli_moe_union": ([_P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "coli_moe_forward": ([_P, _P, ctypes.c_int, _I32, _P, _P, _SZ, _P], ctypes.c_int),
    "coli_moe_forward_ex": ([_P, _P, ctypes.c_int, _I32, _P, _P, ctypes.c_int, _P, _P, _P,
                             _P, _SZ, _P], ctypes.c_int),
    "coli_moe_rmsnorm": ([_P, _I32, _I32, ctypes.c_float, _P, _P], ctypes.c_int),
    "coli_moe_stack_workspace_size": ([_P, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_stack_forward": ([_P, _I32, _P, _I32, ctypes.c_float, ctypes.c_int, _P, _SZ,
                                _P], ctypes.c_int),
    "coli_moe_dequant_debug": ([_P, _I32, _I32, _P, _P], ctypes.c_int),
    "coli_moe_union_readback": ([_P, _I32, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "coli_moe_forward_noalloc": ([_P, _P, ctypes.c_int, _I32, _P, _P], ctypes.c_int),
    "coli_moe_status": ([_P, _I32, _P, ctypes.POINTER(_I32), _P], ctypes.c_int),
    "coli_moe_host_workspace_size": ([_P, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_forward_host": ([_P, _P, ctypes.c_int, _I32, _P, ctypes.c_int, _P, _SZ, _P],
                              ctypes.c_int),
    "coli_moe_stack_host_workspace_size": ([_P, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_stack_forward_host": ([_P, _I32, _P, _P, _I32, ctypes.c_float, ctypes.c_int, _P,
                                     _SZ, _P], ctypes.c_int),
    "coli_moe_sort_workspace_size": ([_I32, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_sort": ([_P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "coli_moe_dispatch": ([_P, ctypes.c_int, _I32, _I32, _I32, _P, _P, _P], ctypes.c_int),
    "coli_moe_dispatch_backward": ([_P, ctypes.c_int, _I32, _I32, _I32, _P, _P, _P], ctypes.c_int),
    "coli_moe_combine": ([_P, ctypes.c_int, _I32, _I32, _I32, _P, _P, _P, _P, ctypes.c_int, _P],
                         ctypes.c_int),
    "coli_moe_combine_backward": ([_P, ctypes.c_int, _P, ctypes.c_int, _I32, _I32, _I32, _P, _P,
                                   _P, _P, _P], ctypes.c_int),
    "coli_moe_block_norm": ([ctypes.POINTER(NormDesc), _P, _P, _P, _I32, _P, _P, _P, _P, _P],
                            ctypes.c_int),
    "coli_moe_block_norm_backward_workspace_size": ([ctypes.POINTER(NormDesc), _I32,
                                                     ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_block_norm_backward": ([ctypes.POINTER(NormDesc), _P, _P, _P, _I32, _P, _P, _P, _P,
                                      _P, _P, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "coli_moe_fp4_bytes": ([ctypes.c_int, _I64, _I32, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)],
                           ctypes.c_int),
    "coli_moe_fp4_quantize": ([ctypes.c_int, _P, ctypes.c_int, _I64, _I64, _I32, ctypes.c_int, _P,
                               _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "coli_moe_fp4_product_workspace_size": ([ctypes.c_int, _I64, _I32, _I32, _I32,
                                             ctypes.POINTER(_SZ)], ctypes.c_int),
    "coli_moe_fp4_product": ([ctypes.c_int, _P, _P, _I64, _I32, _P, _P, _I32, _I32, _P, _P, _P,
                              ctypes.c_int, _P, _SZ, _P], ctypes.c_int),
    "coli_moe_fp4_product_status": ([_P, ctypes.POINTER(_I32), _P], ctypes.c_int),
    "coli_moe_fp4_set_wait_test": ([_I32], ctypes.c_int),
    "coli_moe_block_norm_set_wait_test": ([_I32], ctypes.c_int),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


def coli_moe_last_error() -> str:
    return lib.coli_moe_last_error().decode()


def _ok(rc: int):
    if rc != 0:
        raise ColiError(rc, coli_moe_last_error())


def _ptr(a):
    """Device or host address of a torch tensor / numpy array / int / None."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        assert a.flags["C_CONTIGUOUS"]
        return a.ctypes.data
    assert a.is_contiguous(), "tensors passed to libcolimoe must be contiguous"
    return a.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return s if isinstance(s, int) else s.cuda_stream


def _xtype(x):
    import torch
    if x.dtype == torch.float32:
        return COLI_F32
    if x.dtype == torch.bfloat16:
        return COLI_BF16
    raise TypeError(f"activations must be float32 or bfloat16, got {x.dtype}")


# ---------------------------------------------------------------------------
def coli_moe_quantize(w: np.ndarray, group: int):
    """Host quantiser -> (packed uint8 [R, K/2], scales f32 [R, K/G])."""
    w = np.ascontiguousarray(w, np.float32)
    R, K = w.shape
    ng = 1 if group == 0 else max(K // group, 1)
    packed = np.zeros((R, K // 2), np.uint8)
    scales = np.zeros((R, ng), np.float32)
    _ok(lib.coli_moe_quantize(_ptr(w), R, K, group, _ptr(packed), _ptr(scales)))
    return packed, scales


def coli_moe_expert_bytes(H: int, I: int, group: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_expert_bytes(H, I, group, ctypes.byref(out)))
    return out.value


def coli_moe_pack_expert(H, I, group, gate_codes, gate_scales, up_codes, up_scales,
                         down_codes, down_scales) -> np.ndarray:
    blob = np.zeros((coli_moe_expert_bytes(H, I, group),), np.uint8)
    arrs = [np.ascontiguousarray(a) for a in
            (gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales)]
    _ok(lib.coli_moe_pack_expert(H, I, group, *[_ptr(a) for a in arrs], _ptr(blob)))
    return blob


def coli_moe_quantize8(w: np.ndarray, group: int):
    """Host 8-bit quantiser -> (codes int8 [R, K], scales f32 [R, K/G])."""
    w = np.ascontiguousarray(w, np.float32)
    R, K = w.shape
    ng = 1 if group == 0 else max(K // group, 1)
    codes = np.zeros((R, K), np.int8)
    scales = np.zeros((R, ng), np.float32)
    _ok(lib.coli_moe_quantize8(_ptr(w), R, K, group, _ptr(codes), _ptr(scales)))
    return codes, scales


def coli_moe_expert_bytes8(H: int, I: int, group: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_expert_bytes8(H, I, group, ctypes.byref(out)))
    return out.value


def coli_moe_pack_expert8(H, I, group, gate_codes, gate_scales, up_codes, up_scales,
                          down_codes, down_scales) -> np.ndarray:
    blob = np.zeros((coli_moe_expert_bytes8(H, I, group),), np.uint8)
    arrs = [np.ascontiguousarray(a) for a in
            (gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales)]
    _ok(lib.coli_moe_pack_expert8(H, I, group, *[_ptr(a) for a in arrs], _ptr(blob)))
    return blob


def coli_moe_quantize_expert_device(H, I, group, gate, up, down, blob, stream=None):
    _ok(lib.coli_moe_quantize_expert_device(H, I, group, _ptr(gate), _ptr(up), _ptr(down),
                                            _ptr(blob), _stream(stream)))


def coli_moe_quantize_expert8_device(H, I, group, gate, up, down, blob, stream=None):
    _ok(lib.coli_moe_quantize_expert8_device(H, I, group, _ptr(gate), _ptr(up), _ptr(down),
                                             _ptr(blob), _stream(stream)))


def coli_moe_quantize_expert_fp8_device(H, I, group, gate, up, down, gate_bs, up_bs, down_bs,
                                        blob, stream=None):
    """FP8 E4M3 codes (uint8 device tensors) with 128 x 128 block scales -> int4 blob."""
    _ok(lib.coli_moe_quantize_expert_fp8_device(H, I, group, _ptr(gate), _ptr(up), _ptr(down),
                                                _ptr(gate_bs), _ptr(up_bs), _ptr(down_bs),
                                                _ptr(blob), _stream(stream)))


def coli_moe_layer_create(desc: Desc) -> ctypes.c_void_p:
    h = _P()
    _ok(lib.coli_moe_layer_create(ctypes.byref(desc), ctypes.byref(h)))
    return h


def coli_moe_layer_destroy(layer) -> None:
    _ok(lib.coli_moe_layer_destroy(layer))


def coli_moe_layer_set_wait_test(layer, withhold_stage: int) -> None:
    """Test only: make the fused kernel's bounded waits run out (see the header)."""
    _ok(lib.coli_moe_layer_set_wait_test(layer, withhold_stage))


def coli_moe_layer_set_topp(layer, p: float) -> None:
    _ok(lib.coli_moe_layer_set_topp(layer, p))


def coli_moe_layer_set_partition(layer, e_begin: int, e_end: int, with_shared: bool,
                                 experts) -> None:
    _ok(lib.coli_moe_layer_set_partition(layer, e_begin, e_end, int(bool(with_shared)),
                                         _ptr(experts)))


def coli_moe_workspace_size(layer, T: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_workspace_size(layer, T, ctypes.byref(out)))
    return out.value


def coli_moe_route(layer, x, T, idx, w, ws, stream=None):
    _ok(lib.coli_moe_route(layer, _ptr(x), _xtype(x), T, _ptr(idx), _ptr(w), _ptr(ws),
                           ws.numel() * ws.element_size(), _stream(stream)))


def coli_moe_union(idx, T, k, E, offsets, pair_tok, pair_slot, uniq, n_uniq, stream=None):
    _ok(lib.coli_moe_union(_ptr(idx), T, k, E, _ptr(offsets), _ptr(pair_tok),
                           _ptr(pair_slot), _ptr(uniq), _ptr(n_uniq), _stream(stream)))


def coli_moe_forward(layer, x, T, y, ws, stream=None):
    _ok(lib.coli_moe_forward(layer, _ptr(x), _xtype(x), T, _ptr(y), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)))


COLI_STAGES = 5
STAGE_NAMES = ("router", "union", "gateup", "down", "combine")


def coli_moe_forward_ex(layer, x, T, y, ws, residual=None, path=COLI_PATH_AUTO, idx_out=None,
                        w_out=None, events=None, stream=None):
    """events: None or COLI_STAGES + 1 torch.cuda.Event(enable_timing=True)."""
    ev = None
    if events is not None:
        assert len(events) == COLI_STAGES + 1
        for e in events:          # torch creates the CUDA event on its first record
            if not e.cuda_event:
                e.record()
        ev = (_P * len(events))(*[e.cuda_event for e in events])
    _ok(lib.coli_moe_forward_ex(layer, _ptr(x), _xtype(x), T, _ptr(y), _ptr(residual), path,
                                _ptr(idx_out), _ptr(w_out), ev, _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream)))


def coli_moe_rmsnorm(x, T, H, eps, out, stream=None):
    _ok(lib.coli_moe_rmsnorm(_ptr(x), T, H, eps, _ptr(out), _stream(stream)))


def _layer_array(layers):
    arr = (_P * len(layers))(*[l.value if isinstance(l, _P) else l for l in layers])
    return arr


def coli_moe_stack_workspace_size(layers, T: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_stack_workspace_size(_layer_array(layers), len(layers), T,
                                          ctypes.byref(out)))
    return out.value


def coli_moe_stack_forward(layers, x, T, eps, ws, path=COLI_PATH_AUTO, stream=None):
    _ok(lib.coli_moe_stack_forward(_layer_array(layers), len(layers), _ptr(x), T, eps, path,
                                   _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def coli_moe_host_workspace_size(layer, T: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_host_workspace_size(layer, T, ctypes.byref(out)))
    return out.value


def coli_moe_forward_host(layer, x_host, T, y_host, ws, path=COLI_PATH_AUTO, stream=None):
    """x_host / y_host: host tensors (page-locked for graph capture); ws on the device."""
    _ok(lib.coli_moe_forward_host(layer, _ptr(x_host), _xtype(x_host), T, _ptr(y_host), path,
                                  _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def coli_moe_stack_host_workspace_size(layers, T: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_stack_host_workspace_size(_layer_array(layers), len(layers), T,
                                               ctypes.byref(out)))
    return out.value


def coli_moe_stack_forward_host(layers, x_host, y_host, T, eps, ws, path=COLI_PATH_AUTO,
                                stream=None):
    _ok(lib.coli_moe_stack_forward_host(_layer_array(layers), len(layers), _ptr(x_host),
                                        _ptr(y_host), T, eps, path, _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)))


def coli_moe_status(layer, T: int, ws, stream=None) -> int:
    """Error flags of the last forward on this workspace (raises on a timeout);
    ws None: the built-in scratch array of coli_moe_forward_noalloc."""
    flags = _I32(0)
    _ok(lib.coli_moe_status(layer, T, _ptr(ws), ctypes.byref(flags), _stream(stream)))
    return flags.value


def coli_moe_union_readback(layer, T: int, ws, offsets=None, pair_tok=None, pair_slot=None,
                            uniq=None, n_uniq=None, inv=None, stream=None):
    """Test helper: the union the last forward on ws built (see the header)."""
    _ok(lib.coli_moe_union_readback(layer, T, _ptr(ws), _ptr(offsets), _ptr(pair_tok),
                                    _ptr(pair_slot), _ptr(uniq), _ptr(n_uniq), _ptr(inv),
                                    _stream(stream)))


def coli_moe_dequant_debug(layer, expert: int, which: int, out, stream=None):
    _ok(lib.coli_moe_dequant_debug(layer, expert, which, _ptr(out), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 8 << 20  # COLI_NOALLOC_SCRATCH_BYTES in include/coli_moe.h


def coli_moe_forward_noalloc(layer, x, T, y, stream=None):
    """Forward without a caller workspace, for hosts that cannot allocate device
    memory: the library's built-in scratch array is used instead (see the header
    for its limit and for the rule that overlapping calls must be serialised)."""
    _ok(lib.coli_moe_forward_noalloc(layer, _ptr(x), _xtype(x), T, _ptr(y), _stream(stream)))


# ---------------------------------------------------------------------------
# Operators around the experts (see the header).  Tensors are checked against
# the sizes given, so that a wrong shape raises here instead of reading past a
# buffer on the device.
# ---------------------------------------------------------------------------
_torch = _INT32 = _FLOAT32 = _BFLOAT16 = _UINT8 = None


def _load_torch():
    global _torch, _INT32, _FLOAT32, _BFLOAT16, _UINT8
    import torch
    torch.cuda.init()
    _INT32, _FLOAT32, _BFLOAT16, _UINT8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    _torch = torch


def _device():
    """Index of the current CUDA device."""
    if _torch is None:
        _load_torch()
    return _torch._C._cuda_getDevice()


def _queue(s, dev):
    """Address of the stream s, or of the current one of the device."""
    if s is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    return s if isinstance(s, int) else s.cuda_stream


def _buf(name, a, dtype, count, dev):
    """Address of a contiguous tensor of at least `count` elements of dtype on the CUDA device
    dev (None passes)."""
    if a is None:
        return None
    if a.dtype is dtype and a.get_device() == dev and a.is_contiguous() and a.numel() >= count:
        return a.data_ptr()
    if a.dtype != dtype:
        raise TypeError(f"{name}: {a.dtype}, expected {dtype}")
    if a.get_device() != dev:
        raise ValueError(f"{name}: on {a.device}, expected the current CUDA device {dev}")
    raise ValueError(f"{name}: {tuple(a.shape)} (contiguous: {a.is_contiguous()}), expected {count} contiguous elements")


def _code_of(dtype):
    if dtype is _BFLOAT16:
        return COLI_BF16
    if dtype is _FLOAT32:
        return COLI_F32
    raise TypeError(f"rows must be float32 or bfloat16, got {dtype}")


def _workspace(ws, dev):
    return (None, 0) if ws is None else (_buf("ws", ws, _UINT8, 0, dev), ws.numel())


def coli_moe_sort_workspace_size(T: int, k: int, E: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_sort_workspace_size(T, k, E, ctypes.byref(out)))
    return out.value


def coli_moe_sort(idx, T, k, E, offsets, pair_tok, pair_slot, inv, ws, w=None, stream=None):
    """pair_tok and pair_slot may be None; ws: uint8 of coli_moe_sort_workspace_size bytes."""
    d, n = _device(), T * k
    p, size = _workspace(ws, d)
    _ok(lib.coli_moe_sort(_buf("idx", idx, _INT32, n, d), _buf("w", w, _FLOAT32, n, d), T, k, E,
                          _buf("offsets", offsets, _INT32, E + 1, d), _buf("pair_tok", pair_tok, _INT32, n, d),
                          _buf("pair_slot", pair_slot, _INT32, n, d), _buf("inv", inv, _INT32, n, d), p, size,
                          _queue(stream, d)))


def coli_moe_dispatch(x, T, H, k, inv, xs, stream=None):
    d = _device()
    _ok(lib.coli_moe_dispatch(_buf("x", x, x.dtype, T * H, d), _code_of(x.dtype), T, H, k,
                              _buf("inv", inv, _INT32, T * k, d), _buf("xs", xs, x.dtype, T * k * H, d),
                              _queue(stream, d)))


def coli_moe_dispatch_backward(dxs, T, H, k, inv, dx, stream=None):
    d = _device()
    _ok(lib.coli_moe_dispatch_backward(_buf("dxs", dxs, dxs.dtype, T * k * H, d),
                                       _code_of(dxs.dtype), T, H, k, _buf("inv", inv, _INT32, T * k, d),
                                       _buf("dx", dx, dxs.dtype, T * H, d), _queue(stream, d)))


def coli_moe_combine(o, T, H, k, inv, w, y, residual=None, stream=None):
    d = _device()
    _ok(lib.coli_moe_combine(_buf("o", o, o.dtype, T * k * H, d), _code_of(o.dtype), T, H, k,
                             _buf("inv", inv, _INT32, T * k, d), _buf("w", w, _FLOAT32, T * k, d),
                             _buf("residual", residual, y.dtype, T * H, d),
                             _buf("y", y, y.dtype, T * H, d), _code_of(y.dtype),
                             _queue(stream, d)))


def coli_moe_combine_backward(dy, o, T, H, k, inv, w, d_o, dw, stream=None):
    """o, d_o or dw may be None (see the header)."""
    like = d_o if d_o is not None else o
    if like is None:
        raise ValueError("combine_backward: neither o nor d_o")
    d = _device()
    _ok(lib.coli_moe_combine_backward(_buf("dy", dy, dy.dtype, T * H, d), _code_of(dy.dtype),
                                      _buf("o", o, like.dtype, T * k * H, d),
                                      _code_of(like.dtype), T, H, k, _buf("inv", inv, _INT32, T * k, d),
                                      _buf("w", w, _FLOAT32, T * k, d),
                                      _buf("d_o", d_o, like.dtype, T * k * H, d),
                                      _buf("dw", dw, _FLOAT32, T * k, d), _queue(stream, d)))


def _norm_type(code):
    if code == COLI_F32:
        return _FLOAT32
    if code == COLI_BF16:
        return _BFLOAT16
    raise ValueError(f"NormDesc: bad type {code}")


def _gate_size(desc, T):
    kind = desc.gate_kind
    return (desc.H if kind == COLI_GATE_CHANNEL else T if kind == COLI_GATE_TOKEN
            else T * desc.H if kind == COLI_GATE_FULL else 0)


def coli_moe_block_norm(desc, x, o, T, x_out, n_out, gate=None, rstd_post=None, rstd_pre=None,
                        stream=None):
    d, n = _device(), T * desc.H
    xt, bt = _norm_type(desc.xt), _norm_type(desc.bt)
    _ok(lib.coli_moe_block_norm(desc, _buf("x", x, xt, n, d), _buf("o", o, bt, n, d),
                                _buf("gate", gate, _FLOAT32, _gate_size(desc, T), d), T,
                                _buf("x_out", x_out, xt, n, d), _buf("n_out", n_out, bt, n, d),
                                _buf("rstd_post", rstd_post, _FLOAT32, T, d),
                                _buf("rstd_pre", rstd_pre, _FLOAT32, T, d), _queue(stream, d)))


def coli_moe_block_norm_backward_workspace_size(desc, T: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_block_norm_backward_workspace_size(desc, T, ctypes.byref(out)))
    return out.value


def coli_moe_block_norm_backward(desc, x_out, o, T, dx_out, dn, dx, d_o, ws, gate=None,
                                 rstd_post=None, rstd_pre=None, dpost_gain=None, dgate=None,
                                 dpre_gain=None, stream=None):
    d, n, ng = _device(), T * desc.H, _gate_size(desc, T)
    xt, bt = _norm_type(desc.xt), _norm_type(desc.bt)
    p, size = _workspace(ws, d)
    _ok(lib.coli_moe_block_norm_backward(
        desc, _buf("x_out", x_out, xt, n, d), _buf("o", o, bt, n, d), _buf("gate", gate, _FLOAT32, ng, d), T,
        _buf("rstd_post", rstd_post, _FLOAT32, T, d), _buf("rstd_pre", rstd_pre, _FLOAT32, T, d),
        _buf("dx_out", dx_out, xt, n, d), _buf("dn", dn, bt, n, d), _buf("dx", dx, xt, n, d),
        _buf("d_o", d_o, bt, n, d), _buf("dpost_gain", dpost_gain, _FLOAT32, desc.H, d),
        _buf("dgate", dgate, _FLOAT32, ng, d), _buf("dpre_gain", dpre_gain, _FLOAT32, desc.H, d), p, size,
        _queue(stream, d)))


def coli_moe_block_norm_set_wait_test(withhold: int) -> None:
    """Test of the gradient's bounded waits (see the header); < 0: off."""
    _ok(lib.coli_moe_block_norm_set_wait_test(withhold))


def coli_moe_fp4_bytes(fmt: int, rows: int, K: int):
    """(bytes of the codes, bytes of the scales) of a matrix [rows, K]."""
    nc, ns = _SZ(), _SZ()
    _ok(lib.coli_moe_fp4_bytes(fmt, rows, K, ctypes.byref(nc), ctypes.byref(ns)))
    return nc.value, ns.value


def _fp4_sizes(fmt, rows, K):
    """coli_moe_fp4_bytes without a call: the sizes that tensors are checked against here (the
    library checks fmt, rows and K themselves)."""
    words = -(-K // (64 if fmt == COLI_NVFP4 else 128))
    return rows * K // 2, -(-rows // 128) * words * 512


def coli_moe_fp4_quantize(fmt, x, rows, K, codes, scales, act=COLI_ACT_NONE, src=None, count=None,
                          gscale=None, values=None, stream=None):
    """x: [n, K] rows ([n, 2K] for SwiGLU), n >= rows unless src picks them."""
    d = _device()
    nc, ns = _fp4_sizes(fmt, rows, K)
    n_src = x.numel() // max(1, 2 * K if act == COLI_ACT_SWIGLU else K)
    _ok(lib.coli_moe_fp4_quantize(fmt, _buf("x", x, x.dtype, 0, d), _code_of(x.dtype), n_src, rows,
                                  K, act, _buf("src", src, _INT32, rows, d), _buf("count", count, _INT32, 1, d),
                                  _buf("gscale", gscale, _FLOAT32, 1, d), _buf("codes", codes, _UINT8, nc, d),
                                  _buf("scales", scales, _UINT8, ns, d),
                                  _buf("values", values, x.dtype, rows * K, d),
                                  _queue(stream, d)))


def coli_moe_fp4_product_workspace_size(fmt: int, P: int, K: int, E: int, R: int) -> int:
    out = _SZ()
    _ok(lib.coli_moe_fp4_product_workspace_size(fmt, P, K, E, R, ctypes.byref(out)))
    return out.value


def coli_moe_fp4_product(fmt, x_codes, x_scales, P, K, w_codes, w_scales, E, R, y, ws,
                         offsets=None, alpha=None, stream=None):
    d = _device()
    xc, xs = _fp4_sizes(fmt, P, K)
    wc, wsc = _fp4_sizes(fmt, E * R, K)
    p, n = _workspace(ws, d)
    _ok(lib.coli_moe_fp4_product(fmt, _buf("x_codes", x_codes, _UINT8, xc, d),
                                 _buf("x_scales", x_scales, _UINT8, xs, d), P, K,
                                 _buf("w_codes", w_codes, _UINT8, wc, d),
                                 _buf("w_scales", w_scales, _UINT8, wsc, d), E, R,
                                 _buf("offsets", offsets, _INT32, E + 1, d), _buf("alpha", alpha, _FLOAT32, E, d),
                                 _buf("y", y, y.dtype, P * R, d), _code_of(y.dtype), p, n,
                                 _queue(stream, d)))


def coli_moe_fp4_product_status(ws, stream=None) -> int:
    """0, or raises when a product that used ws gave up a wait since ws was last cleared."""
    flags, d = _I32(0), _device()
    _ok(lib.coli_moe_fp4_product_status(_buf("ws", ws, _UINT8, 8, d), ctypes.byref(flags),
                                        _queue(stream, d)))
    return flags.value


def coli_moe_fp4_set_wait_test(withhold: int) -> None:
    """Test of the product's bounded waits (see the header); < 0: off."""
    _ok(lib.coli_moe_fp4_set_wait_test(withhold))
