"""GB300 MoE token path: Python binding of libmoeroute.so.

The five calls of the MoE token path (route, dispatch layout, pack, receiver
permute, combine) run in hand-written sm_103a kernels behind a C ABI
(``include/moe_route.h``).  This module only marshals torch tensors (device
pointers, sizes, the current CUDA stream) through ctypes, or for the training,
expert and norm calls through compiled entry points; PyTorch supplies
device memory and streams.  There is no fallback: if the library is not
built, importing works but every call raises ``MoeLibraryMissing``.

Function names and argument order follow the C ABI; sizes are read from the
tensor shapes.  bf16 arrays may be torch.bfloat16, torch.int16 or
torch.uint16 tensors (the bits are what matters).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

import numpy as np
import torch

from . import _build

__all__ = [
    "MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_CAPACITY", "MOE_ERR_BAD_EXPERT_ID",
    "MOE_ERR_TIMEOUT", "MOE_ERR_CUDA", "status_bit", "MoeError", "MoeLibraryMissing",
    "build", "load_library", "library_path", "moe_version", "moe_workspace_bytes",
    "moe_dispatch_layout_kernels", "moe_permute_to_experts_kernels", "moe_dispatch_kernels",
    "moe_dispatch", "moe_dispatch_quantized", "moe_dispatch_quantized_kernels",
    "moe_dispatch_pack_permute", "moe_dispatch_pack_permute_kernels",
    "moe_dispatch_pack_permute_masked", "moe_dispatch_pack_permute_masked_kernels",
    "moe_dispatch_masked", "moe_dispatch_masked_kernels", "MOE_FORMAT_MXFP8",
    "MOE_FORMAT_NVFP4",
    "moe_route_topk", "moe_dispatch_layout", "moe_dispatch_pack", "moe_permute_to_experts",
    "moe_combine", "moe_expert_scale", "moe_permute_to_experts_masked", "moe_combine_stage1",
    "moe_combine_stage2", "moe_dispatch_pack_mxfp8", "moe_expert_scale_mxfp8",
    "moe_plan_placement", "moe_workspace_bytes_mapped", "moe_dispatch_layout_mapped", "Placement",
    "moe_dispatch_pack_routed", "moe_routed_expert_stage1", "moe_dispatch_pack_nvfp4",
    "moe_expert_scale_nvfp4", "nvfp4_record_bytes", "mxfp8_record_bytes", "HostPipeline",
    "MOE_TYPE_F32", "MOE_TYPE_BF16", "moe_balance_loss", "moe_balance_loss_workspace_bytes",
    "moe_route_backward", "moe_combine_backward", "moe_w4_bytes", "moe_w4_pack",
    "moe_expert_product_w4", "moe_expert_product_w4_workspace_bytes",
    "moe_expert_product", "moe_expert_product_workspace_bytes", "moe_expert_product_backward",
    "moe_expert_product_backward_workspace_bytes", "moe_rms_norm", "moe_rms_norm_backward",
    "moe_rms_norm_backward_workspace_bytes",
    "MoePath", "trace_enable", "trace_disable", "trace_reset", "trace_records",
]

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_CAPACITY = 2
MOE_ERR_BAD_EXPERT_ID = 3
MOE_ERR_TIMEOUT = 4
MOE_ERR_CUDA = 5
MOE_FORMAT_MXFP8 = 1
MOE_FORMAT_NVFP4 = 2
MOE_TYPE_F32 = 0
MOE_TYPE_BF16 = 1


def status_bit(code: int) -> int:
    """Bit that a data error of kind `code` sets in the device status word."""
    return 1 << code


class MoeError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code


class MoeLibraryMissing(RuntimeError):
    pass


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libmoeroute.so for sm_103a (in-tree) and return its path."""
    return _build.build(force=force, verbose=verbose)


def load_library() -> ctypes.CDLL:
    """Load libmoeroute.so (raises MoeLibraryMissing if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise MoeLibraryMissing(
                f"{path} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        P, i32, sz, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
        sigs = {
            "moe_version": ([], ctypes.c_int),
            "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "moe_last_error_message": ([], ctypes.c_char_p),
            "moe_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
            "moe_dispatch_layout_kernels": ([i32, i32, i32, i32, i32], ctypes.c_int),
            "moe_permute_to_experts_kernels": ([i32, i32, i32, i32, i32], ctypes.c_int),
            "moe_dispatch_kernels": ([i32, i32, i32, i32, i32], ctypes.c_int),
            "moe_dispatch_quantized_kernels": ([i32, i32, i32, i32, i32], ctypes.c_int),
            "moe_dispatch_pack_permute_kernels": ([i32, i32, i32, i32, i32], ctypes.c_int),
            "moe_dispatch_pack_permute_masked_kernels": ([i32, i32, i32, i32, i32, i32],
                                                         ctypes.c_int),
            "moe_dispatch_masked_kernels": ([i32, i32, i32, i32, i32, i32], ctypes.c_int),
            "moe_dispatch_masked": ([P, P, i32, i32, i32, i32, i32, i32, i32, i32, i32, P, P, P, P,
                                     P, P, P, P, P, P, P, P, P, P, sz, P, P], ctypes.c_int),
            "moe_dispatch_pack_permute_masked": ([P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                                  i32, i32, i32, P, P, P, P, P, P, P, P],
                                                 ctypes.c_int),
            "moe_dispatch_pack_permute": ([P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                           i32, i32, P, P, P, P, P, P, P, sz, P, P], ctypes.c_int),
            "moe_dispatch_quantized": ([P, P, i32, i32, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                        i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P, P, P,
                                        sz, P, P], ctypes.c_int),
            "moe_dispatch": ([P, P, i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, P, P, P, P,
                              P, P, P, P, P, P, P, P, P, P, sz, P, P], ctypes.c_int),
            "moe_route_topk": ([P, i32, i32, i32, i32, P, P, P], ctypes.c_int),
            "moe_dispatch_layout": ([P, i32, i32, i32, i32, i32, P, P, P, P, P, P, sz, P, P],
                                    ctypes.c_int),
            "moe_dispatch_layout_static": ([P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P],
                                           ctypes.c_int),
            "moe_dispatch_pack": ([P, i32, i32, i32, i32, P, P, i32, P, P, P, P], ctypes.c_int),
            "moe_permute_to_experts": ([P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                        i32, i32, P, P, P, P, P, sz, P, P], ctypes.c_int),
            "moe_combine": ([P, i32, P, P, i32, i32, i32, i32, P, P, P], ctypes.c_int),
            "moe_combine_stage1": ([P, i32, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32, P,
                                    P, P], ctypes.c_int),
            "moe_combine_stage2": ([P, P, i32, i32, i32, i32, i32, i32, P, P, P], ctypes.c_int),
            "moe_dispatch_pack_mxfp8": ([P, i32, i32, i32, i32, P, P, i32, P, P, P, P],
                                         ctypes.c_int),
            "moe_expert_scale_mxfp8": ([P, P, P, i32, i32, i32, P, P], ctypes.c_int),
            "moe_plan_placement": ([P, i32, i32, i32, P, P, P, P], ctypes.c_int),
            "moe_dispatch_pack_nvfp4": ([P, i32, i32, i32, i32, ctypes.c_float, P, P, i32, P, P, P,
                                         P], ctypes.c_int),
            "moe_expert_scale_nvfp4": ([P, P, P, i32, i32, ctypes.c_float, i32, P, P],
                                       ctypes.c_int),
            "moe_dispatch_pack_routed": ([P, P, P, i32, i32, i32, i32, i32, P, P, i32, P, P, P, P,
                                          P, P], ctypes.c_int),
            "moe_routed_expert_stage1": ([P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32, P, P,
                                          P, P], ctypes.c_int),
            "moe_workspace_bytes_mapped": ([i32, i32, i32, i32, i32, i32], ctypes.c_size_t),
            "moe_dispatch_layout_mapped": ([P, i32, i32, i32, i32, i32, i32, P, P, i32, P, P, P, P,
                                            P, P, P, ctypes.c_size_t, P, P], ctypes.c_int),
            "moe_permute_to_experts_masked": ([P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                               i32, i32, P, P, P, P, P, P], ctypes.c_int),
            "moe_expert_scale": ([P, P, P, i32, i32, i32, P, P], ctypes.c_int),
            "moe_balance_loss_workspace_bytes": ([i32, i32, i32], sz),
            "moe_balance_loss": ([P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, sz, P, P],
                                 ctypes.c_int),
            "moe_route_backward": ([P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P],
                                   ctypes.c_int),
            "moe_combine_backward": ([P, P, i32, P, P, P, i32, i32, i32, i32, P, P, P, P],
                                     ctypes.c_int),
            "moe_w4_pack": ([P, P, i32, i32, i32, i32, P, sz, P], ctypes.c_int),
            "moe_expert_product_w4": ([P, i32, P, P, i32, P, P, i32, i32, i32, i32, P, P, sz, P, P],
                                      ctypes.c_int),
            "moe_w4_bytes": ([i32, i32, i32, i32], sz),
            "moe_expert_product_w4_workspace_bytes": ([i32, i32, i32, i32], sz),
            "moe_expert_product_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
            "moe_expert_product": ([P, i32, P, P, i32, P, i32, i32, i32, i32, P, P, P, sz, P, P],
                                   ctypes.c_int),
            "moe_expert_product_backward_workspace_bytes": ([i32, i32, i32, i32], sz),
            "moe_expert_product_backward": ([P, P, i32, P, P, i32, P, P, i32, i32, i32, P, P, i32, P,
                                             sz, P, P], ctypes.c_int),
            "moe_rms_norm": ([P, P, i32, P, i32, i64, i32, ctypes.c_float, P, P, P, P], ctypes.c_int),
            "moe_rms_norm_backward_workspace_bytes": ([i64, i32], sz),
            "moe_rms_norm_backward": ([P, P, i32, P, i32, P, i64, i32, ctypes.c_float, P, P, P, P, sz,
                                       P], ctypes.c_int),
            "moe_trace_enable": ([ctypes.c_char_p, i32], ctypes.c_int),
            "moe_trace_disable": ([], None),
            "moe_trace_reset": ([], None),
            "moe_trace_count": ([], ctypes.c_int),
            "moe_trace_get": ([i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float)],
                              ctypes.c_int),
        }
        for name, (args, res) in sigs.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def _check(rc: int):
    if rc != MOE_OK:
        lib = load_library()
        raise MoeError(rc, lib.moe_last_error_message().decode())


def _stream(stream) -> ctypes.c_void_p:
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the current stream's handle without a Stream object around it (0.3 instead of 2.8 us a call)
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


_BF16_TYPES = (torch.bfloat16, torch.int16) + ((torch.uint16,) if hasattr(torch, "uint16") else ())


def _dev(t: torch.Tensor, name: str, dtypes, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got shape {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _status_ptr(dev_status):
    if dev_status is None:
        return ctypes.c_void_p(0)
    return _dev(dev_status, "dev_status", (torch.int32,))


_ops_module = None


def _ops():
    """The compiled entry points (csrc/binding.cpp) of the training, expert and norm calls."""
    global _ops_module
    if _ops_module is None:
        load_library()
        if not os.path.exists(_build.OPS_PATH):
            raise MoeLibraryMissing(
                f"{_build.OPS_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        if _build.ops_built_for() != _build.ops_for():
            raise MoeLibraryMissing(
                f"{_build.OPS_PATH} was built for {_build.ops_built_for()}, this is {_build.ops_for()}; "
                "run `python -c 'import __graft_entry__ as g; g.build()'`")
        spec = importlib.util.spec_from_file_location("_moe_ops", _build.OPS_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _ops_module = module
    return _ops_module


def moe_version() -> int:
    return load_library().moe_version()


def moe_workspace_bytes(S: int, T: int, k: int, E: int, P: int) -> int:
    return int(load_library().moe_workspace_bytes(S, T, k, E, P))


def moe_permute_to_experts_kernels(S: int, T: int, k: int, E: int, P: int) -> int:
    """Kernels one moe_permute_to_experts call enqueues (1: map inside the copy, or 2)."""
    n = int(load_library().moe_permute_to_experts_kernels(S, T, k, E, P))
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, f"moe_permute_to_experts_kernels({S}, {T}, {k}, {E}, {P})")
    return n


def moe_dispatch_layout_kernels(S: int, T: int, k: int, E: int, P: int) -> int:
    """Kernels one moe_dispatch_layout call enqueues on the current device (1 or 2)."""
    n = int(load_library().moe_dispatch_layout_kernels(S, T, k, E, P))
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, f"moe_dispatch_layout_kernels({S}, {T}, {k}, {E}, {P})")
    return n


def moe_route_topk(logits, topk_ids, topk_w, stream=None):
    """logits f32 [S,T,E] -> topk_ids i32 [S,T,k], topk_w f32 [S,T,k]."""
    lib = load_library()
    S, T, E = logits.shape
    k = topk_ids.shape[2]
    _check(lib.moe_route_topk(_dev(logits, "logits", (torch.float32,), 3), S, T, E, k,
                              _dev(topk_ids, "topk_ids", (torch.int32,), 3),
                              _dev(topk_w, "topk_w", (torch.float32,), 3), _stream(stream)))


def moe_dispatch_layout(topk_ids, E, P, expert_counts, expert_rank, part_counts, part_offsets,
                        token_slot, ws, dev_status=None, stream=None):
    """topk_ids i32 [S,T,k] -> expert_counts [S,E], expert_rank [S,T,k], part_counts [S,P],
    part_offsets [S,P+1], token_slot [S,T,P] (all int32); ws is a uint8 device tensor."""
    lib = load_library()
    S, T, k = topk_ids.shape
    _check(lib.moe_dispatch_layout(
        _dev(topk_ids, "topk_ids", (torch.int32,), 3), S, T, k, E, P,
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)),
        _dev(part_counts, "part_counts", (torch.int32,)),
        _dev(part_offsets, "part_offsets", (torch.int32,)),
        _dev(token_slot, "token_slot", (torch.int32,)),
        _dev(ws, "ws", (torch.uint8,)), ws.numel(), _status_ptr(dev_status), _stream(stream)))


def moe_dispatch_pack(x, token_slot, part_offsets, send, send_src, dev_status=None, stream=None):
    """x bf16 [S,T,H] -> send bf16 [S,cap_send,H], send_src i32 [S,cap_send]."""
    lib = load_library()
    S, T, H = x.shape
    P = token_slot.shape[2]
    cap_send = send.shape[1]
    _check(lib.moe_dispatch_pack(
        _dev(x, "x", _BF16_TYPES, 3), S, T, H, P, _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(part_offsets, "part_offsets", (torch.int32,)), cap_send,
        _dev(send, "send", _BF16_TYPES, 3), _dev(send_src, "send_src", (torch.int32,)),
        _status_ptr(dev_status), _stream(stream)))


def mxfp8_record_bytes(H: int) -> int:
    """Bytes of one MXFP8 row record: H E4M3 codes, then H/32 E8M0 block scales."""
    return H + H // 32


def nvfp4_record_bytes(H: int) -> int:
    """Bytes of one NVFP4 row record: H/2 bytes of E2M1 codes, then H/16 E4M3 scales."""
    return H // 2 + H // 16


def moe_dispatch_pack_nvfp4(x, token_slot, part_offsets, send_q, send_src, global_scale=1.0,
                            dev_status=None, stream=None):
    """x bf16 [S,T,H] -> send_q uint8 [S,cap_send,H/2+H/16] NVFP4 records, send_src [S,cap_send]."""
    lib = load_library()
    S, T, H = x.shape
    P = token_slot.shape[2]
    cap_send = send_q.shape[1]
    if send_q.shape[2] != nvfp4_record_bytes(H):
        raise ValueError(f"send_q rows must be {nvfp4_record_bytes(H)} bytes for H={H}")
    _check(lib.moe_dispatch_pack_nvfp4(
        _dev(x, "x", _BF16_TYPES, 3), S, T, H, P, float(global_scale),
        _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(part_offsets, "part_offsets", (torch.int32,)), cap_send,
        _dev(send_q, "send_q", (torch.uint8,), 3), _dev(send_src, "send_src", (torch.int32,)),
        _status_ptr(dev_status), _stream(stream)))


def moe_expert_scale_nvfp4(recv_q, expert_offsets, scale, y, global_scale=1.0, stream=None):
    """Stand-in expert on NVFP4 records: y[r] = bf16(scale[e] * dequant(recv_q[r]))."""
    lib = load_library()
    cap_recv, H = y.shape
    if tuple(recv_q.shape) != (cap_recv, nvfp4_record_bytes(H)):
        raise ValueError("recv_q must be [cap_recv, H/2 + H/16] uint8")
    E = scale.shape[0]
    _check(lib.moe_expert_scale_nvfp4(
        _dev(recv_q, "recv_q", (torch.uint8,), 2),
        _dev(expert_offsets, "expert_offsets", (torch.int32,)),
        _dev(scale, "scale", (torch.float32,)), E, H, float(global_scale), cap_recv,
        _dev(y, "y", _BF16_TYPES, 2), _stream(stream)))


def moe_dispatch_pack_mxfp8(x, token_slot, part_offsets, send_q, send_src, dev_status=None,
                            stream=None):
    """x bf16 [S,T,H] -> send_q uint8 [S,cap_send,H+H/32] MXFP8 records, send_src i32 [S,cap_send]."""
    lib = load_library()
    S, T, H = x.shape
    P = token_slot.shape[2]
    cap_send = send_q.shape[1]
    if send_q.shape[2] != mxfp8_record_bytes(H):
        raise ValueError(f"send_q rows must be {mxfp8_record_bytes(H)} bytes for H={H}")
    _check(lib.moe_dispatch_pack_mxfp8(
        _dev(x, "x", _BF16_TYPES, 3), S, T, H, P, _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(part_offsets, "part_offsets", (torch.int32,)), cap_send,
        _dev(send_q, "send_q", (torch.uint8,), 3), _dev(send_src, "send_src", (torch.int32,)),
        _status_ptr(dev_status), _stream(stream)))


def moe_dispatch_pack_routed(x, topk_ids, topk_w, token_slot, part_offsets, send, send_src,
                             send_ids, send_w, dev_status=None, stream=None):
    """moe_dispatch_pack plus each row's routing: send_ids i32 / send_w f32 [S,cap_send,k]."""
    lib = load_library()
    S, T, H = x.shape
    k = topk_ids.shape[2]
    P = token_slot.shape[2]
    cap_send = send.shape[1]
    _check(lib.moe_dispatch_pack_routed(
        _dev(x, "x", _BF16_TYPES, 3), _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(topk_w, "topk_w", (torch.float32,), 3), S, T, H, k, P,
        _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(part_offsets, "part_offsets", (torch.int32,)), cap_send,
        _dev(send, "send", _BF16_TYPES, 3), _dev(send_src, "send_src", (torch.int32,)),
        _dev(send_ids, "send_ids", (torch.int32,), 3), _dev(send_w, "send_w", (torch.float32,), 3),
        _status_ptr(dev_status), _stream(stream)))


def moe_routed_expert_stage1(send, send_ids, send_w, part_offsets, T, E, recv_part, scale, ret,
                             dev_status=None, stream=None):
    """Routed stand-in expert + stage-1 pre-add: ret [S,cap_send,H] per received row;
    T tokens per source; scale None = identity expert."""
    lib = load_library()
    S, cap_send, H = send.shape
    k = send_ids.shape[2]
    P = part_offsets.shape[1] - 1
    sc = None if scale is None else _dev(scale, "scale", (torch.float32,))
    _check(lib.moe_routed_expert_stage1(
        _dev(send, "send", _BF16_TYPES, 3), _dev(send_ids, "send_ids", (torch.int32,), 3),
        _dev(send_w, "send_w", (torch.float32,), 3),
        _dev(part_offsets, "part_offsets", (torch.int32,)), S, T, cap_send, k, E, P, H,
        recv_part, sc, _dev(ret, "ret", _BF16_TYPES, 3), _status_ptr(dev_status),
        _stream(stream)))


class Placement:
    """A placement of E logical experts on P partitions with Lp slots each.

    copy_offsets [E+1] / copy_slots [n] (CSR of each expert's physical slots),
    slot_expert [P*Lp] (-1 = empty) and part_load [P] (predicted pairs), all
    host numpy arrays; `to(device)` gives the device copies the layout reads.
    """

    def __init__(self, copy_offsets, copy_slots, slot_expert, part_load, P, Lp):
        self.copy_offsets = np.ascontiguousarray(copy_offsets, np.int32)
        self.copy_slots = np.ascontiguousarray(copy_slots, np.int32)
        self.slot_expert = np.ascontiguousarray(slot_expert, np.int32)
        self.part_load = np.ascontiguousarray(part_load, np.int64)
        self.E = self.copy_offsets.size - 1
        self.P, self.Lp = P, Lp
        self.E_phys = P * Lp

    def to(self, device):
        d = torch.device(device)
        return (torch.from_numpy(self.copy_offsets).to(d), torch.from_numpy(self.copy_slots).to(d),
                torch.from_numpy(self.slot_expert).to(d))


def moe_plan_placement(load, P: int, R: int) -> Placement:
    """Host planner: load int64 [E] (pairs per logical expert) -> Placement."""
    lib = load_library()
    load = np.ascontiguousarray(load, np.int64)
    E = load.size
    Lp = E // P + R
    co = np.empty(E + 1, np.int32)
    cs = np.empty(E + P * R, np.int32)
    se = np.empty(P * Lp, np.int32)
    pl = np.empty(P, np.int64)
    vp = lambda a: ctypes.c_void_p(a.ctypes.data)  # noqa: E731
    _check(lib.moe_plan_placement(vp(load), E, P, R, vp(co), vp(cs), vp(se), vp(pl)))
    return Placement(co, cs[:co[-1]], se, pl, P, Lp)


def moe_workspace_bytes_mapped(S: int, T: int, k: int, E: int, P: int, Lp: int) -> int:
    return int(load_library().moe_workspace_bytes_mapped(S, T, k, E, P, Lp))


def moe_dispatch_layout_mapped(topk_ids, E, P, Lp, copy_offsets, copy_slots, phys_ids,
                               expert_counts, expert_rank, part_counts, part_offsets, token_slot,
                               ws, dev_status=None, stream=None):
    """Layout over a placement: topk_ids [S,T,k] logical -> phys_ids [S,T,k] physical slots,
    expert_counts [S,P*Lp] and the other outputs of moe_dispatch_layout over phys_ids."""
    lib = load_library()
    S, T, k = topk_ids.shape
    _check(lib.moe_dispatch_layout_mapped(
        _dev(topk_ids, "topk_ids", (torch.int32,), 3), S, T, k, E, P, Lp,
        _dev(copy_offsets, "copy_offsets", (torch.int32,)),
        _dev(copy_slots, "copy_slots", (torch.int32,)), copy_slots.numel(),
        _dev(phys_ids, "phys_ids", (torch.int32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)),
        _dev(part_counts, "part_counts", (torch.int32,)),
        _dev(part_offsets, "part_offsets", (torch.int32,)),
        _dev(token_slot, "token_slot", (torch.int32,), 3), _dev(ws, "ws", (torch.uint8,)),
        ws.numel(), _status_ptr(dev_status), _stream(stream)))


def moe_permute_to_experts(send, token_slot, topk_ids, expert_counts, expert_rank, E, recv_part,
                           align, recv, expert_offsets, pair_row, recv_pair, ws, dev_status=None,
                           stream=None):
    """send bf16 [S,cap_send,H] -> recv bf16 [cap_recv,H] in expert runs, expert_offsets [E+1],
    pair_row [S,T,k], recv_pair [cap_recv]."""
    lib = load_library()
    S, cap_send, H = send.shape
    _, T, P = token_slot.shape
    k = topk_ids.shape[2]
    cap_recv = recv.shape[0]
    _check(lib.moe_permute_to_experts(
        _dev(send, "send", _BF16_TYPES, 3), _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)), S, T, k, E, P, H, recv_part, align,
        cap_send, cap_recv, _dev(recv, "recv", _BF16_TYPES, 2),
        _dev(expert_offsets, "expert_offsets", (torch.int32,)),
        _dev(pair_row, "pair_row", (torch.int32,)), _dev(recv_pair, "recv_pair", (torch.int32,)),
        _dev(ws, "ws", (torch.uint8,)), ws.numel(), _status_ptr(dev_status), _stream(stream)))


def moe_dispatch(logits, x, E, P, recv_part, align, topk_ids, topk_w, expert_counts, expert_rank,
                 part_counts, part_offsets, token_slot, send, send_src, recv, expert_offsets,
                 pair_row, recv_pair, ws, dev_status=None, stream=None):
    """route + layout + pack + permute in one call (the outputs of the four calls).
    logits fp32 [S,T,E], x bf16 [S,T,H] in; the rest as the four calls."""
    lib = load_library()
    S, T, H = x.shape
    k = topk_ids.shape[2]
    cap_send = send.shape[1]
    cap_recv = recv.shape[0]
    _check(lib.moe_dispatch(
        _dev(logits, "logits", (torch.float32,), 3), _dev(x, "x", _BF16_TYPES, 3), S, T, H, E, k,
        P, recv_part, align, cap_send, cap_recv, _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(topk_w, "topk_w", (torch.float32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)),
        _dev(part_counts, "part_counts", (torch.int32,)),
        _dev(part_offsets, "part_offsets", (torch.int32,)),
        _dev(token_slot, "token_slot", (torch.int32,), 3), _dev(send, "send", _BF16_TYPES, 3),
        _dev(send_src, "send_src", (torch.int32,)), _dev(recv, "recv", _BF16_TYPES, 2),
        _dev(expert_offsets, "expert_offsets", (torch.int32,)),
        _dev(pair_row, "pair_row", (torch.int32,)), _dev(recv_pair, "recv_pair", (torch.int32,)),
        _dev(ws, "ws", (torch.uint8,)), ws.numel(), _status_ptr(dev_status), _stream(stream)))


def moe_dispatch_quantized(logits, x, E, P, fmt, global_scale, recv_part, align, topk_ids, topk_w,
                           expert_counts, expert_rank, part_counts, part_offsets, token_slot,
                           send_q, send_src, recv_q, expert_offsets, pair_row, recv_pair, ws,
                           dev_status=None, stream=None):
    """moe_dispatch with MXFP8 (fmt 1) or NVFP4 (fmt 2) records: send_q uint8
    [S,cap_send,rb], recv_q uint8 [cap_recv,rb]; the rest as moe_dispatch."""
    lib = load_library()
    S, T, H = x.shape
    k = topk_ids.shape[2]
    cap_send = send_q.shape[1]
    cap_recv = recv_q.shape[0]
    _check(lib.moe_dispatch_quantized(
        _dev(logits, "logits", (torch.float32,), 3), _dev(x, "x", _BF16_TYPES, 3), S, T, H, E, k,
        P, int(fmt), float(global_scale), recv_part, align, cap_send, cap_recv,
        _dev(topk_ids, "topk_ids", (torch.int32,), 3), _dev(topk_w, "topk_w", (torch.float32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)),
        _dev(part_counts, "part_counts", (torch.int32,)),
        _dev(part_offsets, "part_offsets", (torch.int32,)),
        _dev(token_slot, "token_slot", (torch.int32,), 3), _dev(send_q, "send_q", (torch.uint8,), 3),
        _dev(send_src, "send_src", (torch.int32,)), _dev(recv_q, "recv_q", (torch.uint8,), 2),
        _dev(expert_offsets, "expert_offsets", (torch.int32,)),
        _dev(pair_row, "pair_row", (torch.int32,)), _dev(recv_pair, "recv_pair", (torch.int32,)),
        _dev(ws, "ws", (torch.uint8,)), ws.numel(), _status_ptr(dev_status), _stream(stream)))


def moe_dispatch_pack_permute(x, token_slot, part_offsets, topk_ids, expert_counts, expert_rank,
                              E, recv_part, align, send, send_src, recv, expert_offsets, pair_row,
                              recv_pair, ws, dev_status=None, stream=None):
    """moe_dispatch_pack + moe_permute_to_experts in one call, for a layout already made."""
    lib = load_library()
    S, T, H = x.shape
    P = token_slot.shape[2]
    k = topk_ids.shape[2]
    cap_send = send.shape[1]
    cap_recv = recv.shape[0]
    _check(lib.moe_dispatch_pack_permute(
        _dev(x, "x", _BF16_TYPES, 3), _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(part_offsets, "part_offsets", (torch.int32,)),
        _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)), S, T, k, E, P, H, recv_part, align,
        cap_send, cap_recv, _dev(send, "send", _BF16_TYPES, 3),
        _dev(send_src, "send_src", (torch.int32,)), _dev(recv, "recv", _BF16_TYPES, 2),
        _dev(expert_offsets, "expert_offsets", (torch.int32,)),
        _dev(pair_row, "pair_row", (torch.int32,)), _dev(recv_pair, "recv_pair", (torch.int32,)),
        _dev(ws, "ws", (torch.uint8,)), ws.numel(), _status_ptr(dev_status), _stream(stream)))


def moe_dispatch_pack_permute_kernels(S, T, k, E, P) -> int:
    """Kernels one moe_dispatch_pack_permute call with these sizes enqueues."""
    n = load_library().moe_dispatch_pack_permute_kernels(S, T, k, E, P)
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_permute_kernels: invalid sizes")
    return n


def moe_dispatch_pack_permute_masked(x, token_slot, part_offsets, topk_ids, expert_counts,
                                     expert_rank, E, recv_part, block_rows, send, send_src, recv,
                                     masked_counts, pair_row, recv_pair, dev_status=None,
                                     stream=None):
    """moe_dispatch_pack + moe_permute_to_experts_masked in one call."""
    lib = load_library()
    S, T, H = x.shape
    P = token_slot.shape[2]
    k = topk_ids.shape[2]
    cap_send = send.shape[1]
    _check(lib.moe_dispatch_pack_permute_masked(
        _dev(x, "x", _BF16_TYPES, 3), _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(part_offsets, "part_offsets", (torch.int32,)),
        _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)), S, T, k, E, P, H, recv_part,
        block_rows, cap_send, _dev(send, "send", _BF16_TYPES, 3),
        _dev(send_src, "send_src", (torch.int32,)), _dev(recv, "recv", _BF16_TYPES, 2),
        _dev(masked_counts, "masked_counts", (torch.int32,)),
        _dev(pair_row, "pair_row", (torch.int32,)), _dev(recv_pair, "recv_pair", (torch.int32,)),
        _status_ptr(dev_status), _stream(stream)))


def moe_dispatch_masked(logits, x, E, P, recv_part, block_rows, topk_ids, topk_w, expert_counts,
                        expert_rank, part_counts, part_offsets, token_slot, send, send_src, recv,
                        masked_counts, pair_row, recv_pair, ws, dev_status=None, stream=None):
    """route + layout + pack + masked permute in one call (the outputs of the four
    calls).  logits fp32 [S,T,E], x bf16 [S,T,H] in; the rest as the four calls."""
    lib = load_library()
    S, T, H = x.shape
    k = topk_ids.shape[2]
    cap_send = send.shape[1]
    _check(lib.moe_dispatch_masked(
        _dev(logits, "logits", (torch.float32,), 3), _dev(x, "x", _BF16_TYPES, 3), S, T, H, E, k,
        P, recv_part, block_rows, cap_send, _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(topk_w, "topk_w", (torch.float32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)),
        _dev(part_counts, "part_counts", (torch.int32,)),
        _dev(part_offsets, "part_offsets", (torch.int32,)),
        _dev(token_slot, "token_slot", (torch.int32,), 3), _dev(send, "send", _BF16_TYPES, 3),
        _dev(send_src, "send_src", (torch.int32,)), _dev(recv, "recv", _BF16_TYPES, 2),
        _dev(masked_counts, "masked_counts", (torch.int32,)),
        _dev(pair_row, "pair_row", (torch.int32,)), _dev(recv_pair, "recv_pair", (torch.int32,)),
        _dev(ws, "ws", (torch.uint8,)), ws.numel(), _status_ptr(dev_status), _stream(stream)))


def moe_dispatch_masked_kernels(S, T, k, E, P, recv_part) -> int:
    """Kernels one moe_dispatch_masked call with these sizes enqueues on the current device."""
    n = load_library().moe_dispatch_masked_kernels(S, T, k, E, P, recv_part)
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_dispatch_masked_kernels: invalid sizes")
    return n


def moe_dispatch_pack_permute_masked_kernels(S, T, k, E, P, recv_part) -> int:
    """Kernels one moe_dispatch_pack_permute_masked call with these sizes enqueues."""
    n = load_library().moe_dispatch_pack_permute_masked_kernels(S, T, k, E, P, recv_part)
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_permute_masked_kernels: invalid sizes")
    return n


def moe_dispatch_quantized_kernels(S, T, k, E, P) -> int:
    """Kernels one moe_dispatch_quantized call with these sizes enqueues on the current device."""
    n = load_library().moe_dispatch_quantized_kernels(S, T, k, E, P)
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_dispatch_quantized_kernels: invalid sizes")
    return n


def moe_dispatch_kernels(S, T, k, E, P) -> int:
    """Kernels one moe_dispatch call with these sizes enqueues on the current device."""
    n = load_library().moe_dispatch_kernels(S, T, k, E, P)
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_dispatch_kernels: invalid sizes")
    return n


def moe_permute_to_experts_masked(send, token_slot, topk_ids, expert_counts, expert_rank, E,
                                  recv_part, block_rows, recv, masked_counts, pair_row, recv_pair,
                                  dev_status=None, stream=None):
    """Masked layout: recv bf16 [blocks*block_rows, H] with one fixed block per expert of the
    receiving set, masked_counts [blocks], pair_row [S,T,k], recv_pair [blocks*block_rows]."""
    lib = load_library()
    S, cap_send, H = send.shape
    _, T, P = token_slot.shape
    k = topk_ids.shape[2]
    _check(lib.moe_permute_to_experts_masked(
        _dev(send, "send", _BF16_TYPES, 3), _dev(token_slot, "token_slot", (torch.int32,), 3),
        _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(expert_counts, "expert_counts", (torch.int32,)),
        _dev(expert_rank, "expert_rank", (torch.int32,)), S, T, k, E, P, H, recv_part,
        block_rows, cap_send, _dev(recv, "recv", _BF16_TYPES, 2),
        _dev(masked_counts, "masked_counts", (torch.int32,)),
        _dev(pair_row, "pair_row", (torch.int32,)), _dev(recv_pair, "recv_pair", (torch.int32,)),
        _status_ptr(dev_status), _stream(stream)))


def moe_combine(y, pair_row, topk_w, out, dev_status=None, stream=None):
    """out[s,t] = bf16(sum_j topk_w[s,t,j] * y[pair_row[s,t,j]]) with fp32 accumulation."""
    lib = load_library()
    S, T, k = pair_row.shape
    H = out.shape[2]
    _check(lib.moe_combine(_dev(y, "y", _BF16_TYPES, 2), y.shape[0],
                           _dev(pair_row, "pair_row", (torch.int32,), 3),
                           _dev(topk_w, "topk_w", (torch.float32,), 3), S, T, k, H,
                           _dev(out, "out", _BF16_TYPES, 3), _status_ptr(dev_status),
                           _stream(stream)))


def moe_combine_stage1(y, pair_row, topk_w, topk_ids, token_slot, E, recv_part, ret,
                       dev_status=None, stream=None):
    """Pre-add per (token, partition) slot: ret bf16 [S, cap_send, H] in the send layout."""
    lib = load_library()
    S, T, k = pair_row.shape
    P = token_slot.shape[2]
    _, cap_send, H = ret.shape
    _check(lib.moe_combine_stage1(
        _dev(y, "y", _BF16_TYPES, 2), y.shape[0], _dev(pair_row, "pair_row", (torch.int32,), 3),
        _dev(topk_w, "topk_w", (torch.float32,), 3), _dev(topk_ids, "topk_ids", (torch.int32,), 3),
        _dev(token_slot, "token_slot", (torch.int32,), 3), S, T, k, E, P, H, recv_part, cap_send,
        _dev(ret, "ret", _BF16_TYPES, 3), _status_ptr(dev_status), _stream(stream)))


def moe_combine_stage2(ret, token_slot, out, dev_status=None, stream=None, recv_part=-1):
    """Home-side sum of a token's returned rows (from the receiving set): out bf16 [S, T, H]."""
    lib = load_library()
    S, cap_send, H = ret.shape
    _, T, P = token_slot.shape
    _check(lib.moe_combine_stage2(
        _dev(ret, "ret", _BF16_TYPES, 3), _dev(token_slot, "token_slot", (torch.int32,), 3), S, T,
        P, H, recv_part, cap_send, _dev(out, "out", _BF16_TYPES, 3), _status_ptr(dev_status),
        _stream(stream)))


def moe_expert_scale(recv, expert_offsets, scale, y, stream=None):
    """Stand-in expert (not a step of the method): y[r] = bf16(recv[r] * scale[expert of r])."""
    lib = load_library()
    cap_recv, H = recv.shape
    E = scale.shape[0]
    _check(lib.moe_expert_scale(_dev(recv, "recv", _BF16_TYPES, 2),
                                _dev(expert_offsets, "expert_offsets", (torch.int32,)),
                                _dev(scale, "scale", (torch.float32,)), E, H, cap_recv,
                                _dev(y, "y", _BF16_TYPES, 2), _stream(stream)))


def moe_expert_scale_mxfp8(recv_q, expert_offsets, scale, y, stream=None):
    """Stand-in expert on MXFP8 records: y[r] = bf16(scale[e] * dequant(recv_q[r]))."""
    lib = load_library()
    cap_recv, H = y.shape
    if tuple(recv_q.shape) != (cap_recv, mxfp8_record_bytes(H)):
        raise ValueError("recv_q must be [cap_recv, H + H/32] uint8")
    E = scale.shape[0]
    _check(lib.moe_expert_scale_mxfp8(
        _dev(recv_q, "recv_q", (torch.uint8,), 2),
        _dev(expert_offsets, "expert_offsets", (torch.int32,)),
        _dev(scale, "scale", (torch.float32,)), E, H, cap_recv, _dev(y, "y", _BF16_TYPES, 2),
        _stream(stream)))


def trace_enable(kernel_filter: str | None = None, max_records: int = 4096):
    """Bracket this library's kernel launches (names containing kernel_filter) with CUDA events."""
    lib = load_library()
    _check(lib.moe_trace_enable(kernel_filter.encode() if kernel_filter else None, max_records))


def trace_disable():
    load_library().moe_trace_disable()


def trace_reset():
    load_library().moe_trace_reset()


def trace_records() -> list[tuple[str, float]]:
    """(kernel name, milliseconds) of every traced launch since enable/reset (waits for them)."""
    lib = load_library()
    out = []
    name = ctypes.c_char_p()
    ms = ctypes.c_float()
    for i in range(lib.moe_trace_count()):
        _check(lib.moe_trace_get(i, ctypes.byref(name), ctypes.byref(ms)))
        out.append((name.value.decode(), float(ms.value)))
    return out


def moe_balance_loss_workspace_bytes(S: int, T: int, E: int) -> int:
    return int(load_library().moe_balance_loss_workspace_bytes(S, T, E))


def moe_balance_loss(logits, topk_ids, counts, prob_mean, lse, n_valid, losses, ws,
                     token_mask=None, dev_status=None, stream=None):
    """Router losses: logits f32 or bf16 [S,T,E], topk_ids i32 [S,T,k], token_mask uint8 [S,T]
    (None: all valid) -> counts i32 [S,E], prob_mean f32 [S,E], lse f32 [S,T], n_valid i32 [S],
    losses f32 [2] (balance, z); ws is a uint8 device tensor."""
    rc = _ops().balance_loss(logits, topk_ids, counts, prob_mean, lse, n_valid, losses, ws,
                             token_mask, dev_status, stream)
    if rc:
        _check(rc)


def moe_route_backward(logits, topk_ids, topk_w, d_topk_w, lse, counts, n_valid, d_losses,
                       d_logits, token_mask=None, dev_status=None, stream=None):
    """Gradient in the logits [S,T,E] (f32 or bf16) of the routing weights (topk_w, d_topk_w f32
    [S,T,k], both or neither None) and of the two losses (d_losses f32 [2] with what
    moe_balance_loss wrote, or None) -> d_logits of the logits' type."""
    rc = _ops().route_backward(logits, topk_ids, topk_w, d_topk_w, lse, counts, n_valid, d_losses,
                               d_logits, token_mask, dev_status, stream)
    if rc:
        _check(rc)


def moe_combine_backward(d_out, y, pair_row, topk_w, d_y, d_topk_w, recv_pair=None,
                         dev_status=None, stream=None):
    """Gradient of moe_combine: d_out bf16 [S,T,H], y bf16 [y_rows,H] -> d_y bf16 [y_rows,H],
    d_topk_w f32 [S,T,k]; rows with recv_pair i32 [y_rows] < 0 are set to zero."""
    rc = _ops().combine_backward(d_out, y, pair_row, topk_w, d_y, d_topk_w, recv_pair, dev_status,
                                 stream)
    if rc:
        _check(rc)


def moe_w4_bytes(E: int, N: int, K: int, gated: bool = False) -> int:
    """Bytes of E experts' packed 4-bit weights with N outputs over K columns."""
    n = int(load_library().moe_w4_bytes(E, N, K, int(gated)))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, load_library().moe_last_error_message().decode())
    return n


def moe_w4_pack(codes, scales, w4, gated=False, stream=None):
    """codes uint8 [E,rows,K/2] (E2M1, first value in the low nibble), scales uint8 [E,rows,K/16]
    (E4M3), rows = N or for gated weights 2N (gate, then up) -> w4 uint8 [moe_w4_bytes]."""
    rc = _ops().w4_pack(codes, scales, w4, gated, stream)
    if rc:
        _check(rc)


def moe_expert_product_w4_workspace_bytes(a_rows: int, E: int, N: int, K: int) -> int:
    return int(load_library().moe_expert_product_w4_workspace_bytes(a_rows, E, N, K))


def moe_expert_product_w4(a, w4, w_factor, y, ws, expert_offsets=None, masked_counts=None,
                          block_rows=0, gated=False, dev_status=None, stream=None):
    """a bf16 [rows,K] times every expert's packed 4-bit weights -> y bf16 [rows,N]; the experts'
    rows by expert_offsets i32 [E+1] or by masked_counts i32 [E] with block_rows; w_factor f32 [E]."""
    rc = _ops().expert_product_w4(a, w4, w_factor, y, ws, expert_offsets, masked_counts, block_rows,
                                  gated, dev_status, stream)
    if rc:
        _check(rc)


def moe_expert_product_workspace_bytes(a_rows: int, E: int, N: int, K: int, gated: bool = False) -> int:
    return int(load_library().moe_expert_product_workspace_bytes(a_rows, E, N, K, int(gated)))


def moe_expert_product(a, w, y, ws, expert_offsets=None, masked_counts=None, block_rows=0, gated=False,
                       pre=None, dev_status=None, stream=None):
    """a bf16 [rows,K] times every expert's bf16 weights w [E,N,K] (gated: [E,2N,K], gate rows, then
    up rows) -> y bf16 [rows,N]; the experts' rows by expert_offsets i32 [E+1] or by masked_counts
    i32 [E] with block_rows.  pre bf16 [rows,2N] (gated) takes gate and up for the way back."""
    rc = _ops().expert_product(a, w, y, ws, expert_offsets, masked_counts, block_rows, gated, pre,
                               dev_status, stream)
    if rc:
        _check(rc)


def moe_expert_product_backward_workspace_bytes(a_rows: int, E: int, N: int, K: int) -> int:
    return int(load_library().moe_expert_product_backward_workspace_bytes(a_rows, E, N, K))


def moe_expert_product_backward(d_y, a, w, ws, d_a=None, d_w=None, expert_offsets=None,
                                masked_counts=None, block_rows=0, pre=None, dev_status=None,
                                stream=None):
    """Gradient of y = a W^T: d_y bf16 [rows,N], a bf16 [rows,K], w bf16 [E,N,K] -> d_a bf16 [rows,K]
    and d_w f32 or bf16 [E,N,K], each where it is given (a may be None without d_w).  With pre bf16
    [rows,2K], a was silu(gate) * up of it and d_a [rows,2K] is the gradient in gate and up."""
    rc = _ops().expert_product_backward(d_y, a, w, ws, d_a, d_w, expert_offsets, masked_counts,
                                        block_rows, pre, dev_status, stream)
    if rc:
        _check(rc)


def moe_rms_norm(x, weight, y=None, record=None, residual=None, residual_out=None, eps=1e-6,
                 stream=None):
    """RMS norm of x + residual: x bf16 [...,H], residual f32 or bf16 [...,H], weight f32 or bf16 [H]
    -> y bf16 [...,H], record uint8 [...,H+H/32] (the MXFP8 records of y; H % 32 == 0), residual_out
    (the sum, of the residual's type; may be the residual itself), each where it is given."""
    rc = _ops().rms_norm(x, weight, y, record, residual, residual_out, eps, stream)
    if rc:
        _check(rc)


def moe_rms_norm_backward_workspace_bytes(rows: int, H: int) -> int:
    return int(load_library().moe_rms_norm_backward_workspace_bytes(rows, H))


def moe_rms_norm_backward(d_y, h, weight, d_h, ws=None, d_weight=None, d_residual=None, d_x=None,
                          eps=1e-6, stream=None):
    """Gradient of moe_rms_norm: d_y bf16 [...,H], h f32 or bf16 [...,H] (what was normed:
    residual_out, or x) -> d_h of h's type (+ d_residual of that type), d_x its bf16 copy, d_weight
    f32 [H] (with ws), each but d_h where it is given."""
    rc = _ops().rms_norm_backward(d_y, h, weight, d_h, ws, d_weight, d_residual, d_x, eps, stream)
    if rc:
        _check(rc)


class MoePath:
    """Device buffers for one shape plus the five calls in order.

    Buffers are allocated once (worst-case capacities, fixed addresses), so a
    step enqueues kernels only and can be captured in a CUDA graph.
    """

    def __init__(self, S, T, H, E, k, P, recv_part=-1, align=1, cap_send=None, cap_recv=None,
                 device="cuda", layout="contiguous", block_rows=None, combine="single",
                 quant="none", placement: "Placement | None" = None, nvfp4_scale: float = 1.0,
                 dispatch: str | None = None):
        """layout: "contiguous" (expert runs, moe_permute_to_experts), "masked" (one
        block of block_rows rows per expert, moe_permute_to_experts_masked) or "routed"
        (no permute: rows carry their ids and weights, moe_dispatch_pack_routed, and
        moe_routed_expert_stage1 + moe_combine_stage2 replace the expert and combine).
        combine: "single" (moe_combine) or "two_stage" (moe_combine_stage1 + stage2).
        quant: "none" (bf16 rows), "mxfp8" or "nvfp4" (rows sent as quantized records;
        the receiver's stand-in expert dequantizes them, so every step runs it);
        nvfp4_scale is the NVFP4 per-tensor scale.
        placement: a Placement (moe_plan_placement) -- the layout then maps each
        pair to a physical expert slot and everything after it works on the
        P*Lp physical experts; None keeps expert e in slot e.
        dispatch: "fused" (moe_dispatch, or moe_dispatch_quantized with quantized
        rows: route, layout, pack and permute in one call, one launch for a
        decode-sized batch of bf16 rows; under a placement the mapped layout and
        then moe_dispatch_pack_permute) or "separate" (the four calls); the
        default is "fused" where it applies (the contiguous layout)."""
        if layout not in ("contiguous", "masked", "routed") or combine not in ("single", "two_stage"):
            raise ValueError("layout must be contiguous|masked|routed, combine single|two_stage")
        if layout == "routed":
            if quant != "none":
                raise ValueError("the routed layout carries bf16 rows")
            combine = "two_stage"          # the routed expert produces stage 1 itself
        if quant not in ("none", "mxfp8", "nvfp4"):
            raise ValueError("quant must be none|mxfp8|nvfp4")
        if quant == "mxfp8" and (H % 512 != 0 or layout != "contiguous"):
            raise ValueError("mxfp8 rows need H % 512 == 0 and the contiguous layout")
        if quant == "nvfp4" and (H % 256 != 0 or layout != "contiguous"):
            raise ValueError("nvfp4 rows need H % 256 == 0 and the contiguous layout")
        # moe_dispatch / moe_dispatch_quantized / moe_dispatch_masked without a
        # placement; with one, the layout call and then one pack + permute call (bf16)
        fusable = ((layout == "contiguous" and (placement is None or quant == "none"))
                   or (layout == "masked" and quant == "none"))
        if dispatch is None:
            dispatch = "fused" if fusable else "separate"
        if dispatch not in ("fused", "separate") or (dispatch == "fused" and not fusable):
            raise ValueError("dispatch must be fused|separate; fused needs the contiguous or masked "
                             "layout (and bf16 rows under a placement or in masked blocks)")
        self.dispatch_mode = dispatch
        self.quantized = quant != "none"
        self.nvfp4_scale = float(nvfp4_scale)
        if placement is not None and (placement.E != E or placement.P != P):
            raise ValueError("the placement is for another E or P")
        self.S, self.T, self.H, self.E, self.k, self.P = S, T, H, E, k, P
        self.placement = placement
        # experts as the layout's outputs and every later call see them
        self.Ep = placement.E_phys if placement is not None else E
        self.recv_part, self.align = recv_part, align
        self.layout, self.combine_mode, self.quant = layout, combine, quant
        # row width as the permute sees it: bf16 slots per row
        self.row_bytes = {"mxfp8": mxfp8_record_bytes(H), "nvfp4": nvfp4_record_bytes(H)}.get(quant, 2 * H)
        self.Hp = self.row_bytes // 2
        self.cap_send = T * min(k, P) if cap_send is None else cap_send
        Ep = self.Ep
        self.n_blocks = Ep if recv_part < 0 else Ep // P
        if layout == "masked":
            if block_rows is None:
                raise ValueError("the masked layout needs block_rows")
            self.block_rows = block_rows
            self.cap_recv = self.n_blocks * block_rows
        elif layout == "routed":
            self.block_rows = None
            self.cap_recv = 0              # no receive buffer: rows stay where they arrive
        else:
            self.block_rows = None
            self.cap_recv = S * T * k + Ep * (align - 1) if cap_recv is None else cap_recv
        d = torch.device(device)
        i32 = dict(dtype=torch.int32, device=d)
        self.topk_ids = torch.empty((S, T, k), **i32)
        self.topk_w = torch.empty((S, T, k), dtype=torch.float32, device=d)
        self.expert_counts = torch.empty((S, Ep), **i32)
        # ids of the pairs after the layout: physical slots under a placement
        self.phys_ids = torch.empty((S, T, k), **i32) if placement is not None else self.topk_ids
        if placement is not None:
            self.copy_offsets, self.copy_slots, self.slot_expert = placement.to(d)
        self.expert_rank = torch.empty((S, T, k), **i32)
        self.part_counts = torch.empty((S, P), **i32)
        self.part_offsets = torch.empty((S, P + 1), **i32)
        self.token_slot = torch.empty((S, T, P), **i32)
        row_dt = torch.uint8 if self.quantized else torch.bfloat16
        row_w = self.row_bytes if self.quantized else H
        self.send = torch.empty((S, self.cap_send, row_w), dtype=row_dt, device=d)
        self.send_src = torch.empty((S, self.cap_send), **i32)
        self.recv = torch.empty((self.cap_recv, row_w), dtype=row_dt, device=d)
        self.expert_offsets = torch.empty((Ep + 1,), **i32)
        self.pair_row = torch.empty((S, T, k), **i32)
        self.recv_pair = torch.empty((self.cap_recv,), **i32)
        self.out = torch.empty((S, T, H), dtype=torch.bfloat16, device=d)
        ws = moe_workspace_bytes(S, T, k, Ep, P)
        if placement is not None:
            ws = max(ws, moe_workspace_bytes_mapped(S, T, k, E, P, placement.Lp))
        self.ws = torch.empty((max(ws, 256),), dtype=torch.uint8, device=d)
        self.dev_status = torch.zeros((1,), **i32)
        self.masked_counts = torch.empty((self.n_blocks,), **i32) if layout == "masked" else None
        self.ret = (torch.empty((S, self.cap_send, H), dtype=torch.bfloat16, device=d)
                    if combine == "two_stage" else None)
        if layout == "routed":
            self.send_ids = torch.empty((S, self.cap_send, k), **i32)
            self.send_w = torch.empty((S, self.cap_send, k), dtype=torch.float32, device=d)
        self.y = None
        if self.quantized:
            self.y = torch.empty((self.cap_recv, H), dtype=torch.bfloat16, device=d)
            self.unit_scale = torch.ones((Ep,), dtype=torch.float32, device=d)

    def bind(self, logits, x, stream=None, scale=None):
        """Pre-marshal the calls of one step for fixed input tensors and stream.

        Returns a list of (C function, argument tuple); calling them in order
        is one step (route, layout, pack, permute, [dequantizing stand-in
        expert with MXFP8 rows], combine) with no per-call Python checks, so
        the host enqueues far ahead of the GPU.
        """
        lib = load_library()
        st = _stream(stream)
        S, T, H, E, k, P = self.S, self.T, self.H, self.E, self.k, self.P
        vp = ctypes.c_void_p
        ptr = lambda t, name, dt: _dev(t, name, dt)  # noqa: E731
        if tuple(logits.shape) != (S, T, E) or tuple(x.shape) != (S, T, H):
            raise ValueError("bind: logits / x shapes do not match the path")
        stp = vp(self.dev_status.data_ptr())
        Hp, Ep = self.Hp, self.Ep
        ids_p = vp(self.phys_ids.data_ptr())
        one_call = self.placement is None and self.layout == "contiguous"
        if self.dispatch_mode == "fused" and self.placement is None and self.layout == "masked":
            calls = [(lib.moe_dispatch_masked, (
                ptr(logits, "logits", (torch.float32,)), ptr(x, "x", _BF16_TYPES), S, T, H, E, k, P,
                self.recv_part, self.block_rows, self.cap_send, vp(self.topk_ids.data_ptr()),
                vp(self.topk_w.data_ptr()), vp(self.expert_counts.data_ptr()),
                vp(self.expert_rank.data_ptr()), vp(self.part_counts.data_ptr()),
                vp(self.part_offsets.data_ptr()), vp(self.token_slot.data_ptr()),
                vp(self.send.data_ptr()), vp(self.send_src.data_ptr()), vp(self.recv.data_ptr()),
                vp(self.masked_counts.data_ptr()), vp(self.pair_row.data_ptr()),
                vp(self.recv_pair.data_ptr()), vp(self.ws.data_ptr()), self.ws.numel(), stp, st))]
            return calls + self._bind_combine(lib, self.recv, stp, st, ids_p)
        if self.dispatch_mode == "fused" and one_call and self.quantized:
            fmt = MOE_FORMAT_MXFP8 if self.quant == "mxfp8" else MOE_FORMAT_NVFP4
            calls = [(lib.moe_dispatch_quantized, (
                ptr(logits, "logits", (torch.float32,)), ptr(x, "x", _BF16_TYPES), S, T, H, E, k, P,
                fmt, self.nvfp4_scale if self.quant == "nvfp4" else 1.0, self.recv_part, self.align,
                self.cap_send, self.cap_recv, vp(self.topk_ids.data_ptr()),
                vp(self.topk_w.data_ptr()), vp(self.expert_counts.data_ptr()),
                vp(self.expert_rank.data_ptr()), vp(self.part_counts.data_ptr()),
                vp(self.part_offsets.data_ptr()), vp(self.token_slot.data_ptr()),
                vp(self.send.data_ptr()), vp(self.send_src.data_ptr()), vp(self.recv.data_ptr()),
                vp(self.expert_offsets.data_ptr()), vp(self.pair_row.data_ptr()),
                vp(self.recv_pair.data_ptr()), vp(self.ws.data_ptr()), self.ws.numel(), stp, st))]
            return calls + self._bind_expert_q(lib, scale, stp, st) + \
                self._bind_combine(lib, self.y, stp, st, ids_p)
        if self.dispatch_mode == "fused" and one_call:
            calls = [(lib.moe_dispatch, (
                ptr(logits, "logits", (torch.float32,)), ptr(x, "x", _BF16_TYPES), S, T, H, E, k, P,
                self.recv_part, self.align, self.cap_send, self.cap_recv,
                vp(self.topk_ids.data_ptr()), vp(self.topk_w.data_ptr()),
                vp(self.expert_counts.data_ptr()), vp(self.expert_rank.data_ptr()),
                vp(self.part_counts.data_ptr()), vp(self.part_offsets.data_ptr()),
                vp(self.token_slot.data_ptr()), vp(self.send.data_ptr()),
                vp(self.send_src.data_ptr()), vp(self.recv.data_ptr()),
                vp(self.expert_offsets.data_ptr()), vp(self.pair_row.data_ptr()),
                vp(self.recv_pair.data_ptr()), vp(self.ws.data_ptr()), self.ws.numel(), stp, st))]
            return calls + self._bind_combine(lib, self.recv, stp, st, ids_p)
        calls = [
            (lib.moe_route_topk, (ptr(logits, "logits", (torch.float32,)), S, T, E, k,
                                  vp(self.topk_ids.data_ptr()), vp(self.topk_w.data_ptr()), st)),
        ]
        outs = (vp(self.expert_counts.data_ptr()), vp(self.expert_rank.data_ptr()),
                vp(self.part_counts.data_ptr()), vp(self.part_offsets.data_ptr()),
                vp(self.token_slot.data_ptr()), vp(self.ws.data_ptr()), self.ws.numel(), stp, st)
        if self.placement is not None:
            calls.append((lib.moe_dispatch_layout_mapped, (
                vp(self.topk_ids.data_ptr()), S, T, k, E, P, self.placement.Lp,
                vp(self.copy_offsets.data_ptr()), vp(self.copy_slots.data_ptr()),
                self.copy_slots.numel(), ids_p) + outs))
        else:
            calls.append((lib.moe_dispatch_layout, (vp(self.topk_ids.data_ptr()), S, T, k, E, P)
                          + outs))
        if self.dispatch_mode == "fused" and self.layout == "masked":
            calls.append((lib.moe_dispatch_pack_permute_masked, (
                ptr(x, "x", _BF16_TYPES), vp(self.token_slot.data_ptr()),
                vp(self.part_offsets.data_ptr()), ids_p, vp(self.expert_counts.data_ptr()),
                vp(self.expert_rank.data_ptr()), S, T, k, Ep, P, H, self.recv_part,
                self.block_rows, self.cap_send, vp(self.send.data_ptr()),
                vp(self.send_src.data_ptr()), vp(self.recv.data_ptr()),
                vp(self.masked_counts.data_ptr()), vp(self.pair_row.data_ptr()),
                vp(self.recv_pair.data_ptr()), stp, st)))
            return calls + self._bind_combine(lib, self.recv, stp, st, ids_p)
        if self.dispatch_mode == "fused":
            # under a placement: pack and permute over the physical slots in one pass
            calls.append((lib.moe_dispatch_pack_permute, (
                ptr(x, "x", _BF16_TYPES), vp(self.token_slot.data_ptr()),
                vp(self.part_offsets.data_ptr()), ids_p, vp(self.expert_counts.data_ptr()),
                vp(self.expert_rank.data_ptr()), S, T, k, Ep, P, H, self.recv_part, self.align,
                self.cap_send, self.cap_recv, vp(self.send.data_ptr()),
                vp(self.send_src.data_ptr()), vp(self.recv.data_ptr()),
                vp(self.expert_offsets.data_ptr()), vp(self.pair_row.data_ptr()),
                vp(self.recv_pair.data_ptr()), vp(self.ws.data_ptr()), self.ws.numel(), stp, st)))
            return calls + self._bind_combine(lib, self.recv, stp, st, ids_p)
        if self.layout == "routed":
            calls.append((lib.moe_dispatch_pack_routed, (
                ptr(x, "x", _BF16_TYPES), vp(self.topk_ids.data_ptr()),
                vp(self.topk_w.data_ptr()), S, T, H, k, P, vp(self.token_slot.data_ptr()),
                vp(self.part_offsets.data_ptr()), self.cap_send, vp(self.send.data_ptr()),
                vp(self.send_src.data_ptr()), vp(self.send_ids.data_ptr()),
                vp(self.send_w.data_ptr()), stp, st)))
            self._bound_scale = None if scale is None else self.slot_scale(scale)
            sc = vp(None) if self._bound_scale is None else ptr(self._bound_scale, "scale",
                                                                  (torch.float32,))
            calls.append((lib.moe_routed_expert_stage1, (
                vp(self.send.data_ptr()), vp(self.send_ids.data_ptr()),
                vp(self.send_w.data_ptr()), vp(self.part_offsets.data_ptr()), S, T, self.cap_send,
                k, Ep, P, H, self.recv_part, sc, vp(self.ret.data_ptr()), stp, st)))
            calls.append((lib.moe_combine_stage2, (
                vp(self.ret.data_ptr()), vp(self.token_slot.data_ptr()), S, T, P, H,
                self.recv_part, self.cap_send, vp(self.out.data_ptr()), stp, st)))
            return calls
        if self.quant == "mxfp8":
            calls.append((lib.moe_dispatch_pack_mxfp8, (
                ptr(x, "x", _BF16_TYPES), S, T, H, P, vp(self.token_slot.data_ptr()),
                vp(self.part_offsets.data_ptr()), self.cap_send, vp(self.send.data_ptr()),
                vp(self.send_src.data_ptr()), stp, st)))
        elif self.quant == "nvfp4":
            calls.append((lib.moe_dispatch_pack_nvfp4, (
                ptr(x, "x", _BF16_TYPES), S, T, H, P, self.nvfp4_scale,
                vp(self.token_slot.data_ptr()), vp(self.part_offsets.data_ptr()), self.cap_send,
                vp(self.send.data_ptr()), vp(self.send_src.data_ptr()), stp, st)))
        else:
            calls.append((lib.moe_dispatch_pack, (
                ptr(x, "x", _BF16_TYPES), S, T, H, P, vp(self.token_slot.data_ptr()),
                vp(self.part_offsets.data_ptr()), self.cap_send, vp(self.send.data_ptr()),
                vp(self.send_src.data_ptr()), stp, st)))
        if self.layout == "masked":
            calls.append((lib.moe_permute_to_experts_masked, (
                vp(self.send.data_ptr()), vp(self.token_slot.data_ptr()),
                ids_p, vp(self.expert_counts.data_ptr()),
                vp(self.expert_rank.data_ptr()), S, T, k, Ep, P, H, self.recv_part,
                self.block_rows, self.cap_send, vp(self.recv.data_ptr()),
                vp(self.masked_counts.data_ptr()), vp(self.pair_row.data_ptr()),
                vp(self.recv_pair.data_ptr()), stp, st)))
        else:
            calls.append((lib.moe_permute_to_experts, (
                vp(self.send.data_ptr()), vp(self.token_slot.data_ptr()),
                ids_p, vp(self.expert_counts.data_ptr()),
                vp(self.expert_rank.data_ptr()), S, T, k, Ep, P, Hp, self.recv_part, self.align,
                self.cap_send, self.cap_recv, vp(self.recv.data_ptr()),
                vp(self.expert_offsets.data_ptr()), vp(self.pair_row.data_ptr()),
                vp(self.recv_pair.data_ptr()), vp(self.ws.data_ptr()), self.ws.numel(), stp, st)))
        y = self.recv
        if self.quantized:
            calls += self._bind_expert_q(lib, scale, stp, st)
            y = self.y
        return calls + self._bind_combine(lib, y, stp, st, ids_p)

    def _bind_expert_q(self, lib, scale, stp, st):
        """The bound dequantizing stand-in expert (quantized rows: recv records -> y)."""
        vp = ctypes.c_void_p
        # the bound call keeps a pointer: hold the per-slot scales on the path
        self._bound_scale = self.unit_scale if scale is None else self.slot_scale(scale)
        sc = _dev(self._bound_scale, "scale", (torch.float32,))
        if self.quant == "mxfp8":
            return [(lib.moe_expert_scale_mxfp8, (
                vp(self.recv.data_ptr()), vp(self.expert_offsets.data_ptr()), sc, self.Ep, self.H,
                self.cap_recv, vp(self.y.data_ptr()), st))]
        return [(lib.moe_expert_scale_nvfp4, (
            vp(self.recv.data_ptr()), vp(self.expert_offsets.data_ptr()), sc, self.Ep, self.H,
            self.nvfp4_scale, self.cap_recv, vp(self.y.data_ptr()), st))]

    def _bind_combine(self, lib, y, stp, st, ids_p):
        """The bound combine call(s) reading expert rows y."""
        S, T, H, k, P, Ep = self.S, self.T, self.H, self.k, self.P, self.Ep
        vp = ctypes.c_void_p
        if self.combine_mode == "two_stage":
            return [(lib.moe_combine_stage1, (
                        vp(y.data_ptr()), self.cap_recv, vp(self.pair_row.data_ptr()),
                        vp(self.topk_w.data_ptr()), ids_p,
                        vp(self.token_slot.data_ptr()), S, T, k, Ep, P, H, self.recv_part,
                        self.cap_send, vp(self.ret.data_ptr()), stp, st)),
                    (lib.moe_combine_stage2, (
                        vp(self.ret.data_ptr()), vp(self.token_slot.data_ptr()), S, T, P, H,
                        self.recv_part, self.cap_send, vp(self.out.data_ptr()), stp, st))]
        return [(lib.moe_combine, (
            vp(y.data_ptr()), self.cap_recv, vp(self.pair_row.data_ptr()),
            vp(self.topk_w.data_ptr()), S, T, k, H, vp(self.out.data_ptr()), stp, st))]

    @staticmethod
    def run_bound(calls, upto: int | None = None, start: int = 0):
        """Issue pre-marshalled calls [start, upto); raise on the first non-OK status."""
        for fn, args in calls[start:upto]:
            rc = fn(*args)
            if rc != MOE_OK:
                _check(rc)

    def route(self, logits, stream=None):
        moe_route_topk(logits, self.topk_ids, self.topk_w, stream)

    def dispatch(self, x, stream=None):
        """layout + pack + permute (the receiver's copy epilogue is part of dispatch)."""
        if self.placement is not None:
            moe_dispatch_layout_mapped(self.topk_ids, self.E, self.P, self.placement.Lp,
                                       self.copy_offsets, self.copy_slots, self.phys_ids,
                                       self.expert_counts, self.expert_rank, self.part_counts,
                                       self.part_offsets, self.token_slot, self.ws,
                                       self.dev_status, stream)
        else:
            moe_dispatch_layout(self.topk_ids, self.E, self.P, self.expert_counts,
                                self.expert_rank, self.part_counts, self.part_offsets,
                                self.token_slot, self.ws, self.dev_status, stream)
        if self.dispatch_mode == "fused" and self.layout == "masked":
            moe_dispatch_pack_permute_masked(x, self.token_slot, self.part_offsets, self.phys_ids,
                                             self.expert_counts, self.expert_rank, self.Ep,
                                             self.recv_part, self.block_rows, self.send,
                                             self.send_src, self.recv, self.masked_counts,
                                             self.pair_row, self.recv_pair, self.dev_status, stream)
            return
        if self.dispatch_mode == "fused":
            # under a placement: pack and permute over the physical slots in one pass
            moe_dispatch_pack_permute(x, self.token_slot, self.part_offsets, self.phys_ids,
                                      self.expert_counts, self.expert_rank, self.Ep,
                                      self.recv_part, self.align, self.send, self.send_src,
                                      self.recv, self.expert_offsets, self.pair_row,
                                      self.recv_pair, self.ws, self.dev_status, stream)
            return
        if self.layout == "routed":
            moe_dispatch_pack_routed(x, self.topk_ids, self.topk_w, self.token_slot,
                                     self.part_offsets, self.send, self.send_src, self.send_ids,
                                     self.send_w, self.dev_status, stream)
            return
        if self.quantized:
            if self.quant == "mxfp8":
                moe_dispatch_pack_mxfp8(x, self.token_slot, self.part_offsets, self.send,
                                        self.send_src, self.dev_status, stream)
            else:
                moe_dispatch_pack_nvfp4(x, self.token_slot, self.part_offsets, self.send,
                                        self.send_src, self.nvfp4_scale, self.dev_status, stream)
            moe_permute_to_experts(self.send.view(torch.bfloat16), self.token_slot, self.phys_ids,
                                   self.expert_counts, self.expert_rank, self.Ep, self.recv_part,
                                   self.align, self.recv.view(torch.bfloat16),
                                   self.expert_offsets, self.pair_row, self.recv_pair, self.ws,
                                   self.dev_status, stream)
            return
        moe_dispatch_pack(x, self.token_slot, self.part_offsets, self.send, self.send_src,
                          self.dev_status, stream)
        if self.layout == "masked":
            moe_permute_to_experts_masked(self.send, self.token_slot, self.phys_ids,
                                          self.expert_counts, self.expert_rank, self.Ep,
                                          self.recv_part, self.block_rows, self.recv,
                                          self.masked_counts, self.pair_row, self.recv_pair,
                                          self.dev_status, stream)
        else:
            moe_permute_to_experts(self.send, self.token_slot, self.phys_ids, self.expert_counts,
                                   self.expert_rank, self.Ep, self.recv_part, self.align, self.recv,
                                   self.expert_offsets, self.pair_row, self.recv_pair, self.ws,
                                   self.dev_status, stream)

    def slot_scale(self, scale):
        """Stand-in expert scales per logical expert -> per expert slot (a copy
        computes what its original computes; empty slots get 0)."""
        if self.placement is None:
            return scale
        se = self.slot_expert
        return torch.where(se >= 0, scale[se.clamp(min=0).long()], torch.zeros_like(scale[:1]))

    def expert(self, scale, stream=None):
        if self.layout != "contiguous":
            raise ValueError("the stand-in expert reads contiguous expert runs")
        if self.quantized:
            sc = self.unit_scale if scale is None else self.slot_scale(scale)
            if self.quant == "mxfp8":
                moe_expert_scale_mxfp8(self.recv, self.expert_offsets, sc, self.y, stream)
            else:
                moe_expert_scale_nvfp4(self.recv, self.expert_offsets, sc, self.y,
                                       self.nvfp4_scale, stream)
            return self.y
        if self.y is None:
            self.y = torch.empty_like(self.recv)
        moe_expert_scale(self.recv, self.expert_offsets, self.slot_scale(scale), self.y, stream)
        return self.y

    def combine(self, y=None, stream=None):
        if y is None:
            y = self.y if self.quantized else self.recv
        if self.combine_mode == "two_stage":
            moe_combine_stage1(y, self.pair_row, self.topk_w, self.phys_ids, self.token_slot,
                               self.Ep, self.recv_part, self.ret, self.dev_status, stream)
            moe_combine_stage2(self.ret, self.token_slot, self.out, self.dev_status, stream,
                               recv_part=self.recv_part)
        else:
            moe_combine(y, self.pair_row, self.topk_w, self.out, self.dev_status, stream)

    def routed_combine(self, scale=None, stream=None):
        """Routed layout: the routed stand-in expert with the stage-1 pre-add, then stage 2."""
        sc = None if scale is None else self.slot_scale(scale)
        moe_routed_expert_stage1(self.send, self.send_ids, self.send_w, self.part_offsets, self.T,
                                 self.Ep, self.recv_part, sc, self.ret, self.dev_status, stream)
        moe_combine_stage2(self.ret, self.token_slot, self.out, self.dev_status, stream,
                               recv_part=self.recv_part)

    def dispatch_records(self, logits, record, stream=None):
        """dispatch_fused for rows that are MXFP8 records already, record uint8 [S,T,H+H/32] as
        moe_rms_norm writes them: quantized once per token, then moved.  For quant="mxfp8" paths;
        recv holds what dispatch_fused makes of the rows in bf16."""
        if self.quant != "mxfp8" or self.placement is not None:
            raise ValueError("dispatch_records needs quant='mxfp8' and no placement")
        if tuple(record.shape) != (self.S, self.T, self.row_bytes):
            raise ValueError(f"record must be [{self.S}, {self.T}, {self.row_bytes}] uint8")
        _dev(record, "record", (torch.uint8,), 3)
        rows = torch.bfloat16
        moe_dispatch(logits, record.view(rows), self.E, self.P, self.recv_part, self.align,
                     self.topk_ids, self.topk_w, self.expert_counts, self.expert_rank,
                     self.part_counts, self.part_offsets, self.token_slot, self.send.view(rows),
                     self.send_src, self.recv.view(rows), self.expert_offsets, self.pair_row,
                     self.recv_pair, self.ws, self.dev_status, stream)

    def dispatch_fused(self, logits, x, stream=None):
        """route + layout + pack + permute through one moe_dispatch (with quantized
        rows moe_dispatch_quantized, with the masked layout moe_dispatch_masked) call."""
        if self.layout == "masked":
            moe_dispatch_masked(logits, x, self.E, self.P, self.recv_part, self.block_rows,
                                self.topk_ids, self.topk_w, self.expert_counts, self.expert_rank,
                                self.part_counts, self.part_offsets, self.token_slot, self.send,
                                self.send_src, self.recv, self.masked_counts, self.pair_row,
                                self.recv_pair, self.ws, self.dev_status, stream)
            return
        if self.quantized:
            moe_dispatch_quantized(logits, x, self.E, self.P,
                                   MOE_FORMAT_MXFP8 if self.quant == "mxfp8" else MOE_FORMAT_NVFP4,
                                   self.nvfp4_scale if self.quant == "nvfp4" else 1.0,
                                   self.recv_part, self.align, self.topk_ids, self.topk_w,
                                   self.expert_counts, self.expert_rank, self.part_counts,
                                   self.part_offsets, self.token_slot, self.send, self.send_src,
                                   self.recv, self.expert_offsets, self.pair_row, self.recv_pair,
                                   self.ws, self.dev_status, stream)
            return
        moe_dispatch(logits, x, self.E, self.P, self.recv_part, self.align, self.topk_ids,
                     self.topk_w, self.expert_counts, self.expert_rank, self.part_counts,
                     self.part_offsets, self.token_slot, self.send, self.send_src, self.recv,
                     self.expert_offsets, self.pair_row, self.recv_pair, self.ws,
                     self.dev_status, stream)

    def step(self, logits, x, scale=None, stream=None):
        """route -> layout -> pack -> permute -> [stand-in expert] -> combine; returns out."""
        if (self.dispatch_mode == "fused" and self.placement is None
                and self.layout in ("contiguous", "masked")):
            self.dispatch_fused(logits, x, stream)
        else:
            self.route(logits, stream)
            self.dispatch(x, stream)
        if self.layout == "routed":
            self.routed_combine(scale, stream)
            return self.out
        y = self.expert(scale, stream) if scale is not None or self.quantized else None
        self.combine(y, stream)
        return self.out

    def launches_per_step(self, with_expert=False) -> int:
        """Kernels one step enqueues: route 1, layout 1 or 2 (as the library reports for
        the shape; under a placement plus the replica map, and a logical layout first
        when some expert has copies), pack 1, permute 1 or 2 (the masked form always
        2: map + copy), stand-in expert 1 (always with quantized rows), combine 1
        (2 when split into two stages)."""
        with_expert = with_expert or self.quantized
        if self.dispatch_mode == "fused" and self.placement is None and self.layout == "masked":
            comb = (2 if self.combine_mode == "two_stage" else 1) if self.T > 0 else 0
            return (moe_dispatch_masked_kernels(self.S, self.T, self.k, self.E, self.P,
                                                self.recv_part) + comb + (1 if with_expert else 0))
        if self.dispatch_mode == "fused" and self.placement is None and self.layout == "contiguous":
            comb = 2 if self.combine_mode == "two_stage" else 1
            if self.T == 0:
                comb = 0                   # the combine launches nothing for an empty batch
            count = moe_dispatch_quantized_kernels if self.quantized else moe_dispatch_kernels
            return (count(self.S, self.T, self.k, self.E, self.P) + comb
                    + (1 if with_expert else 0))
        mapped = self.placement is not None
        if mapped:
            layout = moe_dispatch_layout_kernels(self.S, self.T, self.k, self.Ep, self.P)
            if self.T > 0:
                layout += 1                # the replica map (nothing to map at T = 0)
            if self.placement.copy_slots.size > self.E:   # ranks over logical experts first
                layout += moe_dispatch_layout_kernels(self.S, self.T, self.k, self.E, 1)
        else:
            layout = moe_dispatch_layout_kernels(self.S, self.T, self.k, self.E, self.P)
        if self.dispatch_mode == "fused":        # the layout call, then pack + permute in one
            comb = (2 if self.combine_mode == "two_stage" else 1) if self.T > 0 else 0
            if self.layout == "masked":
                pp = moe_dispatch_pack_permute_masked_kernels(self.S, self.T, self.k, self.Ep,
                                                              self.P, self.recv_part)
            else:
                pp = moe_dispatch_pack_permute_kernels(self.S, self.T, self.k, self.Ep, self.P)
            return 1 + layout + pp + comb + (1 if with_expert else 0)
        if self.layout == "routed":
            if self.T == 0:                # the two receive-side calls launch nothing
                return 1 + layout + 1
            return 1 + layout + 1 + 1 + 1
        if self.layout == "masked":
            permute = 2 if self.T > 0 else 1      # nothing to copy at T = 0
        else:
            permute = moe_permute_to_experts_kernels(self.S, self.T, self.k, self.Ep, self.P)
        if self.T == 0:
            return 1 + layout + permute + (1 if with_expert else 0)
        comb = 2 if self.combine_mode == "two_stage" else 1
        return 1 + layout + 1 + permute + comb + (1 if with_expert else 0)


class HostPipeline:
    """Steps fed from and drained to pinned host memory, as a serving loop runs them.

    Each step copies its logits and x in from host buffers, runs the path on
    one of `sets` buffer sets, and copies the output back to a host buffer.
    Copies in, steps and copies out use three streams ordered by events, so
    the copies of one step overlap the steps next to it; a set is reused only
    after its previous step has read its inputs and its output has been copied
    out.  With `graphs` the step of every set is captured once as a CUDA graph.
    """

    def __init__(self, S, T, H, E, k, P, sets=3, graphs=True, device="cuda", **path_kwargs):
        d = torch.device(device)
        self.sets = sets
        self.paths, self.logits, self.x, self.steps = [], [], [], []
        self.s_in = torch.cuda.Stream(device=d)
        self.s_step = torch.cuda.Stream(device=d)
        self.s_out = torch.cuda.Stream(device=d)
        self._graphs = []
        for _ in range(sets):
            p = MoePath(S, T, H, E, k, P, device=d, **path_kwargs)
            lg = torch.zeros((S, T, E), dtype=torch.float32, device=d)
            xx = torch.zeros((S, T, H), dtype=torch.bfloat16, device=d)
            calls = p.bind(lg, xx, self.s_step)
            if graphs:
                # one eager step first: kernels load and the library's one-time
                # device queries run outside the capture
                MoePath.run_bound(calls)
                torch.cuda.synchronize(d)
                g = torch.cuda.CUDAGraph()
                cap = torch.cuda.Stream(device=d)
                with torch.cuda.graph(g, stream=cap):
                    MoePath.run_bound(p.bind(lg, xx, cap))
                self._graphs.append(g)
                self.steps.append(g.replay)
            else:
                self.steps.append(lambda c=calls: MoePath.run_bound(c))
            self.paths.append(p)
            self.logits.append(lg)
            self.x.append(xx)
        self.ev_in = [torch.cuda.Event() for _ in range(sets)]
        self.ev_step = [torch.cuda.Event() for _ in range(sets)]
        self.ev_out = [torch.cuda.Event() for _ in range(sets)]
        self.n = 0

    def submit(self, h_logits, h_x, h_out):
        """Enqueue one step: h_logits fp32 [S,T,E], h_x bf16 (or int16 bits) [S,T,H] in, and
        the output's bf16 bits into h_out (int16 [S,T,H]); all pinned host tensors.  Returns
        the event recorded after the output copy.  h_out must not be reused before that."""
        b = self.n % self.sets
        p = self.paths[b]
        with torch.cuda.stream(self.s_in):
            if self.n >= self.sets:
                self.s_in.wait_event(self.ev_step[b])     # the set's last step read its inputs
            self.logits[b].copy_(h_logits, non_blocking=True)
            self.x[b].view(torch.int16).copy_(h_x.view(torch.int16), non_blocking=True)
            self.ev_in[b].record(self.s_in)
        self.s_step.wait_event(self.ev_in[b])
        if self.n >= self.sets:
            self.s_step.wait_event(self.ev_out[b])        # its output has been copied out
        with torch.cuda.stream(self.s_step):
            self.steps[b]()
            self.ev_step[b].record(self.s_step)
        self.s_out.wait_event(self.ev_step[b])
        with torch.cuda.stream(self.s_out):
            h_out.copy_(p.out.view(torch.int16), non_blocking=True)
            self.ev_out[b].record(self.s_out)
        self.n += 1
        return self.ev_out[b]

    def synchronize(self):
        for s in (self.s_in, self.s_step, self.s_out):
            s.synchronize()

    def release(self):
        """Drop the captured graphs (before the buffers they refer to)."""
        self.synchronize()
        self._graphs = []
        self.steps = []
