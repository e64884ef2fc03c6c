"""B200 (sm_100a) library for the forward and backward pass of a
mixture-of-experts FFN layer with zero-computation (identity) experts: Python
binding.

Every step of the layer runs in the CUDA library ``_lib/libmoe.so`` behind the
C ABI declared in ``include/moe_api.h``. This module only marshals torch CUDA
tensors into that ABI (pointers, sizes, the current stream); it computes
nothing itself and has no fallback: if the library is missing, importing the
binding's functions raises.

All CUDA tensors of a call must live on the current device
(``torch.cuda.set_device``): the library launches its kernels there, on the
given stream or that device's current stream, and they read the tensors
directly.

Build the library with ``python -m expert_routing_dispatch_router_b200.build``.
"""
from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass
from typing import Optional

import torch

from . import build as _build

LIB_PATH = _build.LIB
HEADER = os.path.join(_build.ROOT, "include", "moe_api.h")

MOE_F32, MOE_BF16 = 0, 1
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_CHECK"}


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")
        self.status = status


class MoEConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32),
                ("n_routed", ctypes.c_int32), ("n_zero", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("routed_scale", ctypes.c_float)]


class MoEPIDParams(ctypes.Structure):
    _fields_ = [("target_routed_share", ctypes.c_float), ("kp", ctypes.c_float),
                ("ki", ctypes.c_float), ("kd", ctypes.c_float),
                ("max_step", ctypes.c_float)]


class MoEGrouped(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class MoEAdamW(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("total_blocks", ctypes.c_int64)]


class MoEAdamWParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps",
                                               "weight_decay")]


_DTYPE_CODE = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


@dataclass(frozen=True)
class GroupedShape:
    """Sizes of a grouped matrix product (mirrors moe_grouped_t): the capacity
    of the row buffers, the number of matrices, and their [n_out, n_in]."""
    rows: int
    groups: int
    n_in: int
    n_out: int
    dtype: torch.dtype = torch.bfloat16

    def c(self) -> MoEGrouped:
        """A struct of the caller's own."""
        return MoEGrouped.from_buffer_copy(self._shared())

    def _shared(self) -> MoEGrouped:
        c = self.__dict__.get("_c")  # built once: a frozen shape does not change
        if c is None:
            c = MoEGrouped(self.rows, self.groups, self.n_in, self.n_out,
                           _DTYPE_CODE[self.dtype])
            object.__setattr__(self, "_c", c)
        return c


@dataclass(frozen=True)
class LayerShape:
    """Sizes of one layer call (mirrors moe_config_t)."""
    T: int
    d: int
    n_routed: int
    n_zero: int
    top_k: int
    ffn: int
    act_dtype: torch.dtype = torch.bfloat16
    routed_scale: float = 1.0

    @property
    def E(self) -> int:
        return self.n_routed + self.n_zero

    def c(self) -> MoEConfig:
        """A struct of the caller's own."""
        return MoEConfig.from_buffer_copy(self._shared())

    def _shared(self) -> MoEConfig:
        c = self.__dict__.get("_c")  # built once: a frozen shape does not change
        if c is None:
            c = MoEConfig(self.T, self.d, self.n_routed, self.n_zero, self.top_k, self.ffn,
                          _DTYPE_CODE[self.act_dtype], float(self.routed_scale))
            object.__setattr__(self, "_c", c)
        return c


_lib = None
P = ctypes.c_void_p


def declared_functions():
    """Names of the functions ``include/moe_api.h`` declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:[\w]+\s*\*?\s+)+\*?(moe_\w+)\(", text, re.M)))


def lib():
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"CUDA library {LIB_PATH} is missing; build it with "
                "`python -m expert_routing_dispatch_router_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        C = ctypes.POINTER(MoEConfig)
        G = ctypes.POINTER(MoEGrouped)
        i32 = ctypes.c_int
        sz = ctypes.c_size_t
        sig = {
            "moe_workspace_size": ([C], sz),
            "moe_route": ([C, P, P, P, P, P, P, P, P, sz, P], i32),
            "moe_dispatch": ([C, P, P, P, P, P, P, P, P, sz, P], i32),
            "moe_expert_ffn": ([C, P, P, P, P, P, P, P, sz, P], i32),
            "moe_combine": ([C, P, P, P, P, P, P, P], i32),
            "moe_layer_forward": ([C, P, P, P, P, P, P, P, P, P, sz, P], i32),
            "moe_layer_forward_host": ([C, P, P, P, P, P, P, P, P, P, sz, P], i32),
            "moe_read_device_error": ([P, P, P], i32),
            "moe_selftest_wait_limit": ([P, ctypes.c_size_t, P], i32),
            "moe_route_noalloc": ([C, P, P, P, P, P, P, P, P], i32),
            "moe_bias_pid_update": ([C, P, P, P, ctypes.POINTER(MoEPIDParams), P], i32),
            "moe_layer_launch_count": ([C], ctypes.c_int32),
            "moe_ep_local_experts": ([C, ctypes.c_int32, ctypes.c_int32], ctypes.c_int32),
            "moe_ep_plan": ([C, ctypes.c_int32, ctypes.c_int32, P, P, P, P], i32),
            "moe_ep_dispatch": ([C, ctypes.c_int32, P, P, P, P, P, P], i32),
            "moe_ep_return": ([C, ctypes.c_int32, ctypes.c_int32, P, P, P, P, P, P], i32),
            "moe_grouped_workspace_size": ([G], sz),
            "moe_grouped_matmul": ([G, P, P, P, P, P, sz, P], i32),
            "moe_grouped_matmul_dx": ([G, P, P, P, P, P, sz, P], i32),
            "moe_grouped_matmul_dw": ([G, P, P, P, P, i32, P, sz, P], i32),
            "moe_backward_workspace_size": ([C], sz),
            "moe_combine_backward": ([C] + [P] * 9, i32),
            "moe_expert_ffn_backward": ([C] + [P] * 10 + [i32, P, sz, P], i32),
            "moe_input_backward": ([C] + [P] * 11 + [sz, P], i32),
            "moe_layer_backward": ([C] + [P] * 17 + [i32, P, sz, P], i32),
            "moe_adamw_step": ([ctypes.POINTER(MoEAdamW), ctypes.POINTER(MoEAdamWParams)]
                               + [P] * 7, i32),
            "moe_status_string": ([i32], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is None:  # the handle alone: the Stream object costs 3.5 us
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status, lib().moe_status_string(status).decode())


def _need(t: torch.Tensor, name: str, dtype, shape=None, on_device=True):
    """Checks one tensor argument before its address goes to the library. A
    host tensor where device memory is expected (or the reverse) would be
    dereferenced by a kernel or a copy on the wrong side, so it is refused."""
    if (t.dtype == dtype and t.is_cuda == on_device and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if on_device and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not on_device and t.is_cuda:
        raise ValueError(f"{name}: must be a host tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _ws(ws: torch.Tensor):
    """(address, size in bytes) of a workspace tensor, which must be device
    memory (alloc_workspace gives one)."""
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: must be a contiguous CUDA tensor (use alloc_workspace)")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


def _on(stream, device=None):
    """A context in which the call's stream, an object with its handle in
    `cuda_stream`, is torch's current one."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
    return torch.cuda.stream(stream)


def _new(shape, dtype, device, stream):
    """A new output of a call on `stream`. torch hands out memory stream by
    stream, so it is taken from the call's own: nobody else still uses it when
    the call writes it, and it is not handed out again before the call is done,
    even if the caller drops it at once. The current stream, where the caller
    goes on with it, is noted as a second user."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _out(t, name, dtype, shape, device, stream):
    """An output the caller gave (checked), or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    _need(t, name, dtype, shape)
    return t


def workspace_size(shape: LayerShape) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(shape._shared())))


def alloc_workspace(shape: LayerShape, device="cuda") -> torch.Tensor:
    """Zeroed workspace (the error word must start at zero)."""
    n = workspace_size(shape)
    if n == 0:
        raise ValueError(f"invalid or unsupported shape {shape}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def launch_count(shape: LayerShape) -> int:
    return int(lib().moe_layer_launch_count(ctypes.byref(shape._shared())))


def route(shape: LayerShape, x, w_router, bias, ws, logits=None, flags=None,
          stream=None):
    """Router + top-k + gates -> (topk_idx [T,k] int32, topk_gate [T,k] f32)."""
    T, E, k = shape.T, shape.E, shape.top_k
    _need(x, "x", shape.act_dtype, (T, shape.d))
    _need(w_router, "w_router", torch.float32, (E, shape.d))
    _need(bias, "bias", torch.float32, (E,))
    idx = _new((T, k), torch.int32, x.device, stream)
    gate = _new((T, k), torch.float32, x.device, stream)
    if logits is not None:
        _need(logits, "logits", torch.float32, (T, E))
    if flags is not None:
        _need(flags, "flags", torch.uint8, (T,))
    st = lib().moe_route(ctypes.byref(shape._shared()), _ptr(x), _ptr(w_router), _ptr(bias),
                         _ptr(logits), _ptr(idx), _ptr(gate), _ptr(flags), *_ws(ws),
                         _stream(stream))
    _check("moe_route", st)
    return idx, gate


def route_noalloc(shape: LayerShape, x, w_router, bias, topk_idx, topk_gate,
                  logits=None, flags=None, stream=None):
    """moe_route without a workspace, for callers that cannot allocate device
    memory: every output is caller-provided and the library's own fixed
    scratch array is used (T * E <= 4194304). Calls sharing a device must not
    overlap on the GPU."""
    T, E, k = shape.T, shape.E, shape.top_k
    _need(x, "x", shape.act_dtype, (T, shape.d))
    _need(w_router, "w_router", torch.float32, (E, shape.d))
    _need(bias, "bias", torch.float32, (E,))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(topk_gate, "topk_gate", torch.float32, (T, k))
    if logits is not None:
        _need(logits, "logits", torch.float32, (T, E))
    if flags is not None:
        _need(flags, "flags", torch.uint8, (T,))
    st = lib().moe_route_noalloc(ctypes.byref(shape._shared()), _ptr(x), _ptr(w_router),
                                 _ptr(bias), _ptr(logits), _ptr(topk_idx),
                                 _ptr(topk_gate), _ptr(flags), _stream(stream))
    _check("moe_route_noalloc", st)
    return topk_idx, topk_gate


def dispatch(shape: LayerShape, x, topk_idx, ws, stream=None):
    """-> (counts [E], offsets [N+1], row_token [T*k], slot_row [T*k], x_perm [T*k, d])."""
    T, k = shape.T, shape.top_k
    _need(x, "x", shape.act_dtype, (T, shape.d))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    dev, i32 = x.device, torch.int32
    counts = _new((shape.E,), i32, dev, stream)
    offsets = _new((shape.n_routed + 1,), i32, dev, stream)
    row_token = _new((T * k,), i32, dev, stream)
    slot_row = _new((T * k,), i32, dev, stream)
    x_perm = _new((T * k, shape.d), shape.act_dtype, dev, stream)
    st = lib().moe_dispatch(ctypes.byref(shape._shared()), _ptr(x), _ptr(topk_idx),
                            _ptr(counts), _ptr(offsets), _ptr(row_token),
                            _ptr(slot_row), _ptr(x_perm), *_ws(ws),
                            _stream(stream))
    _check("moe_dispatch", st)
    return counts, offsets, row_token, slot_row, x_perm


def expert_ffn(shape: LayerShape, x_perm, offsets, w_gate, w_up, w_down, ws,
               y_perm=None, stream=None):
    """-> y_perm [T*k, d] in the activation dtype (rows >= R untouched)."""
    T, k, d, F, N = shape.T, shape.top_k, shape.d, shape.ffn, shape.n_routed
    _need(x_perm, "x_perm", shape.act_dtype, (T * k, d))
    _need(offsets, "offsets", torch.int32, (N + 1,))
    for name, w, shp in (("w_gate", w_gate, (N, F, d)), ("w_up", w_up, (N, F, d)),
                         ("w_down", w_down, (N, d, F))):
        _need(w, name, shape.act_dtype, shp)
    y_perm = _out(y_perm, "y_perm", shape.act_dtype, (T * k, d), x_perm.device, stream)
    st = lib().moe_expert_ffn(ctypes.byref(shape._shared()), _ptr(x_perm), _ptr(offsets),
                              _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(y_perm),
                              *_ws(ws), _stream(stream))
    _check("moe_expert_ffn", st)
    return y_perm


def combine(shape: LayerShape, x, y_perm, topk_idx, topk_gate, slot_row, out=None,
            stream=None):
    T, k, d = shape.T, shape.top_k, shape.d
    _need(x, "x", shape.act_dtype, (T, d))
    _need(y_perm, "y_perm", shape.act_dtype, (T * k, d))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(topk_gate, "topk_gate", torch.float32, (T, k))
    _need(slot_row, "slot_row", torch.int32, (T * k,))
    out = _out(out, "out", shape.act_dtype, (T, d), x.device, stream)
    st = lib().moe_combine(ctypes.byref(shape._shared()), _ptr(x), _ptr(y_perm),
                           _ptr(topk_idx), _ptr(topk_gate), _ptr(slot_row), _ptr(out),
                           _stream(stream))
    _check("moe_combine", st)
    return out


def ep_local_experts(shape: LayerShape, rank: int, world: int) -> int:
    """Routed experts rank `rank` owns when the N routed ids are split evenly
    over `world` ranks (the first N % world ranks take one more)."""
    n = int(lib().moe_ep_local_experts(ctypes.byref(shape._shared()), rank, world))
    if n < 0:
        raise ValueError(f"invalid rank {rank} of {world} or shape {shape}")
    return n


def _pointer_array(tensors, dtype, rows_min, d, device):
    """Device array of the data addresses of `tensors` (one per rank)."""
    for r, t in enumerate(tensors):
        _need(t, f"buffer of rank {r}", dtype)
        if t.dim() != 2 or t.shape[1] != d or t.shape[0] < rows_min:
            raise ValueError(f"buffer of rank {r}: shape {tuple(t.shape)}, expected "
                             f"[>= {rows_min}, {d}]")
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device=device)


def ep_plan(shape: LayerShape, rank: int, world: int, counts_all, stream=None):
    """-> (dest_row [N], recv_offsets [n_rank + 1]) from every rank's counts
    (counts_all [world, E] int32, on the device)."""
    N, E = shape.n_routed, shape.E
    _need(counts_all, "counts_all", torch.int32, (world, E))
    dev = counts_all.device
    dest_row = _new((N,), torch.int32, dev, stream)
    recv_offsets = _new((ep_local_experts(shape, rank, world) + 1,), torch.int32, dev, stream)
    st = lib().moe_ep_plan(ctypes.byref(shape._shared()), rank, world, _ptr(counts_all),
                           _ptr(dest_row), _ptr(recv_offsets), _stream(stream))
    _check("moe_ep_plan", st)
    return dest_row, recv_offsets


def ep_dispatch(shape: LayerShape, world: int, x, offsets, row_token, dest_row, recv_bufs,
                stream=None):
    """Sends this rank's routed rows into the owners' receive buffers
    (recv_bufs: one [rows, d] tensor per rank, each with room for every row
    its experts get)."""
    T, k, d, N = shape.T, shape.top_k, shape.d, shape.n_routed
    _need(x, "x", shape.act_dtype, (T, d))
    _need(offsets, "offsets", torch.int32, (N + 1,))
    _need(row_token, "row_token", torch.int32, (T * k,))
    _need(dest_row, "dest_row", torch.int32, (N,))
    if len(recv_bufs) != world:
        raise ValueError("one receive buffer per rank")
    ptrs = _pointer_array(recv_bufs, shape.act_dtype, 0, d, x.device)
    st = lib().moe_ep_dispatch(ctypes.byref(shape._shared()), world, _ptr(x), _ptr(offsets),
                               _ptr(row_token), _ptr(dest_row), _ptr(ptrs), _stream(stream))
    _check("moe_ep_dispatch", st)
    return ptrs  # kept alive by the caller until the stream has run the kernel


def ep_return(shape: LayerShape, rank: int, world: int, y_recv, recv_offsets, counts_all,
              offsets_all, y_homes, stream=None):
    """Sends this rank's expert output rows back into every source rank's
    y_perm (y_homes: one [T*k, d] tensor per rank)."""
    T, k, d, N, E = shape.T, shape.top_k, shape.d, shape.n_routed, shape.E
    _need(y_recv, "y_recv", shape.act_dtype)
    _need(recv_offsets, "recv_offsets", torch.int32,
          (ep_local_experts(shape, rank, world) + 1,))
    _need(counts_all, "counts_all", torch.int32, (world, E))
    _need(offsets_all, "offsets_all", torch.int32, (world, N + 1))
    if len(y_homes) != world:
        raise ValueError("one y_perm per rank")
    ptrs = _pointer_array(y_homes, shape.act_dtype, T * k, d, y_recv.device)
    st = lib().moe_ep_return(ctypes.byref(shape._shared()), rank, world, _ptr(y_recv),
                             _ptr(recv_offsets), _ptr(counts_all), _ptr(offsets_all),
                             _ptr(ptrs), _stream(stream))
    _check("moe_ep_return", st)
    return ptrs


def layer_forward(shape: LayerShape, x, w_router, bias, w_gate, w_up, w_down, ws,
                  out=None, counts=None, stream=None):
    """The whole layer -> out [T, d]; counts [E] (optional) gets slots per expert."""
    T, d, F, N, E = shape.T, shape.d, shape.ffn, shape.n_routed, shape.E
    _need(x, "x", shape.act_dtype, (T, d))
    _need(w_router, "w_router", torch.float32, (E, d))
    _need(bias, "bias", torch.float32, (E,))
    if N > 0:
        for name, w, shp in (("w_gate", w_gate, (N, F, d)), ("w_up", w_up, (N, F, d)),
                             ("w_down", w_down, (N, d, F))):
            _need(w, name, shape.act_dtype, shp)
    out = _out(out, "out", shape.act_dtype, (T, d), x.device, stream)
    if counts is not None:
        _need(counts, "counts", torch.int32, (E,))
    st = lib().moe_layer_forward(ctypes.byref(shape._shared()), _ptr(x), _ptr(w_router),
                                 _ptr(bias), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                 _ptr(out), _ptr(counts), *_ws(ws),
                                 _stream(stream))
    _check("moe_layer_forward", st)
    return out


def layer_forward_host(shape: LayerShape, x_host, w_router, bias, w_gate, w_up,
                       w_down, ws, out_host, counts_host=None, stream=None):
    """The whole layer with x and out in (pinned) host memory; asynchronous:
    synchronise the stream before reading out_host."""
    T, d, E = shape.T, shape.d, shape.E
    F, N = shape.ffn, shape.n_routed
    _need(x_host, "x_host", shape.act_dtype, (T, d), on_device=False)
    _need(out_host, "out_host", shape.act_dtype, (T, d), on_device=False)
    if counts_host is not None:
        _need(counts_host, "counts_host", torch.int32, (E,), on_device=False)
    _need(w_router, "w_router", torch.float32, (E, d))
    _need(bias, "bias", torch.float32, (E,))
    if N > 0:
        for name, w, shp in (("w_gate", w_gate, (N, F, d)), ("w_up", w_up, (N, F, d)),
                             ("w_down", w_down, (N, d, F))):
            _need(w, name, shape.act_dtype, shp)
    st = lib().moe_layer_forward_host(ctypes.byref(shape._shared()), _ptr(x_host),
                                      _ptr(w_router), _ptr(bias), _ptr(w_gate),
                                      _ptr(w_up), _ptr(w_down), _ptr(out_host),
                                      _ptr(counts_host), *_ws(ws),
                                      _stream(stream))
    _check("moe_layer_forward_host", st)
    return out_host


def read_device_error(ws, stream=None) -> int:
    """Waits for the stream; returns (and clears) the workspace error word."""
    code = ctypes.c_int32(0)
    lib().moe_read_device_error(_ws(ws)[0], ctypes.byref(code), _stream(stream))
    return int(code.value)


def selftest_wait_limit(ws, stream=None) -> None:
    """Runs the device-side wait-limit self-test: after ~2 s the workspace
    error word holds 1 (read it with read_device_error)."""
    _check("moe_selftest_wait_limit",
           lib().moe_selftest_wait_limit(*_ws(ws),
                                         _stream(stream)))


def bias_pid_update(shape: LayerShape, counts, bias, state, target: float, kp: float,
                    ki: float = 0.0, kd: float = 0.0, max_step: float = 1.0,
                    stream=None):
    """One PID step on the zero experts' router bias (in place on `bias` and
    `state`), from the per-expert counts of the last layer call."""
    _need(counts, "counts", torch.int32, (shape.E,))
    _need(bias, "bias", torch.float32, (shape.E,))
    _need(state, "state", torch.float64, (2,))
    prm = MoEPIDParams(target, kp, ki, kd, max_step)
    st = lib().moe_bias_pid_update(ctypes.byref(shape._shared()), _ptr(counts), _ptr(bias),
                                   _ptr(state), ctypes.byref(prm), _stream(stream))
    _check("moe_bias_pid_update", st)
    return bias, state


# ------------------------------------------------------------------ training --
def _on_current_device(*tensors):
    """Refuses tensors of another device than the current one, whose kernels
    could not read them."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, but the current device is cuda:{dev}")


def alloc_grouped_workspace(shape: GroupedShape, device="cuda") -> torch.Tensor:
    """Zeroed workspace of the grouped products (the error word and counters)."""
    n = int(lib().moe_grouped_workspace_size(ctypes.byref(shape._shared())))
    if n == 0:
        raise ValueError(f"invalid or unsupported shape {shape}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def grouped_matmul(shape: GroupedShape, x, w, offsets, ws, out=None, stream=None):
    """Ragged products y[r] = w[e] x[r] for the rows r of each segment
    [offsets[e], offsets[e+1]) -> y [rows, n_out] (rows from offsets[groups] on
    untouched)."""
    R, G, I, O = shape.rows, shape.groups, shape.n_in, shape.n_out
    _need(x, "x", shape.dtype, (R, I))
    _need(w, "w", shape.dtype, (G, O, I))
    _need(offsets, "offsets", torch.int32, (G + 1,))
    out = _out(out, "out", shape.dtype, (R, O), x.device, stream)
    _on_current_device(x, w, offsets, ws, out)
    st = lib().moe_grouped_matmul(ctypes.byref(shape._shared()), _ptr(x), _ptr(w), _ptr(offsets),
                                  _ptr(out), *_ws(ws), _stream(stream))
    _check("moe_grouped_matmul", st)
    return out


def grouped_matmul_dx(shape: GroupedShape, dy, w, offsets, ws, out=None, stream=None):
    """Ragged products dx[r] = w[e]^T dy[r] -> dx [rows, n_in]: the input
    gradient of grouped_matmul (rows from offsets[groups] on untouched)."""
    R, G, I, O = shape.rows, shape.groups, shape.n_in, shape.n_out
    _need(dy, "dy", shape.dtype, (R, O))
    _need(w, "w", shape.dtype, (G, O, I))
    _need(offsets, "offsets", torch.int32, (G + 1,))
    out = _out(out, "out", shape.dtype, (R, I), dy.device, stream)
    _on_current_device(dy, w, offsets, ws, out)
    st = lib().moe_grouped_matmul_dx(ctypes.byref(shape._shared()), _ptr(dy), _ptr(w),
                                     _ptr(offsets), _ptr(out), *_ws(ws), _stream(stream))
    _check("moe_grouped_matmul_dx", st)
    return out


def grouped_matmul_dw(shape: GroupedShape, dy, x, offsets, ws, out=None, stream=None):
    """Ragged products dw[e] = sum over e's rows of dy[r] x[r]^T -> dw [groups,
    n_out, n_in]: the weight gradient of grouped_matmul, in the operands' type
    or, when `out` is float32, in fp32. A segment without rows gives zeros."""
    R, G, I, O = shape.rows, shape.groups, shape.n_in, shape.n_out
    _need(dy, "dy", shape.dtype, (R, O))
    _need(x, "x", shape.dtype, (R, I))
    _need(offsets, "offsets", torch.int32, (G + 1,))
    f32 = out is not None and out.dtype == torch.float32
    out = _out(out, "out", torch.float32 if f32 else shape.dtype, (G, O, I), x.device, stream)
    _on_current_device(dy, x, offsets, ws, out)
    st = lib().moe_grouped_matmul_dw(ctypes.byref(shape._shared()), _ptr(dy), _ptr(x),
                                     _ptr(offsets), _ptr(out), _DTYPE_CODE[out.dtype],
                                     *_ws(ws), _stream(stream))
    _check("moe_grouped_matmul_dw", st)
    return out


def alloc_backward_workspace(shape: LayerShape, device="cuda") -> torch.Tensor:
    """Workspace of the backward calls (its first 256 bytes zeroed: the error
    word must start at zero)."""
    n = int(lib().moe_backward_workspace_size(ctypes.byref(shape._shared())))
    if n == 0:
        raise ValueError(f"invalid or unsupported shape {shape}")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def combine_backward(shape: LayerShape, dout, x, y_perm, topk_idx, topk_gate, slot_row,
                     dy_perm=None, dgate=None, stream=None):
    """Gradients of combine -> (dy_perm [T*k, d], dgate [T, k] f32); rows of
    dy_perm behind the routed ones are untouched."""
    T, k, d = shape.T, shape.top_k, shape.d
    _need(dout, "dout", shape.act_dtype, (T, d))
    _need(x, "x", shape.act_dtype, (T, d))
    _need(y_perm, "y_perm", shape.act_dtype, (T * k, d))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(topk_gate, "topk_gate", torch.float32, (T, k))
    _need(slot_row, "slot_row", torch.int32, (T * k,))
    dy_perm = _out(dy_perm, "dy_perm", shape.act_dtype, (T * k, d), x.device, stream)
    dgate = _out(dgate, "dgate", torch.float32, (T, k), x.device, stream)
    _on_current_device(dout, x, y_perm, topk_idx, topk_gate, slot_row, dy_perm, dgate)
    st = lib().moe_combine_backward(ctypes.byref(shape._shared()), _ptr(dout), _ptr(x),
                                    _ptr(y_perm), _ptr(topk_idx), _ptr(topk_gate),
                                    _ptr(slot_row), _ptr(dy_perm), _ptr(dgate),
                                    _stream(stream))
    _check("moe_combine_backward", st)
    return dy_perm, dgate


def _weight_grads(shape, dw_gate, dw_up, dw_down, device, stream):
    """The experts' weight gradients (given or new) and their common type: the
    activation type unless the given ones are float32."""
    N, F, d = shape.n_routed, shape.ffn, shape.d
    given = [t for t in (dw_gate, dw_up, dw_down) if t is not None]
    dtype = given[0].dtype if given else shape.act_dtype
    if dtype not in (shape.act_dtype, torch.float32):
        raise ValueError(f"weight gradients: dtype {dtype}, expected {shape.act_dtype} "
                         "or torch.float32")
    out = tuple(_out(t, n, dtype, s, device, stream) for n, t, s in (
        ("dw_gate", dw_gate, (N, F, d)), ("dw_up", dw_up, (N, F, d)),
        ("dw_down", dw_down, (N, d, F))))
    return out, _DTYPE_CODE[dtype]


def _need_experts(shape, w_gate, w_up, w_down):
    N, F, d = shape.n_routed, shape.ffn, shape.d
    for name, w, shp in (("w_gate", w_gate, (N, F, d)), ("w_up", w_up, (N, F, d)),
                         ("w_down", w_down, (N, d, F))):
        _need(w, name, shape.act_dtype, shp)


def expert_ffn_backward(shape: LayerShape, x_perm, offsets, w_gate, w_up, w_down, dy_perm, ws,
                        dx_perm=None, dw_gate=None, dw_up=None, dw_down=None, stream=None):
    """Gradients of expert_ffn -> (dx_perm [T*k, d], dw_gate, dw_up [N, F, d],
    dw_down [N, d, F]); the pre-activations are computed again. Weight gradients
    come in the activation type, or in float32 when given as such. Rows of
    dx_perm behind the routed ones are untouched."""
    T, k, d = shape.T, shape.top_k, shape.d
    _need(x_perm, "x_perm", shape.act_dtype, (T * k, d))
    _need(offsets, "offsets", torch.int32, (shape.n_routed + 1,))
    _need_experts(shape, w_gate, w_up, w_down)
    _need(dy_perm, "dy_perm", shape.act_dtype, (T * k, d))
    dx_perm = _out(dx_perm, "dx_perm", shape.act_dtype, (T * k, d), x_perm.device, stream)
    dws, code = _weight_grads(shape, dw_gate, dw_up, dw_down, x_perm.device, stream)
    _on_current_device(x_perm, offsets, w_gate, w_up, w_down, dy_perm, ws, dx_perm, *dws)
    st = lib().moe_expert_ffn_backward(ctypes.byref(shape._shared()), _ptr(x_perm), _ptr(offsets),
                                       _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(dy_perm),
                                       _ptr(dx_perm), *[_ptr(t) for t in dws], code,
                                       *_ws(ws), _stream(stream))
    _check("moe_expert_ffn_backward", st)
    return (dx_perm, *dws)


def input_backward(shape: LayerShape, dout, x, w_router, topk_idx, topk_gate, slot_row, dgate,
                   dx_perm, ws, dx=None, dw_router=None, stream=None):
    """Gradients of the layer input (through the experts, the zero experts and
    the router) and of the router weights -> (dx [T, d], dw_router [E, d] f32)."""
    T, k, d, E = shape.T, shape.top_k, shape.d, shape.E
    _need(dout, "dout", shape.act_dtype, (T, d))
    _need(x, "x", shape.act_dtype, (T, d))
    _need(w_router, "w_router", torch.float32, (E, d))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(topk_gate, "topk_gate", torch.float32, (T, k))
    _need(slot_row, "slot_row", torch.int32, (T * k,))
    _need(dgate, "dgate", torch.float32, (T, k))
    _need(dx_perm, "dx_perm", shape.act_dtype, (T * k, d))
    dx = _out(dx, "dx", shape.act_dtype, (T, d), x.device, stream)
    dw_router = _out(dw_router, "dw_router", torch.float32, (E, d), x.device, stream)
    _on_current_device(dout, x, w_router, topk_idx, topk_gate, slot_row, dgate, dx_perm,
                       ws, dx, dw_router)
    st = lib().moe_input_backward(ctypes.byref(shape._shared()), _ptr(dout), _ptr(x),
                                  _ptr(w_router), _ptr(topk_idx), _ptr(topk_gate),
                                  _ptr(slot_row), _ptr(dgate), _ptr(dx_perm), _ptr(dx),
                                  _ptr(dw_router), *_ws(ws), _stream(stream))
    _check("moe_input_backward", st)
    return dx, dw_router


def layer_backward(shape: LayerShape, dout, x, w_router, w_gate, w_up, w_down, topk_idx,
                   topk_gate, offsets, slot_row, x_perm, y_perm, ws, dx=None, dw_router=None,
                   dw_gate=None, dw_up=None, dw_down=None, stream=None):
    """The whole layer's backward pass, from what route, dispatch and expert_ffn
    gave in the forward pass -> (dx, dw_router, dw_gate, dw_up, dw_down).
    combine_backward, expert_ffn_backward and input_backward in one call, bit
    for bit."""
    T, k, d, E, N = shape.T, shape.top_k, shape.d, shape.E, shape.n_routed
    _need(dout, "dout", shape.act_dtype, (T, d))
    _need(x, "x", shape.act_dtype, (T, d))
    _need(w_router, "w_router", torch.float32, (E, d))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(topk_gate, "topk_gate", torch.float32, (T, k))
    _need(slot_row, "slot_row", torch.int32, (T * k,))
    if N > 0:
        _need_experts(shape, w_gate, w_up, w_down)
        _need(offsets, "offsets", torch.int32, (N + 1,))
        _need(x_perm, "x_perm", shape.act_dtype, (T * k, d))
        _need(y_perm, "y_perm", shape.act_dtype, (T * k, d))
    dx = _out(dx, "dx", shape.act_dtype, (T, d), x.device, stream)
    dw_router = _out(dw_router, "dw_router", torch.float32, (E, d), x.device, stream)
    dws, code = _weight_grads(shape, dw_gate, dw_up, dw_down, x.device, stream)
    _on_current_device(dout, x, w_router, w_gate, w_up, w_down, topk_idx, topk_gate, offsets,
                       slot_row, x_perm, y_perm, ws, dx, dw_router, *dws)
    st = lib().moe_layer_backward(ctypes.byref(shape._shared()), _ptr(dout), _ptr(x),
                                  _ptr(w_router), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                  _ptr(topk_idx), _ptr(topk_gate), _ptr(offsets),
                                  _ptr(slot_row), _ptr(x_perm), _ptr(y_perm), _ptr(dx),
                                  _ptr(dw_router), *[_ptr(t) for t in dws], code, *_ws(ws),
                                  _stream(stream))
    _check("moe_layer_backward", st)
    return (dx, dw_router, *dws)


ADAMW_BLOCK = 256  # elements per state block
_DATA_PTR = torch.Tensor.data_ptr


def _capturing(stream=None) -> bool:
    """Whether the call's stream is being captured into a graph."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with _on(stream):
        return torch.cuda.is_current_stream_capturing()


class AdamW:
    """The states of an AdamW optimizer over fixed weights and gradient buffers
    (step it with adamw_step). The tensors are kept alive and updated in place.
    Weights, masters and states stay in the memory they had at construction: a
    step refuses one that has moved since (a replayed step cannot).

    A step reads what the tensors of ``grads`` hold then. One that lies in other
    memory than at the step before (its ``data`` assigned, or another tensor put
    in its place) is checked anew and taken up, for which the step waits for the
    device; a step under capture refuses it. A replayed step reads the memory of
    its capture, which is kept alive.

    params: float32 or bfloat16 CUDA tensors, one type for all; grads: tensors
    of the same sizes, one type for all. master: float32 copies of bfloat16
    weights that the steps update instead (the weights get them rounded).
    state_bits 32 keeps both moments in float32 (``m``, ``v``); 8 keeps e4m3
    codes and one scale per 256 elements (``m`` and ``v`` are then (codes,
    scales); v holds the root of the second moment). The buffers are flat, each
    tensor padded to whole blocks of 256.
    """

    def __init__(self, params, grads, state_bits: int = 32, master=None):
        params, grads = list(params), list(grads)
        master = list(master) if master is not None else [None] * len(params)
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits: {state_bits}, expected 8 or 32")
        if not params or len(grads) != len(params) or len(master) != len(params):
            raise ValueError("one gradient (and master) per weight, and at least one weight")
        pdt, gdt = params[0].dtype, grads[0].dtype
        for what, dt in (("params", pdt), ("grads", gdt)):
            if dt not in _DTYPE_CODE:
                raise ValueError(f"{what}: dtype {dt}, expected float32 or bfloat16")
        if any(w is not None for w in master) and pdt != torch.bfloat16:
            raise ValueError("master: only for bfloat16 weights")
        self._check_tensors(params, grads, master, pdt, gdt)
        self.params, self.grads, self.master = params, grads, master
        self.state_bits = state_bits
        self._mastered = any(w is not None for w in master)
        dev = params[0].device
        self._memory = [t.detach() for t in params + master if t is not None]
        sizes = [p.numel() for p in params]
        at = sum(-(-n // ADAMW_BLOCK) for n in sizes)
        self.total_blocks = at
        self._c = MoEAdamW(sum(n > 0 for n in sizes), state_bits, _DTYPE_CODE[pdt],
                           _DTYPE_CODE[gdt], at)
        self._kept = []  # what captured steps read, once the gradients have moved
        self._captured = False
        n = at * ADAMW_BLOCK
        if state_bits == 32:
            self.m = torch.zeros(n, device=dev)
            self.v = torch.zeros(n, device=dev)
        else:
            self.m, self.v = ((torch.zeros(n, dtype=torch.float8_e4m3fn, device=dev),
                               torch.zeros(at, device=dev)) for _ in range(2))
        self.state = torch.zeros(2, dtype=torch.int64, device=dev)  # step count, scratch
        self._memory += [t.detach() for t in (*((self.m, self.v) if state_bits == 32 else
                                                (*self.m, *self.v)), self.state)]
        self._take_gradients()
        self._addresses = self._lie_at()

    @classmethod
    def _check_tensors(cls, params, grads, master, pdt, gdt):
        for i, (p, g, w) in enumerate(zip(params, grads, master)):
            _need(p, f"params[{i}]", pdt)
            _need(g, f"grads[{i}]", gdt, p.shape)
            if w is not None:
                _need(w, f"master[{i}]", torch.float32, p.shape)
            for t in (p, g) if w is None else (p, g, w):
                if t.device != params[0].device:
                    raise ValueError("all tensors must be on one device")
                if t.data_ptr() % 16:
                    raise ValueError("every tensor must be 16-byte aligned")
        cls._refuse_overlaps([t for t in params + master if t is not None], grads)

    def _take_gradients(self):
        """The table of all tensors, with the gradients where they lie now."""
        rows, at = [], 0
        for p, g, w in zip(self.params, self.grads, self.master):
            rows.append([p.data_ptr(), 0 if w is None else w.data_ptr(), g.data_ptr(),
                         p.numel(), at, 0])
            at += -(-p.numel() // ADAMW_BLOCK)
        # a tensor without elements has no block: it is left out of the table
        rows = [r for r in rows if r[3] > 0]
        self._table = torch.tensor(rows, dtype=torch.int64).reshape(-1, 6).to(
            self.params[0].device)
        self._grad_memory = [g.detach() for g in self.grads]
        (m, ms), (v, vs) = ((self.m, None), (self.v, None)) if self.state_bits == 32 else (
            self.m, self.v)
        self._pointers = tuple(map(_ptr, (self._table, m, ms, v, vs, self.state)))

    def _moved(self, now, capturing):
        """Something lies in other memory (`now`) than at the last step: only
        gradients may."""
        n = len(self.grads)
        if now[n:] != self._addresses[len(self._grad_memory):]:
            raise ValueError("a weight, master or state has moved to other memory")
        if capturing:
            raise ValueError("a gradient has moved to other memory, which a step under "
                             "capture cannot follow")
        if n != len(self.params):
            raise ValueError("one gradient per weight")
        self._check_tensors(self.params, self.grads, self.master, self.params[0].dtype,
                            self._grad_memory[0].dtype)
        if self._captured:
            self._kept.append((self._table, self._grad_memory))
            self._captured = False
        elif self._table.is_cuda:  # steps in flight still read the table
            torch.cuda.synchronize(self._table.device)
        self._take_gradients()
        self._addresses = now

    def _lie_at(self):
        """Where the gradients and everything that a step writes lie now."""
        states = (self.m, self.v) if self.state_bits == 32 else (*self.m, *self.v)
        masters = [w for w in self.master if w is not None] if self._mastered else ()
        return list(map(_DATA_PTR, [*self.grads, *self.params, *masters, *states, self.state]))

    @staticmethod
    def _refuse_overlaps(written, read):
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), out)
                       for out, ts in ((1, written), (0, read)) for t in ts if t.numel())
        end, end_out = 0, 0  # the furthest end so far, of all spans and of written ones
        for lo, hi, out in spans:
            if lo < (end if out else end_out):
                raise ValueError("a weight or master overlaps another tensor")
            end, end_out = max(end, hi), max(end_out, hi if out else 0)

    def load_state(self, m, v, step: int):
        """Sets the states (in the layout of ``m`` and ``v``) and the number of
        steps taken."""
        pairs = []
        for mine, new, name in ((self.m, m, "m"), (self.v, v, "v")):
            mine, new = (mine, new) if self.state_bits == 8 else ((mine,), (new,))
            if not isinstance(new, (tuple, list)) or len(mine) != len(new):
                raise ValueError(f"{name}: expected (codes, scales)")
            for a, b in zip(mine, new):
                _need(b, name, a.dtype, a.shape)
                pairs.append((a, b))
        if step < 0:
            raise ValueError(f"step: {step}, expected >= 0")
        for a, b in pairs:  # nothing is set unless all of it can be
            a.copy_(b)
        self.state[0] = step


def adamw_step(opt: AdamW, lr: float, beta1: float = 0.9, beta2: float = 0.999,
               eps: float = 1e-8, weight_decay: float = 0.0, stream=None):
    """One AdamW step of every tensor of `opt`, in place, from what its gradients
    hold. The step count lives on the device, so a step captured in a
    CUDA graph counts on when it is replayed (its lr and betas are those of the
    capture)."""
    hyper = MoEAdamWParams(lr, beta1, beta2, eps, weight_decay)
    capturing, now = _capturing(stream), opt._lie_at()
    if now != opt._addresses:
        opt._moved(now, capturing)
    if capturing:
        opt._captured = True
    _on_current_device(opt._table)
    st = lib().moe_adamw_step(opt._c, ctypes.byref(hyper), *opt._pointers, _stream(stream))
    _check("moe_adamw_step", st)
    return opt
