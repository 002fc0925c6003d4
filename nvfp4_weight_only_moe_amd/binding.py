"""Thin ctypes binding of libmoe_w4a16.so (C ABI in include/moe_w4a16.h).

Argument marshalling only: every step of the layer runs in the HIP library.
PyTorch supplies device memory and the current HIP stream.  The entry points
keep the C names; each checks the returned status and raises ``MoeError``.
There is no CPU fallback: if the library is missing, loading raises.
"""

import ctypes
import functools
import os
import re
from dataclasses import dataclass
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_w4a16.so")
HEADER_PATH = os.path.join(os.path.dirname(HERE), "include", "moe_w4a16.h")

MOE_OK = 0
STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_SHAPE", -3: "MOE_ERR_ALIGN",
          -4: "MOE_ERR_UNSUPPORTED", -5: "MOE_ERR_NONFINITE", -6: "MOE_ERR_BAD_SCALE",
          -7: "MOE_ERR_WORKSPACE", -8: "MOE_ERR_HIP"}


class MoeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class NVFP4TensorC(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p)]


class Int4TensorC(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_S = ctypes.c_size_t
_TP = ctypes.POINTER(NVFP4TensorC)
_IP = ctypes.POINTER(Int4TensorC)

_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_w4a16_version": (_I, []),
    "moe_w4a16_quantize_pack": (_I, [_P, _I, _I, _I, _TP, _P]),
    "moe_w4a16_dequantize": (_I, [_TP, _P, _P]),
    "moe_w4a16_validate": (_I, [_TP, _P, _P]),
    "moe_route_workspace_size": (_S, [_I, _I, _I]),
    "moe_route_topk": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_w4a16_workspace_size": (_S, [_I, _I, _I, _I, _I]),
    "moe_w4a16_forward": (_I, [_P, _I, _I, _I, _I, _I, _TP, _TP, _TP, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_w4a16_route_forward": (_I, [_P, _P, _I, _I, _I, _I, _I, _TP, _TP, _TP, _P, _P, _P, _P, _P, _P, _P, _P,
                                     _S, _P]),
    "moe_w4a16_linear_workspace_size": (_S, [_I, _I, _I]),
    "moe_w4a16_linear": (_I, [_P, _I, _I, _I, _TP, _P, _P, _S, _P]),
    "moe_router_logits": (_I, [_P, _I, _I, _P, _I, _P, _P]),
    "moe_w4a16_shared_expert_workspace_size": (_S, [_I, _I, _I]),
    "moe_w4a16_shared_expert": (_I, [_P, _I, _I, _I, _TP, _TP, _TP, _P, _P, _S, _P]),
    "moe_debug_set_prefill_variant": (_I, [_I]),
    "moe_bench_stream_read": (_I, [_P, _S, _P, _P]),
    "moe_nvfp4_quantize_activations": (_I, [_P, _I, _I, ctypes.c_float, _P, _P, _P]),
    "moe_w4a4_workspace_size": (_S, [_I, _I, _I, _I, _I]),
    "moe_w4a4_forward": (_I, [_P, _I, _I, _I, _I, _I, _TP, _TP, _TP, ctypes.c_float, ctypes.c_float,
                              _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_w4a4_route_forward": (_I, [_P, _P, _I, _I, _I, _I, _I, _TP, _TP, _TP, ctypes.c_float, ctypes.c_float,
                                    _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_w4a16_route_forward_noalloc": (_I, [_P, _P, _I, _I, _I, _I, _I, _TP, _TP, _TP, _P, _P, _P, _P, _P, _P, _P,
                                             _P]),
    "moe_router_route_workspace_size": (_S, [_I, _I, _I]),
    "moe_router_route_topk": (_I, [_P, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_grouped_workspace_size": (_S, [_I, _I, _I, _I, _I]),
    "moe_grouped_linear": (_I, [_P, _I, _I, _P, _I, _I, _P, _P, _I, _I, _P, _P, _S, _P]),
    "moe_grouped_swiglu": (_I, [_P, _I, _I, _P, _P, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _S, _P]),
    "moe_grouped_linear_dgrad": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _S, _P]),
    "moe_grouped_swiglu_dgrad": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _S, _P]),
    "moe_grouped_linear_wgrad_workspace_size": (_S, [_I, _I, _I, _I]),
    "moe_grouped_linear_wgrad": (_I, [_P, _I, _I, _P, _I, _I, _I, _P, _P, _I, _I, _P, _P, _S, _P]),
    "moe_int4_quantize_pack": (_I, [_P, _IP, _P]),
    "moe_int4_dequantize": (_I, [_IP, _P, _P]),
    "moe_int4_linear": (_I, [_P, _I, _IP, _P, _P, _I, _I, _P, _P]),
    "moe_combine": (_I, [_P, _I, _I, _P, _P, _I, _I, _P, _P]),
    "moe_combine_backward": (_I, [_P, _I, _I, _P, _I, _P, _P, _P, _I, _I, _P, _P, _P, _P]),
    "moe_profile_begin": (_I, [_I]),
    "moe_profile_end": (_I, [_P, _P, _P, _I]),
}


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def header_symbols():
    """Names of the functions include/moe_w4a16.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_\w+)\s*\(", text)))


def status_string(status):
    return lib().moe_status_string(int(status)).decode()


def _check(status, where):
    if status != MOE_OK:
        raise MoeError(status, where)


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


_BITS16 = (torch.int16, torch.uint16, torch.bfloat16) if hasattr(torch, "uint16") else (torch.int16, torch.bfloat16)


def _dev_tensor(t, name, dtype=None, shape=None, min_bytes=None):
    """The C ABI takes bare pointers and (for outputs) no sizes, so the
    binding checks every tensor before the call: a device tensor,
    contiguous, of the expected dtype(s) and exact shape (or at least
    `min_bytes`).  Raises ValueError instead of calling into the library."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: expected a device (cuda) tensor, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None:
        ok = dtype if isinstance(dtype, tuple) else (dtype,)
        if t.dtype not in ok:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in ok)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if min_bytes is not None and t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, at least {min_bytes} needed")
    return t


@dataclass
class NVFP4Tensor:
    """E experts of an [N, K] NVFP4 projection in canonical layout (device)."""
    codes: torch.Tensor         # uint8 [E, N, K/2]
    scales: torch.Tensor        # uint8 [E, N, K/16]
    global_scale: torch.Tensor  # float32 [E]

    @property
    def shape(self):
        E, N, half = self.codes.shape
        return E, N, half * 2

    def check(self, name="tensor"):
        E, N, K = self.shape
        _dev_tensor(self.codes, f"{name}.codes", torch.uint8, (E, N, K // 2))
        _dev_tensor(self.scales, f"{name}.scales", torch.uint8, (E, N, K // 16))
        _dev_tensor(self.global_scale, f"{name}.global_scale", torch.float32, (E,))
        return self

    def cstruct(self):
        self.check()
        E, N, K = self.shape
        return NVFP4TensorC(E, N, K, self.codes.data_ptr(), self.scales.data_ptr(),
                            self.global_scale.data_ptr())

    @staticmethod
    def empty(E, N, K, device="cuda"):
        return NVFP4Tensor(torch.empty((E, N, K // 2), dtype=torch.uint8, device=device),
                           torch.empty((E, N, K // 16), dtype=torch.uint8, device=device),
                           torch.empty((E,), dtype=torch.float32, device=device))


def moe_w4a16_version():
    return int(lib().moe_w4a16_version())


def moe_w4a16_quantize_pack(w, out=None, stream=None):
    """fp32 masters [E, N, K] (device) -> NVFP4Tensor."""
    _dev_tensor(w, "w", torch.float32)
    E, N, K = w.shape
    out = NVFP4Tensor.empty(E, N, K, w.device) if out is None else out
    if out.shape != (E, N, K):
        raise ValueError(f"out: shape {out.shape}, expected {(E, N, K)}")
    st = out.cstruct()
    _check(lib().moe_w4a16_quantize_pack(_ptr(w), E, N, K, ctypes.byref(st), _stream(stream)),
           "moe_w4a16_quantize_pack")
    return out


def moe_w4a16_dequantize(t, out=None, stream=None):
    E, N, K = t.shape
    out = torch.empty((E, N, K), dtype=torch.float32, device=t.codes.device) if out is None else out
    _dev_tensor(out, "out", torch.float32, (E, N, K))
    st = t.cstruct()
    _check(lib().moe_w4a16_dequantize(ctypes.byref(st), _ptr(out), _stream(stream)), "moe_w4a16_dequantize")
    return out


def moe_w4a16_validate(t, flag=None, stream=None):
    """Synchronises; raises MoeError on a bad scale.  `flag`: an optional
    caller-owned device tensor of at least 4 bytes (allocated here if None)."""
    flag = torch.empty((4,), dtype=torch.int32, device=t.codes.device) if flag is None else flag
    _dev_tensor(flag, "flag", min_bytes=4)
    st = t.cstruct()
    _check(lib().moe_w4a16_validate(ctypes.byref(st), _ptr(flag), _stream(stream)), "moe_w4a16_validate")


def moe_route_workspace_size(T, E, k):
    return int(lib().moe_route_workspace_size(T, E, k))


def moe_w4a16_workspace_size(T, H, I, E, k):
    return int(lib().moe_w4a16_workspace_size(T, H, I, E, k))


@dataclass
class Routing:
    topk_ids: torch.Tensor      # int32 [T, k]
    topk_w: torch.Tensor        # float32 [T, k]
    counts: torch.Tensor        # int32 [E]
    offsets: torch.Tensor       # int32 [E + 1]
    sorted_slots: torch.Tensor  # int32 [T * k]
    slot_pos: torch.Tensor      # int32 [T * k]
    ws: torch.Tensor            # uint8 workspace

    @staticmethod
    def empty(T, E, k, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        return Routing(torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=device),
                       torch.empty((E,), **i32), torch.empty((E + 1,), **i32),
                       torch.empty((T * k,), **i32), torch.empty((T * k,), **i32),
                       torch.empty((max(moe_route_workspace_size(T, E, k), 16),), dtype=torch.uint8,
                                   device=device))

    def check(self, T, E, k):
        i32 = torch.int32
        _dev_tensor(self.topk_ids, "routing.topk_ids", i32, (T, k))
        _dev_tensor(self.topk_w, "routing.topk_w", torch.float32, (T, k))
        _dev_tensor(self.counts, "routing.counts", i32, (E,))
        _dev_tensor(self.offsets, "routing.offsets", i32, (E + 1,))
        _dev_tensor(self.sorted_slots, "routing.sorted_slots", i32, (T * k,))
        _dev_tensor(self.slot_pos, "routing.slot_pos", i32, (T * k,))
        _dev_tensor(self.ws, "routing.ws", torch.uint8, min_bytes=moe_route_workspace_size(T, E, k))
        return self


def moe_route_topk(logits, k, out=None, stream=None):
    """fp32 logits [T, E] (device) -> Routing."""
    _dev_tensor(logits, "logits", torch.float32)
    T, E = logits.shape
    r = Routing.empty(T, E, k, logits.device) if out is None else out
    r.check(T, E, k)
    _check(lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(r.topk_ids), _ptr(r.topk_w), _ptr(r.counts),
                                _ptr(r.offsets), _ptr(r.sorted_slots), _ptr(r.slot_pos), _ptr(r.ws),
                                r.ws.numel(), _stream(stream)), "moe_route_topk")
    return r


def forward_workspace(T, H, I, E, k, device="cuda"):
    """A forward workspace (needs no initialisation)."""
    return torch.empty((max(moe_w4a16_workspace_size(T, H, I, E, k), 256),), dtype=torch.uint8, device=device)


def moe_bench_stream_read(src, nbytes, sink, stream=None):
    """Stream-read the first nbytes of the device tensor src (a benchmark
    reference; see the header); sink: a device int32/uint32 tensor of >= 1
    element."""
    _dev_tensor(src, "src", min_bytes=nbytes)
    _dev_tensor(sink, "sink", min_bytes=4)
    _check(lib().moe_bench_stream_read(_ptr(src), int(nbytes), _ptr(sink), _stream(stream)), "moe_bench_stream_read")


def moe_debug_set_prefill_variant(variant):
    _check(lib().moe_debug_set_prefill_variant(int(variant)), "moe_debug_set_prefill_variant")


def moe_w4a16_forward(x_bits, gate, up, down, routing, out=None, ws=None, stream=None):
    """bf16 activations (int16/uint16 bit patterns or torch.bfloat16) [T, H] ->
    bf16 bits [T, H] (int16 tensor; view as torch.bfloat16 for values)."""
    _dev_tensor(x_bits, "x", _BITS16)
    T, H = x_bits.shape
    E, I, _ = gate.shape
    k = routing.topk_ids.shape[1]
    routing.check(T, E, k)
    out = torch.empty((T, H), dtype=torch.int16, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", _BITS16, (T, H))
    ws = forward_workspace(T, H, I, E, k, x_bits.device) if ws is None else ws
    _dev_tensor(ws, "ws", min_bytes=moe_w4a16_workspace_size(T, H, I, E, k))
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().moe_w4a16_forward(_ptr(x_bits), T, H, I, E, k, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                   _ptr(routing.topk_ids), _ptr(routing.topk_w), _ptr(routing.counts),
                                   _ptr(routing.offsets), _ptr(routing.sorted_slots), _ptr(routing.slot_pos),
                                   _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "moe_w4a16_forward")
    return out


def moe_w4a16_route_forward(logits, x_bits, gate, up, down, k, routing=None, out=None, ws=None, stream=None):
    """Route (as moe_route_topk, outputs stored in `routing`) and run the
    layer (with one token the gate/up kernel routes itself).  Returns
    (out, routing)."""
    _dev_tensor(x_bits, "x", _BITS16)
    T, H = x_bits.shape
    E, I, _ = gate.shape
    _dev_tensor(logits, "logits", torch.float32, (T, E))
    routing = Routing.empty(T, E, k, x_bits.device) if routing is None else routing
    routing.check(T, E, k)
    out = torch.empty((T, H), dtype=torch.int16, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", _BITS16, (T, H))
    ws = forward_workspace(T, H, I, E, k, x_bits.device) if ws is None else ws
    _dev_tensor(ws, "ws", min_bytes=moe_w4a16_workspace_size(T, H, I, E, k))
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().moe_w4a16_route_forward(_ptr(logits), _ptr(x_bits), T, H, I, E, k, ctypes.byref(g), ctypes.byref(u),
                                         ctypes.byref(d), _ptr(routing.topk_ids), _ptr(routing.topk_w),
                                         _ptr(routing.counts), _ptr(routing.offsets), _ptr(routing.sorted_slots),
                                         _ptr(routing.slot_pos), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_w4a16_route_forward")
    return out, routing


def moe_profile_begin(max_launches=4096):
    _check(lib().moe_profile_begin(max_launches), "moe_profile_begin")


def moe_profile_end(max_names=64):
    """Synchronises; returns {kernel name: (launches, total ms)}."""
    names = (ctypes.c_char * 64 * max_names)()
    counts = (ctypes.c_int32 * max_names)()
    ms = (ctypes.c_double * max_names)()
    n = lib().moe_profile_end(ctypes.cast(names, ctypes.c_void_p), ctypes.cast(counts, ctypes.c_void_p),
                              ctypes.cast(ms, ctypes.c_void_p), max_names)
    return {names[i].value.decode(): (int(counts[i]), float(ms[i])) for i in range(n)}


def moe_router_logits(x_bits, wr_bits, out=None, stream=None):
    """Router logits: bf16 bits x [T, H] and router weight [E, H] (int16
    tensors) -> fp32 [T, E]."""
    _dev_tensor(x_bits, "x", _BITS16)
    _dev_tensor(wr_bits, "wr", _BITS16)
    T, H = x_bits.shape
    E, H2 = wr_bits.shape
    if H2 != H:
        raise ValueError(f"wr: {H2} columns, x has {H}")
    out = torch.empty((T, E), dtype=torch.float32, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", torch.float32, (T, E))
    _check(lib().moe_router_logits(_ptr(x_bits), T, H, _ptr(wr_bits), E, _ptr(out), _stream(stream)),
           "moe_router_logits")
    return out


def moe_w4a16_linear(x_bits, w, out=None, ws=None, stream=None):
    """Dense projection: bf16 bits [T, K] and an NVFP4 tensor with E = 1,
    shape [1, N, K] -> bf16 bits [T, N] (int16 tensor)."""
    _dev_tensor(x_bits, "x", _BITS16)
    T, K = x_bits.shape
    E, N, K2 = w.shape
    if E != 1 or K2 != K:
        raise ValueError(f"w: shape {(E, N, K2)}, expected (1, N, {K})")
    out = torch.empty((T, N), dtype=torch.int16, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", _BITS16, (T, N))
    if ws is None:
        ws = torch.empty((max(lib().moe_w4a16_linear_workspace_size(max(T, 1), K, N), 256),), dtype=torch.uint8,
                         device=x_bits.device)
    _dev_tensor(ws, "ws", min_bytes=lib().moe_w4a16_linear_workspace_size(T, K, N))
    c = w.cstruct()
    _check(lib().moe_w4a16_linear(_ptr(x_bits), T, K, N, ctypes.byref(c), _ptr(out), _ptr(ws), ws.numel(),
                                  _stream(stream)), "moe_w4a16_linear")
    return out


def moe_w4a16_shared_expert(x_bits, gate, up, down, out=None, ws=None, stream=None):
    """The shared expert (one SwiGLU FFN for every token): bf16 bits [T, H]
    and NVFP4 tensors with E = 1 -> bf16 bits [T, H] (int16 tensor)."""
    _dev_tensor(x_bits, "x", _BITS16)
    T, H = x_bits.shape
    E, I, _ = gate.shape
    if E != 1:
        raise ValueError(f"gate: {E} experts, the shared expert has 1")
    out = torch.empty((T, H), dtype=torch.int16, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", _BITS16, (T, H))
    if ws is None:
        ws = torch.empty((max(lib().moe_w4a16_shared_expert_workspace_size(max(T, 1), H, I), 256),),
                         dtype=torch.uint8, device=x_bits.device)
    _dev_tensor(ws, "ws", min_bytes=lib().moe_w4a16_shared_expert_workspace_size(T, H, I))
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().moe_w4a16_shared_expert(_ptr(x_bits), T, H, I, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                         _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_w4a16_shared_expert")
    return out


def _input_scale(s, name):
    """A W4A4 input scale as a Python float; None (a missing scale) is
    refused here, everything else is checked by the library."""
    if s is None:
        raise ValueError(f"{name} is missing: a W4A4 layer needs its static input scale")
    return float(s)


def moe_nvfp4_quantize_activations(x_bits, input_scale, codes=None, scales=None, stream=None):
    """bf16 bits [T, K] -> (codes uint8 [T, K/2], scales uint8 [T, K/16])."""
    s = _input_scale(input_scale, "input_scale")
    _dev_tensor(x_bits, "x", _BITS16)
    T, K = x_bits.shape
    codes = torch.empty((T, K // 2), dtype=torch.uint8, device=x_bits.device) if codes is None else codes
    scales = torch.empty((T, K // 16), dtype=torch.uint8, device=x_bits.device) if scales is None else scales
    _dev_tensor(codes, "codes", torch.uint8, (T, K // 2))
    _dev_tensor(scales, "scales", torch.uint8, (T, K // 16))
    _check(lib().moe_nvfp4_quantize_activations(_ptr(x_bits), T, K, s, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_nvfp4_quantize_activations")
    return codes, scales


def moe_w4a4_workspace_size(T, H, I, E, k):
    return int(lib().moe_w4a4_workspace_size(T, H, I, E, k))


def moe_w4a4_forward(x_bits, gate, up, down, routing, input_scale_x, input_scale_h, out=None, ws=None,
                     stream=None):
    """The W4A4 layer: bf16 bits [T, H] -> bf16 bits [T, H] (int16 tensor)."""
    sx = _input_scale(input_scale_x, "input_scale_x")
    sh = _input_scale(input_scale_h, "input_scale_h")
    _dev_tensor(x_bits, "x", _BITS16)
    T, H = x_bits.shape
    E, I, _ = gate.shape
    k = routing.topk_ids.shape[1]
    routing.check(T, E, k)
    out = torch.empty((T, H), dtype=torch.int16, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", _BITS16, (T, H))
    need = moe_w4a4_workspace_size(T, H, I, E, k)
    ws = torch.empty((max(need, 256),), dtype=torch.uint8, device=x_bits.device) if ws is None else ws
    _dev_tensor(ws, "ws", min_bytes=need)
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().moe_w4a4_forward(_ptr(x_bits), T, H, I, E, k, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                  sx, sh, _ptr(routing.topk_ids), _ptr(routing.topk_w), _ptr(routing.counts),
                                  _ptr(routing.offsets), _ptr(routing.sorted_slots), _ptr(routing.slot_pos),
                                  _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "moe_w4a4_forward")
    return out


def moe_w4a4_route_forward(logits, x_bits, gate, up, down, k, input_scale_x, input_scale_h, routing=None,
                           out=None, ws=None, stream=None):
    """Route (as moe_route_topk, outputs stored in `routing`) and run the W4A4
    layer (with one token the gate/up kernel routes itself).  Returns
    (out, routing)."""
    sx = _input_scale(input_scale_x, "input_scale_x")
    sh = _input_scale(input_scale_h, "input_scale_h")
    _dev_tensor(x_bits, "x", _BITS16)
    T, H = x_bits.shape
    E, I, _ = gate.shape
    _dev_tensor(logits, "logits", torch.float32, (T, E))
    routing = Routing.empty(T, E, k, x_bits.device) if routing is None else routing
    routing.check(T, E, k)
    out = torch.empty((T, H), dtype=torch.int16, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", _BITS16, (T, H))
    need = moe_w4a4_workspace_size(T, H, I, E, k)
    ws = torch.empty((max(need, 256),), dtype=torch.uint8, device=x_bits.device) if ws is None else ws
    _dev_tensor(ws, "ws", min_bytes=need)
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().moe_w4a4_route_forward(_ptr(logits), _ptr(x_bits), T, H, I, E, k, ctypes.byref(g), ctypes.byref(u),
                                        ctypes.byref(d), sx, sh, _ptr(routing.topk_ids), _ptr(routing.topk_w),
                                        _ptr(routing.counts), _ptr(routing.offsets), _ptr(routing.sorted_slots),
                                        _ptr(routing.slot_pos), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_w4a4_route_forward")
    return out, routing


def moe_w4a16_route_forward_noalloc(logits, x_bits, gate, up, down, k, routing=None, out=None, stream=None):
    """moe_w4a16_route_forward with the library's own device array as the
    workspace (no workspace argument, no allocation in the call).  Returns
    (out, routing)."""
    _dev_tensor(x_bits, "x", _BITS16)
    T, H = x_bits.shape
    E, I, _ = gate.shape
    _dev_tensor(logits, "logits", torch.float32, (T, E))
    routing = Routing.empty(T, E, k, x_bits.device) if routing is None else routing
    routing.check(T, E, k)
    out = torch.empty((T, H), dtype=torch.int16, device=x_bits.device) if out is None else out
    _dev_tensor(out, "out", _BITS16, (T, H))
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().moe_w4a16_route_forward_noalloc(_ptr(logits), _ptr(x_bits), T, H, I, E, k, ctypes.byref(g),
                                                 ctypes.byref(u), ctypes.byref(d), _ptr(routing.topk_ids),
                                                 _ptr(routing.topk_w), _ptr(routing.counts), _ptr(routing.offsets),
                                                 _ptr(routing.sorted_slots), _ptr(routing.slot_pos), _ptr(out),
                                                 _stream(stream)), "moe_w4a16_route_forward_noalloc")
    return out, routing


def router_route_workspace(T, E, k, device="cuda"):
    """A workspace for moe_router_route_topk, zero-filled (its ticket word
    must start at zero; every call leaves it zero)."""
    n = int(lib().moe_router_route_workspace_size(T, E, k))
    return torch.zeros((max(n, 256),), dtype=torch.uint8, device=device)


def moe_router_route_topk(x_bits, wr_bits, k, logits=None, routing=None, ws=None, stream=None):
    """Router logits and the route in one call: bf16 bits x [T, H], router
    weight [E, H] -> (fp32 logits [T, E], Routing)."""
    _dev_tensor(x_bits, "x", _BITS16)
    _dev_tensor(wr_bits, "wr", _BITS16)
    T, H = x_bits.shape
    E, H2 = wr_bits.shape
    if H2 != H:
        raise ValueError(f"wr: {H2} columns, x has {H}")
    logits = torch.empty((T, E), dtype=torch.float32, device=x_bits.device) if logits is None else logits
    _dev_tensor(logits, "logits", torch.float32, (T, E))
    routing = Routing.empty(T, E, k, x_bits.device) if routing is None else routing
    routing.check(T, E, k)
    ws = router_route_workspace(T, E, k, x_bits.device) if ws is None else ws
    _dev_tensor(ws, "ws", min_bytes=int(lib().moe_router_route_workspace_size(T, E, k)))
    _check(lib().moe_router_route_topk(_ptr(x_bits), T, H, _ptr(wr_bits), E, k, _ptr(logits), _ptr(routing.topk_ids),
                                       _ptr(routing.topk_w), _ptr(routing.counts), _ptr(routing.offsets),
                                       _ptr(routing.sorted_slots), _ptr(routing.slot_pos), _ptr(ws), ws.numel(),
                                       _stream(stream)), "moe_router_route_topk")
    return logits, routing


# ---------------------------------------------------------------- unquantized and 4-bit integer experts
def _entry(fn):
    """Runs an entry point on the device of its first tensor and on `stream`
    (default: that device's current stream): outputs and workspaces that the
    call allocates belong to the stream that the kernels run on."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, (torch.Tensor, Int4Tensor)):
            raise ValueError(f"{fn.__name__}: {name}: expected a torch.Tensor, got {type(first).__name__}")
        dev = first.get_device()
        if dev < 0:
            raise ValueError(f"{fn.__name__}: expected a device (cuda) tensor, got {first.device}")
        if stream is None:
            if dev == _current_device():
                return fn(*args, **kw)
            with torch.cuda.device(dev):
                return fn(*args, **kw)
        if stream.device != first.device:
            raise ValueError(f"stream: on {stream.device}, the tensors are on {first.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


_I32, _F32, _U8 = (torch.int32,), (torch.float32,), (torch.uint8,)


def _same(t, name, like, dtypes, shape):
    """A contiguous tensor on `like`'s device, of one of the dtypes and of that
    shape; its address.  (One expression for the case that holds: these calls
    are as short as a launch.)"""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.is_contiguous()
            and t.get_device() == like.get_device()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != like.device:
        raise ValueError(f"{name}: on {t.device}, expected {like.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name}: expected a {n}-dimensional torch.Tensor")
    return t.shape


def _new(out, name, like, dtype, shape):
    """`out` checked, or a new tensor."""
    if out is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    _same(out, name, like, _BITS16 if dtype in _BITS16 else (dtype,), shape)
    return out


def _here(t):
    """The current stream of t's device, as the C ABI takes it."""
    return _raw_stream(t.get_device())


# torch.cuda.current_stream() builds an object for the same answer (2.8 us
# against 0.1), torch.cuda.current_device() initialises first (0.26)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _rows(x, sorted_slots):
    """(rows of the result, address of the sorted slots or None)."""
    if sorted_slots is None:
        return x.shape[0], None
    M, = _dims(sorted_slots, "sorted_slots", 1)
    return M, _same(sorted_slots, "sorted_slots", x, _I32, (M,))


GROUPED_ONE, GROUPED_PAIR, GROUPED_SWIGLU = 1, 2, 3


@functools.lru_cache(maxsize=4096)
def moe_grouped_workspace_size(M, E, R, C, products=GROUPED_ONE):
    """Workspace bytes of a grouped product (a function of its sizes alone)."""
    return int(lib().moe_grouped_workspace_size(M, E, R, C, products))


def _workspace(ws, need, like):
    """(address, bytes) of a workspace of at least `need` bytes on `like`'s
    device (allocated if None), and the tensor, to be kept until the launch."""
    if ws is None:
        if not need:
            return None, 0, None
        ws = like.new_empty((need,), dtype=torch.uint8)
    _dev_tensor(ws, "ws", min_bytes=need)
    return _same(ws, "ws", like, (ws.dtype,), ws.shape), ws.numel() * ws.element_size(), ws


@_entry
def moe_grouped_linear(x, w, offsets, sorted_slots=None, k=1, out=None, ws=None):
    """y = x . W^T by expert: x bf16 [X, K] (values or bits), w [E, N, K],
    offsets int32 [E + 1]; with sorted_slots (int32 [M]) row p of the result
    reads x's row sorted_slots[p] // k.  Returns [M, N] in x's dtype.  ws (here
    and below): a workspace of moe_grouped_workspace_size bytes, allocated if
    None."""
    (X, K), (E, N, _) = _dims(x, "x", 2), _dims(w, "w", 3)
    px, pw = _same(x, "x", x, _BITS16, (X, K)), _same(w, "w", x, _BITS16, (E, N, K))
    po = _same(offsets, "offsets", x, _I32, (E + 1,))
    M, ps = _rows(x, sorted_slots)
    out = _new(out, "out", x, x.dtype, (M, N))
    L = lib()
    pws, nws, ws = _workspace(ws, moe_grouped_workspace_size(M, E, K, N, GROUPED_ONE), x)
    _check(L.moe_grouped_linear(px, X, K, pw, E, N, po, ps, k, M, out.data_ptr(), pws, nws, _here(x)),
           "moe_grouped_linear")
    return out


@_entry
def moe_grouped_swiglu(x, gate, up, offsets, sorted_slots=None, k=1, h=None, a=None, b=None, save=False,
                       ws=None):
    """h = silu(x . gate^T) * (x . up^T) by expert, rows as in
    moe_grouped_linear.  Returns h, or (h, a, b) with save (or with a and b
    given): the two products, for moe_grouped_swiglu_dgrad."""
    (X, K), (E, N, _) = _dims(x, "x", 2), _dims(gate, "gate", 3)
    px = _same(x, "x", x, _BITS16, (X, K))
    pg, pu = _same(gate, "gate", x, _BITS16, (E, N, K)), _same(up, "up", x, _BITS16, (E, N, K))
    po = _same(offsets, "offsets", x, _I32, (E + 1,))
    M, ps = _rows(x, sorted_slots)
    save = save or a is not None or b is not None
    h = _new(h, "h", x, x.dtype, (M, N))
    if save:
        a, b = _new(a, "a", x, x.dtype, (M, N)), _new(b, "b", x, x.dtype, (M, N))
    L = lib()
    pws, nws, ws = _workspace(ws, moe_grouped_workspace_size(M, E, K, N, GROUPED_SWIGLU), x)
    _check(L.moe_grouped_swiglu(px, X, K, pg, pu, E, N, po, ps, k, M, h.data_ptr(), a.data_ptr() if save else None,
                                b.data_ptr() if save else None, pws, nws, _here(x)), "moe_grouped_swiglu")
    return (h, a, b) if save else h


@_entry
def moe_grouped_linear_dgrad(dy, w, offsets, dy2=None, w2=None, out=None, ws=None):
    """dx = dy . W (+ dy2 . W2) by expert: dy [M, N], w [E, N, K] -> [M, K]
    in dy's dtype."""
    (M, N), (E, _, K) = _dims(dy, "dy", 2), _dims(w, "w", 3)
    pd, pw = _same(dy, "dy", dy, _BITS16, (M, N)), _same(w, "w", dy, _BITS16, (E, N, K))
    po = _same(offsets, "offsets", dy, _I32, (E + 1,))
    if (dy2 is None) != (w2 is None):
        raise ValueError("dy2 and w2 go together")
    pd2 = pw2 = None
    if dy2 is not None:
        pd2, pw2 = _same(dy2, "dy2", dy, _BITS16, (M, N)), _same(w2, "w2", dy, _BITS16, (E, N, K))
    out = _new(out, "out", dy, dy.dtype, (M, K))
    L = lib()
    pws, nws, ws = _workspace(ws, moe_grouped_workspace_size(M, E, N, K, GROUPED_ONE if dy2 is None else GROUPED_PAIR),
                              dy)
    _check(L.moe_grouped_linear_dgrad(pd, pw, pd2, pw2, M, N, E, K, po, out.data_ptr(), pws, nws, _here(dy)),
           "moe_grouped_linear_dgrad")
    return out


@_entry
def moe_grouped_swiglu_dgrad(dy, w, a, b, offsets, da=None, db=None, ws=None):
    """(da, db): the gradient through the down projection w [E, N, K] and
    SwiGLU, with a and b [M, K] as moe_grouped_swiglu saved them."""
    (M, N), (E, _, K) = _dims(dy, "dy", 2), _dims(w, "w", 3)
    pd, pw = _same(dy, "dy", dy, _BITS16, (M, N)), _same(w, "w", dy, _BITS16, (E, N, K))
    pa, pb = _same(a, "a", dy, _BITS16, (M, K)), _same(b, "b", dy, _BITS16, (M, K))
    po = _same(offsets, "offsets", dy, _I32, (E + 1,))
    da, db = _new(da, "da", dy, dy.dtype, (M, K)), _new(db, "db", dy, dy.dtype, (M, K))
    L = lib()
    pws, nws, ws = _workspace(ws, moe_grouped_workspace_size(M, E, N, K, GROUPED_ONE), dy)
    _check(L.moe_grouped_swiglu_dgrad(pd, pw, M, N, E, K, po, pa, pb, da.data_ptr(), db.data_ptr(), pws, nws, _here(dy)),
           "moe_grouped_swiglu_dgrad")
    return da, db


@_entry
def moe_grouped_linear_wgrad(dy, x, offsets, sorted_slots=None, k=1, out=None, accumulate=False, ws=None):
    """dW[e] = sum over e's rows of dy[p]^T x[p] (x's row sorted_slots[p] // k
    if given): dy [M, N], x [X, K] -> fp32 [E, N, K].  accumulate adds to
    `out`, which must be given.  ws: a workspace of
    moe_grouped_linear_wgrad_workspace_size bytes (allocated if None)."""
    (M, N), (X, K), E = _dims(dy, "dy", 2), _dims(x, "x", 2), _dims(offsets, "offsets", 1)[0] - 1
    pd, px = _same(dy, "dy", dy, _BITS16, (M, N)), _same(x, "x", dy, _BITS16, (X, K))
    po = _same(offsets, "offsets", dy, _I32, (E + 1,))
    rows, ps = _rows(x, sorted_slots)
    if rows != M:
        raise ValueError(f"dy has {M} rows, {'x' if sorted_slots is None else 'sorted_slots'} {rows}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out = _new(out, "out", dy, torch.float32, (E, N, K))
    L = lib()
    pws, nws, ws = _workspace(ws, moe_grouped_linear_wgrad_workspace_size(M, N, K, E), dy)
    _check(L.moe_grouped_linear_wgrad(pd, M, N, px, X, K, E, po, ps, k, int(bool(accumulate)), out.data_ptr(), pws, nws,
                                      _here(dy)), "moe_grouped_linear_wgrad")
    return out


@functools.lru_cache(maxsize=4096)
def moe_grouped_linear_wgrad_workspace_size(M, N, K, E):
    """Workspace bytes of a weight gradient (a function of its sizes alone)."""
    return int(lib().moe_grouped_linear_wgrad_workspace_size(M, N, K, E))


@dataclass
class Int4Tensor:
    """E experts of an [N, K] 4-bit integer projection (device)."""
    codes: torch.Tensor                     # uint8 [E, N, K/2]
    scales: torch.Tensor                    # bf16 (values or bits) [E, N, K/group]
    zeros: Optional[torch.Tensor] = None    # uint8 [E, N, K/group], None: 8 everywhere

    @property
    def device(self):
        return self.codes.device

    def get_device(self):
        return self.codes.get_device()

    @property
    def shape(self):
        E, N, half = self.codes.shape
        return E, N, half * 2

    @property
    def group(self):
        return self.shape[2] // max(self.scales.shape[-1], 1)

    def cstruct(self, like=None):
        codes, scales, zeros = self.codes, self.scales, self.zeros
        like = codes if like is None else like
        (E, N, half), (_, _, groups) = _dims(codes, "codes", 3), _dims(scales, "scales", 3)
        K = half * 2
        if groups < 1 or K % groups:
            raise ValueError(f"scales: {groups} groups for {K} columns")
        return Int4TensorC(E, N, K, K // groups, _same(codes, "codes", like, _U8, (E, N, half)),
                           _same(scales, "scales", like, _BITS16, (E, N, groups)),
                           None if zeros is None else _same(zeros, "zeros", like, _U8, (E, N, groups)))

    @staticmethod
    def empty(E, N, K, group=128, zeros=True, device="cuda"):
        def u8(*s):
            return torch.empty(s, dtype=torch.uint8, device=device)
        return Int4Tensor(u8(E, N, K // 2), torch.empty((E, N, K // group), dtype=torch.bfloat16, device=device),
                          u8(E, N, K // group) if zeros else None)


@_entry
def moe_int4_quantize_pack(w, group=128, zeros=True, out=None):
    """fp32 masters [E, N, K] -> Int4Tensor (with zero points, or symmetric)."""
    E, N, K = _dims(w, "w", 3)
    pw = _same(w, "w", w, _F32, (E, N, K))
    if out is None:
        if group not in (32, 64, 128) or K % 128:
            raise ValueError(f"group {group} of {K} columns: groups of 32, 64 or 128, columns a multiple of 128")
        out = Int4Tensor.empty(E, N, K, group, zeros, w.device)
    if out.shape != (E, N, K):
        raise ValueError(f"out: shape {out.shape}, expected {(E, N, K)}")
    st = out.cstruct(w)
    _check(lib().moe_int4_quantize_pack(pw, ctypes.byref(st), _here(w)), "moe_int4_quantize_pack")
    return out


@_entry
def moe_int4_dequantize(t, out=None):
    """Int4Tensor -> fp32 [E, N, K]."""
    st = t.cstruct()
    out = _new(out, "out", t.codes, torch.float32, t.shape)
    _check(lib().moe_int4_dequantize(ctypes.byref(st), out.data_ptr(), _here(t.codes)), "moe_int4_dequantize")
    return out


@_entry
def moe_int4_linear(x, w, offsets=None, sorted_slots=None, k=1, out=None):
    """bf16 rows times a 4-bit integer projection: x [X, K], w an Int4Tensor.
    Without offsets a dense projection (E = 1); with them rows by expert, as
    in moe_grouped_linear.  Returns [M, N] in x's dtype."""
    X, K = _dims(x, "x", 2)
    px = _same(x, "x", x, _BITS16, (X, K))
    if not isinstance(w, Int4Tensor):
        raise ValueError(f"w: expected an Int4Tensor, got {type(w).__name__}")
    st = w.cstruct(x)
    if st.K != K:
        raise ValueError(f"w: {st.K} columns, x has {K}")
    po = None if offsets is None else _same(offsets, "offsets", x, _I32, (st.E + 1,))
    M, ps = _rows(x, sorted_slots)
    out = _new(out, "out", x, x.dtype, (M, st.N))
    _check(lib().moe_int4_linear(px, X, ctypes.byref(st), po, ps, k, M, out.data_ptr(), _here(x)), "moe_int4_linear")
    return out


def _tokens(slot_pos, like, k):
    n, = _dims(slot_pos, "slot_pos", 1)
    if k < 1 or n % k:
        raise ValueError(f"slot_pos: {n} entries, not a multiple of k = {k}")
    return n // k, _same(slot_pos, "slot_pos", like, _I32, (n,))


@_entry
def moe_combine(y, slot_pos, k, w=None, out=None):
    """out[t] = sum_j w[t, j] * y[slot_pos[t * k + j]]: y [M, H] rows by
    expert, w fp32 [T, k] (None: all 1) -> [T, H] in y's dtype."""
    M, H = _dims(y, "y", 2)
    py = _same(y, "y", y, _BITS16, (M, H))
    T, pp = _tokens(slot_pos, y, k)
    pw = None if w is None else _same(w, "w", y, _F32, (T, k))
    out = _new(out, "out", y, y.dtype, (T, H))
    _check(lib().moe_combine(py, M, H, pp, pw, T, k, out.data_ptr(), _here(y)), "moe_combine")
    return out


@_entry
def moe_combine_backward(dout, y, slot_pos, w, ids=None, E=0, dy=None, dw=None, dlogits=None):
    """Gradients of moe_combine: (dy [M, H] in dout's dtype, dw fp32 [T, k]),
    and with ids (int32 [T, k]) and E the router logits' gradient through the
    softmax over the k selected: (dy, dw, dlogits fp32 [T, E]).  Rows of dy
    that slot_pos does not name are not written."""
    (T, H), (M, _), (_, k) = _dims(dout, "dout", 2), _dims(y, "y", 2), _dims(w, "w", 2)
    pd, py = _same(dout, "dout", dout, _BITS16, (T, H)), _same(y, "y", dout, _BITS16, (M, H))
    pp = _same(slot_pos, "slot_pos", dout, _I32, (T * k,))
    pw = _same(w, "w", dout, _F32, (T, k))
    dy, dw = _new(dy, "dy", dout, dout.dtype, (M, H)), _new(dw, "dw", dout, torch.float32, (T, k))
    pi = pl = None
    if ids is not None:
        pi = _same(ids, "ids", dout, _I32, (T, k))
        dlogits = _new(dlogits, "dlogits", dout, torch.float32, (T, E))
        pl = dlogits.data_ptr()
    _check(lib().moe_combine_backward(pd, T, H, py, M, pp, pw, pi, k, E, dy.data_ptr(), dw.data_ptr(), pl, _here(dout)),
           "moe_combine_backward")
    return (dy, dw) if ids is None else (dy, dw, dlogits)
