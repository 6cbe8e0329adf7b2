"""Python binding of the C ABI in ``include/e4b.h`` and ``include/e4b_operators.h`` (ctypes; argument marshalling
only).

Every function here forwards to the entry point of the same name in
``libe4b.so``; all computation runs in that library's CUDA kernels.  Tensors
are torch CUDA tensors (PyTorch supplies device memory and streams).  A
non-OK status raises :class:`E4BError`.  There is no fallback: if the library
is missing, :func:`lib` raises.

The library sees raw device addresses only, so before each call the binding
checks what the addresses cannot carry: every tensor is a contiguous CUDA
tensor of the dtype the header names, on one device, holding at least the
elements the call reads or writes (``TypeError`` / ``ValueError`` otherwise).
Alignment, shapes the build refuses and workspace size are the library's own
checks.
"""

from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libe4b.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "e4b.h")
OPERATORS_HEADER = os.path.join(os.path.dirname(PKG), "include", "e4b_operators.h")

c_i32, c_i64, c_f32, c_vp, c_sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t

STATUS = {0: "E4B_OK", 1: "E4B_ERR_INVALID_ARG", 2: "E4B_ERR_UNSUPPORTED",
          3: "E4B_ERR_WORKSPACE_TOO_SMALL", 4: "E4B_ERR_CUDA", 5: "E4B_ERR_DEVICE_TIMEOUT"}
E4B_OK, E4B_ERR_INVALID_ARG, E4B_ERR_UNSUPPORTED = 0, 1, 2
E4B_ERR_WORKSPACE_TOO_SMALL, E4B_ERR_CUDA, E4B_ERR_DEVICE_TIMEOUT = 3, 4, 5
ROW_ALIGN = 128


class E4BError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().e4b_status_string(status).decode()
        super().__init__("%s failed: %s" % (where, msg))


class MoeDims(ctypes.Structure):
    _fields_ = [("E", c_i32), ("H", c_i32), ("I", c_i32), ("top_k", c_i32), ("r", c_i32),
                ("alpha", c_f32), ("blocksize", c_i32), ("act", c_i32)]


class Nf4Experts(ctypes.Structure):
    _fields_ = [("gate_up_nf4", c_vp), ("gate_up_absmax", c_vp), ("down_nf4", c_vp), ("down_absmax", c_vp)]


class Lora(ctypes.Structure):
    _fields_ = [("A_gu", c_vp), ("B_gu", c_vp), ("A_d", c_vp), ("B_d", c_vp)]


class Routing(ctypes.Structure):
    _fields_ = [("topk_ids", c_vp), ("topk_w", c_vp), ("counts", c_vp), ("offsets", c_vp),
                ("row_of_slot", c_vp), ("slot_of_row", c_vp), ("tiles", c_vp)]


class FwdBuffers(ctypes.Structure):
    _fields_ = [("x_perm", c_vp), ("p_gu", c_vp), ("gu", c_vp), ("act", c_vp), ("p_d", c_vp), ("y_perm", c_vp)]


class BwdBuffers(ctypes.Structure):
    _fields_ = [("dyw", c_vp), ("q_d", c_vp), ("dgu", c_vp), ("q_gu", c_vp), ("dx_perm", c_vp)]


class Sizes(ctypes.Structure):
    _fields_ = [("slots", c_i64), ("rows_cap", c_i64), ("tiles_cap", c_i64), ("workspace_bytes", c_sz)]


class ProjDimsC(ctypes.Structure):
    _fields_ = [("K", c_i32), ("N", c_i32), ("n_adapters", c_i32), ("r", c_i32), ("blocksize", c_i32)]


class Nf4Matrix(ctypes.Structure):
    _fields_ = [("nf4", c_vp), ("absmax", c_vp)]


class AdapterFactors(ctypes.Structure):
    _fields_ = [("A", c_vp), ("B", c_vp), ("scale", c_vp)]


class AdapterGroups(ctypes.Structure):
    _fields_ = [("order", c_vp), ("offsets", c_vp), ("steps", c_vp)]


class ProjSizes(ctypes.Structure):
    _fields_ = [("rows_cap", c_i64), ("steps_cap", c_i64), ("workspace_bytes", c_sz),
                ("serve_workspace_bytes", c_sz)]


class BalanceDims(ctypes.Structure):
    _fields_ = [("E", c_i32), ("top_k", c_i32), ("S", c_i32), ("balance_coef", c_f32), ("z_coef", c_f32)]


class BalanceStats(ctypes.Structure):
    _fields_ = [("counts", c_vp), ("prob_sum", c_vp), ("tokens", c_vp), ("lse", c_vp)]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", c_i64), ("total_ms", ctypes.c_double)]


_LIB: Optional[ctypes.CDLL] = None

_SIGNATURES = {
    "e4b_status_string": (ctypes.c_char_p, [c_i32]),
    "e4b_version": (ctypes.c_char_p, []),
    "e4b_nf4_levels": (None, [ctypes.POINTER(c_f32)]),
    "e4b_get_sizes": (c_i32, [ctypes.POINTER(MoeDims), c_i32, ctypes.POINTER(Sizes)]),
    "e4b_workspace_init": (c_i32, [c_vp, c_sz, c_vp]),
    "e4b_check_device_error": (c_i32, [c_vp, c_vp]),
    "e4b_route_permute": (c_i32, [ctypes.POINTER(MoeDims), c_i32, c_vp, c_vp, ctypes.POINTER(Routing), c_vp,
                                  c_vp, c_sz, c_vp]),
    "e4b_route_permute_noalloc": (c_i32, [ctypes.POINTER(MoeDims), c_i32, c_vp, c_vp, ctypes.POINTER(Routing),
                                          c_vp, c_vp]),
    "e4b_grouped_nf4_lora_fwd": (c_i32, [ctypes.POINTER(MoeDims), c_i32, ctypes.POINTER(Routing),
                                         ctypes.POINTER(Nf4Experts), ctypes.POINTER(Lora), c_vp,
                                         ctypes.POINTER(FwdBuffers), c_vp, c_vp, c_sz, c_vp]),
    "e4b_grouped_nf4_lora_dgrad": (c_i32, [ctypes.POINTER(MoeDims), c_i32, ctypes.POINTER(Routing),
                                           ctypes.POINTER(Nf4Experts), ctypes.POINTER(Lora),
                                           ctypes.POINTER(FwdBuffers), c_vp, ctypes.POINTER(BwdBuffers), c_vp,
                                           c_vp, c_sz, c_vp]),
    "e4b_lora_wgrad": (c_i32, [ctypes.POINTER(MoeDims), c_i32, ctypes.POINTER(Routing),
                               ctypes.POINTER(FwdBuffers), ctypes.POINTER(BwdBuffers), c_vp, c_vp, c_vp, c_vp,
                               c_vp, c_sz, c_vp]),
    "e4b_moe_serve_fwd": (c_i32, [ctypes.POINTER(MoeDims), c_i32, c_vp, c_vp, ctypes.POINTER(Routing),
                                  ctypes.POINTER(Nf4Experts), ctypes.POINTER(Lora), ctypes.POINTER(FwdBuffers), c_vp,
                                  c_vp, c_sz, c_vp]),
    "e4b_router_backward": (c_i32, [ctypes.POINTER(MoeDims), c_i32, ctypes.POINTER(Routing), c_vp, c_vp, c_vp,
                                    c_vp, c_vp]),
    "e4b_nf4_dequant": (c_i32, [c_vp, c_vp, c_i64, c_vp, c_vp]),
    "e4b_nf4_quantize": (c_i32, [c_vp, c_i64, c_vp, c_vp, c_vp]),
    "e4b_proj_get_sizes": (c_i32, [ctypes.POINTER(ProjDimsC), c_i32, ctypes.POINTER(ProjSizes)]),
    "e4b_adapter_group": (c_i32, [ctypes.POINTER(ProjDimsC), c_i32, c_vp, ctypes.POINTER(AdapterGroups), c_vp]),
    "e4b_multi_lora_serve_fwd": (c_i32, [ctypes.POINTER(ProjDimsC), c_i32, c_vp, c_vp, ctypes.POINTER(Nf4Matrix),
                                         ctypes.POINTER(AdapterFactors), c_vp, c_vp, c_sz, c_vp]),
    "e4b_multi_lora_fwd": (c_i32, [ctypes.POINTER(ProjDimsC), c_i32, ctypes.POINTER(AdapterGroups), c_vp,
                                   ctypes.POINTER(Nf4Matrix), ctypes.POINTER(AdapterFactors), c_vp, c_vp, c_vp, c_sz,
                                   c_vp]),
    "e4b_multi_lora_dgrad": (c_i32, [ctypes.POINTER(ProjDimsC), c_i32, ctypes.POINTER(AdapterGroups), c_vp,
                                     ctypes.POINTER(Nf4Matrix), ctypes.POINTER(AdapterFactors), c_vp, c_vp, c_vp,
                                     c_sz, c_vp]),
    "e4b_multi_lora_wgrad": (c_i32, [ctypes.POINTER(ProjDimsC), c_i32, ctypes.POINTER(AdapterGroups), c_vp, c_vp,
                                     c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "e4b_balance_get_sizes": (c_i32, [ctypes.POINTER(BalanceDims), c_i32, ctypes.POINTER(c_sz)]),
    "e4b_balance_fwd": (c_i32, [ctypes.POINTER(BalanceDims), c_i32, c_vp, c_vp, c_vp, c_vp,
                                ctypes.POINTER(BalanceStats), c_vp, c_vp, c_sz, c_vp]),
    "e4b_balance_bwd": (c_i32, [ctypes.POINTER(BalanceDims), c_i32, c_vp, c_vp, c_vp, ctypes.POINTER(BalanceStats),
                                c_vp, c_i32, c_vp, c_vp]),
    "e4b_debug_watchdog": (c_i32, [c_vp, c_sz, c_i64, c_vp]),
    "e4b_profiler_enable": (c_i32, [c_i32]),
    "e4b_profiler_read": (c_i32, [ctypes.POINTER(KernelTime), c_i32, ctypes.POINTER(c_i32)]),
    "e4b_launch_count": (c_i64, []),
}


def lib() -> ctypes.CDLL:
    """Loads ``libe4b.so`` (built in-tree by ``grouped_nf4_expert_b200.build``)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libe4b.so is not built; run `python -m grouped_nf4_expert_b200.build`")
        so = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(so, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = so
    return _LIB


def header_symbols():
    """Names of the entry points ``include/e4b.h`` declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^(?:const\s+)?[\w\s\*]*?\b(e4b_\w+)\s*\(", text, flags=re.M)))


def _check(status: int, where: str):
    if status != E4B_OK:
        raise E4BError(status, where)


def _ptr(t) -> Optional[int]:
    """Device address of a tensor's first element; for an empty view, the address it would have in its
    storage (torch reports 0 for empty tensors)."""
    if t is None:
        return None
    if t.numel() == 0:
        return t.untyped_storage().data_ptr() + t.storage_offset() * t.element_size() or None
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "u8": torch.uint8}[name]


def _dev(t, dtype: str, min_numel: int, name: str, device=None, optional=None, where=True) -> Optional[int]:
    """Device address of ``t`` after checking that it is a contiguous CUDA tensor of ``dtype``
    holding at least ``min_numel`` elements (on ``device`` when given).  ``None`` passes where the
    header allows NULL: by default where nothing is read or written (``min_numel == 0``)."""
    import torch
    if optional is None:
        optional = min_numel == 0
    if t is None:
        if optional:
            return None
        raise ValueError("%s: a tensor is required" % name)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %s" % (name, type(t).__name__))
    if t.dtype != _torch_dtype(dtype):
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, _torch_dtype(dtype)))
    if not t.is_contiguous():
        raise ValueError("%s: must be contiguous" % name)
    if t.numel() < min_numel:
        raise ValueError("%s: %d elements, the call needs %d" % (name, t.numel(), min_numel))
    if not where:  # the caller checks the devices of all its tensors together (_one_cuda_device)
        return _ptr(t)
    if t.device.type != "cuda":
        raise ValueError("%s: must be a CUDA tensor, got one on %s" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s: on %s, expected %s" % (name, t.device, device))
    return _ptr(t)


def _numel_of(t, name: str) -> int:
    import torch
    if t is None:
        raise ValueError("%s: a tensor is required" % name)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %s" % (name, type(t).__name__))
    return t.numel()


def _one_cuda_device(**tensors):
    """The one CUDA device that all the given tensors are on (None entries are skipped)."""
    devs = set()
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError("%s: must be a CUDA tensor, got one on %s" % (name, t.device))
        devs.add(t.device)
    if len(devs) > 1:
        raise ValueError("tensors on several devices: %s" % sorted(str(d) for d in devs))
    return devs.pop() if devs else None


@dataclass(frozen=True)
class Dims:
    E: int
    H: int
    I: int  # noqa: E741
    top_k: int
    r: int
    alpha: float

    def c(self) -> MoeDims:
        return MoeDims(self.E, self.H, self.I, self.top_k, self.r, float(self.alpha), 64, 0)


def e4b_get_sizes(dims: Dims, T: int) -> Sizes:
    out = Sizes()
    d = dims.c()
    _check(lib().e4b_get_sizes(ctypes.byref(d), T, ctypes.byref(out)), "e4b_get_sizes")
    return out


def e4b_nf4_levels():
    buf = (c_f32 * 16)()
    lib().e4b_nf4_levels(buf)
    return [buf[i] for i in range(16)]


def e4b_workspace_init(ws, stream=None):
    p = _dev(ws, "u8", 1, "ws")
    _check(lib().e4b_workspace_init(p, ws.numel(), _stream(stream)), "e4b_workspace_init")


def e4b_check_device_error(ws, stream=None) -> int:
    """Synchronises the stream; returns the status (does not raise)."""
    return lib().e4b_check_device_error(_dev(ws, "u8", 1, "ws"), _stream(stream))


def e4b_nf4_dequant(packed, absmax, out, stream=None):
    """packed NF4 codes [n/2] u8 and absmax [n/64] f32 -> bf16 [n] (n = out.numel())."""
    n = _numel_of(out, "out")
    pp = _dev(packed, "u8", n // 2, "packed", where=False)
    pa = _dev(absmax, "f32", n // 64, "absmax", where=False)
    po = _dev(out, "bf16", 0, "out", optional=False, where=False)
    _one_cuda_device(packed=packed, absmax=absmax, out=out)
    _check(lib().e4b_nf4_dequant(pp, pa, n, po, _stream(stream)), "e4b_nf4_dequant")


def e4b_nf4_quantize(w, packed, absmax, stream=None):
    """bf16 weights (n elements, n % 64 == 0) -> packed NF4 codes [n/2] u8 and absmax [n/64] f32."""
    n = _numel_of(w, "w")
    pp = _dev(packed, "u8", n // 2, "packed", where=False)
    pa = _dev(absmax, "f32", n // 64, "absmax", where=False)
    pw = _dev(w, "bf16", 0, "w", optional=False, where=False)
    _one_cuda_device(w=w, packed=packed, absmax=absmax)
    _check(lib().e4b_nf4_quantize(pw, n, pp, pa, _stream(stream)), "e4b_nf4_quantize")


def e4b_debug_watchdog(ws, timeout_ns: int, stream=None):
    p = _dev(ws, "u8", 1, "ws")
    _check(lib().e4b_debug_watchdog(p, ws.numel(), int(timeout_ns), _stream(stream)), "e4b_debug_watchdog")


def e4b_profiler_enable(on: bool):
    _check(lib().e4b_profiler_enable(1 if on else 0), "e4b_profiler_enable")


def e4b_profiler_read():
    """Per-kernel {name: (launches, total_ms)} recorded since the last read (waits for the events)."""
    cap = 64
    buf = (KernelTime * cap)()
    n = c_i32(0)
    _check(lib().e4b_profiler_read(buf, cap, ctypes.byref(n)), "e4b_profiler_read")
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms)) for i in range(min(n.value, cap))}


def e4b_launch_count() -> int:
    return int(lib().e4b_launch_count())


def e4b_proj_get_sizes(dims: "ProjDims", T: int) -> ProjSizes:
    out = ProjSizes()
    d = dims.c()
    _check(lib().e4b_proj_get_sizes(ctypes.byref(d), T, ctypes.byref(out)), "e4b_proj_get_sizes")
    return out


def e4b_balance_get_sizes(dims: BalanceDims, T: int) -> int:
    out = c_sz(0)
    _check(lib().e4b_balance_get_sizes(ctypes.byref(dims), T, ctypes.byref(out)), "e4b_balance_get_sizes")
    return int(out.value)


class Block:
    """Device buffers of one block problem (``dims``, ``T`` tokens), allocated with torch.

    Holds the routing arrays, the forward activations, the backward
    intermediates, the workspace and the outputs, laid out as ``include/e4b.h``
    requires, and calls the four entry points on them.
    """

    def __init__(self, dims: Dims, T: int, device="cuda"):
        import torch
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.dims, self.T, self.device = dims, T, dev
        sz = e4b_get_sizes(dims, T)
        self.sizes = sz
        E, H, I, k, r = dims.E, dims.H, dims.I, dims.top_k, dims.r
        R = sz.rows_cap
        dev = self.device

        def z(shape, dtype):
            n = 1
            for s in shape:
                n *= s
            return torch.zeros(max(n, 8), dtype=dtype, device=dev)[:n].view(*shape)

        bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
        self.topk_ids, self.topk_w = z((T, k), i32), z((T, k), f32)
        self.counts, self.offsets = z((E,), i32), z((E + 1,), i32)
        self.row_of_slot, self.slot_of_row, self.tiles = z((T * k,), i32), z((R,), i32), z((sz.tiles_cap,), i32)
        self.x_perm, self.p_gu, self.gu = z((R, H), bf), z((R, r), bf), z((R, 2 * I), bf)
        self.act, self.p_d, self.y_perm = z((R, I), bf), z((R, r), bf), z((R, H), bf)
        self.dyw, self.q_d, self.dgu = z((R, H), bf), z((R, r), bf), z((R, 2 * I), bf)
        self.q_gu, self.dx_perm = z((R, r), bf), z((R, H), bf)
        self.y, self.dx = z((T, H), bf), z((T, H), bf)
        # the four LoRA gradients are views of one flat buffer, so that a data-parallel step sums them
        # with one collective and no packing copy (every size is a multiple of 8 elements: r % 8 == 0)
        gshapes = ((E, r, H), (E, 2 * I, r), (E, r, I), (E, H, r))
        gsizes = [a * b * c for a, b, c in gshapes]
        self.lora_grads = z((sum(gsizes),), bf)
        views, o = [], 0
        for shp, n in zip(gshapes, gsizes):
            views.append(self.lora_grads[o:o + n].view(*shp))
            o += n
        self.dA_gu, self.dB_gu, self.dA_d, self.dB_d = views
        self.ws = z((int(sz.workspace_bytes),), torch.uint8)
        e4b_workspace_init(self.ws)
        self._dims_c = dims.c()
        self._routing = Routing(*(_ptr(t) for t in (self.topk_ids, self.topk_w, self.counts, self.offsets,
                                                      self.row_of_slot, self.slot_of_row, self.tiles)))
        self._fwd = FwdBuffers(*(_ptr(t) for t in (self.x_perm, self.p_gu, self.gu, self.act, self.p_d,
                                                    self.y_perm)))
        self._fwd_nogu = FwdBuffers(self.x_perm.data_ptr(), self.p_gu.data_ptr(), None, self.act.data_ptr(),
                                    self.p_d.data_ptr(), self.y_perm.data_ptr())
        self._bwd = BwdBuffers(*(t.data_ptr() for t in (self.dyw, self.q_d, self.dgu, self.q_gu, self.dx_perm)))

    # -- argument checks (see the module docstring) ----------------------------
    def _rows(self, t, dtype, cols, name, required=True):
        """A [T, cols] token tensor of this problem (at least T * cols elements)."""
        return _dev(t, dtype, self.T * cols, name, self.device, optional=not required or self.T == 0)

    def _base(self, base: Nf4Experts):
        """The NF4 base struct; when made by :func:`nf4_experts`, its sizes and device are checked
        against this problem."""
        d = self.dims
        need = {"gate_up_nf4": d.E * 2 * d.I * d.H // 2, "gate_up_absmax": d.E * 2 * d.I * d.H // 64,
                "down_nf4": d.E * d.H * d.I // 2, "down_absmax": d.E * d.H * d.I // 64}
        _check_struct(base, need, self.device, "base")
        return ctypes.byref(base)

    def _lora(self, lora: Lora):
        d = self.dims
        need = {"A_gu": d.E * d.r * d.H, "B_gu": d.E * 2 * d.I * d.r, "A_d": d.E * d.r * d.I,
                "B_d": d.E * d.H * d.r}
        _check_struct(lora, need, self.device, "lora")
        return ctypes.byref(lora)

    # -- the four hot-path calls -------------------------------------------------
    def e4b_route_permute(self, logits, x, gather=True, stream=None):
        """Routing tables; with ``gather`` also ``x_perm`` (else the forward gathers, given ``x``)."""
        pl = self._rows(logits, "f32", self.dims.E, "logits")
        px = self._rows(x, "bf16", self.dims.H, "x", required=gather)
        _check(lib().e4b_route_permute(ctypes.byref(self._dims_c), self.T, pl, px,
                                       ctypes.byref(self._routing), _ptr(self.x_perm) if gather else None,
                                       _ptr(self.ws), self.ws.numel(), _stream(stream)), "e4b_route_permute")

    def e4b_route_permute_noalloc(self, logits, x, gather=True, stream=None):
        """As ``e4b_route_permute``, with the library's fixed scratch instead of ``ws`` (capturable in
        a global-mode CUDA graph once a first call on the device has been made)."""
        pl = self._rows(logits, "f32", self.dims.E, "logits")
        px = self._rows(x, "bf16", self.dims.H, "x", required=gather)
        _check(lib().e4b_route_permute_noalloc(ctypes.byref(self._dims_c), self.T, pl, px,
                                               ctypes.byref(self._routing), _ptr(self.x_perm) if gather else None,
                                               _stream(stream)), "e4b_route_permute_noalloc")

    def e4b_grouped_nf4_lora_fwd(self, base: Nf4Experts, lora: Lora, x=None, stream=None):
        """Forward; with ``x`` the call also writes ``x_perm`` (fused with the first projection)."""
        px = self._rows(x, "bf16", self.dims.H, "x", required=False)
        _check(lib().e4b_grouped_nf4_lora_fwd(ctypes.byref(self._dims_c), self.T, ctypes.byref(self._routing),
                                              self._base(base), self._lora(lora), px,
                                              ctypes.byref(self._fwd), _ptr(self.y), _ptr(self.ws),
                                              self.ws.numel(), _stream(stream)), "e4b_grouped_nf4_lora_fwd")

    def e4b_grouped_nf4_lora_dgrad(self, base: Nf4Experts, lora: Lora, dY, stream=None):
        pdy = self._rows(dY, "bf16", self.dims.H, "dY")
        _check(lib().e4b_grouped_nf4_lora_dgrad(ctypes.byref(self._dims_c), self.T, ctypes.byref(self._routing),
                                                self._base(base), self._lora(lora), ctypes.byref(self._fwd),
                                                pdy, ctypes.byref(self._bwd), _ptr(self.dx), _ptr(self.ws),
                                                self.ws.numel(), _stream(stream)), "e4b_grouped_nf4_lora_dgrad")

    def e4b_lora_wgrad(self, stream=None):
        _check(lib().e4b_lora_wgrad(ctypes.byref(self._dims_c), self.T, ctypes.byref(self._routing),
                                    ctypes.byref(self._fwd), ctypes.byref(self._bwd), _ptr(self.dA_gu),
                                    _ptr(self.dB_gu), _ptr(self.dA_d), _ptr(self.dB_d), _ptr(self.ws),
                                    self.ws.numel(), _stream(stream)), "e4b_lora_wgrad")

    def e4b_moe_serve_fwd(self, logits, x, base: Nf4Experts, lora: Lora, keep_gu=None, stream=None):
        """Routing + forward for inference into ``self.y``.  ``keep_gu=False`` passes no gu buffer,
        which the call allows for decode-sized batches only (at most 16 * E routed slots; larger ones
        run the training forward, which writes gu); ``None`` keeps gu exactly when it is required."""
        if keep_gu is None:
            keep_gu = self.T * self.dims.top_k > 16 * self.dims.E
        fwd = self._fwd if keep_gu else self._fwd_nogu
        pl = self._rows(logits, "f32", self.dims.E, "logits")
        px = self._rows(x, "bf16", self.dims.H, "x")
        _check(lib().e4b_moe_serve_fwd(ctypes.byref(self._dims_c), self.T, pl, px,
                                       ctypes.byref(self._routing), self._base(base), self._lora(lora),
                                       ctypes.byref(fwd), _ptr(self.y), _ptr(self.ws), self.ws.numel(),
                                       _stream(stream)), "e4b_moe_serve_fwd")

    def e4b_router_backward(self, dY, d_logits, dw=None, stream=None):
        pdy = self._rows(dY, "bf16", self.dims.H, "dY")
        pdl = self._rows(d_logits, "f32", self.dims.E, "d_logits")
        pdw = self._rows(dw, "f32", self.dims.top_k, "dw", required=False)
        _check(lib().e4b_router_backward(ctypes.byref(self._dims_c), self.T, ctypes.byref(self._routing),
                                         _ptr(self.y_perm), pdy, pdl, pdw, _stream(stream)),
               "e4b_router_backward")

    def check_device_error(self, stream=None) -> int:
        return e4b_check_device_error(self.ws, stream)


def _make_struct(cls, tensors, dtypes):
    """A pointer struct over contiguous CUDA tensors on one device.  The struct keeps the tensors
    alive (it holds their raw addresses) and records their sizes for the calls' checks."""
    names = [f[0] for f in cls._fields_]
    st = cls(*(_dev(t, dt, 1, n, where=False) for t, dt, n in zip(tensors, dtypes, names)))
    dev = _one_cuda_device(**dict(zip(names, tensors)))
    st._keep, st._device = tuple(tensors), dev
    st._numel = {n: t.numel() for n, t in zip(names, tensors)}
    return st


def _check_struct(st, need, device, what):
    """Sizes and device of a struct made by :func:`nf4_experts` / :func:`lora_factors` against a
    problem (a struct built field by field carries no sizes and is passed as is)."""
    numel = getattr(st, "_numel", None)
    if numel is None:
        return
    if st._device != device:
        raise ValueError("%s: tensors on %s, the problem is on %s" % (what, st._device, device))
    for name, n in need.items():
        if numel[name] < n:
            raise ValueError("%s.%s: %d elements, the dims need %d" % (what, name, numel[name], n))


def nf4_experts(gate_up_nf4, gate_up_absmax, down_nf4, down_absmax) -> Nf4Experts:
    """The frozen NF4 base: codes u8 [E,2I,H/2] and [E,H,I/2], block absmax f32 [E,2I,H/64] and
    [E,H,I/64]."""
    return _make_struct(Nf4Experts, (gate_up_nf4, gate_up_absmax, down_nf4, down_absmax), ("u8", "f32", "u8", "f32"))


def lora_factors(A_gu, B_gu, A_d, B_d) -> Lora:
    """The per-expert LoRA factors, bf16 [E,r,H], [E,2I,r], [E,r,I], [E,H,r]."""
    return _make_struct(Lora, (A_gu, B_gu, A_d, B_d), ("bf16",) * 4)


def _cuda_device(device):
    import torch
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("device: a CUDA device is required, got %s" % dev)
    return dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())


def _alloc(shape, dtype, device, zero=True):
    """Zeroed tensor of ``shape`` whose address is valid (and 16-byte aligned) even when it is empty; with ``zero``
    false its values are left as they come, for what a call writes whole."""
    import torch
    n = 1
    for d in shape:
        n *= d
    return (torch.zeros if zero else torch.empty)(max(n, 8), dtype=dtype, device=device)[:n].view(*shape)


class _OnDevice:
    """Calls on the object's device, whatever device is current: its current stream by default, or a
    stream of that device (a stream of another device is refused)."""

    def _arg(self, t, dtype, numel, name, optional=False):
        """Device address of ``t`` after the checks of :func:`_dev`; the tests a sound tensor passes come
        first, since a small batch's call costs the host more than the GPU."""
        if (type(t) is self._tensor and t.dtype is dtype[1] and t.get_device() == self._index and t.is_contiguous()
                and t.numel() >= numel > 0):
            return t.data_ptr()
        return _dev(t, dtype[0], numel, name, self.device, optional=optional or self.T == 0)

    def _on(self, device):
        import torch
        self.device = _cuda_device(device)
        self._index = self.device.index
        self._tensor = torch.Tensor
        self._raw_stream = torch._C._cuda_getCurrentRawStream  # the handle, without a Stream object a call
        torch.cuda.init()
        self._current_device = torch._C._cuda_getDevice
        self._bf16, self._f32 = ("bf16", torch.bfloat16), ("f32", torch.float32)
        self._i32, self._u8 = ("i32", torch.int32), ("u8", torch.uint8)
        self._fns = {}
        return self.device

    def _call(self, name, stream, *args):
        index = self._index
        if stream is None:
            handle = self._raw_stream(index)
        elif stream.device != self.device:
            raise ValueError("stream: on %s, the problem is on %s" % (stream.device, self.device))
        else:
            handle = stream.cuda_stream
        fn = self._fns.get(name)
        if fn is None:
            # structs go in by address: a handle of its own converts its arguments in two thirds of the time
            fn = self._fns[name] = lib()[name]
            fn.restype, args_of = _SIGNATURES[name]
            fn.argtypes = [c_vp if issubclass(a, ctypes._Pointer) else a for a in args_of]
        if self._current_device() == index:
            status = fn(*args, handle)
        else:
            import torch
            with torch.cuda.device(self.device):
                status = fn(*args, handle)
        if status != E4B_OK:
            raise E4BError(status, name)

    def check_device_error(self, stream=None) -> int:
        """Synchronises the stream; the status of the object's calls so far (does not raise)."""
        import torch
        with torch.cuda.device(self.device):
            return e4b_check_device_error(self.ws, stream)


@dataclass(frozen=True)
class ProjDims:
    """A projection W [N, K] with ``n_adapters`` adapters of rank ``r`` beside it."""
    K: int
    N: int
    n_adapters: int
    r: int

    def c(self) -> ProjDimsC:
        return ProjDimsC(self.K, self.N, self.n_adapters, self.r, 64)


class Projection(_OnDevice):
    """Device buffers of one NF4 projection with adapters for ``T`` tokens, allocated with torch.

    Serving: :meth:`e4b_multi_lora_serve_fwd` into ``y``.  Training (``train=True``, the default):
    :meth:`e4b_adapter_group`, then :meth:`e4b_multi_lora_fwd` (``y``), :meth:`e4b_multi_lora_dgrad`
    (``dx``) and :meth:`e4b_multi_lora_wgrad` (``dA``, ``dB``).  Calls on one object share its buffers
    and workspace, so they must not overlap on the GPU; the buffers are filled on the current stream, which
    another stream has to wait for before its first call.
    """

    def __init__(self, dims: ProjDims, T: int, device="cuda", train: bool = True):
        import torch
        self.dims, self.T, self.train = dims, T, train
        self._done = 0
        sz = e4b_proj_get_sizes(dims, T)
        self.sizes = sz
        dev = self._on(device)
        n, r, R = dims.n_adapters, dims.r, sz.rows_cap
        bf, i32 = torch.bfloat16, torch.int32
        self.y = _alloc((T, dims.N), bf, dev, zero=False)
        self.ws = _alloc((int(max(sz.workspace_bytes, sz.serve_workspace_bytes)),), torch.uint8, dev, zero=False)
        self._dims_c = dims.c()
        self._dims_p = ctypes.addressof(self._dims_c)
        self._base_need = {"nf4": dims.N * dims.K // 2, "absmax": dims.N * dims.K // 64}
        self._adapters_need = {"A": n * r * dims.K, "B": n * dims.N * r, "scale": n}
        self._y_p, self._ws_p, self._ws_n = _ptr(self.y), _ptr(self.ws), self.ws.numel()
        if train:
            self.order, self.offsets = _alloc((R,), i32, dev), _alloc((n + 2,), i32, dev)
            self.steps = _alloc((sz.steps_cap,), i32, dev)
            # by row: the values cut to bf16 (p, q), then what the cut left
            self._p_pairs, self._q_pairs = (_alloc((R, 2, r), bf, dev, zero=False) for _ in range(2))
            self.p, self.q = self._p_pairs[:, 0], self._q_pairs[:, 0]
            self.dx = _alloc((T, dims.K), bf, dev, zero=False)
            # the two gradients are views of one flat buffer (one collective in a data-parallel step)
            na, nb = n * r * dims.K, n * dims.N * r
            self.lora_grads = _alloc((na + nb,), bf, dev)
            self.dA = self.lora_grads[:na].view(n, r, dims.K)
            self.dB = self.lora_grads[na:].view(n, dims.N, r)
            self._groups = AdapterGroups(_ptr(self.order), _ptr(self.offsets), _ptr(self.steps))
            self._groups_p = ctypes.addressof(self._groups)
            self._low_p = (_ptr(self._p_pairs), _ptr(self._q_pairs))
            self._dx_p, self._grad_p = _ptr(self.dx), (_ptr(self.dA), _ptr(self.dB))
        self._call("e4b_workspace_init", None, self._ws_p, self._ws_n)

    def _structs(self, base: Nf4Matrix, ad: AdapterFactors):
        """Addresses of the call's structs, after their checks."""
        if type(base) is not Nf4Matrix:
            raise TypeError("base: an Nf4Matrix (nf4_matrix) is required, got %s" % type(base).__name__)
        if type(ad) is not AdapterFactors:
            raise TypeError("adapters: AdapterFactors (adapter_factors) are required, got %s" % type(ad).__name__)
        _check_struct(base, self._base_need, self.device, "base")
        _check_struct(ad, self._adapters_need, self.device, "adapters")
        return ctypes.addressof(base), ctypes.addressof(ad)

    def _training(self):
        if not self.train:
            raise ValueError("made with train=False: no training buffers")

    def _after(self, needs):
        """Refuses a training call ahead of those whose results it reads (1: the grouping, 2: the forward, 4: the
        input gradient)."""
        missing = needs & ~self._done
        if missing and self.T:
            raise ValueError("call %s first" % ", ".join(
                name for bit, name in ((1, "e4b_adapter_group"), (2, "e4b_multi_lora_fwd"),
                                       (4, "e4b_multi_lora_dgrad")) if missing & bit))

    def e4b_multi_lora_serve_fwd(self, ids, x, base: Nf4Matrix, adapters: AdapterFactors, stream=None):
        """Serving forward into ``self.y`` (ids int32 [T], any id outside [0, n) for no adapter)."""
        pi = self._arg(ids, self._i32, self.T, "ids")
        px = self._arg(x, self._bf16, self.T * self.dims.K, "x")
        pb, pa = self._structs(base, adapters)
        self._call("e4b_multi_lora_serve_fwd", stream, self._dims_p, self.T, pi, px, pb, pa, self._y_p, self._ws_p,
                   self._ws_n)

    def e4b_adapter_group(self, ids, stream=None):
        """Groups the step's tokens by adapter for the training calls."""
        self._training()
        self._call("e4b_adapter_group", stream, self._dims_p, self.T, self._arg(ids, self._i32, self.T, "ids"),
                   self._groups_p)
        self._done = 1

    def e4b_multi_lora_fwd(self, x, base: Nf4Matrix, adapters: AdapterFactors, stream=None):
        """``y`` of the grouped tokens; keeps ``p`` for the adapter gradients."""
        self._training()
        px = self._arg(x, self._bf16, self.T * self.dims.K, "x")
        pb, pa = self._structs(base, adapters)
        self._after(1)
        self._call("e4b_multi_lora_fwd", stream, self._dims_p, self.T, self._groups_p, px, pb, pa,
                   self._low_p[0], self._y_p, self._ws_p, self._ws_n)
        self._done |= 2

    def e4b_multi_lora_dgrad(self, dY, base: Nf4Matrix, adapters: AdapterFactors, stream=None):
        """``dx``; keeps ``q`` for the adapter gradients."""
        self._training()
        pd = self._arg(dY, self._bf16, self.T * self.dims.N, "dY")
        pb, pa = self._structs(base, adapters)
        self._after(1)
        self._call("e4b_multi_lora_dgrad", stream, self._dims_p, self.T, self._groups_p, pd, pb, pa,
                   self._low_p[1], self._dx_p, self._ws_p, self._ws_n)
        self._done |= 4

    def e4b_multi_lora_wgrad(self, x, dY, stream=None):
        """Adapter gradients from the ``p`` and ``q`` of the forward and the input gradient."""
        self._training()
        px = self._arg(x, self._bf16, self.T * self.dims.K, "x")
        pd = self._arg(dY, self._bf16, self.T * self.dims.N, "dY")
        self._after(7)
        self._call("e4b_multi_lora_wgrad", stream, self._dims_p, self.T, self._groups_p, px, pd,
                   *self._low_p, *self._grad_p, self._ws_p, self._ws_n)


class RouterBalance(_OnDevice):
    """Device buffers of the router's balance loss: ``E`` experts, ``top_k``, ``T`` tokens in ``S`` sequences.

    :meth:`e4b_balance_fwd` writes ``loss`` (float32 [3]: loss, balance, z), ``counts`` (int32 [S, E]),
    ``prob_sum`` (float32 [S, E]), ``tokens`` (int32 [S]) and ``lse``; :meth:`e4b_balance_bwd` the gradient
    of the logits.  Calls on one object share its buffers, so they must not overlap on the GPU; the
    buffers are filled on the current stream, which another stream has to wait for before its first call.
    """

    def __init__(self, E: int, top_k: int, T: int, S: int = 1, device="cuda"):
        import torch
        self.E, self.top_k, self.T, self.S = E, top_k, T, S
        self._done = False
        self._dims_c = BalanceDims(E, top_k, S, 0.0, 0.0)
        self._dims_p = ctypes.addressof(self._dims_c)
        ws_bytes = e4b_balance_get_sizes(self._dims_c, T)
        dev = self._on(device)
        f32, i32 = torch.float32, torch.int32
        self.counts, self.prob_sum = _alloc((S, E), i32, dev), _alloc((S, E), f32, dev)
        self._tokens = _alloc((S + 2,), i32, dev)
        self.tokens = self._tokens[:S]
        self.lse, self.loss = _alloc((T,), f32, dev), _alloc((3,), f32, dev)
        self.ws = _alloc((ws_bytes,), torch.uint8, dev, zero=False)
        self._stats = BalanceStats(*(_ptr(t) for t in (self.counts, self.prob_sum, self._tokens, self.lse)))
        self._stats_p = ctypes.addressof(self._stats)
        self._loss_p, self._ws_p, self._ws_n = _ptr(self.loss), _ptr(self.ws), self.ws.numel()
        self._call("e4b_workspace_init", None, self._ws_p, self._ws_n)

    def _inputs(self, logits, seq_offsets, token_mask):
        pl = self._arg(logits, self._f32, self.T * self.E, "logits")
        if seq_offsets is None and self.S != 1:
            raise ValueError("seq_offsets: required for %d sequences" % self.S)
        ps = self._arg(seq_offsets, self._i32, self.S + 1, "seq_offsets", optional=True)
        pm = self._arg(token_mask, self._u8, self.T, "token_mask", optional=True)
        return pl, ps, pm

    def e4b_balance_fwd(self, logits, topk_ids, seq_offsets=None, token_mask=None, balance_coef=1.0, z_coef=0.0,
                        stream=None):
        """Loss and per-expert counts.  seq_offsets: int32 [S + 1] ascending (None: one sequence of all
        tokens); token_mask: uint8 [T], 0 for tokens that take no part."""
        pl, ps, pm = self._inputs(logits, seq_offsets, token_mask)
        pi = self._arg(topk_ids, self._i32, self.T * self.top_k, "topk_ids")
        self._dims_c.balance_coef, self._dims_c.z_coef = balance_coef, z_coef
        self._call("e4b_balance_fwd", stream, self._dims_p, self.T, pl, pi, ps, pm, self._stats_p, self._loss_p,
                   self._ws_p, self._ws_n)
        self._done = True

    def e4b_balance_bwd(self, logits, d_logits, seq_offsets=None, token_mask=None, balance_coef=1.0, z_coef=0.0,
                        dloss=None, accumulate=False, stream=None):
        """d_logits = dloss * dloss/dlogits (dloss: float32 [1], None for 1), or += with ``accumulate``; after
        :meth:`e4b_balance_fwd`, whose counts and lse it reads."""
        pl, ps, pm = self._inputs(logits, seq_offsets, token_mask)
        pd = self._arg(d_logits, self._f32, self.T * self.E, "d_logits")
        pg = self._arg(dloss, self._f32, 1, "dloss", optional=True)
        if not self._done and self.T:
            raise ValueError("call e4b_balance_fwd first")
        self._dims_c.balance_coef, self._dims_c.z_coef = balance_coef, z_coef
        self._call("e4b_balance_bwd", stream, self._dims_p, self.T, pl, ps, pm, self._stats_p, pg,
                   1 if accumulate else 0, pd)


def nf4_matrix(nf4, absmax) -> Nf4Matrix:
    """A frozen NF4 projection: codes u8 [N, K/2], block absmax f32 [N, K/64]."""
    return _make_struct(Nf4Matrix, (nf4, absmax), ("u8", "f32"))


def adapter_factors(A, B, scale) -> AdapterFactors:
    """Adapters of a projection: bf16 A [n, r, K] and B [n, N, r], scale f32 [n]."""
    return _make_struct(AdapterFactors, (A, B, scale), ("bf16", "bf16", "f32"))
