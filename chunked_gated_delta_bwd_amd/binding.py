"""Python binding of the C ABI in include/gdr.h (argument marshalling only).

Every computation runs in the HIP library ``libgdr.so``; this module only
turns torch tensors into pointers and the current torch stream into a
``hipStream_t``.  If the library is missing the import of the entry points
fails loudly: there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdr.so")
_lib = None

GDR_OK, GDR_EINVAL, GDR_EUNSUPPORTED, GDR_EWORKSPACE, GDR_EHIP = 0, 1, 2, 3, 4
GDR_GATE_SCALAR, GDR_GATE_CHANNEL, GDR_GATE_CHANNEL_SIGMOID = 0, 1, 2
GDR_BF16, GDR_F32 = 0, 1
GDR_WS_STATE, GDR_WS_DSTATE, GDR_WS_U, GDR_WS_A, GDR_WS_GAMMA = 0, 1, 2, 3, 4

GDR_STAGE_PREP, GDR_STAGE_CHAIN_FWD, GDR_STAGE_CHAIN_BWD, GDR_STAGE_CHAIN_BOTH = 0, 1, 2, 3
GDR_STAGE_GRADS, GDR_STAGE_FINISH = 4, 5
STAGE_NAMES = {GDR_STAGE_PREP: "prep", GDR_STAGE_CHAIN_FWD: "chain_fwd", GDR_STAGE_CHAIN_BWD: "chain_bwd",
               GDR_STAGE_CHAIN_BOTH: "chain_both", GDR_STAGE_GRADS: "grads", GDR_STAGE_FINISH: "finish"}

SYMBOLS = ("gdr_workspace_bytes", "gdr_fwd_recompute", "gdr_fwd", "gdr_bwd", "gdr_fwd_bwd",
           "gdr_workspace_region", "gdr_run_stage", "gdr_fwd_bwd_noalloc", "gdr_step",
           "gdr_scan_workspace_bytes", "gdr_scan_fwd", "gdr_scan_bwd", "gdr_scan_step",
           "gdr_norm_fwd", "gdr_norm_quant", "gdr_norm_workspace_bytes", "gdr_norm_bwd", "gdr_last_error")
# the device array gdr_fwd_bwd_noalloc uses as its workspace (128 MiB per GPU)
NOALLOC_WORKSPACE_BYTES = 128 << 20


class GdrError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"gdr status {status}: {message}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32), ("N", ctypes.c_int32),
                ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int64)),
                ("gate", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("gate_scale", ctypes.c_float), ("Hk", ctypes.c_int32), ("seq_split", ctypes.c_int32)]


class Inputs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("beta_logit", ctypes.c_void_p),
                ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("h0", ctypes.c_void_p)]


class Grads(ctypes.Structure):
    _fields_ = [("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
                ("dg", ctypes.c_void_p), ("dbeta", ctypes.c_void_p), ("dh0", ctypes.c_void_p),
                ("dA_log", ctypes.c_void_p), ("ddt_bias", ctypes.c_void_p)]


class ScanShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("N", ctypes.c_int32), ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int64)),
                ("gate", ctypes.c_int32), ("dtype", ctypes.c_int32), ("gate_scale", ctypes.c_float),
                ("convex", ctypes.c_int32)]


class ScanInputs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("g", ctypes.c_void_p), ("A_log", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("h0", ctypes.c_void_p)]


class ScanGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dg", ctypes.c_void_p), ("dh0", ctypes.c_void_p),
                ("dA_log", ctypes.c_void_p), ("ddt_bias", ctypes.c_void_p)]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("group", ctypes.c_int32)]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libgdr.so (built by ``build.build()``); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with chunked_gated_delta_bwd_amd.build.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.POINTER
    lib.gdr_workspace_bytes.argtypes = [P(Shape), P(ctypes.c_size_t)]
    lib.gdr_fwd_recompute.argtypes = [P(Shape), P(Inputs), ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.gdr_fwd.argtypes = [P(Shape), P(Inputs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p,
                            ctypes.c_void_p]
    lib.gdr_bwd.argtypes = [P(Shape), P(Inputs), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                            ctypes.c_size_t, P(Grads), ctypes.c_void_p]
    lib.gdr_fwd_bwd.argtypes = [P(Shape), P(Inputs), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_size_t, P(Grads), ctypes.c_void_p, ctypes.c_void_p]
    lib.gdr_workspace_region.argtypes = [P(Shape), ctypes.c_int32, P(ctypes.c_size_t), P(ctypes.c_size_t)]
    lib.gdr_run_stage.argtypes = [P(Shape), P(Inputs), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_size_t, P(Grads), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    lib.gdr_fwd_bwd_noalloc.argtypes = [P(Shape), P(Inputs), ctypes.c_void_p, ctypes.c_void_p, P(Grads),
                                        ctypes.c_void_p, ctypes.c_void_p]
    ptr, size = ctypes.c_void_p, ctypes.c_size_t
    lib.gdr_step.argtypes = [P(Shape), P(Inputs), ptr, ctypes.c_int32, ptr, ptr, ptr]
    lib.gdr_scan_workspace_bytes.argtypes = [P(ScanShape), P(size)]
    lib.gdr_scan_fwd.argtypes = [P(ScanShape), P(ScanInputs), ptr, size, ptr, ptr, ptr]
    lib.gdr_scan_bwd.argtypes = [P(ScanShape), P(ScanInputs), ptr, ptr, ptr, size, P(ScanGrads), ptr]
    lib.gdr_scan_step.argtypes = [P(ScanShape), P(ScanInputs), ptr, ctypes.c_int32, ptr, ptr, ptr]
    lib.gdr_norm_fwd.argtypes = [P(NormShape), ptr, ptr, ptr, ptr, ptr, ptr]
    lib.gdr_norm_quant.argtypes = [P(NormShape), ptr, ptr, ptr, ptr, ptr, ptr, ptr]
    lib.gdr_norm_workspace_bytes.argtypes = [P(NormShape), P(size)]
    lib.gdr_norm_bwd.argtypes = [P(NormShape), ptr, ptr, ptr, ptr, ptr, size, ptr, ptr, ptr]
    lib.gdr_last_error.argtypes = []
    lib.gdr_last_error.restype = ctypes.c_char_p
    for name in SYMBOLS[:-1]:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != GDR_OK:
        raise GdrError(status, load_library().gdr_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Problem:
    """Host-side description of one problem: the C shape plus the tensors.

    ``tensors`` holds device tensors q k v g b (and optionally A_log dt_bias h0);
    ``cu_seqlens`` (host int64, or None for dense) is kept alive here because the
    C shape points into it.
    """

    def __init__(self, B: int, T: int, H: int, D: int, N: int, gate: int, dtype: int, scale: float,
                 cu_seqlens=None, gate_scale: float = 0.0, Hk: int = 0, seq_split: int = 0):
        self.cu = None
        if cu_seqlens is not None:
            cu = torch.as_tensor(cu_seqlens, dtype=torch.int64).contiguous().cpu()
            self.cu = cu
        self.shape = Shape(B, T, H, D, D, N,
                           None if self.cu is None else ctypes.cast(self.cu.data_ptr(), ctypes.POINTER(ctypes.c_int64)),
                           gate, dtype, scale, gate_scale, Hk, seq_split)

    @staticmethod
    def from_inputs(inp: Dict, varlen: Optional[bool] = None, seq_split: int = 0) -> "Problem":
        lengths = inp["lengths"]
        if varlen is None:
            varlen = inp["B"] == 1 and (len(lengths) > 1 or lengths[0] != inp["T"])
        dtype = GDR_BF16 if inp["dtype"] == "bf16" else GDR_F32
        gs = float(inp.get("gate_scale", 0.0))
        hk = int(inp.get("Hk") or 0)
        if varlen:
            return Problem(1, inp["T"], inp["H"], inp["K"], inp["N"], inp["gate"], dtype, inp["scale"],
                           cu_seqlens=inp["cu_seqlens"], gate_scale=gs, Hk=hk, seq_split=seq_split)
        return Problem(inp["B"], inp["T"], inp["H"], inp["K"], inp["N"], inp["gate"], dtype, inp["scale"],
                       gate_scale=gs, Hk=hk, seq_split=seq_split)


def gdr_workspace_bytes(prob: Problem) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gdr_workspace_bytes(ctypes.byref(prob.shape), ctypes.byref(out)))
    return out.value


def gdr_workspace_region(prob: Problem, which: int):
    off, n = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load_library().gdr_workspace_region(ctypes.byref(prob.shape), which, ctypes.byref(off), ctypes.byref(n)))
    return off.value, n.value


def _inputs(t: Dict) -> Inputs:
    return Inputs(_ptr(t["q"]), _ptr(t["k"]), _ptr(t["v"]), _ptr(t["g"]), _ptr(t["b"]),
                  _ptr(t.get("A_log")), _ptr(t.get("dt_bias")), _ptr(t.get("h0")))


def _grads(o: Dict) -> Grads:
    return Grads(_ptr(o["dq"]), _ptr(o["dk"]), _ptr(o["dv"]), _ptr(o["dg"]), _ptr(o["db"]),
                 _ptr(o.get("dh0")), _ptr(o.get("dA_log")), _ptr(o.get("ddt_bias")))


def gdr_fwd_recompute(prob: Problem, t: Dict, ws: torch.Tensor, ht: Optional[torch.Tensor] = None,
                      o: Optional[torch.Tensor] = None, stream=None) -> None:
    inp = _inputs(t)
    _check(load_library().gdr_fwd_recompute(ctypes.byref(prob.shape), ctypes.byref(inp), _ptr(ws),
                                            ws.numel() * ws.element_size(), _ptr(o), _ptr(ht), _stream(stream)))


def gdr_fwd(prob: Problem, t: Dict, ws: torch.Tensor, o: torch.Tensor, ht: Optional[torch.Tensor] = None,
            stream=None) -> None:
    inp = _inputs(t)
    _check(load_library().gdr_fwd(ctypes.byref(prob.shape), ctypes.byref(inp), _ptr(ws),
                                  ws.numel() * ws.element_size(), _ptr(o), _ptr(ht), _stream(stream)))


def gdr_bwd(prob: Problem, t: Dict, dO: torch.Tensor, dht: Optional[torch.Tensor], ws: torch.Tensor,
            out: Dict, stream=None) -> None:
    inp, gr = _inputs(t), _grads(out)
    _check(load_library().gdr_bwd(ctypes.byref(prob.shape), ctypes.byref(inp), _ptr(dO), _ptr(dht), _ptr(ws),
                                  ws.numel() * ws.element_size(), ctypes.byref(gr), _stream(stream)))


def gdr_fwd_bwd(prob: Problem, t: Dict, dO: torch.Tensor, dht: Optional[torch.Tensor], ws: torch.Tensor,
                out: Dict, ht: Optional[torch.Tensor] = None, stream=None) -> None:
    inp, gr = _inputs(t), _grads(out)
    _check(load_library().gdr_fwd_bwd(ctypes.byref(prob.shape), ctypes.byref(inp), _ptr(dO), _ptr(dht),
                                      _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(gr), _ptr(ht),
                                      _stream(stream)))


def gdr_fwd_bwd_noalloc(prob: Problem, t: Dict, dO: torch.Tensor, dht: Optional[torch.Tensor], out: Dict,
                        ht: Optional[torch.Tensor] = None, stream=None) -> None:
    inp, gr = _inputs(t), _grads(out)
    _check(load_library().gdr_fwd_bwd_noalloc(ctypes.byref(prob.shape), ctypes.byref(inp), _ptr(dO), _ptr(dht),
                                              ctypes.byref(gr), _ptr(ht), _stream(stream)))


def gdr_run_stage(prob: Problem, t: Dict, dO: torch.Tensor, dht: Optional[torch.Tensor], ws: torch.Tensor,
                  out: Dict, stage: int, ht: Optional[torch.Tensor] = None, stream=None) -> None:
    inp, gr = _inputs(t), _grads(out)
    _check(load_library().gdr_run_stage(ctypes.byref(prob.shape), ctypes.byref(inp), _ptr(dO), _ptr(dht),
                                        _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(gr), _ptr(ht),
                                        stage, _stream(stream)))


# ---------------------------------------------------------------------------
# the operators around the delta rule: the single-token steps, the gated linear
# recurrence and the row norm.  These entry points check their tensors (type,
# size, layout, device) before the library is called; its own checks follow.
# ---------------------------------------------------------------------------

_DTYPE = {GDR_BF16: torch.bfloat16, GDR_F32: torch.float32}


def _bad(message: str) -> None:
    raise GdrError(GDR_EINVAL, message)


def _check_range(bits: int, **fields) -> None:
    """ctypes keeps the low bits of a number that a C integer of that width cannot hold."""
    for name, value in fields.items():
        if not -(1 << (bits - 1)) <= value < 1 << (bits - 1):
            raise GdrError(GDR_EUNSUPPORTED, f"{name} ({value}) is beyond {bits} bits")


def _check_tensors(specs) -> None:
    """specs: (name, tensor or None, numel, dtype).  Every tensor given has that type
    and size, is contiguous, and lies on the current GPU, where the call is enqueued."""
    first = other = None
    for name, t, numel, dtype in specs:
        if t is None:
            continue
        if t.dtype is not dtype:
            _bad(f"{name} is {t.dtype}, expected {dtype}")
        if t.numel() != numel:
            _bad(f"{name} has {t.numel()} elements, expected {numel}")
        if not t.is_contiguous():
            _bad(f"{name} is not contiguous")
        d = t.get_device()
        if first is None:
            first = d
        elif d != first:
            other = d
    if first is None:
        return
    if other is not None:
        _bad(f"tensors are on several devices: {first} and {other} (-1: the CPU)")
    if first < 0:
        _bad("tensors are on the CPU, expected a GPU")
    if first != torch.cuda.current_device():
        _bad(f"tensors are on cuda:{first}, the current device is cuda:{torch.cuda.current_device()}")


def _stream_here(stream) -> Optional[int]:
    """The stream's handle; it has to be the current device's, where _check_tensors found the tensors."""
    here = getattr(stream, "device_index", None)
    if here is not None and here != torch.cuda.current_device():
        _bad(f"the stream is on cuda:{here}, the current device is cuda:{torch.cuda.current_device()}")
    return _stream(stream)


def _check_workspace(ws: Optional[torch.Tensor], like: Optional[torch.Tensor]) -> int:
    if ws is None:
        return 0
    if not ws.is_contiguous():
        _bad("the workspace is not contiguous")
    if like is not None and ws.get_device() != like.get_device():
        _bad(f"the workspace is on {ws.device}, the tensors are on {like.device}")
    return ws.numel() * ws.element_size()


def _pool_size(state: torch.Tensor, per_state: int) -> int:
    """Number of states in a pool [P, ...] of per_state elements each."""
    if state.dim() < 1 or state.numel() != state.shape[0] * per_state:
        _bad(f"state has shape {tuple(state.shape)}, expected [P, ...] with {per_state} elements a state")
    _check_range(32, **{"state's first dimension": state.shape[0]})
    return state.shape[0]


class ScanProblem:
    """Host-side description of one gated linear recurrence (gdr_scan_shape)."""

    def __init__(self, B: int, T: int, H: int, D: int, N: int, gate: int, dtype: int, cu_seqlens=None,
                 gate_scale: float = 0.0, convex: bool = False):
        _check_range(32, B=B, T=T, H=H, D=D, N=N, gate=gate, dtype=dtype, convex=convex)
        self.cu = None
        if cu_seqlens is not None:
            self.cu = torch.as_tensor(cu_seqlens, dtype=torch.int64).contiguous().cpu()
            if self.cu.numel() != N + 1:
                _bad(f"cu_seqlens has {self.cu.numel()} entries, expected {N + 1}")
        self.shape = ScanShape(B, T, H, D, N,
                               None if self.cu is None else ctypes.cast(self.cu.data_ptr(),
                                                                        ctypes.POINTER(ctypes.c_int64)),
                               gate, dtype, gate_scale if gate == GDR_GATE_CHANNEL_SIGMOID else 0.0, int(convex))
        self.ref = ctypes.byref(self.shape)
        tokens = B * T
        self.x_numel = tokens * H * D
        self.g_numel = tokens * H if gate == GDR_GATE_SCALAR else self.x_numel
        self.state_numel, self.per_state, self.D, self.H = N * H * D, H * D, D, H
        self.rows, self.io = N, _DTYPE.get(dtype)

    def input_specs(self, t: Dict):
        return (("x", t["x"], self.x_numel, self.io), ("g", t["g"], self.g_numel, self.io),
                ("A_log", t.get("A_log"), self.H, torch.float32),
                ("dt_bias", t.get("dt_bias"), self.per_state, torch.float32),
                ("h0", t.get("h0"), self.state_numel, torch.float32))


def _scan_inputs(t: Dict) -> ScanInputs:
    return ScanInputs(_ptr(t["x"]), _ptr(t["g"]), _ptr(t.get("A_log")), _ptr(t.get("dt_bias")), _ptr(t.get("h0")))


def gdr_scan_workspace_bytes(prob: ScanProblem) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gdr_scan_workspace_bytes(prob.ref, ctypes.byref(out)))
    return out.value


def alloc_scan_workspace(prob: ScanProblem, device="cuda") -> torch.Tensor:
    return torch.empty(max(gdr_scan_workspace_bytes(prob), 256), dtype=torch.uint8, device=device)


def gdr_scan_fwd(prob: ScanProblem, t: Dict, ws: torch.Tensor, y: torch.Tensor, ht: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    _check_tensors(prob.input_specs(t) + (("y", y, prob.x_numel, prob.io), ("ht", ht, prob.state_numel, torch.float32)))
    n = _check_workspace(ws, y)
    inp = _scan_inputs(t)
    _check(load_library().gdr_scan_fwd(prob.ref, ctypes.byref(inp), _ptr(ws), n, _ptr(y), _ptr(ht), _stream_here(stream)))


def gdr_scan_bwd(prob: ScanProblem, t: Dict, dy: torch.Tensor, dht: Optional[torch.Tensor], ws: torch.Tensor,
                 out: Dict, stream=None) -> None:
    """out: dx, dg, and optionally dh0; for the per-channel gates dA_log and ddt_bias."""
    f32 = torch.float32
    _check_tensors(prob.input_specs(t) + (
        ("dy", dy, prob.x_numel, prob.io), ("dht", dht, prob.state_numel, f32), ("dx", out["dx"], prob.x_numel, prob.io),
        ("dg", out["dg"], prob.g_numel, prob.io), ("dh0", out.get("dh0"), prob.state_numel, f32),
        ("dA_log", out.get("dA_log"), prob.H, f32), ("ddt_bias", out.get("ddt_bias"), prob.per_state, f32)))
    n = _check_workspace(ws, dy)
    inp = _scan_inputs(t)
    gr = ScanGrads(_ptr(out["dx"]), _ptr(out["dg"]), _ptr(out.get("dh0")), _ptr(out.get("dA_log")),
                   _ptr(out.get("ddt_bias")))
    _check(load_library().gdr_scan_bwd(prob.ref, ctypes.byref(inp), _ptr(dy), _ptr(dht), _ptr(ws), n, ctypes.byref(gr),
                                       _stream_here(stream)))


def gdr_scan_step(prob: ScanProblem, t: Dict, state: torch.Tensor, y: torch.Tensor,
                  slots: Optional[torch.Tensor] = None, stream=None) -> None:
    P = _pool_size(state, prob.per_state)
    _check_tensors(prob.input_specs(t) + (("y", y, prob.x_numel, prob.io), ("state", state, state.numel(), torch.float32),
                                          ("slots", slots, prob.rows, torch.int32)))
    inp = _scan_inputs(t)
    _check(load_library().gdr_scan_step(prob.ref, ctypes.byref(inp), _ptr(state), P, _ptr(slots), _ptr(y),
                                        _stream_here(stream)))


def gdr_step(prob: Problem, t: Dict, state: torch.Tensor, o: torch.Tensor, slots: Optional[torch.Tensor] = None,
             stream=None) -> None:
    """prob: Problem(N, 1, H, D, N, ...); t: q k v g b (and A_log, dt_bias)."""
    s = prob.shape
    N, H, D, io = s.B * s.T, s.H, s.Dk, _DTYPE.get(s.dtype)
    qk = N * (s.Hk or H) * D
    gn = N * H if s.gate == GDR_GATE_SCALAR else N * H * D
    P = _pool_size(state, H * D * D)
    _check_tensors((("q", t["q"], qk, io), ("k", t["k"], qk, io), ("v", t["v"], N * H * D, io), ("g", t["g"], gn, io),
                    ("b", t["b"], N * H, io), ("A_log", t.get("A_log"), H, torch.float32),
                    ("dt_bias", t.get("dt_bias"), H * D, torch.float32), ("o", o, N * H * D, io),
                    ("state", state, state.numel(), torch.float32), ("slots", slots, N, torch.int32)))
    inp = _inputs(t)
    _check(load_library().gdr_step(ctypes.byref(s), ctypes.byref(inp), _ptr(state), P, _ptr(slots), _ptr(o),
                                   _stream_here(stream)))


class NormProblem:
    """Host-side description of one row norm (gdr_norm_shape)."""

    def __init__(self, rows: int, width: int, dtype: int, eps: float = 1e-6, group: int = 0):
        _check_range(64, rows=rows)
        _check_range(32, width=width, dtype=dtype, group=group)
        self.shape = NormShape(rows, width, dtype, eps, group)
        self.ref = ctypes.byref(self.shape)
        self.numel, self.width, self.io = rows * width, width, _DTYPE.get(dtype)
        self.scales_numel = rows * (-(-width // group) if group > 0 else 1)


def gdr_norm_workspace_bytes(prob: NormProblem) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gdr_norm_workspace_bytes(prob.ref, ctypes.byref(out)))
    return out.value


def alloc_norm_workspace(prob: NormProblem, device="cuda") -> torch.Tensor:
    return torch.empty(max(gdr_norm_workspace_bytes(prob), 256), dtype=torch.uint8, device=device)


def gdr_norm_fwd(prob: NormProblem, x: torch.Tensor, w: Optional[torch.Tensor], y: torch.Tensor,
                 res: Optional[torch.Tensor] = None, res_out: Optional[torch.Tensor] = None, stream=None) -> None:
    n, io = prob.numel, prob.io
    _check_tensors((("x", x, n, io), ("w", w, prob.width, torch.float32), ("y", y, n, io), ("res", res, n, io),
                    ("res_out", res_out, n, io)))
    _check(load_library().gdr_norm_fwd(prob.ref, _ptr(x), _ptr(res), _ptr(w), _ptr(y), _ptr(res_out), _stream_here(stream)))


def gdr_norm_quant(prob: NormProblem, x: torch.Tensor, w: Optional[torch.Tensor], q: torch.Tensor,
                   scales: torch.Tensor, res: Optional[torch.Tensor] = None, res_out: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    n, io = prob.numel, prob.io
    _check_tensors((("x", x, n, io), ("w", w, prob.width, torch.float32), ("q", q, n, torch.float8_e4m3fn),
                    ("scales", scales, prob.scales_numel, torch.float32), ("res", res, n, io),
                    ("res_out", res_out, n, io)))
    _check(load_library().gdr_norm_quant(prob.ref, _ptr(x), _ptr(res), _ptr(w), _ptr(q), _ptr(scales), _ptr(res_out),
                                         _stream_here(stream)))


def gdr_norm_bwd(prob: NormProblem, r: torch.Tensor, w: Optional[torch.Tensor], dy: torch.Tensor, dx: torch.Tensor,
                 dw: Optional[torch.Tensor], ws: Optional[torch.Tensor], dres: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    n, io = prob.numel, prob.io
    _check_tensors((("r", r, n, io), ("w", w, prob.width, torch.float32), ("dy", dy, n, io), ("dx", dx, n, io),
                    ("dw", dw, prob.width, torch.float32), ("dres", dres, n, io)))
    _check(load_library().gdr_norm_bwd(prob.ref, _ptr(r), _ptr(w), _ptr(dy), _ptr(dres), _ptr(ws),
                                       _check_workspace(ws, dy), _ptr(dx), _ptr(dw), _stream_here(stream)))


# ---------------------------------------------------------------------------
# convenience for tests and the benchmark: device copies and output buffers
# ---------------------------------------------------------------------------

def to_device(inp: Dict, device="cuda") -> Dict:
    """Device copies of the generator's tensors (same bytes)."""
    out = {}
    for key in ("q", "k", "v", "g", "b", "dO", "A_log", "dt_bias", "h0", "dht"):
        x = inp.get(key)
        out[key] = None if x is None else x.to(device).contiguous()
    return out


def alloc_outputs(inp: Dict, dev: Dict, want_dh0: bool = True) -> Dict:
    """Output tensors of the right shapes/dtypes on the inputs' device."""
    q, g = dev["q"], dev["g"]
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(dev["k"]), "dv": torch.empty_like(dev["v"]),
           "dg": torch.empty_like(g), "db": torch.empty_like(dev["b"])}
    N, H, K, V = inp["N"], inp["H"], inp["K"], inp["V"]
    out["dh0"] = torch.empty((N, H, V, K), dtype=torch.float32, device=q.device) if want_dh0 else None
    if inp["gate"] != GDR_GATE_SCALAR:
        out["dA_log"] = torch.empty((H,), dtype=torch.float32, device=q.device)
        out["ddt_bias"] = torch.empty((H, K), dtype=torch.float32, device=q.device)
    return out


def alloc_workspace(prob: Problem, device="cuda") -> torch.Tensor:
    n = gdr_workspace_bytes(prob)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)
