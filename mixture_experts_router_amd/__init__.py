"""Python binding of the MI355X MoE-layer library (libmoe_amd.so).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  PyTorch provides device memory and the current stream.  The names
mirror the C ABI in include/moe.h:

    route, topk_from_logits, layer_forward, fuse_gate_up,
    layer_workspace_size, route_workspace_size,
    gate, gate_from_logits, gate_backward, layer_forward_gated, lora_add

If the library is not built this module raises on first use; there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_amd.so")

MOE_F16, MOE_BF16, MOE_F32 = 1, 2, 3
MOE_K_ENTROPY = -1
MOE_K_ENTROPY_CAP = 3
FLAG_UNFUSED, FLAG_FORCE_GEMV, FLAG_FORCE_MFMA = 0x1, 0x2, 0x4

STATUS = {0: "MOE_OK", -1: "MOE_ERR_NULL", -2: "MOE_ERR_SHAPE", -3: "MOE_ERR_DTYPE", -4: "MOE_ERR_ALIGN",
          -5: "MOE_ERR_K", -6: "MOE_ERR_QUANT", -7: "MOE_ERR_INCOMPATIBLE", -8: "MOE_ERR_WORKSPACE",
          -9: "MOE_ERR_DEVICE", -10: "MOE_ERR_HIP", -11: "MOE_ERR_INTERNAL", -12: "MOE_ERR_OPTION",
          -13: "MOE_ERR_SCRATCH"}
NOALLOC_SCRATCH_BYTES = 64 << 20

EXPORTS = ("moe_route_workspace_size", "moe_route", "moe_route_ex", "moe_topk_from_logits",
           "moe_topk_from_logits_ex", "moe_layer_workspace_size", "moe_layer_forward", "moe_layer_forward_ex",
           "moe_layer_forward_noalloc", "moe_layer_forward_gated",
           "moe_gate_workspace_size", "moe_gate", "moe_gate_from_logits", "moe_gate_backward",
           "moe_lora_add",
           "moe_expert_load_stats", "moe_fuse_gate_up", "moe_packed_sb_bytes", "moe_pack_sb", "moe_packed_q_bytes", "moe_pack_q", "moe_status_string",
           "moe_debug_set_events",
           "moe_debug_last_plan", "moe_debug_set_tuning", "moe_debug_stream_read")


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__("%s failed: %s (%s)" % (what, self.name, _status_text(status)))


class CWeights(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
                ("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("expert_stride_rows", ctypes.c_int64), ("packed_sb", ctypes.c_void_p),
                ("format", ctypes.c_int32), ("tensor_scale", ctypes.c_float), ("packed_q", ctypes.c_void_p)]


FMT_AFFINE, FMT_NVFP4 = 0, 1


class CRouteOpts(ctypes.Structure):
    _fields_ = [("health", ctypes.c_void_p), ("alpha", ctypes.c_float), ("groups", ctypes.c_int32),
                ("capacity", ctypes.c_int32)]


class CGateOpts(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int32),
                ("group_k", ctypes.c_int32), ("group_best", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("scale", ctypes.c_float), ("capacity", ctypes.c_int32)]


class CLora(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("K", ctypes.c_int32),
                ("N", ctypes.c_int32)]


class CTaps(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("logits", "topk_idx", "topk_w", "k_used", "entropy", "counts", "offsets", "perm", "h",
                 "gate_up_preact")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe_amd.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libmoe_amd.so is not built; run `python -m mixture_experts_router_amd.build` "
                           "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    u32 = ctypes.c_uint32
    L.moe_route_workspace_size.argtypes = [i32, i32, i32]
    L.moe_route_workspace_size.restype = sz
    L.moe_route.argtypes = [vp, i32, i32, i32, vp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_route.restype = i32
    L.moe_topk_from_logits.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.moe_topk_from_logits.restype = i32
    ropt = ctypes.POINTER(CRouteOpts)
    L.moe_route_ex.argtypes = [vp, i32, i32, i32, vp, i32, i32, ropt, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_route_ex.restype = i32
    L.moe_topk_from_logits_ex.argtypes = [vp, i32, i32, i32, ropt, vp, vp, vp, vp, vp, sz, vp]
    L.moe_topk_from_logits_ex.restype = i32
    L.moe_layer_forward_ex.argtypes = [vp, i32, i32, i32, vp, i32, i32, ropt, ctypes.POINTER(CWeights),
                                       ctypes.POINTER(CWeights), ctypes.POINTER(CWeights), ctypes.POINTER(CWeights),
                                       vp, u32, ctypes.POINTER(CTaps), vp, sz, vp]
    L.moe_layer_forward_ex.restype = i32
    L.moe_layer_forward_noalloc.argtypes = [vp, i32, i32, i32, vp, i32, i32, ropt, ctypes.POINTER(CWeights),
                                            ctypes.POINTER(CWeights), ctypes.POINTER(CWeights),
                                            ctypes.POINTER(CWeights), vp, u32, ctypes.POINTER(CTaps), vp]
    L.moe_layer_forward_noalloc.restype = i32
    gopt = ctypes.POINTER(CGateOpts)
    L.moe_gate_workspace_size.argtypes = [i32, i32]
    L.moe_gate_workspace_size.restype = sz
    L.moe_gate.argtypes = [vp, i32, i32, i32, vp, i32, i32, gopt, vp, vp, vp, vp, sz, vp]
    L.moe_gate.restype = i32
    L.moe_gate_from_logits.argtypes = [vp, i32, i64, i32, i32, i32, gopt, vp, vp, vp]
    L.moe_gate_from_logits.restype = i32
    L.moe_gate_backward.argtypes = [vp, i32, i64, i32, i32, i32, gopt, vp, vp, vp, i64, vp]
    L.moe_gate_backward.restype = i32
    L.moe_layer_forward_gated.argtypes = [vp, i32, i32, i32, vp, vp, i32, i32, gopt, ctypes.POINTER(CWeights),
                                          ctypes.POINTER(CWeights), ctypes.POINTER(CWeights),
                                          ctypes.POINTER(CWeights), vp, u32, ctypes.POINTER(CTaps), vp, sz, vp]
    L.moe_layer_forward_gated.restype = i32
    L.moe_lora_add.argtypes = [vp, i32, i64, i32, ctypes.POINTER(CLora), vp, vp, i64, vp, i64, i32, vp]
    L.moe_lora_add.restype = i32
    L.moe_expert_load_stats.argtypes = [vp, i32, vp, vp, vp]
    L.moe_expert_load_stats.restype = i32
    L.moe_layer_workspace_size.argtypes = [i32, i32, i32, i32, i32, u32]
    L.moe_layer_workspace_size.restype = sz
    L.moe_layer_forward.argtypes = [vp, i32, i32, i32, vp, i32, i32, ctypes.POINTER(CWeights),
                                    ctypes.POINTER(CWeights), ctypes.POINTER(CWeights), ctypes.POINTER(CWeights),
                                    vp, u32, ctypes.POINTER(CTaps), vp, sz, vp]
    L.moe_layer_forward.restype = i32
    L.moe_fuse_gate_up.argtypes = [ctypes.POINTER(CWeights), ctypes.POINTER(CWeights), vp, vp, vp, vp]
    L.moe_fuse_gate_up.restype = i32
    L.moe_packed_sb_bytes.argtypes = [i32, ctypes.c_int64, i32]
    L.moe_packed_sb_bytes.restype = sz
    L.moe_pack_sb.argtypes = [ctypes.POINTER(CWeights), vp, vp]
    L.moe_packed_q_bytes.argtypes = [i32, ctypes.c_int64, i32, i32]
    L.moe_packed_q_bytes.restype = sz
    L.moe_pack_q.argtypes = [ctypes.POINTER(CWeights), vp, vp]
    L.moe_pack_sb.restype = i32
    L.moe_status_string.argtypes = [i32]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_debug_set_events.argtypes = [vp, i32]
    L.moe_debug_set_events.restype = None
    L.moe_debug_last_plan.argtypes = [ctypes.c_char_p, sz]
    L.moe_debug_last_plan.restype = i32
    L.moe_debug_set_tuning.argtypes = [i32, i32]
    L.moe_debug_set_tuning.restype = None
    L.moe_debug_stream_read.argtypes = [vp, sz, vp, vp]
    L.moe_debug_stream_read.restype = i32
    _lib = L
    return L


def _status_text(s: int) -> str:
    try:
        return lib().moe_status_string(s).decode()
    except Exception:  # pragma: no cover
        return "?"


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MoeError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return MOE_F16
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError("activations must be float16 or bfloat16, got %s" % t.dtype)


@dataclasses.dataclass
class Weights:
    """Device weight tensor [E, N, K] in the library's layout (see include/moe.h).

    bits 4: q uint8 [E, N, K/2]; bits 5 / 6: q uint8 [E, N, 5K/8] / [E, N, 3K/4]
    (code k at bits b*k..b*k+b-1 of the row's little-endian bit stream, b =
    bits; the batched path takes 5-bit rows when hidden and inter are multiples
    of 128); bits 8: q uint8 [E, N, K];
    bits 16: q float16 [E, N, K].  scales/biases float16 [E, N, K/64] (None for bits 16).
    ``fmt="nvfp4"`` (bits 4, group_size 16): q uint8 [E, N, K/2] E2M1 codes
    (even column in the low nibble), scales uint8 [E, N, K/16] E4M3 block
    scales, biases None, ``tensor_scale`` the fp32 per-tensor scale.
    ``row_offset``/``stride`` describe a view (the gate or up half of a fused
    tensor): rows start ``row_offset`` rows in, experts are ``stride`` rows apart.
    ``packed_sb`` (optional, uint8): the scales and biases repacked by pack_sb
    for the batched path (the whole tensor's; views share it).  ``packed_q``
    (optional, uint8): the codes repacked by pack_q for the batched path (the
    whole tensor's; views share it).
    """

    q: torch.Tensor
    scales: Optional[torch.Tensor]
    biases: Optional[torch.Tensor]
    E: int
    N: int
    K: int
    bits: int
    group_size: int = 64
    stride: Optional[int] = None
    row_offset: int = 0
    packed_sb: Optional[torch.Tensor] = None
    fmt: str = "affine"  # "affine" | "nvfp4"
    tensor_scale: float = 1.0
    packed_q: Optional[torch.Tensor] = None

    _cstruct: Optional[CWeights] = dataclasses.field(default=None, repr=False, compare=False)

    def c(self) -> CWeights:
        if self._cstruct is not None:
            return self._cstruct
        stride = self.N if self.stride is None else self.stride
        rb = self.K * self.bits // 8
        ng = self.K // self.group_size
        f4 = self.fmt == "nvfp4"
        srb = ng if f4 else ng * 2  # scale bytes per row
        q = self.q.data_ptr() + self.row_offset * rb
        s = None if self.scales is None else self.scales.data_ptr() + self.row_offset * srb
        b = None if self.biases is None else self.biases.data_ptr() + self.row_offset * srb
        sb = None if self.packed_sb is None else self.packed_sb.data_ptr() + self.row_offset * 8
        pq = None
        if self.packed_q is not None:
            ug = 1 if self.bits in (6, 16) else 2  # groups per unit
            nu = (self.K + 64 * ug - 1) // (64 * ug)
            pq = self.packed_q.data_ptr() + self.row_offset // 32 * nu * 32 * 8 * self.bits * ug
        self._cstruct = CWeights(q, s, b, self.E, self.N, self.K, self.bits, self.group_size, stride, sb,
                                 FMT_NVFP4 if f4 else FMT_AFFINE, float(self.tensor_scale), pq)
        return self._cstruct

    def split_gate_up(self):
        """(gate, up) views of a fused [E, 2I, K] tensor, gate rows first."""
        I = self.N // 2
        g = dataclasses.replace(self, N=I, stride=self.N, row_offset=0, _cstruct=None)
        u = dataclasses.replace(self, N=I, stride=self.N, row_offset=I, _cstruct=None)
        return g, u


def route_workspace_size(T: int, E: int, k: int) -> int:
    return int(lib().moe_route_workspace_size(T, E, k))


def layer_workspace_size(T: int, H: int, E: int, k: int, inter: int, flags: int = 0) -> int:
    return int(lib().moe_layer_workspace_size(T, H, E, k, inter, flags))


def _kcap(k: int) -> int:
    return k if k > 0 else MOE_K_ENTROPY_CAP


def _opts(health: Optional[torch.Tensor], alpha: float, groups: int, capacity: int = 0):
    """moe_route_opts for the *_ex entry points, or None when no option is set."""
    if health is None and not groups and not capacity:
        return None
    if health is not None:
        assert health.dtype == torch.float32 and health.is_contiguous()
    return CRouteOpts(_ptr(health), float(alpha), int(groups), int(capacity))


def route(x: torch.Tensor, router_w: torch.Tensor, k: int, want_logits: bool = False, stream=None,
          health: Optional[torch.Tensor] = None, alpha: float = 0.0, groups: int = 0):
    """Router + selection.  Returns dict(idx [T,kcap] int32, w [T,kcap] fp32,
    k_used [1] int32, entropy [1] fp32[, logits [T,E] fp32]).  health/alpha:
    load-aware correction of the logits; groups: at most one expert per group
    of E/groups consecutive experts (moe_route_opts)."""
    T, H = x.shape
    E = router_w.shape[0]
    dev = x.device
    kc = _kcap(k)
    idx = torch.empty((T, kc), dtype=torch.int32, device=dev)
    w = torch.empty((T, kc), dtype=torch.float32, device=dev)
    ku = torch.zeros(1, dtype=torch.int32, device=dev)
    ent = torch.zeros(1, dtype=torch.float32, device=dev)
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None
    ws = torch.empty(max(route_workspace_size(T, E, k), 256), dtype=torch.uint8, device=dev)
    o = _opts(health, alpha, groups)
    if o is None:
        st = lib().moe_route(_ptr(x), _dtype_code(x), T, H, _ptr(router_w), E, k, _ptr(idx), _ptr(w), _ptr(ku),
                             _ptr(ent), _ptr(logits), _ptr(ws), ws.numel(), _stream(stream))
    else:
        st = lib().moe_route_ex(_ptr(x), _dtype_code(x), T, H, _ptr(router_w), E, k, ctypes.byref(o), _ptr(idx),
                                _ptr(w), _ptr(ku), _ptr(ent), _ptr(logits), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "moe_route")
    out = dict(idx=idx, w=w, k_used=ku, entropy=ent)
    if logits is not None:
        out["logits"] = logits
    return out


def topk_from_logits(logits: torch.Tensor, k: int, stream=None, groups: int = 0):
    T, E = logits.shape
    dev = logits.device
    kc = _kcap(k)
    idx = torch.empty((T, kc), dtype=torch.int32, device=dev)
    w = torch.empty((T, kc), dtype=torch.float32, device=dev)
    ku = torch.zeros(1, dtype=torch.int32, device=dev)
    ent = torch.zeros(1, dtype=torch.float32, device=dev)
    lg = logits.contiguous()
    if not groups:
        st = lib().moe_topk_from_logits(_ptr(lg), T, E, k, _ptr(idx), _ptr(w), _ptr(ku), _ptr(ent), None, 0,
                                        _stream(stream))
    else:
        o = CRouteOpts(None, 0.0, int(groups), 0)
        st = lib().moe_topk_from_logits_ex(_ptr(lg), T, E, k, ctypes.byref(o), _ptr(idx), _ptr(w), _ptr(ku),
                                           _ptr(ent), None, 0, _stream(stream))
    _check(st, "moe_topk_from_logits")
    return dict(idx=idx, w=w, k_used=ku, entropy=ent)


TAP_NAMES = ("logits", "topk_idx", "topk_w", "k_used", "entropy", "counts", "offsets", "perm", "h",
             "gate_up_preact")


def make_taps(T: int, E: int, k: int, inter: int, device, names: Sequence[str] = TAP_NAMES):
    """Allocate tap buffers (logits, routing, sort results, SwiGLU rows, fp32
    gate+up pre-activations)."""
    kc = _kcap(k)
    P = T * kc
    spec = dict(logits=((T, E), torch.float32), topk_idx=((T, kc), torch.int32), topk_w=((T, kc), torch.float32),
                k_used=((1,), torch.int32), entropy=((1,), torch.float32), counts=((E,), torch.int32),
                offsets=((E + 1,), torch.int32), perm=((P,), torch.int32), h=((P, inter), torch.float16),
                gate_up_preact=((P, 2 * inter), torch.float32))
    return {n: torch.zeros(spec[n][0], dtype=spec[n][1], device=device) for n in names}


def layer_forward(x: torch.Tensor, router_w: torch.Tensor, k: int, down: Weights, gate_up: Optional[Weights] = None,
                  gate: Optional[Weights] = None, up: Optional[Weights] = None, flags: int = 0,
                  taps: Optional[dict] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None, health: Optional[torch.Tensor] = None,
                  alpha: float = 0.0, groups: int = 0, capacity: int = 0) -> torch.Tensor:
    """The whole layer: y [T, H] in the activation dtype (routing options as in
    route(); capacity > 0: at most that many pairs per expert, moe_route_opts)."""
    T, H = x.shape
    E = router_w.shape[0]
    inter = down.K
    y = torch.empty_like(x) if out is None else out
    need = layer_workspace_size(T, H, E, k, inter, flags)
    ws = workspace
    if ws is None or ws.numel() < need:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    ctaps = None
    if taps:
        ctaps = CTaps(*[(taps[n].data_ptr() if n in taps and taps[n] is not None else None) for n in TAP_NAMES])
    cgu = gate_up.c() if gate_up is not None else None
    cg = gate.c() if gate is not None else None
    cu = up.c() if up is not None else None
    cd = down.c()
    wargs = (ctypes.byref(cgu) if cgu is not None else None, ctypes.byref(cg) if cg is not None else None,
             ctypes.byref(cu) if cu is not None else None, ctypes.byref(cd), _ptr(y), flags,
             ctypes.byref(ctaps) if ctaps is not None else None, _ptr(ws), ws.numel(), _stream(stream))
    o = _opts(health, alpha, groups, capacity)
    if o is None:
        st = lib().moe_layer_forward(_ptr(x), _dtype_code(x), T, H, _ptr(router_w), E, k, *wargs)
    else:
        st = lib().moe_layer_forward_ex(_ptr(x), _dtype_code(x), T, H, _ptr(router_w), E, k, ctypes.byref(o),
                                        *wargs)
    _check(st, "moe_layer_forward")
    return y


def layer_forward_noalloc(x: torch.Tensor, router_w: torch.Tensor, k: int, down: Weights,
                          gate_up: Optional[Weights] = None, gate: Optional[Weights] = None,
                          up: Optional[Weights] = None, flags: int = 0, taps: Optional[dict] = None,
                          out: Optional[torch.Tensor] = None, stream=None, health: Optional[torch.Tensor] = None,
                          alpha: float = 0.0, groups: int = 0, capacity: int = 0) -> torch.Tensor:
    """layer_forward through moe_layer_forward_noalloc: no workspace argument,
    the library's per-device scratch array instead (calls on one GPU must not
    overlap).  With `out` given, nothing is allocated."""
    T, H = x.shape
    E = router_w.shape[0]
    y = torch.empty_like(x) if out is None else out
    ctaps = None
    if taps:
        ctaps = CTaps(*[(taps[n].data_ptr() if n in taps and taps[n] is not None else None) for n in TAP_NAMES])
    ref = lambda w: ctypes.byref(w.c()) if w is not None else None
    o = _opts(health, alpha, groups, capacity)
    st = lib().moe_layer_forward_noalloc(_ptr(x), _dtype_code(x), T, H, _ptr(router_w), E, k,
                                         ctypes.byref(o) if o is not None else None, ref(gate_up), ref(gate),
                                         ref(up), ref(down), _ptr(y), flags,
                                         ctypes.byref(ctaps) if ctaps is not None else None, _stream(stream))
    _check(st, "moe_layer_forward_noalloc")
    return y


# ------------------------------------------------------ gate and adapters --

SCORES = {"softmax": 0, "sigmoid": 1}
_TYPES = {torch.float16: MOE_F16, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}


def _elsewhere(t: torch.Tensor, stream):
    """The context for a call that is not on tensor `t`'s GPU or not on `stream`
    yet.  Under `stream`, what the call allocates belongs to that stream."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on the GPU, got one on %s" % t.device)
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != t.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
    return torch.cuda.stream(stream)


# the current device and stream's handle without Python objects (2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# a dense tensor on the current GPU: half of new_empty's time (0.6 against 1.2 us)
_empty_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _new(like: torch.Tensor, rows: int, columns: int, dtype):
    """A dense tensor [rows, columns] beside `like`, which is on the current GPU."""
    if _empty_cuda is not None:
        return _empty_cuda((rows, columns), (columns, 1), dtype)
    return like.new_empty((rows, columns), dtype=dtype)


def _here(t: torch.Tensor, stream) -> bool:
    """Whether `t` is on the current GPU and no other stream is asked for."""
    dev = t.get_device()
    return stream is None and dev >= 0 and dev == _raw_device()


def _current(dev: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _operand(t: Optional[torch.Tensor], name: str, dev: int, dtype, shape):
    """Address of a dense tensor of that type and shape on GPU `dev` (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        raise ValueError("%s must be dense on GPU %d with shape %s, got shape %s on %s" %
                         (name, dev, tuple(shape), tuple(t.shape), t.device))
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str):
    """(t, T, columns, elements between rows) of a matrix whose rows are dense and
    do not overlap: `t` itself or, if it is none, a copy."""
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions, got shape %s" % (name, tuple(t.shape)))
    T, n = t.shape
    ld, step = t.stride()
    if step == 1 and (ld >= n or T < 2):
        return t, T, n, ld if T > 1 else n
    return t.contiguous(), T, n, n


def _out_rows(t: torch.Tensor, name: str, dev: int, dtype, shape) -> int:
    """Elements between the dense rows of the caller's output."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape or t.get_device() != dev:
        raise ValueError("%s must have shape %s on GPU %d, got %s on %s" %
                         (name, tuple(shape), dev, tuple(t.shape), t.device))
    ld, step = t.stride()
    if shape[0] < 2:
        ld = shape[1]
    if (step != 1 and shape[1] > 1) or ld < shape[1]:
        raise ValueError("%s: rows must be dense and apart" % name)
    return ld


def _gate_opts(dev: int, E: int, score: str, bias, groups: int, group_k: int, group_best: int, renorm: bool,
               scale: float, capacity: int = 0) -> CGateOpts:
    kind = SCORES.get(score)
    if kind is None:
        raise ValueError("score must be one of %s, got %r" % (sorted(SCORES), score))
    return CGateOpts(kind, _operand(bias, "bias", dev, torch.float32, (E,)), groups, group_k, group_best,
                     1 if renorm else 0, scale, capacity)


def _gate_type(logits: torch.Tensor) -> int:
    code = _TYPES.get(logits.dtype)
    if code is None:
        raise TypeError("logits must be float32, float16 or bfloat16, got %s" % logits.dtype)
    return code


def _routing_out(like: torch.Tensor, T: int, k: int, out):
    """The (idx, w) tensors of a gate call, new or the caller's."""
    if out is None:
        k = max(k, 0)
        return _new(like, T, k, torch.int32), _new(like, T, k, torch.float32)
    idx, w = out
    dev = like.get_device()
    _operand(idx, "out[0]", dev, torch.int32, (T, k))
    _operand(w, "out[1]", dev, torch.float32, (T, k))
    return idx, w


def _no_graph(name: str) -> None:
    """Refuses inputs that autograd follows: the call has no backward pass, and a
    result without a graph would drop their gradient silently."""
    if torch.is_grad_enabled():
        raise RuntimeError("%s has no backward pass, and an input requires grad: call it under torch.no_grad() or on "
                           "detached tensors" % name)


class _GateFromLogits(torch.autograd.Function):
    """gate_from_logits for logits that require grad, with gate_backward as its gradient."""

    @staticmethod
    def forward(ctx, logits, k, opts):
        r = gate_from_logits(logits, k, **opts)  # grad mode is off in here
        ctx.mark_non_differentiable(r["idx"])
        ctx.save_for_backward(logits, r["idx"])
        ctx.opts = {n: opts[n] for n in ("score", "renorm", "scale")}
        return r["idx"], r["w"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, grad_w):
        logits, idx = ctx.saved_tensors
        return gate_backward(logits, idx, grad_w.contiguous(), **ctx.opts), None, None


def gate_from_logits(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                     groups: int = 0, group_k: int = 0, group_best: int = 1, renorm: bool = True, scale: float = 1.0,
                     out=None, stream=None):
    """The routing gate on logits [T, E] (float32, float16 or bfloat16): dict(idx
    [T, k] int32, w [T, k] float32).  score "softmax" or "sigmoid"; bias [E]
    float32 is added to the scores for the selection only; groups: only the
    experts of the group_k best of `groups` groups can be chosen, a group being
    worth the sum of its group_best best keys; renorm: the weights of a token
    sum to `scale` (moe_gate_opts).  out: (idx, w) to write into.  For logits
    that require grad (and no `out`) w carries the graph of gate_backward, of
    first order; refused while the stream is captured."""
    if not _here(logits, stream):
        with _elsewhere(logits, stream):
            return gate_from_logits(logits, k, score=score, bias=bias, groups=groups, group_k=group_k,
                                    group_best=group_best, renorm=renorm, scale=scale, out=out)
    if logits.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise RuntimeError("gate_from_logits: `out` has no graph, and the logits require grad")
        if torch.cuda.is_current_stream_capturing():
            # its backward pass would be captured too, which an eager graph of the same leaves can make an abort
            raise RuntimeError("gate_from_logits: while a stream is captured, call it under torch.no_grad() with "
                               "gate_backward for the gradient")
        idx, w = _GateFromLogits.apply(logits, k, dict(score=score, bias=bias, groups=groups, group_k=group_k,
                                                       group_best=group_best, renorm=renorm, scale=scale))
        return dict(idx=idx, w=w)
    code = _gate_type(logits)
    logits, T, E, ld = _rows(logits, "logits")
    dev = logits.get_device()
    o = _gate_opts(dev, E, score, bias, groups, group_k, group_best, renorm, scale)
    idx, w = _routing_out(logits, T, k, out)
    _check(lib().moe_gate_from_logits(logits.data_ptr(), code, ld, T, E, k, o, idx.data_ptr(), w.data_ptr(),
                                      _current(dev)), "moe_gate_from_logits")
    return dict(idx=idx, w=w)


def gate(x: torch.Tensor, router_w: torch.Tensor, k: int, *, score: str = "softmax",
         bias: Optional[torch.Tensor] = None, groups: int = 0, group_k: int = 0, group_best: int = 1,
         renorm: bool = True, scale: float = 1.0, want_logits: bool = False, out=None, stream=None):
    """Router projection of x [T, H] and the gate on its fp32 logits (options as
    in gate_from_logits): dict(idx, w[, logits]).  Refuses x and router_w that
    require grad in grad mode."""
    if not _here(x, stream):
        with _elsewhere(x, stream):
            return gate(x, router_w, k, score=score, bias=bias, groups=groups, group_k=group_k,
                        group_best=group_best, renorm=renorm, scale=scale, want_logits=want_logits, out=out)
    if x.requires_grad or router_w.requires_grad:
        _no_graph("gate")
    code = _dtype_code(x)
    if x.dim() != 2 or router_w.dim() != 2:
        raise ValueError("x and router_w must have two dimensions")
    (T, H), E = x.shape, router_w.shape[0]
    x = x.contiguous()
    dev = x.get_device()
    o = _gate_opts(dev, E, score, bias, groups, group_k, group_best, renorm, scale)
    pw = _operand(router_w, "router_w", dev, x.dtype, (E, H))
    idx, w = _routing_out(x, T, k, out)
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _check(lib().moe_gate(x.data_ptr(), code, T, H, pw, E, k, o, idx.data_ptr(), w.data_ptr(), logits.data_ptr(), None,
                          0, _current(dev)), "moe_gate")
    r = dict(idx=idx, w=w)
    if want_logits:
        r["logits"] = logits
    return r


def gate_backward(logits: torch.Tensor, idx: torch.Tensor, grad_w: torch.Tensor, *, score: str = "softmax",
                  renorm: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """The gradient [T, E] of the gate's weights with respect to the logits, in
    their type: idx [T, k] int32 as the gate returned it, grad_w [T, k] float32,
    score, renorm and scale as in the forward call (a bias and groups only
    select: they change nothing here).  The result has no graph of its own; `out`
    must not overlap the inputs."""
    if not _here(logits, stream):
        with _elsewhere(logits, stream):
            return gate_backward(logits, idx, grad_w, score=score, renorm=renorm, scale=scale, out=out)
    code = _gate_type(logits)
    logits, T, E, ld = _rows(logits, "logits")
    if idx.dim() != 2:
        raise ValueError("idx must have two dimensions")
    k = idx.shape[1]
    dev = logits.get_device()
    pi = _operand(idx, "idx", dev, torch.int32, (T, k))
    pg = _operand(grad_w, "grad_w", dev, torch.float32, (T, k))
    if out is None:
        g, ldg = _new(logits, T, E, logits.dtype), E
    else:
        g, ldg = out, _out_rows(out, "out", dev, logits.dtype, (T, E))
    o = _gate_opts(dev, E, score, None, 0, 0, 1, renorm, scale)
    _check(lib().moe_gate_backward(logits.data_ptr(), code, ld, T, E, k, o, pi, pg, g.data_ptr(), ldg, _current(dev)),
           "moe_gate_backward")
    return g


def layer_forward_gated(x: torch.Tensor, router_w: Optional[torch.Tensor], k: int, down: Weights,
                        gate_up: Optional[Weights] = None, gate: Optional[Weights] = None,
                        up: Optional[Weights] = None, flags: int = 0, taps: Optional[dict] = None,
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None, *,
                        logits: Optional[torch.Tensor] = None, score: str = "softmax",
                        bias: Optional[torch.Tensor] = None, groups: int = 0, group_k: int = 0, group_best: int = 1,
                        renorm: bool = True, scale: float = 1.0, capacity: int = 0) -> torch.Tensor:
    """layer_forward with the gate's routing (options as in gate_from_logits).
    logits [T, E] float32, with router_w None: the caller's router logits.
    Refuses x, router_w and logits that require grad in grad mode."""
    if not _here(x, stream):
        with _elsewhere(x, stream):
            return layer_forward_gated(x, router_w, k, down, gate_up, gate, up, flags, taps, out, workspace,
                                       logits=logits, score=score, bias=bias, groups=groups, group_k=group_k,
                                       group_best=group_best, renorm=renorm, scale=scale, capacity=capacity)
    if any(t is not None and t.requires_grad for t in (x, router_w, logits)):
        _no_graph("layer_forward_gated")
    code = _dtype_code(x)
    T, H = x.shape
    E = down.E
    dev = x.get_device()
    _operand(x, "x", dev, x.dtype, (T, H))
    pw = _operand(router_w, "router_w", dev, x.dtype, (E, H))
    pl = _operand(logits, "logits", dev, torch.float32, (T, E))
    o = _gate_opts(dev, E, score, bias, groups, group_k, group_best, renorm, scale, capacity)
    y = torch.empty_like(x) if out is None else out
    _operand(y, "out", dev, x.dtype, (T, H))
    need = layer_workspace_size(T, H, E, k, down.K, flags)
    ws = workspace
    if ws is None or ws.numel() < need:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    ctaps = None
    if taps:
        ctaps = CTaps(*[(taps[n].data_ptr() if n in taps and taps[n] is not None else None) for n in TAP_NAMES])
    ref = lambda w: w.c() if w is not None else None
    _check(lib().moe_layer_forward_gated(x.data_ptr(), code, T, H, pw, pl, E, k, o, ref(gate_up), ref(gate), ref(up),
                                         down.c(), y.data_ptr(), flags, ctaps, ws.data_ptr(), ws.numel(), _current(dev)),
           "moe_layer_forward_gated")
    return y


def lora_add(x: torch.Tensor, base: torch.Tensor, ids: torch.Tensor, a: torch.Tensor, b: torch.Tensor, *,
             scale: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """base [T, N] + scale[i] * (x [T, K] a[i]^T) b[i]^T with i = ids[t] (moe_lora):
    the low-rank adapters of many requests beside a projection they share, whose
    output `base` is (x's type, or float32: e.g. router logits).  a [L, R, K]
    and b [L, N, R] in x's type; ids [T] int32 in any order, outside [0, L) for a
    token without an adapter; scale [L] float32; ranks [L] int32, the ranks in
    use of adapters smaller than R.  out: written instead of a new tensor; pass
    base itself to add in place (otherwise it must not overlap base, nor ever x).
    Refuses inputs that require grad in grad mode."""
    if not _here(x, stream):
        with _elsewhere(x, stream):
            return lora_add(x, base, ids, a, b, scale=scale, ranks=ranks, out=out)
    if (x.requires_grad or base.requires_grad or a.requires_grad or b.requires_grad or
            (scale is not None and scale.requires_grad)):
        _no_graph("lora_add")
    dtype, odt = x.dtype, base.dtype
    code = _dtype_code(x)
    if odt is not dtype and odt is not torch.float32:
        raise TypeError("base must be %s or float32, got %s" % (dtype, odt))
    if a.dim() != 3 or b.dim() != 3 or base.dim() != 2:
        raise ValueError("a and b must have three dimensions, base two")
    x, T, K, ldx = _rows(x, "x")
    if ldx % 8 or x.data_ptr() % 16:
        x, ldx = x.clone(memory_format=torch.contiguous_format), K
    dev = x.get_device()
    (L, R, _), N = a.shape, base.shape[1]
    if base.shape[0] != T or base.get_device() != dev:
        raise ValueError("base must have a row for each of x, on its device")
    lora = CLora(_operand(a, "a", dev, dtype, (L, R, K)), _operand(b, "b", dev, dtype, (L, N, R)),
                 _operand(scale, "scale", dev, torch.float32, (L,)), _operand(ranks, "ranks", dev, torch.int32, (L,)),
                 L, R, K, N)
    pids = _operand(ids, "ids", dev, torch.int32, (T,))
    if out is None:
        base, _, _, ldb = _rows(base, "base")
        out, ldo = _new(base, T, N, odt), N
    else:
        ldo = _out_rows(out, "out", dev, odt, (T, N))
        if out is base:
            ldb = ldo
        else:
            base, _, _, ldb = _rows(base, "base")
    _check(lib().moe_lora_add(x.data_ptr(), code, ldx, T, lora, pids, base.data_ptr(), ldb, out.data_ptr(), ldo,
                              _TYPES[odt], _current(dev)), "moe_lora_add")
    return out


def expert_load_stats(counts: torch.Tensor, stream=None):
    """(least-used expert [1] int32, standard deviation [1] fp32) of int32 counts [E] on the device."""
    assert counts.dtype == torch.int32 and counts.dim() == 1 and counts.is_contiguous()
    lu = torch.empty(1, dtype=torch.int32, device=counts.device)
    sd = torch.empty(1, dtype=torch.float32, device=counts.device)
    _check(lib().moe_expert_load_stats(_ptr(counts), counts.numel(), _ptr(lu), _ptr(sd), _stream(stream)),
           "moe_expert_load_stats")
    return lu, sd


def fuse_gate_up(gate: Weights, up: Weights, stream=None) -> Weights:
    """Pack gate [E, I, K] and up [E, I, K] into a new fused [E, 2I, K] tensor."""
    E, I, K, bits = gate.E, gate.N, gate.K, gate.bits
    dev = gate.q.device
    qshape = (E, 2 * I) + tuple(gate.q.shape[2:])
    q = torch.empty(qshape, dtype=gate.q.dtype, device=dev)
    s = b = None
    if gate.scales is not None:
        sdt = torch.uint8 if gate.fmt == "nvfp4" else torch.float16
        s = torch.empty((E, 2 * I, K // gate.group_size), dtype=sdt, device=dev)
    if gate.biases is not None:
        b = torch.empty((E, 2 * I, K // gate.group_size), dtype=torch.float16, device=dev)
    cg, cu = gate.c(), up.c()
    st = lib().moe_fuse_gate_up(ctypes.byref(cg), ctypes.byref(cu), _ptr(q), _ptr(s), _ptr(b), _stream(stream))
    _check(st, "moe_fuse_gate_up")
    return Weights(q, s, b, E, 2 * I, K, bits, gate.group_size, fmt=gate.fmt, tensor_scale=gate.tensor_scale)


def pack_sb(w: Weights, stream=None) -> Weights:
    """The same weights with packed_sb filled (scales and biases in the batched
    path's layout; a one-time repack, like fusing gate and up)."""
    if w.bits == 16 or w.row_offset != 0:
        raise ValueError("pack_sb: needs a whole quantised tensor")
    stride = w.N if w.stride is None else w.stride
    nbytes = int(lib().moe_packed_sb_bytes(w.E, stride, w.K))
    out = torch.empty(nbytes, dtype=torch.uint8, device=w.q.device)
    _check(lib().moe_pack_sb(ctypes.byref(w.c()), _ptr(out), _stream(stream)), "moe_pack_sb")
    return dataclasses.replace(w, packed_sb=out, _cstruct=None)


def pack_q(w: Weights, stream=None) -> Weights:
    """The same weights with packed_q filled (the codes in the batched path's
    block layout; a one-time repack, a second copy of the codes)."""
    if w.row_offset != 0:
        raise ValueError("pack_q: needs a whole tensor")
    stride = w.N if w.stride is None else w.stride
    nbytes = int(lib().moe_packed_q_bytes(w.E, stride, w.K, w.bits))
    if nbytes == 0:
        raise ValueError("pack_q: rows per expert and N must be multiples of 32")
    out = torch.empty(nbytes, dtype=torch.uint8, device=w.q.device)
    _check(lib().moe_pack_q(ctypes.byref(w.c()), _ptr(out), _stream(stream)), "moe_pack_q")
    return dataclasses.replace(w, packed_q=out, _cstruct=None)


def debug_set_events(events: Optional[Sequence]) -> None:
    """Record the given torch.cuda.Events around each kernel of later calls on this thread."""
    if not events:
        lib().moe_debug_set_events(None, 0)
        debug_set_events._keep = None
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    debug_set_events._keep = arr  # keep the array alive while the library holds it
    lib().moe_debug_set_events(ctypes.cast(arr, ctypes.c_void_p), len(events))


def debug_set_tuning(key: int, value: int) -> None:
    """Launch-shape knob (0: decode gate+up waves/CU, 1: decode down waves/CU, 2: GEMM row tiles per group,
    3: GEMM row tile 32/64/128 (else automatic), 4: GEMM K groups per stage (1 or 2), 5: GEMM N subtiles
    per wave (2 or 4), 6: GEMM waves per column block (1 or 2), 7: GEMM workgroups per CU at 32/64-row
    tiles (1 or 2; 3 for 4-bit and NVFP4 weights at 64-row tiles), 8: decode gate+up waves per pair (2: from the wave target alone, else equal iterations
    per wave), 9: tokens per small-batch router workgroup at eight experts each (1, 2 or 4; default 2))."""
    lib().moe_debug_set_tuning(int(key), int(value))


STREAM_READ_WAVES = 8192


def debug_stream_read(src: torch.Tensor, sink: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The streaming-read reference over all of `src` (see moe_debug_stream_read);
    returns the int32 sink [STREAM_READ_WAVES] of per-wave XORs."""
    if sink is None:
        sink = torch.empty(STREAM_READ_WAVES, dtype=torch.int32, device=src.device)
    nbytes = src.numel() * src.element_size()
    _check(lib().moe_debug_stream_read(_ptr(src), nbytes, _ptr(sink), _stream(stream)), "moe_debug_stream_read")
    return sink


def source_hash() -> str:
    """sha256 over the library's sources (identifies which kernels a profile measured)."""
    import hashlib
    h = hashlib.sha256()
    csrc = os.path.join(_HERE, "csrc")
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name), "rb") as f:
            h.update(name.encode() + b"\0" + f.read())
    return h.hexdigest()[:16]


def last_plan() -> list:
    buf = ctypes.create_string_buffer(1024)
    lib().moe_debug_last_plan(buf, 1024)
    s = buf.value.decode()
    return s.split(",") if s else []
