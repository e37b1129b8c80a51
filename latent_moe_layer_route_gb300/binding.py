"""Thin binding of libklt.so, with the same names as the C ABI in include/klt.h.

Argument marshalling only: every step of the tail runs in the library's CUDA kernels.
PyTorch supplies device memory and the stream.  There is no fallback path: if the
library cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Dict, Optional

from .build import LIB_PATH, MARSHAL_PATH

KLT_OK = 0
KLT_ERR_INVALID_ARG = 1
KLT_ERR_UNSUPPORTED = 2
KLT_ERR_ALIGN = 3
KLT_ERR_CUDA = 4
KLT_ERR_DEVICE_TIMEOUT = 5
KLT_ERR_OOM = 6
KLT_ERR_TOO_LARGE = 7
KLT_NOALLOC_MAX_PAIRS = 65536
KLT_FMT_FP8_B128 = 0
KLT_FMT_NVFP4 = 1
KLT_FMT_MXFP8 = 2
KLT_FMT_NVFP4_W4A4 = 3
KLT_FLAG_NO_PDL = 1
KLT_FLAG_PHASED = 2
KLT_FLAG_DETERMINISTIC = 4
KLT_DT_BF16 = 0
KLT_DT_F32 = 1
KLT_DT_E4M3 = 2
KLT_ACT_NONE = 0
KLT_ACT_SWIGLU = 1
KLT_BLOCK_NORM_MAX_H = 16384
KLT_ROPE_HALVES = 0
KLT_ROPE_NEIGHBOURS = 1

EXPORTS = ("klt_create", "klt_forward", "klt_forward_hidden", "klt_status", "klt_destroy",
           "klt_strerror", "klt_launch_count", "klt_gemm_tile", "klt_route_noalloc",
           "klt_quantize", "klt_block_norm", "klt_linear_create", "klt_linear_forward",
           "klt_linear_tile", "klt_linear_status", "klt_linear_destroy", "klt_latent_create",
           "klt_latent_append", "klt_latent_workspace", "klt_latent_attend",
           "klt_latent_prefill", "klt_latent_status", "klt_latent_destroy")


class KltDims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("L", ctypes.c_int32), ("E", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("I", ctypes.c_int32), ("Is", ctypes.c_int32),
                ("routed_fmt", ctypes.c_int32), ("eps", ctypes.c_float),
                ("max_tokens", ctypes.c_int32)]


class KltWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w13", "w13_scale", "w13_global", "w2", "w2_scale", "w2_global", "ws13", "ws2",
        "w_up", "gamma", "w_lat", "w_gate")]


class KltRouting(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "ids", "weights", "cnt", "off", "gidx", "slot", "pos")]


class KltDebug(ctypes.Structure):
    _fields_ = [("zq", ctypes.c_void_p), ("zs", ctypes.c_void_p), ("aq", ctypes.c_void_p),
                ("as_", ctypes.c_void_p), ("r", ctypes.c_void_p), ("n", ctypes.c_void_p),
                ("a_s", ctypes.c_void_p), ("events", ctypes.c_void_p * 8),
                ("stall_after_kblocks", ctypes.c_int32), ("timeout_ms", ctypes.c_int32),
                ("trace", ctypes.c_void_p), ("trace_entries", ctypes.c_int32),
                ("force_bn", ctypes.c_int32), ("z", ctypes.c_void_p),
                ("logits", ctypes.c_void_p), ("zsx", ctypes.c_void_p)]


class KltBlockNormArgs(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("H", ctypes.c_int32), ("h_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32),
                ("gate_sigmoid", ctypes.c_int32), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("branch_scale", ctypes.c_float)] + [
        (n, ctypes.c_void_p) for n in ("h", "y", "gate", "gamma_post", "gamma_pre", "h_out",
                                       "n", "q", "s")] + [
        (n, ctypes.c_int64) for n in ("ld_h", "ld_y", "gate_row", "gate_col", "ld_h_out",
                                      "ld_n", "ld_q")]


class KltLinearDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("act", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class KltLinearDebug(ctypes.Structure):
    _fields_ = [("stall_after_kblocks", ctypes.c_int32), ("timeout_ms", ctypes.c_int32),
                ("force_tile", ctypes.c_int32), ("force_split", ctypes.c_int32)]


class KltLatentDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads", "latent", "rope", "nope", "value", "page",
                                              "pairs")] + [
        ("eps", ctypes.c_float), ("scale", ctypes.c_float)]


class KltLatentDebug(ctypes.Structure):
    _fields_ = [("stall_after_tiles", ctypes.c_int32), ("timeout_ms", ctypes.c_int32)]


class KltLatentAppendArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)] + [
        (n, ctypes.c_void_p) for n in ("kv", "positions", "slots", "cache", "kv_out", "q",
                                       "q_out")] + [
        (n, ctypes.c_int64) for n in ("pages", "ld_kv", "page_stride", "row_stride", "ld_kv_out",
                                      "q_token", "q_head", "q_out_token", "q_out_head")]


class KltLatentAttendArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "max_pages")] + [
        (n, ctypes.c_void_p) for n in ("q", "cache", "block_table", "seq_lens", "cu_q", "out",
                                       "lse", "workspace")] + [
        ("workspace_bytes", ctypes.c_uint64)] + [
        (n, ctypes.c_int64) for n in ("pages", "q_token", "q_head", "page_stride", "row_stride",
                                      "ld_table", "out_token", "out_head")]


class KltLatentPrefillArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "S", "causal")] + [
        (n, ctypes.c_void_p) for n in ("q", "k", "v", "k_rope", "cu_q", "cu_k", "out", "lse")] + [
        (n, ctypes.c_int64) for n in ("q_token", "q_head", "k_token", "k_head", "v_token",
                                      "v_head", "ld_k_rope", "out_token", "out_head")]


_LIB: Optional[ctypes.CDLL] = None
_LIB_FILE: Optional[str] = None
_marshal = None  # the CPython module of the operators around the tail, loaded by their first use


class KltError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libklt.so (built by ``build.build()``); raises if it is missing."""
    global _LIB, _LIB_FILE
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libklt.so not built at {path}; run "
                           "latent_moe_layer_route_gb300.build.build() first")
    lib = ctypes.CDLL(path)
    lib.klt_create.argtypes = [ctypes.POINTER(KltDims), ctypes.POINTER(KltWeights),
                               ctypes.c_uint32, ctypes.POINTER(ctypes.c_void_p)]
    lib.klt_create.restype = ctypes.c_int
    lib.klt_forward.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                ctypes.POINTER(KltRouting), ctypes.POINTER(KltDebug),
                                ctypes.c_void_p]
    lib.klt_forward.restype = ctypes.c_int
    lib.klt_forward_hidden.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.POINTER(KltRouting),
                                       ctypes.POINTER(KltDebug), ctypes.c_void_p]
    lib.klt_forward_hidden.restype = ctypes.c_int
    lib.klt_status.argtypes = [ctypes.c_void_p]
    lib.klt_status.restype = ctypes.c_int
    lib.klt_destroy.argtypes = [ctypes.c_void_p]
    lib.klt_destroy.restype = ctypes.c_int
    lib.klt_strerror.argtypes = [ctypes.c_int]
    lib.klt_strerror.restype = ctypes.c_char_p
    lib.klt_launch_count.argtypes = [ctypes.c_void_p, ctypes.c_int32]
    lib.klt_launch_count.restype = ctypes.c_int
    lib.klt_gemm_tile.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32]
    lib.klt_gemm_tile.restype = ctypes.c_int
    lib.klt_route_noalloc.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_int32] + [ctypes.c_void_p] * 8
    lib.klt_route_noalloc.restype = ctypes.c_int
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.klt_quantize.argtypes = [vp, i32, i64, i32, i32, vp, i64, vp, vp]
    lib.klt_quantize.restype = ctypes.c_int
    lib.klt_block_norm.argtypes = [ctypes.POINTER(KltBlockNormArgs), vp]
    lib.klt_block_norm.restype = ctypes.c_int
    lib.klt_linear_create.argtypes = [ctypes.POINTER(KltLinearDims), vp, vp,
                                      ctypes.POINTER(vp)]
    lib.klt_linear_create.restype = ctypes.c_int
    lib.klt_linear_forward.argtypes = [vp, vp, i64, vp, i32, vp, i64, vp,
                                       ctypes.POINTER(KltLinearDebug), vp]
    lib.klt_linear_forward.restype = ctypes.c_int
    lib.klt_linear_tile.argtypes = [vp, i32]
    lib.klt_linear_tile.restype = ctypes.c_int
    lib.klt_linear_status.argtypes = [vp]
    lib.klt_linear_status.restype = ctypes.c_int
    lib.klt_linear_destroy.argtypes = [vp]
    lib.klt_linear_destroy.restype = ctypes.c_int
    P = ctypes.POINTER
    lib.klt_latent_create.argtypes = [P(KltLatentDims), vp, vp, P(vp)]
    lib.klt_latent_append.argtypes = [vp, P(KltLatentAppendArgs), vp]
    lib.klt_latent_workspace.argtypes = [vp, i32, i32, P(ctypes.c_uint64)]
    lib.klt_latent_attend.argtypes = [vp, P(KltLatentAttendArgs), P(KltLatentDebug), vp]
    lib.klt_latent_prefill.argtypes = [vp, P(KltLatentPrefillArgs), P(KltLatentDebug), vp]
    lib.klt_latent_status.argtypes = [vp]
    lib.klt_latent_destroy.argtypes = [vp]
    for name in EXPORTS:
        if name.startswith("klt_latent_"):
            getattr(lib, name).restype = ctypes.c_int
    _LIB, _LIB_FILE = lib, os.path.realpath(path)
    return lib


def _load_marshal():
    """Load the module that the operators' calls go through.  It is linked to the libklt.so beside
    it, so it works with that copy of the library alone."""
    global _marshal
    load_library()
    if _LIB_FILE != os.path.realpath(LIB_PATH):
        raise RuntimeError(f"the operators work with {LIB_PATH} only; loaded is {_LIB_FILE}")
    if not os.path.exists(MARSHAL_PATH):
        raise RuntimeError(f"the operators' module is not built at {MARSHAL_PATH}; run "
                           "latent_moe_layer_route_gb300.build.build() first")
    import torch  # noqa: F401  (the module links to its libraries)

    from . import _marshal as marshal
    _marshal = marshal


def strerror(code: int) -> str:
    return load_library().klt_strerror(code).decode()


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _memory_of(stream: Optional[int], like):
    """Context in which torch allocates the outputs of a call on `stream` (a handle, or None for
    the current one): on the current stream's memory, work queued there may still be running."""
    if stream is None or not like.is_cuda:
        return contextlib.nullcontext()
    import torch
    if stream in (0, 1):  # the legacy default stream
        return torch.cuda.stream(torch.cuda.default_stream(like.device))
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device))


def dims_of(cfg, max_tokens: Optional[int] = None) -> KltDims:
    fmt = {"nvfp4": KLT_FMT_NVFP4, "mxfp8": KLT_FMT_MXFP8,
           "nvfp4_w4a4": KLT_FMT_NVFP4_W4A4}.get(cfg.routed_fmt, KLT_FMT_FP8_B128)
    return KltDims(cfg.H, cfg.L, cfg.E, cfg.topk, cfg.I, cfg.Is, fmt, cfg.eps,
                   cfg.M if max_tokens is None else max_tokens)


def weights_of(w: Dict) -> KltWeights:
    """Weight dict (CUDA tensors, names as produced by ``inputs.make_weights``, plus the
    optional ``w_lat``/``w_gate`` of ``inputs.make_projection_weights``)."""
    proj = (_ptr(w.get("w_lat")), _ptr(w.get("w_gate")))
    if "w13_sx" in w:  # MXFP8: UE8M0 scale bytes per 32 K-elements
        return KltWeights(_ptr(w["w13_q"]), _ptr(w["w13_sx"]), None, _ptr(w["w2_q"]),
                          _ptr(w["w2_sx"]), None, _ptr(w["ws13"]), _ptr(w["ws2"]),
                          _ptr(w["w_up"]), _ptr(w["gamma"]), *proj)
    if "w13_s" in w:
        return KltWeights(_ptr(w["w13_q"]), _ptr(w["w13_s"]), None, _ptr(w["w2_q"]),
                          _ptr(w["w2_s"]), None, _ptr(w["ws13"]), _ptr(w["ws2"]),
                          _ptr(w["w_up"]), _ptr(w["gamma"]), *proj)
    return KltWeights(_ptr(w["w13_q"]), _ptr(w["w13_sb"]), _ptr(w["w13_g"]), _ptr(w["w2_q"]),
                      _ptr(w["w2_sb"]), _ptr(w["w2_g"]), _ptr(w["ws13"]), _ptr(w["ws2"]),
                      _ptr(w["w_up"]), _ptr(w["gamma"]), *proj)


def klt_create(dims: KltDims, weights: KltWeights, flags: int = 0) -> ctypes.c_void_p:
    lib = load_library()
    h = ctypes.c_void_p()
    rc = lib.klt_create(ctypes.byref(dims), ctypes.byref(weights), flags, ctypes.byref(h))
    if rc != KLT_OK:
        raise KltError(rc, "klt_create")
    return h


def klt_forward(h, x, z, logits, M: int, out, routing: Optional[KltRouting] = None,
                debug: Optional[KltDebug] = None, stream: Optional[int] = None) -> int:
    lib = load_library()
    return lib.klt_forward(h, _ptr(x), _ptr(z), _ptr(logits), M, _ptr(out),
                           ctypes.byref(routing) if routing is not None else None,
                           ctypes.byref(debug) if debug is not None else None,
                           stream)


def klt_forward_hidden(h, x, M: int, out, routing: Optional[KltRouting] = None,
                       debug: Optional[KltDebug] = None, stream: Optional[int] = None) -> int:
    lib = load_library()
    return lib.klt_forward_hidden(h, _ptr(x), M, _ptr(out),
                                  ctypes.byref(routing) if routing is not None else None,
                                  ctypes.byref(debug) if debug is not None else None, stream)


def klt_status(h) -> int:
    return load_library().klt_status(h)


def klt_destroy(h) -> int:
    return load_library().klt_destroy(h)


def klt_launch_count(h, M: int) -> int:
    return load_library().klt_launch_count(h, M)


def klt_gemm_tile(h, M: int, force_bn: int = 0) -> int:
    return load_library().klt_gemm_tile(h, M, force_bn)


def klt_route_noalloc(logits, topk: int, ids, weights, cnt, off, gidx, slot, pos,
                      stream: Optional[int] = None) -> int:
    """Routing + permutation with no device allocation (fixed internal scratch); tensors
    are caller-owned CUDA tensors with the klt_routing layouts."""
    M, E = logits.shape
    return load_library().klt_route_noalloc(
        _ptr(logits), M, E, topk, _ptr(ids), _ptr(weights), _ptr(cnt), _ptr(off), _ptr(gidx),
        _ptr(slot), _ptr(pos), stream)


class LatentMoETail:
    """One tail layer on the current CUDA device (owns a klt handle)."""

    def __init__(self, cfg, weights: Dict, max_tokens: Optional[int] = None, flags: int = 0):
        self.cfg = cfg
        self.max_tokens = cfg.M if max_tokens is None else max_tokens
        self.handle = klt_create(dims_of(cfg, self.max_tokens), weights_of(weights), flags)

    def forward(self, x, z, logits, out=None, routing: Optional[KltRouting] = None,
                debug: Optional[KltDebug] = None, stream=None):
        import torch
        M = x.shape[0]
        if out is None:
            with _memory_of(stream, x):
                out = torch.empty((M, self.cfg.H), dtype=torch.bfloat16, device=x.device)
        if stream is None:
            stream = torch.cuda.current_stream(x.device).cuda_stream
        rc = klt_forward(self.handle, x, z, logits, M, out, routing, debug, stream)
        if rc != KLT_OK:
            raise KltError(rc, "klt_forward")
        return out

    __call__ = forward

    def forward_hidden(self, x, out=None, routing: Optional[KltRouting] = None,
                       debug: Optional[KltDebug] = None, stream=None):
        """The step before the tail (latent input and router logits from x), then the
        tail; the handle must have been created with ``w_lat`` and ``w_gate``."""
        import torch
        M = x.shape[0]
        if out is None:
            with _memory_of(stream, x):
                out = torch.empty((M, self.cfg.H), dtype=torch.bfloat16, device=x.device)
        if stream is None:
            stream = torch.cuda.current_stream(x.device).cuda_stream
        rc = klt_forward_hidden(self.handle, x, M, out, routing, debug, stream)
        if rc != KLT_OK:
            raise KltError(rc, "klt_forward_hidden")
        return out

    def status(self) -> int:
        return klt_status(self.handle)

    def launch_count(self, M: int) -> int:
        return klt_launch_count(self.handle, M)

    def gemm_tile(self, M: int, force_bn: int = 0) -> int:
        """256 for the token-major engine, else the feature-major engine's token tile."""
        return klt_gemm_tile(self.handle, M, force_bn)

    def close(self):
        if self.handle is not None and self.handle.value:
            klt_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- operators around the tail
#
# The checks that C cannot make of bare pointers (types, shapes, devices) and the calls are in
# the _marshal module; what is here allocates what the caller did not give.  `stream` is a
# stream's handle, or None for torch's current stream; outputs that a call allocates belong to the
# stream it runs on, and inputs given from another stream's memory must outlive the call's work.

def fp8_codes(M: int, K: int, device):
    """An uninitialised e4m3 tensor [M, K] whose rows start on 16 bytes, as the linear layer
    reads and the quantiser and the norms may write it."""
    import torch
    wide = torch.empty((M, -(-K // 16) * 16), dtype=torch.float8_e4m3fn, device=device)
    return wide[:, :K]


def quantize_fp8(x, q=None, s=None, stream: Optional[int] = None):
    """e4m3 codes q [M, K] and fp32 scales s [M, ceil(K/128)] of x [M, K] (bf16 or fp32; rows
    may be strided) per row and 128 columns (klt_quantize)."""
    if _marshal is None:
        _load_marshal()
    if q is None or s is None:
        import torch
        if x.dim() != 2:
            raise ValueError("x: not a matrix")
        M, K = x.shape
        with _memory_of(stream, x):
            if q is None:
                q = fp8_codes(M, K, x.device)
            if s is None:
                s = torch.empty((M, -(-K // 128)), dtype=torch.float32, device=x.device)
    rc = _marshal.quantize(x, q, s, stream)
    if rc:
        raise KltError(rc, "klt_quantize")
    return q, s


class BlockNorm:
    """The norms before and after a block with its gate and residual scale (klt_block_norm).

    gamma_post, gamma_pre: bf16 [H] or None (that norm is left out).  The object keeps the
    weights and scales; it has no other state.  New weights are copied into the tensors it was
    given, or go into a new object."""

    def __init__(self, H: int, gamma_post=None, gamma_pre=None, eps: float = 1e-6,
                 res_scale: float = 1.0, branch_scale: float = 1.0,
                 gate_sigmoid: bool = False):
        import torch
        if _marshal is None:
            _load_marshal()
        if not 1 <= H <= KLT_BLOCK_NORM_MAX_H:  # here: ctypes would cut it to 32 bits
            raise KltError(KLT_ERR_INVALID_ARG if H < 1 else KLT_ERR_UNSUPPORTED, "BlockNorm")
        self._H, self._gamma_post, self._gamma_pre = H, gamma_post, gamma_pre
        self._device = -1
        for name, g in (("gamma_post", gamma_post), ("gamma_pre", gamma_pre)):
            if g is None:
                continue
            if g.dtype != torch.bfloat16 or tuple(g.shape) != (H,) or not g.is_contiguous() \
                    or not g.is_cuda:
                raise ValueError(f"{name}: not a contiguous bf16 CUDA vector of {H}")
            if self._device >= 0 and g.get_device() != self._device:
                raise ValueError("gamma_post and gamma_pre are on different devices")
            self._device = g.get_device()
        self._args = KltBlockNormArgs(H=H, gate_sigmoid=int(gate_sigmoid), eps=eps,
                                      res_scale=res_scale, branch_scale=branch_scale,
                                      gamma_post=_ptr(gamma_post), gamma_pre=_ptr(gamma_pre))
        self._address = ctypes.addressof(self._args)

    # read-only: the calls read the weights at the addresses in _args
    H = property(lambda self: self._H)
    gamma_post = property(lambda self: self._gamma_post)
    gamma_pre = property(lambda self: self._gamma_pre)

    def forward(self, h, y=None, gate=None, *, h_out=None, n=None, q=None, s=None,
                stream: Optional[int] = None):
        """h [M, H] bf16/fp32 residual stream, y [M, H] bf16/fp32 block output or None, gate
        broadcastable to [M, H] or None.  Writes the outputs that are given: h_out (h's
        dtype; may be h), n (bf16; may be y), q and s (e4m3 codes and fp32 scales of n);
        when none is given, h_out (with y) and n are allocated.  Without y the norm after
        the block is skipped.  Returns (h_out, n, q, s)."""
        if h_out is None and n is None and q is None and s is None:
            import torch
            with _memory_of(stream, h):
                if y is not None:
                    h_out = torch.empty((h.shape[0], self.H), dtype=h.dtype, device=h.device)
                n = torch.empty((h.shape[0], self.H), dtype=torch.bfloat16, device=h.device)
        rc = _marshal.block_norm(self._address, self._device, h, y, gate, h_out, n, q, s, stream)
        if rc:
            raise KltError(rc, "klt_block_norm")
        return h_out, n, q, s

    __call__ = forward


class Fp8Linear:
    """y = x W^T with e4m3 weights and a scale per 128 x 128 block (klt_linear_*); owns a
    handle with its own copy of the weights, on the weights' device.  Threads may share it, but
    close() must not overlap a call.

    w_q: e4m3 (or uint8 codes) [N, K]; w_s: fp32 [ceil(N/128), ceil(K/128)].  act "none" or
    "swiglu" (gate rows first; N/2 outputs); out "bf16", "f32" or, for SwiGLU, "fp8"."""

    def __init__(self, w_q, w_s, act: str = "none", out: str = "bf16"):
        import torch
        self.handle = None
        if _marshal is None:
            _load_marshal()
        self._lib = _LIB
        acts = {"none": KLT_ACT_NONE, "swiglu": KLT_ACT_SWIGLU}
        outs = {"bf16": KLT_DT_BF16, "f32": KLT_DT_F32, "fp8": KLT_DT_E4M3}
        if act not in acts or out not in outs:
            raise ValueError(f"act {act!r}, out {out!r}: not known")
        if w_q.dim() != 2 or w_q.dtype not in (torch.float8_e4m3fn, torch.uint8) or \
                not w_q.is_cuda or not w_q.is_contiguous():
            raise ValueError("w_q: not a contiguous CUDA matrix of e4m3 codes")
        self.device = w_q.get_device()
        self.N, self.K = w_q.shape
        blocks = (-(-self.N // 128), -(-self.K // 128))
        if tuple(w_s.shape) != blocks or w_s.dtype != torch.float32 or \
                w_s.get_device() != self.device or not w_s.is_contiguous():
            raise ValueError(f"w_s: not a contiguous fp32 matrix {blocks} on the weights' device")
        self.width = self.N // 2 if act == "swiglu" else self.N
        self.fp8 = out == "fp8"
        self._dtype = outs[out]
        self._torch_dtype = torch.float32 if out == "f32" else torch.bfloat16
        if max(self.N, self.K) > 0x7FFFFFFF:  # ctypes would cut it to 32 bits
            raise KltError(KLT_ERR_UNSUPPORTED, "klt_linear_create")
        d = KltLinearDims(self.N, self.K, acts[act], outs[out])
        h = ctypes.c_void_p()
        # the create copies on the legacy default stream; what wrote the weights may have run
        # on another
        torch.cuda.current_stream(self.device).synchronize()
        with torch.cuda.device(self.device):
            rc = self._lib.klt_linear_create(ctypes.byref(d), w_q.data_ptr(), w_s.data_ptr(),
                                             ctypes.byref(h))
        if rc != KLT_OK:
            raise KltError(rc, "klt_linear_create")
        self.handle = h
        self._address = h.value

    def forward(self, xq, xs, out=None, out_s=None, stream: Optional[int] = None,
                debug: Optional[KltLinearDebug] = None):
        """xq e4m3 (or uint8) [M, K] whose rows start on 16 bytes, xs fp32 [M, ceil(K/128)].
        Returns out [M, N] (SwiGLU: [M, N/2]), or (codes, scales) with out "fp8"."""
        if out is None or (self.fp8 and out_s is None):
            import torch
            M = xq.shape[0]
            with _memory_of(stream, xq):
                if out is None:
                    out = fp8_codes(M, self.width, xq.device) if self.fp8 else \
                        torch.empty((M, self.width), dtype=self._torch_dtype, device=xq.device)
                if self.fp8 and out_s is None:
                    out_s = torch.empty((M, self.width // 128), dtype=torch.float32,
                                        device=xq.device)
        rc = _marshal.linear(self._address, self.device, self.K, self.width, self._dtype, xq, xs,
                             out, out_s, 0 if debug is None else ctypes.addressof(debug), stream)
        if rc:
            raise KltError(rc, "klt_linear_forward")
        return (out, out_s) if self.fp8 else out

    __call__ = forward

    def tile(self, M: int) -> int:
        """Token tile plus 1000 times the K split that a call with M tokens uses."""
        return self._lib.klt_linear_tile(self.handle, M)

    def status(self) -> int:
        return self._lib.klt_linear_status(self.handle)

    def close(self):
        if self.handle is not None and self.handle.value:
            self._lib.klt_linear_destroy(self.handle)
        self.handle, self._address = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class LatentAttention:
    """Latent attention of one layer (klt_latent_*): the step that fills the paged cache of latent
    rows, attention over it in absorbed form, and attention in expanded form.  Owns a handle with
    its own copy of inv_freq and gamma, on inv_freq's device.  Threads may share it, but close()
    must not overlap a call, and graphs captured from its calls need it while they are replayed.
    Forward only: results carry no gradient.

    inv_freq: fp32 [rope / 2], the angle of pair i at position p is p * inv_freq[i]; gamma: bf16
    [latent] or None; scale: of the scores, None for 1 / sqrt(nope + rope); pairs "halves" (element
    i turns with i + rope / 2) or "neighbours" (2 i with 2 i + 1).  A cache is bf16
    [pages, page, latent + rope]."""

    def __init__(self, heads: int, latent: int = 512, rope: int = 64, nope: int = 128,
                 value: int = 128, page: int = 64, *, inv_freq, gamma=None,
                 scale: Optional[float] = None, eps: float = 1e-6, pairs: str = "halves"):
        import torch
        self.handle = None
        if _marshal is None:
            _load_marshal()
        self._lib = _LIB
        kinds = {"halves": KLT_ROPE_HALVES, "neighbours": KLT_ROPE_NEIGHBOURS}
        if pairs not in kinds:
            raise ValueError(f"pairs {pairs!r}: not known")
        sizes = (heads, latent, rope, nope, value, page)
        if not all(0 <= v <= 0x7FFFFFFF for v in sizes):  # ctypes would cut it to 32 bits
            raise KltError(KLT_ERR_INVALID_ARG, "klt_latent_create")
        for name, t, n, dtype in (("inv_freq", inv_freq, rope // 2, torch.float32),
                                  ("gamma", gamma, latent, torch.bfloat16)):
            if t is None and name == "gamma":
                continue
            if t.dtype != dtype or tuple(t.shape) != (n,) or not t.is_cuda or \
                    not t.is_contiguous():
                raise ValueError(f"{name}: not a contiguous CUDA vector of {n}, {dtype}")
        self.device = inv_freq.get_device()
        if gamma is not None and gamma.get_device() != self.device:
            raise ValueError("inv_freq and gamma are on different devices")
        if scale is None:
            scale = max(nope + rope, 1) ** -0.5
        self.dims = KltLatentDims(*sizes, kinds[pairs], eps, scale)
        h = ctypes.c_void_p()
        # the create copies on the legacy default stream; what wrote the vectors may have run on
        # another
        torch.cuda.current_stream(self.device).synchronize()
        with torch.cuda.device(self.device):
            rc = self._lib.klt_latent_create(ctypes.byref(self.dims), _ptr(inv_freq), _ptr(gamma),
                                             ctypes.byref(h))
        if rc != KLT_OK:
            raise KltError(rc, "klt_latent_create")
        self.handle = h
        self._address, self._dims = h.value, ctypes.addressof(self.dims)

    def append(self, kv, positions, slots=None, cache=None, *, kv_out=None, q=None, q_out=None,
               stream: Optional[int] = None):
        """Rows kv [T, latent + rope] (bf16 or fp32) of tokens at `positions` (int64 [T]), normed
        and rotated, into `slots` (int64 [T]; outside of the cache: not stored) of the cache
        and/or into kv_out (bf16 [T, latent + rope]); q [T, heads, rope] (bf16) rotated into q_out
        (may be q).  Allocates q_out when q is given without it, and kv_out when there is no cache.
        Returns (kv_out, q_out)."""
        if (kv_out is None and cache is None) or (q is not None and q_out is None):
            import torch
            with _memory_of(stream, kv):
                if kv_out is None and cache is None:
                    kv_out = torch.empty(kv.shape, dtype=torch.bfloat16, device=kv.device)
                if q is not None and q_out is None:
                    q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        rc = _marshal.latent_append(self._address, self._dims, self.device, kv, positions, slots,
                                    cache, kv_out, q, q_out, stream)
        if rc:
            raise KltError(rc, "klt_latent_append")
        return kv_out, q_out

    def workspace(self, B: int, T: Optional[int] = None):
        """A workspace for attend() calls of B sequences and T queries (None: B), uint8.  Calls
        that may overlap need one each, and so do two captured graphs that may run at once."""
        import torch
        n = self._workspace_bytes(B, B if T is None else T)
        return torch.empty(n, dtype=torch.uint8, device=f"cuda:{self.device}")

    def _workspace_bytes(self, B: int, T: int) -> int:
        n = ctypes.c_uint64()
        if not (0 <= B <= 0x7FFFFFFF and 0 <= T <= 0x7FFFFFFF):
            raise KltError(KLT_ERR_INVALID_ARG, "klt_latent_workspace")
        rc = self._lib.klt_latent_workspace(self.handle, B, T, ctypes.byref(n))
        if rc:
            raise KltError(rc, "klt_latent_workspace")
        return n.value

    def attend(self, q, cache, block_table, seq_lens, cu_q=None, *, out=None, lse=None,
               workspace=None, stream: Optional[int] = None,
               debug: Optional[KltLatentDebug] = None):
        """q bf16 [T, heads, latent + rope] over the cache; block_table int32 [B, max_pages],
        seq_lens int32 [B] (the queries' own tokens counted), cu_q int32 [B + 1] or None for one
        query a sequence.  Returns out bf16 [T, heads, latent] and lse fp32 [T, heads]; what is
        allocated here is zeros and minus infinity outside of cu_q's ranges, so with cu_q it is
        filled on every call (prefill() says what that costs)."""
        if out is None or lse is None or workspace is None:
            import torch
            T = q.shape[0]
            with _memory_of(stream, q):
                shape = (T, self.dims.heads, self.dims.latent)
                if out is None:
                    out = torch.empty(shape, dtype=torch.bfloat16, device=q.device) \
                        if cu_q is None else \
                        torch.zeros(shape, dtype=torch.bfloat16, device=q.device)
                if lse is None:
                    lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device) \
                        if cu_q is None else \
                        torch.full(shape[:2], -float("inf"), dtype=torch.float32, device=q.device)
                if workspace is None:
                    workspace = torch.empty(self._workspace_bytes(seq_lens.shape[0], T),
                                            dtype=torch.uint8, device=q.device)
        rc = _marshal.latent_attend(self._address, self._dims, self.device, q, cache, block_table,
                                    seq_lens, cu_q, out, lse, workspace,
                                    0 if debug is None else ctypes.addressof(debug), stream)
        if rc:
            raise KltError(rc, "klt_latent_attend")
        return out, lse

    def prefill(self, q, k, v, k_rope, cu_q, cu_k, *, causal: bool = True, out=None, lse=None,
                stream: Optional[int] = None, debug: Optional[KltLatentDebug] = None):
        """q bf16 [T, heads, nope + rope], k bf16 [S, heads, nope], v bf16 [S, heads, value], k_rope
        bf16 [S, rope], cu_q and cu_k int32 [B + 1].  Returns out bf16 [T, heads, value] and lse
        fp32 [T, heads]; what is allocated here is zeros and minus infinity outside of cu_q's
        ranges: filled on every call (27 us of host time, 30 us of the GPU's at 8192 tokens of 64
        heads), so a loop passes out and lse of its own."""
        if out is None or lse is None:
            import torch
            shape = (q.shape[0], self.dims.heads, self.dims.value)
            with _memory_of(stream, q):
                if out is None:
                    out = torch.zeros(shape, dtype=torch.bfloat16, device=q.device)
                if lse is None:
                    lse = torch.full(shape[:2], -float("inf"), dtype=torch.float32,
                                     device=q.device)
        rc = _marshal.latent_prefill(self._address, self._dims, self.device, q, k, v, k_rope, cu_q,
                                     cu_k, bool(causal), out, lse,
                                     0 if debug is None else ctypes.addressof(debug), stream)
        if rc:
            raise KltError(rc, "klt_latent_prefill")
        return out, lse

    def status(self) -> int:
        return self._lib.klt_latent_status(self.handle)

    def close(self):
        if self.handle is not None and self.handle.value:
            self._lib.klt_latent_destroy(self.handle)
        self.handle, self._address = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
