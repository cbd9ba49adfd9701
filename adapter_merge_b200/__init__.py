"""Python binding of libadafuse.so (the AdaFuse fused gated multi-LoRA path on
B200).  Argument marshalling only (through ctypes; for the operators between
the adapted linears, which run once per layer and token, through the extension
module _binding): every step of the path runs in the CUDA kernels behind the C
ABI declared in include/adafuse.h.  PyTorch supplies device memory and streams.
There is no fallback: if the shared library is missing or fails to load,
importing the binding's entry points raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

__all__ = [
    "AdafuseError", "lib", "library_path", "pregate", "segments", "Plan", "PointerArrays",
    "RENORM", "POOL_MEAN", "STATUS_BAD_INDEX", "STATUS_TIMEOUT", "PLAN_Y_F32", "round_bf16",
    "project", "gated_project", "epilogue", "rotary", "rotary_frequencies",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libadafuse.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_WORKSPACE_TOO_SMALL = 3
ERR_CUDA = 4
ERR_TIMEOUT = 5
ERR_DEVICE = 6
RENORM = 1 << 0
POOL_MEAN = 1 << 1
STATUS_BAD_INDEX = 1 << 0
STATUS_TIMEOUT = 1 << 1
PLAN_Y_F32 = 1 << 0
PLAN_TEST_STALL = 1 << 31
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
OUT_F32 = 1 << 4
IN_F32 = 1 << 5
PAIRS = 1 << 6
POS_I32 = 1 << 7
TEST_STALL = 1 << 31

# Every entry point the header declares.
EXPORTS = (
    "adafuse_plan_create", "adafuse_plan_destroy", "adafuse_pregate", "adafuse_merge",
    "adafuse_switch", "adafuse_merge_per_linear", "adafuse_segments",
    "adafuse_apply_workspace_bytes", "adafuse_apply", "adafuse_plan_status",
    "adafuse_plan_last_launches", "adafuse_strerror", "adafuse_version",
    "adafuse_apply_noalloc", "adafuse_round_bf16", "adafuse_project", "adafuse_gated_project",
    "adafuse_epilogue", "adafuse_rotary",
)


class AdafuseError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = _lib.adafuse_strerror(code).decode() if _lib is not None else str(code)
        super().__init__(f"{where}: {msg} (code {code})")


class Linear(ctypes.Structure):
    _fields_ = [
        ("W", ctypes.c_void_p), ("W_out", ctypes.c_void_p),
        ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
        ("d_out", ctypes.c_int32), ("d_in", ctypes.c_int32),
        ("a_expert_stride", ctypes.c_int64), ("b_expert_stride", ctypes.c_int64),
    ]


class Heads(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("in_token_stride", ctypes.c_int64), ("in_head_stride", ctypes.c_int64),
        ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("heads", ctypes.c_int32),
    ]


_lib = None
_native = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libadafuse.so (built by adapter_merge_b200.build); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libadafuse.so not built ({_LIB_PATH}); run adapter_merge_b200.build.build()")
    L = ctypes.CDLL(_LIB_PATH)
    P, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
    L.adafuse_plan_create.argtypes = [ctypes.POINTER(P), ctypes.POINTER(Linear), i32, i32, i32, u32]
    L.adafuse_plan_destroy.argtypes = [P]
    L.adafuse_plan_destroy.restype = None
    L.adafuse_pregate.argtypes = [P, i64, i32, i64, P, P, i32, i32, u32, P, P, P]
    L.adafuse_merge.argtypes = [P, P, P, i32, P]
    L.adafuse_switch.argtypes = [P, P, P, P, P, i32, P]
    L.adafuse_merge_per_linear.argtypes = [P, P, P, i32, P]
    L.adafuse_segments.argtypes = [P, i64, i32, i32, P, P, P, P, P]
    L.adafuse_apply_workspace_bytes.argtypes = [P, i64, i32]
    L.adafuse_apply_workspace_bytes.restype = ctypes.c_size_t
    L.adafuse_apply.argtypes = [P, P, P, i64, P, P, i32, P, ctypes.c_size_t, P]
    L.adafuse_apply_noalloc.argtypes = [P, P, P, i64, P, P, i32, P]
    L.adafuse_round_bf16.argtypes = [P, P, i64, P]
    L.adafuse_project.argtypes = [P, i64, i32, i64, P, i32, i64, P, P, i64, P, i64, u32, P, P]
    L.adafuse_gated_project.argtypes = [P, i64, i32, i64, P, P, i32, i64, P, P, P, i64, u32, P, P]
    L.adafuse_epilogue.argtypes = [P, i64, i64, i64, P, P, i64, P, i64, P, i64, u32, P]
    L.adafuse_rotary.argtypes = [P, P, i64, i32, i32, P, P,
                                 ctypes.c_float, ctypes.c_float, u32, P]
    L.adafuse_plan_status.argtypes = [P, P, ctypes.POINTER(i32)]
    L.adafuse_plan_last_launches.argtypes = [P]
    L.adafuse_plan_last_launches.restype = i32
    L.adafuse_strerror.argtypes = [ctypes.c_int]
    L.adafuse_strerror.restype = ctypes.c_char_p
    L.adafuse_version.restype = i32
    for name in EXPORTS:
        getattr(L, name)
    _lib = L
    return L


def _check(rc: int, where: str):
    if rc != OK:
        raise AdafuseError(rc, where)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def pregate(x, W_r, k: int, b_r=None, renorm: bool = False, pool: bool = False,
            idx=None, gate=None, stream=None):
    """Token-level pre-gating: returns (idx int32 [T,k], gate fp32 [T,k]) on the
    device ([1,k] with pool=True).  x bf16 [T, H] (rows may be strided)."""
    import torch
    T, H = x.shape
    E = W_r.shape[0]
    rows = 1 if pool else T
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=x.device)
    if gate is None:
        gate = torch.empty((rows, k), dtype=torch.float32, device=x.device)
    flags = (RENORM if renorm else 0) | (POOL_MEAN if pool else 0)
    _check(lib().adafuse_pregate(_ptr(x), T, H, x.stride(0), _ptr(W_r), _ptr(b_r), E, k, flags,
                                 _ptr(idx), _ptr(gate), _stream(stream)), "adafuse_pregate")
    return idx, gate


def segments(idx, E: int, status=None, stream=None):
    """Stable segment build: (offsets [E+1], perm [T*k], used [E+1]) on the device."""
    import torch
    T, k = idx.shape
    offsets = torch.empty(E + 1, dtype=torch.int32, device=idx.device)
    perm = torch.full((T * k,), -1, dtype=torch.int32, device=idx.device)
    used = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    _check(lib().adafuse_segments(_ptr(idx), T, k, E, _ptr(offsets), _ptr(perm), _ptr(used),
                                  _ptr(status), _stream(stream)), "adafuse_segments")
    return offsets, perm, used


def round_bf16(src, out=None, stream=None):
    """bf16 round-to-nearest-even of an fp32 device tensor into `out` (a new
    bf16 tensor of src's shape if None); returns out."""
    import torch
    if src.dtype != torch.float32 or not src.is_contiguous():
        raise ValueError("round_bf16 takes a contiguous fp32 tensor")
    if out is None:
        out = torch.empty(src.shape, dtype=torch.bfloat16, device=src.device)
    if out.dtype != torch.bfloat16 or not out.is_contiguous() or out.numel() != src.numel():
        raise ValueError("round_bf16 writes a contiguous bf16 tensor of src's size")
    _check(lib().adafuse_round_bf16(_ptr(src), _ptr(out), src.numel(), _stream(stream)), "adafuse_round_bf16")
    return out


# ---------------------------------------------------------------- operators
# The operators between the adapted linears.  Each runs on its tensors' device
# and, unless `stream` is given, on that device's current stream; a result that
# the call allocates belongs to the stream it is computed on.  The arguments
# are checked and passed on by the extension module _binding: bad tensors raise
# ValueError, the library's error codes AdafuseError.  They have no backward
# pass: a tensor that requires grad is taken as its values, and no result has a
# gradient function.

def _operators():
    """The extension module, with the library's entry points installed."""
    global _native
    if _native is None:
        import importlib.util

        import torch  # noqa: F401  (its libraries, which the module links)

        from .build import binding_path
        L, path = lib(), binding_path()
        if not os.path.exists(path):
            raise RuntimeError(f"the operators' binding is not built for this Python and torch ({path}); run "
                               "adapter_merge_b200.build.build()")
        spec = importlib.util.spec_from_file_location(__name__ + "._binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.install(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.adafuse_project, L.adafuse_gated_project, L.adafuse_epilogue, L.adafuse_rotary)))
        _native = module
    return _native


def _activation(name) -> int:
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation {name!r} is none of {[a for a in ACTIVATIONS if a]}") from None


def _raw(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def project(x, W, bias=None, activation=None, residual=None, out=None, out_dtype=None, status=None, stream=None):
    """act(x W^T + bias) + residual in one launch, e.g. with a W_out that
    Plan.merge wrote: x bf16 [T, d_in], W bf16 [d_out, d_in], bias bf16 [d_out],
    residual bf16 [T, d_out] (rows may be strided or one expanded row; may be
    `out` itself).  activation: "relu", "silu", "gelu", "gelu_tanh" or None.
    Returns `out`, bf16 [T, d_out]; out_dtype=torch.float32 leaves the fp32
    result unrounded (a row-parallel rank's partial sums).  STATUS_TIMEOUT is
    OR-ed into `status` (int32 [1]) when a device-side wait gave up.  Forward
    only: gradients do not pass through the call."""
    r = (_native or _operators()).project(x, W, bias, _activation(activation), residual, out, out_dtype, status,
                                          _raw(stream))
    if r.__class__ is int:
        raise AdafuseError(r, "adafuse_project")
    return r if out is None else out


def gated_project(x, W_gate, W_up, bias_gate=None, bias_up=None, activation="silu", out=None, status=None,
                  stream=None):
    """act(x W_gate^T + bias_gate) * (x W_up^T + bias_up) in one launch: the
    feed-forward block's two projections, activation and product.  Weights bf16
    [d_out, d_in] with the same row stride; everything else as project.  Forward
    only: gradients do not pass through the call."""
    r = (_native or _operators()).gated_project(x, W_gate, W_up, bias_gate, bias_up, _activation(activation), out,
                                                status, _raw(stream))
    if r.__class__ is int:
        raise AdafuseError(r, "adafuse_gated_project")
    return r if out is None else out


def epilogue(y, bias=None, activation=None, up=None, residual=None, out=None, out_dtype=None, stream=None):
    """act(y + bias) * up + residual of outputs that exist already, in one
    launch, rounded once: silu(gate) * up of an unmerged apply, an apply's
    output plus the residual stream, or all-reduced fp32 sums.  y and up
    [T, n], both bf16 or both fp32; bias bf16 [n]; residual bf16 [T, n].  Rows
    may be strided, those of y, up and residual one expanded row.  Returns
    `out`, bf16 [T, n] (or fp32); it may be y, up or residual itself.  Forward
    only: gradients do not pass through the call."""
    r = (_native or _operators()).epilogue(y, bias, _activation(activation), up, residual, out, out_dtype,
                                           _raw(stream))
    if r.__class__ is int:
        raise AdafuseError(r, "adafuse_epilogue")
    return r if out is None else out


def rotary_frequencies(dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       original_length: int = 4096, fast_turns: float = 32.0, slow_turns: float = 1.0, device=None):
    """(freq fp64 [dim/2], value factor) for `rotary`: freq[i] = base^(-2i/dim)
    radians per position, scaled for contexts `factor` times as long:
      None          as they are
      "linear"      every frequency divided by the factor (positions squeezed)
      "base"        the base times factor^(dim / (dim - 2)): the slowest pair is
                    slowed by the factor, the fastest keeps its frequency
      "wavelength"  by the turns that a pair makes within original_length
                    positions: at least fast_turns keeps its frequency, at most
                    slow_turns is slowed by the factor, a linear ramp over the
                    pairs between, whose end may lie beyond the slowest pair
                    (and whose start is the first one at the earliest); rotated
                    values are scaled by 0.1 ln(factor) + 1 (Peng et al. 2023,
                    "YaRN").  Needs a base above 1."""
    import math

    import torch
    if dim < 2 or dim % 2:
        raise ValueError(f"dim {dim} is not a positive even number")
    if base <= 0 or factor <= 0:
        raise ValueError("base and factor are positive")
    i = torch.arange(0, dim, 2, dtype=torch.float64)
    if scaling == "base":
        if dim == 2:
            raise ValueError("scaling by the base needs more than one pair")
        base = base * factor ** (dim / (dim - 2))
    freq, mult = base ** (-i / dim), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "wavelength":
        if base <= 1 or original_length < 1 or not fast_turns > slow_turns > 0:
            raise ValueError("scaling by wavelength needs a base above 1, original_length >= 1 and "
                             "fast_turns > slow_turns > 0")
        pair = lambda turns: dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast_turns)), 0), math.ceil(pair(slow_turns))
        # hi <= 0: even the first pair makes at most slow_turns
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1) if hi > 0 else torch.ones_like(i)
        freq = freq / factor * ramp + freq * (1 - ramp)
        mult = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling {scaling!r} is none of None, 'linear', 'base', 'wavelength'")
    return freq.to(device) if device is not None else freq, mult


def rotary(q, k, positions, freq, layout: str = "half", factor: float = 1.0, q_weight=None, k_weight=None,
           eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Rotates queries and keys by their positions, after an RMS norm of each
    head where a weight is given, in one launch.  q bf16 [T, heads, D], k
    likewise (or None), any token and head strides; positions int64 or int32
    [T], any sign; freq fp64 [rot/2] (rotary_frequencies), rot <= D: the
    elements from rot on are not rotated.  layout "half" rotates elements i and
    i + rot/2, "interleaved" 2i and 2i + 1; `factor` scales the rotated
    elements.  q_weight / k_weight bf16 [D].  Returns (q_out, k_out), new
    contiguous tensors unless given; q_out may be q itself, k_out k.  Forward
    only: gradients do not pass through the call."""
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout {layout!r} is neither 'half' nor 'interleaved'")
    r = (_native or _operators()).rotary(q, k, positions, freq, 0 if layout == "half" else PAIRS, factor, q_weight,
                                         k_weight, eps, q_out, k_out, _raw(stream))
    if r.__class__ is int:
        raise AdafuseError(r, "adafuse_rotary")
    return r[0] if q_out is None else q_out, r[1] if k_out is None else k_out


class Plan:
    """A plan over a list of targeted linears sharing E rank-r adapters.

    `linears` is a sequence of (W, W_out, A, B) device tensors per linear:
    W, W_out bf16 [d_out, d_in]; A bf16 [E, r, d_in]; B bf16 [E, d_out, r]
    (any expert stride, row-major inside an expert).  The tensors must stay
    alive while the plan exists.  `flags`: PLAN_Y_F32 makes apply write fp32
    outputs (the row-parallel partials of tensor parallelism).
    """

    def __init__(self, linears: Sequence, E: int, r: int, flags: int = 0):
        arr = (Linear * len(linears))()
        for i, (W, W_out, A, B) in enumerate(linears):
            d_out, d_in = W.shape
            for t, inner in ((W, (d_in, 1)), (W_out, (d_in, 1)), (A, (d_in, 1)), (B, (r, 1))):
                if tuple(t.stride()[-2:]) != inner and t.shape[-2] > 1:
                    raise ValueError(f"linear {i}: tensors must be row-major inside each expert "
                                     f"(strides {tuple(t.stride())})")
            a_es = A.stride(0) if A.shape[0] > 1 else r * d_in
            b_es = B.stride(0) if B.shape[0] > 1 else d_out * r
            arr[i] = Linear(W.data_ptr(), W_out.data_ptr(), A.data_ptr(), B.data_ptr(),
                            d_out, d_in, a_es, b_es)
        self._keep = list(linears)
        self.E, self.r, self.n_lin = E, r, len(linears)
        h = ctypes.c_void_p()
        _check(lib().adafuse_plan_create(ctypes.byref(h), arr, len(linears), E, r, flags), "adafuse_plan_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def merge(self, idx, gate, k: Optional[int] = None, stream=None):
        k = idx.numel() if k is None else k
        _check(lib().adafuse_merge(self._h, _ptr(idx), _ptr(gate), k, _stream(stream)), "adafuse_merge")

    def switch(self, idx_new, gate_new, idx_old, gate_old, k: Optional[int] = None, stream=None):
        k = idx_new.numel() if k is None else k
        _check(lib().adafuse_switch(self._h, _ptr(idx_new), _ptr(gate_new), _ptr(idx_old), _ptr(gate_old), k,
                                    _stream(stream)), "adafuse_switch")

    def merge_per_linear(self, idx, gate, k: Optional[int] = None, stream=None):
        k = idx.numel() if k is None else k
        _check(lib().adafuse_merge_per_linear(self._h, _ptr(idx), _ptr(gate), k, _stream(stream)),
               "adafuse_merge_per_linear")

    def workspace_bytes(self, T: int, k: int) -> int:
        return int(lib().adafuse_apply_workspace_bytes(self._h, T, k))

    def apply(self, xs, ys, T: int, idx, gate, workspace, stream=None):
        """Segmented-gather apply over every linear.  xs / ys: per-linear device
        tensors (x_l [T, d_in], y_l [T, d_out]) or a PointerArrays built once
        from them (cheaper per call)."""
        k = idx.shape[1]
        ptrs = xs if isinstance(xs, PointerArrays) else PointerArrays(xs, ys)
        _check(lib().adafuse_apply(self._h, ptrs.x, ptrs.y, T, _ptr(idx), _ptr(gate), k,
                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "adafuse_apply")

    def apply_noalloc(self, xs, ys, T: int, idx, gate, stream=None) -> int:
        """As apply, with the library's own fixed device scratch instead of a
        workspace (for callers that cannot allocate device memory).  Returns the
        C return code (ADAFUSE_ERR_WORKSPACE_TOO_SMALL when the call does not
        fit the scratch) instead of raising, so callers can fall back to apply."""
        k = idx.shape[1]
        ptrs = xs if isinstance(xs, PointerArrays) else PointerArrays(xs, ys)
        return int(lib().adafuse_apply_noalloc(self._h, ptrs.x, ptrs.y, T, _ptr(idx), _ptr(gate), k,
                                               _stream(stream)))

    def status(self, stream=None):
        """(return code, device status bits); clears the status word."""
        v = ctypes.c_int32(0)
        rc = lib().adafuse_plan_status(self._h, _stream(stream), ctypes.byref(v))
        return rc, v.value

    @property
    def last_launches(self) -> int:
        return int(lib().adafuse_plan_last_launches(self._h))

    def destroy(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().adafuse_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class PointerArrays:
    """Host arrays of the device pointers of x_l and y_l, in linear order."""

    def __init__(self, xs, ys):
        addr = lambda t: t if isinstance(t, int) else t.data_ptr()
        self.x = (ctypes.c_void_p * len(xs))(*[addr(t) for t in xs])
        self.y = (ctypes.c_void_p * len(ys))(*[addr(t) for t in ys])
        self._keep = (list(xs), list(ys))
