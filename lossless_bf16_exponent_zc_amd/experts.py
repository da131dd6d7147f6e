"""Binding of the expert operators (the C ABI in include/zc_experts.h).

Around the compressed all-to-all: ``ExpertPlan`` sorts tokens by expert
(route, dispatch, dispatch_fp8), brings rows back with the router's weights
(combine) and takes the gradients of both (combine_backward; the gradient of
dispatch is combine without weights).  ``quantize_rows`` / ``_weights`` /
``_columns`` cast to 8-bit blocks of 128; ``expert_product`` and
``expert_weight_grad`` multiply such blocks, expert by expert.

Argument marshalling and checks only, as in ``binding``: every buffer is the
caller's, every call enqueues on the current (or the given) stream.  The
kernels of small calls take less time than checking a call's tensors from
Python would, so the calls are made by the module ``zc_experts_binding``
(csrc/zc_experts_binding.cpp), built with the library; there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import ZC_ERR_INVALID_ARG, ZC_ERR_UNSUPPORTED, ZcError

# Every symbol include/zc_experts.h declares.
EXPERT_EXPORTS = (
    "zc_route_rows", "zc_route_workspace_bytes", "zc_route", "zc_dispatch", "zc_dispatch_fp8",
    "zc_combine", "zc_combine_backward", "zc_quantize_rows", "zc_quantize_weights",
    "zc_quantize_columns", "zc_expert_product", "zc_expert_weight_grad",
    "zc_expert_weight_grad_workspace_bytes",
)

BLOCK = 128  # values per scale
_FP8, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu

_lib = None


class _Calls:
    """The binding module's functions as attributes, set on the first use."""

    def __getattr__(self, name):
        lib()
        return object.__getattribute__(self, name)


_zc = _Calls()


def lib() -> ctypes.CDLL:
    """libzc.so with the expert operators' signatures set."""
    global _lib
    if _lib is not None:
        return _lib
    L = binding.lib()
    vp, u32, u64, i = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int
    args = {
        "zc_route_rows": [u64, u32, u32, u32],
        "zc_route_workspace_bytes": [u64, u32, u32],
        "zc_route": [vp, u64, u32, u32, u32, vp, vp, vp, vp, u64, vp, u64, vp],
        "zc_dispatch": [vp, u64, u32, u64, u32, u32, u32, vp, vp, vp, vp, u64, u64, vp],
        "zc_dispatch_fp8": [vp, u64, u32, u64, u32, u32, u32, vp, vp, vp, vp, vp, u64, vp],
        "zc_combine": [vp, u64, vp, u32, u64, u32, u32, vp, u64, vp, u64, vp],
        "zc_combine_backward": [vp, u64, vp, u64, vp, u32, u64, u32, u32, u32, vp, vp, vp, u64, vp, u64, vp, vp],
        "zc_quantize_rows": [vp, u64, u32, u64, u32, vp, vp, vp, vp],
        "zc_quantize_weights": [vp, u32, u32, u32, u32, i, vp, vp, vp],
        "zc_quantize_columns": [vp, u64, u32, u64, u32, vp, vp, vp, vp],
        "zc_expert_product": [vp, vp, u64, vp, vp, u32, u32, u32, vp, vp, vp, u64, u32, vp],
        "zc_expert_weight_grad": [vp, vp, vp, vp, u64, u32, u32, u32, vp, vp, u32, vp, u64, vp],
        "zc_expert_weight_grad_workspace_bytes": [u64, u32, u32, u32],
    }
    for name in EXPERT_EXPORTS:
        f = getattr(L, name)
        f.argtypes = args[name]
        f.restype = u64 if name.endswith(("_rows", "_bytes")) and not name.startswith("zc_quantize") else i
    try:
        from . import zc_experts_binding as calls
    except ImportError as e:
        raise ImportError(f"{e}: build the package with `python -c 'import __graft_entry__ as g; g.build()'`") from e
    calls.bind(ZcError, {name: ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in EXPERT_EXPORTS})
    for name in ("route", "dispatch", "dispatch_fp8", "combine", "combine_backward", "quantize_rows", "quantize_weights",
                 "quantize_columns", "expert_product", "expert_weight_grad"):
        setattr(_zc, name, getattr(calls, name))
    _lib = L
    return L


def _bad(what: str, why: str, code: int = ZC_ERR_INVALID_ARG):
    raise ZcError(code, f"{what}: {why}")


def _up(n: int, m: int) -> int:
    return -(-n // m) * m


class Fp8Blocks(NamedTuple):
    """A matrix (or one per expert) in 8-bit blocks of 128: ``data`` E4M3
    [..., rows, up(cols, 128)], ``scale`` E8M0 [..., scale rows,
    up(ceil(cols / 128), 4)], ``cols`` the columns that hold values."""
    data: torch.Tensor
    scale: torch.Tensor
    cols: int

    def float(self, rows_per_scale: int = 1) -> torch.Tensor:
        """The values the blocks stand for, in 32 bits (128 rows per scale
        for weights)."""
        s = self.scale.float()[..., :self.data.shape[-1] // BLOCK]
        if rows_per_scale > 1:
            s = s.repeat_interleave(rows_per_scale, -2)[..., :self.data.shape[-2], :]
        v = self.data.float().unflatten(-1, (-1, BLOCK)) * s[..., None]
        return v.flatten(-2)[..., :self.cols]


def _empty_blocks(lead, scale_lead, cols: int, device) -> Fp8Blocks:
    return Fp8Blocks(torch.zeros(*lead, _up(cols, BLOCK), dtype=_FP8, device=device),
                     torch.zeros(*scale_lead, _up(-(-cols // BLOCK), 4), dtype=torch.uint8,
                                 device=device).view(_E8M0), cols)


def empty_fp8_rows(rows: int, cols: int, device="cuda") -> Fp8Blocks:
    """A blocked [rows, cols] for quantize_rows and dispatch_fp8 (1 x 128)."""
    return _empty_blocks((rows,), (rows,), cols, device)


def empty_fp8_weights(experts: int, n: int, k: int, device="cuda") -> Fp8Blocks:
    """A blocked [experts, n, k] for quantize_weights (128 x 128)."""
    return _empty_blocks((experts, n), (experts, -(-n // BLOCK)), k, device)


class Fp8Columns(NamedTuple):
    """A [rows, cols] matrix in 8-bit blocks of 128 rows of a column: ``data``
    E4M3 [ceil(rows / 128), cols, 128], ``scale`` E8M0 [ceil(rows / 128),
    up(cols, 4)]."""
    data: torch.Tensor
    scale: torch.Tensor
    rows: int
    cols: int

    def float(self) -> torch.Tensor:
        """The values the blocks stand for, in 32 bits, as [rows, cols]."""
        v = self.data.float() * self.scale.float()[:, :self.cols, None]
        return v.transpose(1, 2).flatten(0, 1)[:self.rows]


def empty_fp8_columns(rows: int, cols: int, device="cuda") -> Fp8Columns:
    """Storage for quantize_columns of a [rows, cols] matrix."""
    blocks = -(-rows // BLOCK)
    return Fp8Columns(torch.zeros(blocks, cols, BLOCK, dtype=_FP8, device=device),
                      torch.zeros(blocks, _up(cols, 4), dtype=torch.uint8, device=device).view(_E8M0), rows, cols)


class Routing(NamedTuple):
    """Where slots go: ``offsets`` [experts + 1] (first row of each expert's
    segment, and the end), ``counts`` [experts], ``row`` [tokens, topk] (-1
    without a row), ``slot`` [rows] (-1 for a padding row); int32."""
    offsets: torch.Tensor
    counts: torch.Tensor
    row: torch.Tensor
    slot: torch.Tensor


class ExpertPlan:
    """Sizes of one routing: tokens, choices per token, experts, and the
    multiple that segments begin at (1 packs them, as a codec ``Plan`` with
    one segment per expert wants them; ``expert_weight_grad`` wants 128)."""

    def __init__(self, tokens: int, topk: int, experts: int, align: int = 1):
        self.tokens, self.topk, self.experts, self.align = int(tokens), int(topk), int(experts), int(align)
        if min(self.tokens, self.topk, self.experts, self.align) < 0:
            _bad("ExpertPlan", "negative size")
        if self.tokens >> 64 or max(self.topk, self.experts, self.align) >> 32:  # ctypes would cut them short
            _bad("ExpertPlan", "size past the library's types", ZC_ERR_UNSUPPORTED)
        self.rows = lib().zc_route_rows(self.tokens, self.topk, self.experts, self.align)
        self.workspace_bytes = lib().zc_route_workspace_bytes(self.tokens, self.topk, self.experts)
        if self.workspace_bytes == 0 or (self.rows == 0 and self.tokens):
            _bad("ExpertPlan", f"{tokens} tokens, {topk} choices, {experts} experts, align {align}",
                 ZC_ERR_UNSUPPORTED)
        self._sizes = (self.tokens, self.topk, self.experts, self.align, self.rows, self.workspace_bytes)
        if self.align & (self.align - 1) or not 1 <= self.align <= 1024:
            _bad("ExpertPlan", f"align {align}", ZC_ERR_UNSUPPORTED)

    # buffers (torch allocation only) -------------------------------------
    def empty_routing(self, device="cuda") -> Routing:
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)
        return Routing(z(self.experts + 1), z(self.experts), z(self.tokens, self.topk), z(self.rows))

    def empty_workspace(self, device="cuda"):
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)

    def empty_rows(self, hidden: int, dtype=torch.bfloat16, device="cuda"):
        return torch.zeros(self.rows, hidden, dtype=dtype, device=device)

    def empty_fp8(self, hidden: int, device="cuda") -> Fp8Blocks:
        return empty_fp8_rows(self.rows, hidden, device)

    # calls ----------------------------------------------------------------
    def route(self, ids, routing: Routing, ws, stream=None):
        """Enqueue the sorting of ids (int32 [tokens, topk]; outside
        0..experts-1: no row) into routing."""
        _zc.route(self._sizes, ids, routing, ws, stream)

    def dispatch(self, x, routing: Routing, rows, stream=None):
        """Enqueue rows[row of (t, k)] = x[t]; padding rows are zeros."""
        _zc.dispatch(self._sizes, x, routing, rows, stream)

    def dispatch_fp8(self, x, routing: Routing, out: Fp8Blocks, stream=None):
        """Enqueue dispatch with the rows stored as 1 x 128 blocks."""
        _zc.dispatch_fp8(self._sizes, x, routing, out, stream)

    def combine(self, rows, weights, routing: Routing, y, stream=None):
        """Enqueue y[t] = sum over k of weights[t, k] * rows[row of (t, k)];
        weights None: ones, which makes it the gradient of dispatch."""
        _zc.combine(self._sizes, rows, weights, routing, y, stream)

    def combine_backward(self, dy, rows, weights, routing: Routing, drows, dweights, stream=None):
        """Enqueue the gradient of combine: drows (padding rows zeros) and
        dweights (float32 [tokens, topk]); either may be None, and rows with
        dweights."""
        _zc.combine_backward(self._sizes, dy, rows, weights, routing, drows, dweights, stream)


def quantize_rows(x, out: Fp8Blocks, used=None, stream=None):
    """Enqueue the cast of x [rows, cols] to 1 x 128 blocks.  used: None or a
    device int32 (e.g. ``routing.offsets[-1:]``); rows from there on are left."""
    _zc.quantize_rows(x, out, used, stream)


def quantize_weights(w, out: Fp8Blocks, transpose: bool = False, stream=None):
    """Enqueue the cast of w [experts, n, k] (transpose: [experts, k, n]) to
    the 128 x 128 blocks of [experts, n, k]."""
    _zc.quantize_weights(w, out, transpose, stream)


def quantize_columns(x, out: Fp8Columns, used=None, stream=None):
    """Enqueue the cast of x [rows, cols] in blocks of 128 rows of a column."""
    _zc.quantize_columns(x, out, used, stream)


def expert_product(a: Fp8Blocks, w: Fp8Blocks, out, offsets=None, counts=None, stream=None):
    """Enqueue out[r] = A[r] W[e]^T for the rows r of every expert's segment;
    a: 1 x 128 blocks [rows, k], w: 128 x 128 blocks [experts, n, k], out
    [rows, n].  offsets None: one expert, all rows.  Results in 32 bits are off
    by about 2e-5 of their root mean square (the 8-bit matrix unit's rounding,
    here and in expert_weight_grad); where that matters, ``a.float()`` and
    ``w.float(128)`` give the values to multiply in 32 bits."""
    _zc.expert_product(a, w, out, offsets, counts, stream)


def expert_weight_grad_workspace_bytes(rows: int, experts: int, n: int, k: int) -> int:
    """Bytes expert_weight_grad uses to sum long segments in parts (or 0)."""
    if any(v < 0 or v >> 32 for v in (rows, experts, n, k)):  # past every limit; ctypes would cut them short
        return 0
    return lib().zc_expert_weight_grad_workspace_bytes(rows, experts, n, k)


def expert_weight_grad(y: Fp8Columns, x: Fp8Columns, dw, offsets=None, ws=None, stream=None):
    """Enqueue dw[e] = Y_e^T X_e over the rows of every expert's segment
    (segments begin at multiples of 128, and get NaN where they do not); y: columns of [rows, n], x: columns
    of [rows, k], dw [experts, n, k].  ws: the workspace for long segments;
    without one it is taken from torch's allocator, on the call's stream."""
    if ws is None and stream is not None:
        with torch.cuda.stream(stream):
            _zc.expert_weight_grad(y, x, dw, offsets, None, None)
    else:
        _zc.expert_weight_grad(y, x, dw, offsets, ws, stream)
