"""ctypes binding of the expert operators (the C ABI in include/zc_experts.h).

Around the compressed all-to-all: ``ExpertPlan`` sorts tokens by expert
(route, dispatch, dispatch_fp8), brings rows back with the router's weights
(combine) and takes the gradients of both (combine_backward; the gradient of
dispatch is combine without weights).  ``quantize_rows`` / ``_weights`` /
``_columns`` cast to 8-bit blocks of 128; ``expert_product`` and
``expert_weight_grad`` multiply such blocks, expert by expert.

Argument marshalling and checks only, as in ``binding``: every buffer is the
caller's, every call enqueues on the current (or the given) stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import ZC_ERR_CAPACITY, ZC_ERR_INVALID_ARG, ZC_ERR_UNSUPPORTED, ZcError

# Every symbol include/zc_experts.h declares.
EXPERT_EXPORTS = (
    "zc_route_rows", "zc_route_workspace_bytes", "zc_route", "zc_dispatch", "zc_dispatch_fp8",
    "zc_combine", "zc_combine_backward", "zc_quantize_rows", "zc_quantize_weights",
    "zc_quantize_columns", "zc_expert_product", "zc_expert_weight_grad",
    "zc_expert_weight_grad_workspace_bytes",
)

BLOCK = 128  # values per scale
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_FP8, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_I32, _F32 = torch.int32, torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent where torch has no GPU support
_device = getattr(torch._C, "_cuda_getDevice", None)

_lib = None


class _Calls:
    """The library's functions as attributes, set on the first use."""

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
        setattr(_zc, name, f)
    _lib = L
    return L


# The checks below run before every call, and a call's kernels take a few
# microseconds on small inputs: they read each attribute once and say what is
# wrong only when something is.

def _bad(what: str, why: str, code: int = ZC_ERR_INVALID_ARG):
    raise ZcError(code, f"{what}: {why}")


def _failed(rc: int, name: str):
    raise ZcError(rc, name)


def _stream(stream):
    # current_stream() builds a Stream object, 3 us; its handle alone is 0.1
    return _raw_stream(_device()) if stream is None else stream.cuda_stream


def _matrix(t, what: str, rows: int, dtype=None, width=None):
    """(pointer, row stride, rows, width) of a GPU matrix that is contiguous
    along its columns, of `dtype` (or one of the three row types), with at
    least `rows` rows and exactly `width` columns."""
    if not getattr(t, "is_cuda", False):
        _bad(what, "not a GPU tensor")
    d = t.dtype
    if d is not dtype and (dtype is not None or d not in _DTYPES):
        _bad(what, f"type {d}" + (f", {dtype} expected" if dtype is not None else ""))
    shape = t.shape
    if len(shape) != 2 or (width is not None and shape[1] != width):
        _bad(what, f"shape {tuple(shape)}, (rows, {'columns' if width is None else width}) expected")
    n, w = shape
    s, one = t.stride()
    if s < w:
        if n > 1:
            _bad(what, f"strides {(s, one)}: rows overlap")
        s = w
    if one != 1 and w > 1:
        _bad(what, f"strides {(s, one)}: columns must be contiguous")
    if n < rows:
        _bad(what, f"{n} rows, {rows} needed", ZC_ERR_CAPACITY)
    return t.data_ptr(), s, n, w


def _flat(t, what: str, dtype, count: int):
    """Pointer of a contiguous GPU tensor of `dtype` with at least `count`
    elements."""
    if not getattr(t, "is_cuda", False):
        _bad(what, "not a GPU tensor")
    if t.dtype is not dtype:
        _bad(what, f"type {t.dtype}, {dtype} expected")
    if not t.is_contiguous():
        _bad(what, "not contiguous")
    if t.numel() < count:
        _bad(what, f"{t.numel()} elements, {count} needed", ZC_ERR_CAPACITY)
    return t.data_ptr()


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


def _part(t, what: str, dtype, dims, width: int):
    if not getattr(t, "is_cuda", False):
        _bad(what, "not a GPU tensor")
    if t.dtype is not dtype:
        _bad(what, f"type {t.dtype}, {dtype} expected")
    if not t.is_contiguous():
        _bad(what, "not contiguous")
    shape = t.shape
    if len(shape) != len(dims) + 1 or shape[-1] != width or (len(dims) > 1 and shape[1] != dims[1]):
        _bad(what, f"shape {tuple(shape)}, {tuple(dims) + (width,)} expected")
    if shape[0] < dims[0]:
        _bad(what, f"{shape[0]} rows, {dims[0]} needed", ZC_ERR_CAPACITY)
    return t.data_ptr()


def _blocks(f: Fp8Blocks, what: str, cols: int, lead, scale_lead=None):
    """Pointers of data and scale of blocks of the given shape.  The first
    dimension may be longer."""
    data, scale, have = f
    if have != cols:
        _bad(what, f"{have} columns, {cols} expected")
    return (_part(data, what, _FP8, lead, (cols + 127) // 128 * 128),
            _part(scale, what, _E8M0, scale_lead or lead, (cols + 511) // 512 * 4))


def _columns(f: Fp8Columns, what: str, rows: int, cols: int):
    """Pointers of data and scale of the columns of a [rows, cols] matrix."""
    data, scale, r, c = f
    if r != rows or c != cols:
        _bad(what, f"columns of {(r, c)}, {(rows, cols)} expected")
    blocks = (rows + 127) // 128
    return _part(data, what, _FP8, (blocks, cols), 128), _part(scale, what, _E8M0, (blocks,), (cols + 3) // 4 * 4)


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
        self.rows = lib().zc_route_rows(self.tokens, self.topk, self.experts, self.align)
        self.workspace_bytes = lib().zc_route_workspace_bytes(self.tokens, self.topk, self.experts)
        if self.workspace_bytes == 0 or (self.rows == 0 and self.tokens):
            _bad("ExpertPlan", f"{tokens} tokens, {topk} choices, {experts} experts, align {align}",
                 ZC_ERR_UNSUPPORTED)
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

    # checks ---------------------------------------------------------------
    def _routing(self, r: Routing):
        """Pointers of offsets, counts and row; packed segments have no
        padding rows, which the library is told by counts 0."""
        row = _flat(r[2], "row", _I32, self.tokens * self.topk)
        if self.align == 1:
            return 0, 0, row
        return _flat(r[0], "offsets", _I32, self.experts + 1), _flat(r[1], "counts", _I32, self.experts), row

    def _weights(self, w):
        return 0 if w is None else _flat(w, "weights", _F32, self.tokens * self.topk)

    # calls ----------------------------------------------------------------
    def route(self, ids, routing: Routing, ws, stream=None):
        """Enqueue the sorting of ids (int32 [tokens, topk]; outside
        0..experts-1: no row) into routing."""
        p = _flat(ids, "ids", _I32, self.tokens * self.topk)
        off = _flat(routing[0], "offsets", _I32, self.experts + 1)
        cnt = _flat(routing[1], "counts", _I32, self.experts)
        row, slot = _flat(routing[2], "row", _I32, self.tokens * self.topk), routing[3]
        s = _flat(slot, "slot", _I32, self.rows)
        w = _flat(ws, "workspace", torch.uint8, self.workspace_bytes)
        rc = _zc.zc_route(p, self.tokens, self.topk, self.experts, self.align, off, cnt, row, s, slot.numel(), w,
                          ws.numel(), _stream(stream))
        if rc:
            _failed(rc, "zc_route")

    def dispatch(self, x, routing: Routing, rows, stream=None):
        """Enqueue rows[row of (t, k)] = x[t]; padding rows are zeros."""
        p, stride, _, hidden = _matrix(x, "x", self.tokens)
        d = x.dtype
        q, out_stride, n, _ = _matrix(rows, "rows", self.rows, d, hidden)
        off, cnt, row = self._routing(routing)
        rc = _zc.zc_dispatch(p, stride, _DTYPES[d], self.tokens, self.topk, self.experts, hidden, off, cnt, row, q,
                             out_stride, n, _stream(stream))
        if rc:
            _failed(rc, "zc_dispatch")

    def dispatch_fp8(self, x, routing: Routing, out: Fp8Blocks, stream=None):
        """Enqueue dispatch with the rows stored as 1 x 128 blocks."""
        p, stride, _, hidden = _matrix(x, "x", self.tokens)
        data, scale = _blocks(out, "out", hidden, (self.rows,))
        off, cnt, row = self._routing(routing)
        rc = _zc.zc_dispatch_fp8(p, stride, _DTYPES[x.dtype], self.tokens, self.topk, self.experts, hidden, off, cnt,
                                 row, data, scale, min(out[0].shape[0], out[1].shape[0]), _stream(stream))
        if rc:
            _failed(rc, "zc_dispatch_fp8")

    def combine(self, rows, weights, routing: Routing, y, stream=None):
        """Enqueue y[t] = sum over k of weights[t, k] * rows[row of (t, k)];
        weights None: ones, which makes it the gradient of dispatch."""
        q, y_stride, _, hidden = _matrix(y, "y", self.tokens)
        d = y.dtype
        p, stride, n, _ = _matrix(rows, "rows", self.rows, d, hidden)
        row = _flat(routing[2], "row", _I32, self.tokens * self.topk)
        rc = _zc.zc_combine(p, stride, self._weights(weights), _DTYPES[d], self.tokens, self.topk, hidden, row, n, q,
                            y_stride, _stream(stream))
        if rc:
            _failed(rc, "zc_combine")

    def combine_backward(self, dy, rows, weights, routing: Routing, drows, dweights, stream=None):
        """Enqueue the gradient of combine: drows (padding rows zeros) and
        dweights (float32 [tokens, topk]); either may be None, and rows with
        dweights."""
        p, stride, _, hidden = _matrix(dy, "dy", self.tokens)
        d = dy.dtype
        off, cnt, row = self._routing(routing)
        if drows is None and dweights is None:
            _bad("combine_backward", "no gradient asked for")
        q = q_stride = r = r_stride = 0
        n = m = 1 << 31
        if drows is not None:
            q, q_stride, n, _ = _matrix(drows, "drows", self.rows, d, hidden)
        if dweights is not None:
            if rows is None:
                _bad("combine_backward", "dweights needs rows")
            r, r_stride, m, _ = _matrix(rows, "rows", self.rows, d, hidden)
        rc = _zc.zc_combine_backward(p, stride, r, r_stride, self._weights(weights), _DTYPES[d], self.tokens,
                                     self.topk, self.experts, hidden, off, cnt, row, min(n, m), q, q_stride,
                                     self._weights(dweights), _stream(stream))
        if rc:
            _failed(rc, "zc_combine_backward")


def _used(used):
    return 0 if used is None else _flat(used, "used", _I32, 1)


def quantize_rows(x, out: Fp8Blocks, used=None, stream=None):
    """Enqueue the cast of x [rows, cols] to 1 x 128 blocks.  used: None or a
    device int32 (e.g. ``routing.offsets[-1:]``); rows from there on are left."""
    p, stride, rows, cols = _matrix(x, "x", 0)
    data, scale = _blocks(out, "out", cols, (rows,))
    rc = _zc.zc_quantize_rows(p, stride, _DTYPES[x.dtype], rows, cols, _used(used), data, scale, _stream(stream))
    if rc:
        _failed(rc, "zc_quantize_rows")


def quantize_weights(w, out: Fp8Blocks, transpose: bool = False, stream=None):
    """Enqueue the cast of w [experts, n, k] (transpose: [experts, k, n]) to
    the 128 x 128 blocks of [experts, n, k]."""
    if w.dim() != 3 or w.dtype not in _DTYPES:
        _bad("w", f"shape {tuple(w.shape)}, type {w.dtype}")
    e, n, k = w.shape
    if transpose:
        n, k = k, n
    p = _flat(w, "w", w.dtype, 0)
    data, scale = _blocks(out, "out", k, (e, n), (e, (n + 127) // 128))
    rc = _zc.zc_quantize_weights(p, _DTYPES[w.dtype], e, n, k, 1 if transpose else 0, data, scale, _stream(stream))
    if rc:
        _failed(rc, "zc_quantize_weights")


def quantize_columns(x, out: Fp8Columns, used=None, stream=None):
    """Enqueue the cast of x [rows, cols] in blocks of 128 rows of a column."""
    p, stride, rows, cols = _matrix(x, "x", 0)
    data, scale = _columns(out, "out", rows, cols)
    rc = _zc.zc_quantize_columns(p, stride, _DTYPES[x.dtype], rows, cols, _used(used), data, scale, _stream(stream))
    if rc:
        _failed(rc, "zc_quantize_columns")


def expert_product(a: Fp8Blocks, w: Fp8Blocks, out, offsets=None, counts=None, stream=None):
    """Enqueue out[r] = A[r] W[e]^T for the rows r of every expert's segment;
    a: 1 x 128 blocks [rows, k], w: 128 x 128 blocks [experts, n, k], out
    [rows, n].  offsets None: one expert, all rows."""
    shape, k = w[0].shape, w[2]
    if len(shape) != 3:
        _bad("expert_product", "a is [rows, k], w is [experts, n, k]")
    experts, n = shape[0], shape[1]
    q, stride, rows, _ = _matrix(out, "out", 0, None, n)
    ap, asp = _blocks(a, "a", k, (rows,))
    wp, wsp = _blocks(w, "w", k, (experts, n), (experts, (n + 127) // 128))
    off = 0 if offsets is None else _flat(offsets, "offsets", _I32, experts + 1)
    cnt = 0 if counts is None else _flat(counts, "counts", _I32, experts)
    rc = _zc.zc_expert_product(ap, asp, rows, wp, wsp, experts, n, k, off, cnt, q, stride, _DTYPES[out.dtype],
                               _stream(stream))
    if rc:
        _failed(rc, "zc_expert_product")


def expert_weight_grad_workspace_bytes(rows: int, experts: int, n: int, k: int) -> int:
    """Bytes expert_weight_grad uses to sum long segments in parts (or 0)."""
    return _zc.zc_expert_weight_grad_workspace_bytes(rows, experts, n, k)


def expert_weight_grad(y: Fp8Columns, x: Fp8Columns, dw, offsets=None, ws=None, stream=None):
    """Enqueue dw[e] = Y_e^T X_e over the rows of every expert's segment
    (segments begin at multiples of 128); y: columns of [rows, n], x: columns
    of [rows, k], dw [experts, n, k].  ws: the workspace for long segments;
    without one it is taken from torch's allocator, on the call's stream."""
    shape = dw.shape
    if len(shape) != 3 or dw.dtype not in _DTYPES:
        _bad("dw", f"shape {tuple(shape)}, type {dw.dtype}")
    experts, n, k = shape
    rows = x[2]
    p = _flat(dw, "dw", dw.dtype, 0)
    yp, ysp = _columns(y, "y", rows, n)
    xp, xsp = _columns(x, "x", rows, k)
    off = 0 if offsets is None else _flat(offsets, "offsets", _I32, experts + 1)
    need = _zc.zc_expert_weight_grad_workspace_bytes(rows, experts, n, k)
    w = 0
    if need:
        if ws is None:
            if stream is None:
                ws = torch.empty(need, dtype=torch.uint8, device=dw.device)
            else:
                with torch.cuda.stream(stream):
                    ws = torch.empty(need, dtype=torch.uint8, device=dw.device)
        w = _flat(ws, "workspace", torch.uint8, need)
    rc = _zc.zc_expert_weight_grad(yp, ysp, xp, xsp, rows, experts, n, k, off, p, _DTYPES[dw.dtype], w, need,
                                   _stream(stream))
    if rc:
        _failed(rc, "zc_expert_weight_grad")
