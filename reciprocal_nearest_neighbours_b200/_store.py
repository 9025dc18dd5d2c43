"""ctypes binding of the token store calls of libfastnn.so: argument marshalling only.

A stream of images keeps its tokens (descriptors, patch features) in pages:
``k_pages`` [n_pages, heads, page, d] and ``v_pages`` [n_pages, heads, page, dv]
(bfloat16 or float16), addressed through ``page_table`` [n_seqs, width] int32.
New tokens come as a ragged batch: rows ``cu[s] .. cu[s + 1] - 1`` belong to
sequence ``s``; ``max_new`` bounds the number of new tokens of one sequence (a
host number, which sizes the launches). ``lens`` are the positions held, before
the call for ``fastnn_store_append`` and including the batch's tokens for the
others:

    fastnn_store_append(k, v, k_pages, v_pages, page_table, lens, cu, max_new, ...)
    lens += cu[1:] - cu[:-1]
    out, lse = fastnn_attend(q, k_pages, v_pages, page_table, lens, cu, max_new)
"""

from __future__ import annotations

import ctypes
import math

import torch

from ._lib import FASTNN_BF16, FASTNN_F16, FastNNError, _check, library

FASTNN_ROTARY_HALF = 0
FASTNN_ROTARY_INTERLEAVED = 1
FASTNN_STORE_APPEND_WORKSPACE = 256

_LAYOUTS = {"half": FASTNN_ROTARY_HALF, "interleaved": FASTNN_ROTARY_INTERLEAVED}
_CODES = {torch.bfloat16: FASTNN_BF16, torch.float16: FASTNN_F16}


class _Store(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_mean", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("cu", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("n_seqs", ctypes.c_int), ("table_width", ctypes.c_int), ("page", ctypes.c_int),
                ("heads", ctypes.c_int), ("d", ctypes.c_int), ("dv", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class _Rotation(ctypes.Structure):
    _fields_ = [("pos", ctypes.c_void_p), ("freq", ctypes.c_void_p), ("axes", ctypes.c_int),
                ("rot", ctypes.c_int), ("layout", ctypes.c_int), ("scale", ctypes.c_float)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = library()
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        S, R, F = ctypes.POINTER(_Store), ctypes.POINTER(_Rotation), ctypes.c_float
        for name, args, res in (
                ("fastnn_rotary", [P, I64, I64, I, I, I, R, I, P, I64, P], I),
                ("fastnn_store_append", [S, P, I64, P, I64, I64, I, R, P, SZ, P], I),
                ("fastnn_attend_workspace_size", [S, I64, I, I, I], SZ),
                ("fastnn_attend", [S, P, I64, I64, I, I, I, F, P, I, P, P, P, SZ, P], I),
                ("fastnn_select_workspace_size", [S, I64], SZ),
                ("fastnn_select_pages", [S, P, I64, I64, I, I, I, I, I, I, P, P, SZ, P], I)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _bound = lib
    return _bound


def _code(t: torch.Tensor) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"tokens must be bfloat16 or float16, got {t.dtype}")
    return code


def _rows(t: torch.Tensor, what: str, heads: int, d: int) -> int:
    """Token stride of ``t`` [n, heads, d], whose heads lie one after the other."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{what} must be [tokens, {heads}, {d}], got {tuple(t.shape)}")
    stride, head, one = t.stride()
    if t.shape[0] < 2:
        stride = max(stride, heads * d)
    if (one != 1 and d > 1) or (head != d and heads > 1) or stride < heads * d:
        raise ValueError(f"{what}: the heads of a token must lie one after the other")
    return stride


def _index(t: torch.Tensor, what: str, dims: int, dev):
    if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of {dims} dimension(s)")
    if t.device != dev:
        raise ValueError(f"{what} is on {t.device}, the tokens on {dev}")


def _same(dev, dtype, **tensors):
    for what, t in tensors.items():
        if t.device != dev:
            raise ValueError(f"{what} is on {t.device}, the tokens on {dev}")
        if t.dtype != dtype:
            raise TypeError(f"{what} is {t.dtype}, the tokens {dtype}")


class _On:
    """The tensors' device as the current one, and the stream to launch on."""

    def __init__(self, dev, stream):
        if dev.type != "cuda":
            raise ValueError("tensors must be CUDA tensors")
        self.guard = None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
        s = torch.cuda.current_stream(dev) if stream is None else stream
        if s.device != dev:
            raise ValueError(f"the stream is on {s.device}, the tokens on {dev}")
        self.stream = s.cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, dv, k=None, v=None,
              mean=None) -> _Store:
    _index(page_table, "page_table", 2, dev)
    _index(lens, "lens", 1, dev)
    _index(cu, "cu", 1, dev)
    seqs, width = page_table.shape
    if lens.shape[0] != seqs or cu.shape[0] != seqs + 1:
        raise ValueError("page_table [n_seqs, width], lens [n_seqs] and cu [n_seqs + 1] disagree")
    return _Store(k, v, mean, page_table.data_ptr(), lens.data_ptr(), cu.data_ptr(), n_pages, seqs,
                  width, page, heads, d, dv, code)


def _pages(k_pages, v_pages):
    if k_pages.dim() != 4 or v_pages.dim() != 4 or k_pages.shape[:3] != v_pages.shape[:3]:
        raise ValueError("k_pages [n_pages, heads, page, d] and v_pages [n_pages, heads, page, dv] "
                         f"disagree: {tuple(k_pages.shape)}, {tuple(v_pages.shape)}")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    return k_pages.shape


def _new(shape, dtype, dev, stream):
    """A tensor that a launch on ``stream`` (None: the current one) writes: on another stream
    than the one it was allocated on, its memory must not go round before that launch is done."""
    t = torch.empty(shape, dtype=dtype, device=dev)
    if stream is not None:
        t.record_stream(stream)
    return t


def _scratch(need: int, dev, workspace, what: str, stream):
    if need == 0:
        raise FastNNError(-1, what)
    if workspace is None:
        return _new(need, torch.uint8, dev, stream)
    if workspace.device != dev:
        raise ValueError(f"the workspace is on {workspace.device}, the tokens on {dev}")
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise FastNNError(-3, "workspace")
    return workspace


def _rotation(pos, freq, layout, scale, n, dev) -> _Rotation:
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    if pos.dim() == 1:
        pos = pos.unsqueeze(1)
    _index(pos, "pos", 2, dev)
    if freq.dtype != torch.float64 or freq.dim() != 1 or not freq.is_contiguous() or \
            freq.device != dev:
        raise ValueError(f"freq must be a contiguous float64 vector on {dev}")
    axes = pos.shape[1]
    if pos.shape[0] != n or axes not in (1, 2):
        raise ValueError(f"pos must be [tokens] or [tokens, 1 or 2] for {n} tokens, "
                         f"got {tuple(pos.shape)}")
    return _Rotation(pos.data_ptr(), freq.data_ptr(), axes, 2 * axes * freq.shape[0],
                     _LAYOUTS[layout], scale)


def fastnn_rotary_frequencies(rot: int, base: float = 10000.0, axes: int = 1, stretch: float = 1.0,
                              long_base: float | None = None, device="cuda") -> torch.Tensor:
    """Radians per position of each pair of one axis, float64 [rot / (2 * axes)].

    ``base ** (-j / count)`` for pair ``j`` of ``count``, divided by ``stretch``: positions
    interpolated, for contexts ``stretch`` times longer than those seen in training.
    ``long_base`` (optional) replaces ``base`` instead, which stretches the slow pairs
    and leaves the fast ones. Any other float64 table serves the calls as well.
    """
    if axes not in (1, 2) or rot < 1 or rot % (2 * axes):
        raise ValueError(f"rot must be a multiple of 2 * axes, got {rot} for {axes} axes")
    count = rot // (2 * axes)
    j = torch.arange(count, dtype=torch.float64)
    return ((base if long_base is None else long_base) ** (-j / count) / stretch).to(device)


def fastnn_rotary(x: torch.Tensor, pos: torch.Tensor, freq: torch.Tensor, layout: str = "half",
                  scale: float = 1.0, inverse: bool = False, out=None, stream=None):
    """Rotate ``x`` [tokens, heads, d] by the tokens' positions; returns ``out`` (same shape).

    ``pos`` int32 [tokens] or [tokens, axes], ``freq`` float64 [rot / (2 * axes)] radians
    per position: the first ``rot`` elements of every head turn, the rest stay. Layout
    "half" pairs element j with j + half of its axis' elements, "interleaved" 2j with
    2j + 1. ``inverse`` turns back: applied to a gradient of the result it gives that of
    ``x``. ``out`` may be ``x``.
    """
    code = _code(x)
    if x.dim() != 3:
        raise ValueError(f"x must be [tokens, heads, d], got {tuple(x.shape)}")
    n, heads, d = x.shape
    dev = x.device
    xs = _rows(x, "x", heads, d)
    rot = _rotation(pos, freq, layout, scale, n, dev)
    if out is None:
        out = _new((n, heads, d), x.dtype, dev, stream)
        os = heads * d
    else:
        _same(dev, x.dtype, out=out)
        if out.shape != x.shape:
            raise ValueError(f"out must be {tuple(x.shape)}, got {tuple(out.shape)}")
        os = _rows(out, "out", heads, d)
    with _On(dev, stream) as st:
        rc = _lib().fastnn_rotary(x.data_ptr(), xs, n, heads, d, code, rot, int(inverse),
                                  out.data_ptr(), os, st)
    _check(rc, "fastnn_rotary")
    return out


def fastnn_store_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                        v_pages: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                        cu: torch.Tensor, max_new: int, k_mean=None, pos=None, freq=None,
                        layout: str = "half", scale: float = 1.0, workspace=None, stream=None):
    """Put new keys ``k`` [tokens, heads, d] and values ``v`` [tokens, heads, dv] into the store.

    Token i of sequence s becomes position ``lens[s] + i``; ``lens`` itself is the
    caller's to advance. ``pos`` and ``freq`` (both or neither) rotate the keys on the
    way, as ``fastnn_rotary`` does. ``k_mean`` [n_pages, heads, d] receives the mean key
    of every page that the call touches. ``fastnn_device_status(workspace)`` tells
    whether each token found a place.
    """
    code = _code(k)
    n_pages, heads, page, d = _pages(k_pages, v_pages)
    dv = v_pages.shape[3]
    dev = k.device
    _same(dev, k.dtype, v=v, k_pages=k_pages, v_pages=v_pages)
    ks, vs = _rows(k, "k", heads, d), _rows(v, "v", heads, dv)
    n = k.shape[0]
    if v.shape[0] != n:
        raise ValueError(f"k has {n} tokens, v {v.shape[0]}")
    mean = None
    if k_mean is not None:
        _same(dev, k.dtype, k_mean=k_mean)
        if k_mean.shape != (n_pages, heads, d) or not k_mean.is_contiguous():
            raise ValueError(f"k_mean must be contiguous [{n_pages}, {heads}, {d}]")
        mean = k_mean.data_ptr()
    store = _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, dv,
                      k_pages.data_ptr(), v_pages.data_ptr(), mean)
    if (pos is None) != (freq is None):
        raise ValueError("pos and freq come together")
    rot = None if pos is None else _rotation(pos, freq, layout, scale, n, dev)
    ws = _scratch(FASTNN_STORE_APPEND_WORKSPACE, dev, workspace, "fastnn_store_append", stream)
    with _On(dev, stream) as st:
        rc = _lib().fastnn_store_append(store, k.data_ptr(), ks, v.data_ptr(), vs, n, max_new, rot,
                                        ws.data_ptr(), FASTNN_STORE_APPEND_WORKSPACE, st)
    _check(rc, "fastnn_store_append")


def fastnn_attend_workspace_size(n: int, heads_q: int, heads: int, d: int, dv: int, n_seqs: int,
                                 max_new: int, table_width: int, page: int, select: int = 0,
                                 dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of ``fastnn_attend`` for these sizes (0: no call would accept them)."""
    store = _Store(None, None, None, None, None, None, 1, n_seqs, table_width, page, heads, d, dv,
                   _CODES.get(dtype, -1))
    return int(_lib().fastnn_attend_workspace_size(store, n, heads_q, max_new, select))


def fastnn_attend(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                  page_table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor, max_new: int,
                  causal: bool = True, scale: float | None = None, pages=None, out=None, lse=None,
                  workspace=None, stream=None):
    """Attention of the tokens ``q`` [tokens, heads_q, d] over their sequences in the store.

    ``lens`` count the batch's own tokens (append first); with ``causal`` a token sees the
    positions up to its own, without it all of its sequence. ``scale`` defaults to
    ``d ** -0.5``. ``pages`` (int32 [tokens, heads, select] from ``fastnn_select_pages``)
    restricts each token to the listed pages of its sequence. Returns ``(out [tokens,
    heads_q, dv], lse float32 [tokens, heads_q])``; a token that sees nothing has zeros
    and -inf.
    """
    code = _code(q)
    n_pages, heads, page, d = _pages(k_pages, v_pages)
    dv = v_pages.shape[3]
    dev = q.device
    _same(dev, q.dtype, k_pages=k_pages, v_pages=v_pages)
    if q.dim() != 3 or q.shape[1] % heads:
        raise ValueError(f"q must be [tokens, a multiple of {heads}, {d}], got {tuple(q.shape)}")
    n, hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", hq, d)
    store = _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, dv,
                      k_pages.data_ptr(), v_pages.data_ptr())
    select, listed = 0, None
    if pages is not None:
        _index(pages, "pages", 3, dev)
        if pages.shape[0] != n or pages.shape[1] != heads or pages.shape[2] < 1:
            raise ValueError(f"pages must be [{n}, {heads}, select], got {tuple(pages.shape)}")
        select, listed = pages.shape[2], pages.data_ptr()
    if out is None:
        out = _new((n, hq, dv), q.dtype, dev, stream)
    else:
        _same(dev, q.dtype, out=out)
        if out.shape != (n, hq, dv) or not out.is_contiguous():
            raise ValueError(f"out must be contiguous [{n}, {hq}, {dv}]")
    if lse is None:
        lse = _new((n, hq), torch.float32, dev, stream)
    else:
        _same(dev, torch.float32, lse=lse)
        if lse.shape != (n, hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{n}, {hq}]")
    lib = _lib()
    need = lib.fastnn_attend_workspace_size(store, n, hq, max_new, select)
    ws = _scratch(need, dev, workspace, "fastnn_attend_workspace_size", stream)
    with _On(dev, stream) as st:
        rc = lib.fastnn_attend(store, q.data_ptr(), qs, n, hq, max_new, int(causal),
                               1.0 / math.sqrt(d) if scale is None else scale, listed, select,
                               out.data_ptr(), lse.data_ptr(), ws.data_ptr(), need, st)
    _check(rc, "fastnn_attend")
    return out, lse


def fastnn_select_pages(q: torch.Tensor, k_mean: torch.Tensor, page_table: torch.Tensor,
                        lens: torch.Tensor, cu: torch.Tensor, max_new: int, page: int, select: int,
                        keep_first: int = 0, keep_last: int = 1, causal: bool = True, out=None,
                        workspace=None, stream=None):
    """The ``select`` pages of each token's sequence that score best by their mean key.

    A page's score for a token and key head is the dot product of its ``k_mean``
    [n_pages, heads, d] with the sum of the group's queries. The first ``keep_first``
    and last ``keep_last`` visible pages are always taken. Returns int32 [tokens, heads,
    select]: logical page numbers in ascending order, -1 behind the last.
    """
    code = _code(q)
    dev = q.device
    _same(dev, q.dtype, k_mean=k_mean)
    if k_mean.dim() != 3 or not k_mean.is_contiguous():
        raise ValueError("k_mean must be contiguous [n_pages, heads, d]")
    n_pages, heads, d = k_mean.shape
    if q.dim() != 3 or heads < 1 or q.shape[1] % heads:
        raise ValueError(f"q must be [tokens, a multiple of {heads}, {d}], got {tuple(q.shape)}")
    n, hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", hq, d)
    store = _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, 8, None, None,
                      k_mean.data_ptr())
    if out is None:
        out = _new((n, heads, select), torch.int32, dev, stream)
    else:
        _index(out, "out", 3, dev)
        if out.shape != (n, heads, select):
            raise ValueError(f"out must be [{n}, {heads}, {select}]")
    lib = _lib()
    need = lib.fastnn_select_workspace_size(store, n)
    ws = _scratch(need, dev, workspace, "fastnn_select_workspace_size", stream)
    with _On(dev, stream) as st:
        rc = lib.fastnn_select_pages(store, q.data_ptr(), qs, n, hq, max_new, int(causal),
                                     keep_first, keep_last, select, out.data_ptr(), ws.data_ptr(),
                                     need, st)
    _check(rc, "fastnn_select_pages")
    return out
