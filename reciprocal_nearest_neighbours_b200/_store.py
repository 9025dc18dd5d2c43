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

A call with ``stream`` launches there: outputs and scratch that it makes are of that
stream's memory (outputs are also held for the stream that is current). The inputs are the
caller's to order and to keep until that stream is done with them.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from ._lib import FASTNN_BF16, FASTNN_F16, FastNNError, library

FASTNN_ROTARY_HALF = 0
FASTNN_ROTARY_INTERLEAVED = 1
FASTNN_STORE_APPEND_WORKSPACE = 256

_LAYOUTS = {"half": FASTNN_ROTARY_HALF, "interleaved": FASTNN_ROTARY_INTERLEAVED}
_CODES = {torch.bfloat16: FASTNN_BF16, torch.float16: FASTNN_F16}


# fastnn_store and fastnn_rotation, packed as the C compiler lays them out (a call passes
# the bytes: cheaper than filling a ctypes structure field by field).
_STORE = struct.Struct("@PPPPPPqiiiiiii")
_ROTATION = struct.Struct("@PPiiif")

_STATUS = 256  # bytes of a workspace that holds nothing but the status word

_bound = None
_I32 = torch.int32
# What torch.cuda.current_stream and current_device come down to, without their wrapping (3 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _lib():
    global _bound
    if _bound is None:
        lib = library()
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        B, F = ctypes.c_char_p, ctypes.c_float
        for name, args, res in (
                ("fastnn_rotary", [P, I64, I64, I, I, I, B, I, P, I64, P], I),
                ("fastnn_store_append", [B, P, I64, P, I64, I64, I, B, P, SZ, P], I),
                ("fastnn_attend_workspace_size", [B, I64, I, I, I], SZ),
                ("fastnn_attend", [B, P, I64, I64, I, I, I, F, P, I, P, P, P, SZ, P], I),
                ("fastnn_select_workspace_size", [B, I64, I, I], SZ),
                ("fastnn_select_pages", [B, P, I64, I64, I, I, I, I, I, I, P, P, SZ, P], I)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _bound = lib
    return _bound


def _code(t: torch.Tensor) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"tokens must be bfloat16 or float16, got {t.dtype}")
    return code


def _rows(t: torch.Tensor, what: str, n: int, heads: int, d: int) -> int:
    """Token stride of ``t`` [n, heads, d], whose heads lie one after the other."""
    if t.shape != (n, heads, d):
        raise ValueError(f"{what} must be [{n}, {heads}, {d}], got {tuple(t.shape)}")
    stride, head, one = t.stride()
    if n < 2:
        stride = max(stride, heads * d)
    if (one != 1 and d > 1) or (head != d and heads > 1) or stride < heads * d:
        raise ValueError(f"{what}: the heads of a token must lie one after the other")
    return stride


def _index(t: torch.Tensor, what: str, dims: int, dev: int) -> int:
    """Address of an int32 index array."""
    if t.dtype is not _I32 or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of {dims} dimension(s)")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, the tokens on cuda:{dev}")
    return t.data_ptr()


def _same(dev: int, dtype, what: str, t: torch.Tensor) -> int:
    """Address of ``t``, which must be of the tokens' device and type."""
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, the tokens on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{what} is {t.dtype}, the tokens {dtype}")
    return t.data_ptr()


def _device(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    return t.get_device()


def _launch(what: str, dev: int, stream, *args):
    """Call the library with the tensors' device current, on ``stream`` (None: the device's
    current one)."""
    if stream is None:
        raw = _raw_stream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tokens on cuda:{dev}")
        raw = stream.cuda_stream
    fn = getattr(_bound, what)
    if _current_device() == dev:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc:
        raise FastNNError(rc, what)


def _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, dv, k=None, v=None,
              mean=None) -> bytes:
    t, n, c = (_index(page_table, "page_table", 2, dev), _index(lens, "lens", 1, dev),
               _index(cu, "cu", 1, dev))
    seqs, width = page_table.shape
    if lens.shape[0] != seqs or cu.shape[0] != seqs + 1:
        raise ValueError("page_table [n_seqs, width], lens [n_seqs] and cu [n_seqs + 1] disagree")
    return _STORE.pack(k or 0, v or 0, mean or 0, t, n, c, n_pages, seqs, width, page, heads, d, dv,
                       code)


def _pages(k_pages, v_pages, dev, dtype):
    """Shape [n_pages, heads, page, d], dv, and the addresses of both."""
    kp, vp = _same(dev, dtype, "k_pages", k_pages), _same(dev, dtype, "v_pages", v_pages)
    shape, other = k_pages.shape, v_pages.shape
    if len(shape) != 4 or len(other) != 4 or shape[:3] != other[:3]:
        raise ValueError("k_pages [n_pages, heads, page, d] and v_pages [n_pages, heads, page, dv] "
                         f"disagree: {tuple(shape)}, {tuple(other)}")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    return shape, other[3], kp, vp


def _new(like, shape, dtype, stream):
    """A tensor on the device of ``like`` that a launch on ``stream`` (None: the current one) is
    the first to use. It is made of that stream's memory: the current stream's may just have
    been given back by a call whose kernel is still running there. Hold it until the launch."""
    if stream is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _result(like, shape, dtype, stream):
    """As ``_new``, for what the caller gets and will use on the current stream."""
    t = _new(like, shape, dtype, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _scratch(need: int, like, dev, workspace, what: str, stream):
    """The call's workspace, None for none: _STATUS bytes hold no more than the status word,
    which nobody reads where the caller brings no workspace. The caller of this holds what it
    returns until after the launch."""
    if need == 0:
        raise FastNNError(-1, what)
    if workspace is None:
        return None if need == _STATUS else _new(like, need, torch.uint8, stream)
    if workspace.get_device() != dev:
        raise ValueError(f"the workspace is on {workspace.device}, the tokens on cuda:{dev}")
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise FastNNError(-3, "workspace")
    return workspace


def _address(t) -> int:
    return 0 if t is None else t.data_ptr()


def _rotation(pos, freq, layout, scale, n, dev) -> bytes:
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    dims = pos.dim()
    at = _index(pos, "pos", 1 if dims == 1 else 2, dev)
    if freq.dtype is not torch.float64 or freq.dim() != 1 or not freq.is_contiguous() or \
            freq.get_device() != dev:
        raise ValueError(f"freq must be a contiguous float64 vector on cuda:{dev}")
    axes = 1 if dims == 1 else pos.shape[1]
    if pos.shape[0] != n or axes not in (1, 2):
        raise ValueError(f"pos must be [tokens] or [tokens, 1 or 2] for {n} tokens, "
                         f"got {tuple(pos.shape)}")
    return _ROTATION.pack(at, freq.data_ptr(), axes, 2 * axes * freq.shape[0], code, scale)


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
    dev = _device(x)
    n, heads, d = x.shape
    xs = _rows(x, "x", n, heads, d)
    rot = _rotation(pos, freq, layout, scale, n, dev)
    if out is None:
        out = _result(x, (n, heads, d), x.dtype, stream)
        to, os = out.data_ptr(), heads * d
    else:
        to, os = _same(dev, x.dtype, "out", out), _rows(out, "out", n, heads, d)
    _bound or _lib()
    _launch("fastnn_rotary", dev, stream, x.data_ptr(), xs, n, heads, d, code, rot, inverse, to, os)
    return out


def fastnn_store_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                        v_pages: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                        cu: torch.Tensor, max_new: int, k_mean=None, pos=None, freq=None,
                        layout: str = "half", scale: float = 1.0, workspace=None, stream=None):
    """Put new keys ``k`` [tokens, heads, d] and values ``v`` [tokens, heads, dv] into the store.

    Token i of sequence s becomes position ``lens[s] + i``; ``lens`` itself is the
    caller's to advance. ``pos`` and ``freq`` (both or neither) rotate the keys on the
    way, as ``fastnn_rotary`` does. ``k_mean`` [n_pages, heads, d] receives the mean key
    of every page that the call touches. With a ``workspace`` (256 bytes),
    ``fastnn_device_status(workspace)`` tells whether each token found a place.
    """
    code = _code(k)
    dev = _device(k)
    dtype = k.dtype
    (n_pages, heads, page, d), dv, kp, vp = _pages(k_pages, v_pages, dev, dtype)
    n = k.shape[0]
    ks, vs = _rows(k, "k", n, heads, d), _rows(v, "v", n, heads, dv)
    at_v = _same(dev, dtype, "v", v)
    mean = None
    if k_mean is not None:
        mean = _same(dev, dtype, "k_mean", k_mean)
        if k_mean.shape != (n_pages, heads, d) or not k_mean.is_contiguous():
            raise ValueError(f"k_mean must be contiguous [{n_pages}, {heads}, {d}]")
    store = _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, dv, kp, vp, mean)
    if (pos is None) != (freq is None):
        raise ValueError("pos and freq come together")
    rot = None if pos is None else _rotation(pos, freq, layout, scale, n, dev)
    ws = None
    if workspace is not None:
        ws = _scratch(FASTNN_STORE_APPEND_WORKSPACE, k, dev, workspace, "", stream)
    _bound or _lib()
    _launch("fastnn_store_append", dev, stream, store, k.data_ptr(), ks, at_v, vs, n, max_new, rot,
            _address(ws), FASTNN_STORE_APPEND_WORKSPACE)


def fastnn_attend_workspace_size(n: int, heads_q: int, heads: int, d: int, dv: int, n_seqs: int,
                                 max_new: int, table_width: int, page: int, select: int = 0,
                                 dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of ``fastnn_attend`` for these sizes (0: no call would accept them)."""
    store = _STORE.pack(0, 0, 0, 0, 0, 0, 1, n_seqs, table_width, page, heads, d, dv,
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
    dev = _device(q)
    dtype = q.dtype
    (n_pages, heads, page, d), dv, kp, vp = _pages(k_pages, v_pages, dev, dtype)
    if q.dim() != 3 or heads < 1 or q.shape[1] % heads:
        raise ValueError(f"q must be [tokens, a multiple of {heads}, {d}], got {tuple(q.shape)}")
    n, hq, _ = q.shape
    qs = _rows(q, "q", n, hq, d)
    store = _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, dv, kp, vp)
    select, listed = 0, None
    if pages is not None:
        listed = _index(pages, "pages", 3, dev)
        if pages.shape[0] != n or pages.shape[1] != heads or pages.shape[2] < 1:
            raise ValueError(f"pages must be [{n}, {heads}, select], got {tuple(pages.shape)}")
        select = pages.shape[2]
    if out is None:
        out = _result(q, (n, hq, dv), dtype, stream)
    else:
        _same(dev, dtype, "out", out)
        if out.shape != (n, hq, dv) or not out.is_contiguous():
            raise ValueError(f"out must be contiguous [{n}, {hq}, {dv}]")
    if lse is None:
        lse = _result(q, (n, hq), torch.float32, stream)
    else:
        _same(dev, torch.float32, "lse", lse)
        if lse.shape != (n, hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{n}, {hq}]")
    lib = _bound or _lib()
    # listed pages need no scratch
    need = lib.fastnn_attend_workspace_size(store, n, hq, max_new, select) \
        if pages is None or workspace is not None else _STATUS
    ws = _scratch(need, q, dev, workspace, "fastnn_attend_workspace_size", stream)
    _launch("fastnn_attend", dev, stream, store, q.data_ptr(), qs, n, hq, max_new, causal,
            d ** -0.5 if scale is None else scale, listed, select, out.data_ptr(), lse.data_ptr(),
            _address(ws), need)
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
    dev = _device(q)
    mean = _same(dev, q.dtype, "k_mean", k_mean)
    if k_mean.dim() != 3 or not k_mean.is_contiguous():
        raise ValueError("k_mean must be contiguous [n_pages, heads, d]")
    n_pages, heads, d = k_mean.shape
    if q.dim() != 3 or heads < 1 or q.shape[1] % heads:
        raise ValueError(f"q must be [tokens, a multiple of {heads}, {d}], got {tuple(q.shape)}")
    n, hq, _ = q.shape
    qs = _rows(q, "q", n, hq, d)
    store = _describe(code, dev, page_table, lens, cu, n_pages, heads, page, d, 8, None, None, mean)
    if out is None:
        out = _result(q, (n, heads, select), _I32, stream)
    else:
        _index(out, "out", 3, dev)
        if out.shape != (n, heads, select):
            raise ValueError(f"out must be [{n}, {heads}, {select}]")
    need = (_bound or _lib()).fastnn_select_workspace_size(store, n, hq, max_new)
    ws = _scratch(need, q, dev, workspace, "fastnn_select_workspace_size", stream)
    _launch("fastnn_select_pages", dev, stream, store, q.data_ptr(), qs, n, hq, max_new, causal,
            keep_first, keep_last, select, out.data_ptr(), _address(ws), need)
    return out
