"""Host-side checks of the token store calls (no GPU): refusals and workspace sizes."""

from __future__ import annotations

import ctypes
import weakref

import pytest
import torch

import reciprocal_nearest_neighbours_b200 as fnn
from reciprocal_nearest_neighbours_b200 import _store, build as fnn_build

P = ctypes.c_void_p
FAKE = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    fnn_build.build()
    return _store._lib()


def _desc(**kw):
    """fastnn_store as the C compiler lays it out."""
    f = dict(k_pages=FAKE, v_pages=FAKE, k_mean=FAKE, page_table=FAKE, lens=FAKE, cu=FAKE, n_pages=9,
             n_seqs=2, table_width=4, page=16, heads=2, d=64, dv=64, dtype=fnn.FASTNN_BF16)
    f.update(kw)
    return _store._STORE.pack(*(f[k] or 0 for k in (
        "k_pages", "v_pages", "k_mean", "page_table", "lens", "cu", "n_pages", "n_seqs", "table_width",
        "page", "heads", "d", "dv", "dtype")))


def _rot(**kw):
    f = dict(pos=FAKE, freq=FAKE, axes=1, rot=64, layout=0, scale=1.0)
    f.update(kw)
    return _store._ROTATION.pack(*(f[k] or 0 for k in ("pos", "freq", "axes", "rot", "layout", "scale")))


STORE_FAULTS = [
    (dict(dtype=fnn.FASTNN_I8), -2), (dict(dtype=fnn.FASTNN_F32_L2), -2), (dict(dtype=9), -2),
    (dict(d=0), -2), (dict(d=12), -2), (dict(d=136), -2), (dict(dv=4), -2), (dict(dv=256), -2),
    (dict(page=8), -2), (dict(page=48), -2), (dict(page=256), -2), (dict(page=0), -2),
    (dict(n_seqs=0), -1), (dict(n_seqs=65535), -1), (dict(heads=0), -1), (dict(heads=1025), -1),
    (dict(n_pages=0), -1), (dict(n_pages=1 << 31), -1), (dict(table_width=0), -1),
    (dict(table_width=1 << 27), -1),
]


@pytest.mark.parametrize("change,status", STORE_FAULTS)
def test_store_sizes_are_refused(lib, change, status):
    s, heads = _desc(**change), max(1, change.get("heads", 2))
    big = 1 << 40
    assert lib.fastnn_store_append(s, FAKE, 8192, FAKE, 8192, 5, 3, None, FAKE, 256, None) == status
    assert lib.fastnn_attend(s, FAKE, 8192, 5, 2 * heads, 3, 1, 1.0, None, 0, FAKE, FAKE, FAKE,
                             big, None) == status
    assert lib.fastnn_select_pages(s, FAKE, 8192, 5, 2 * heads, 3, 1, 0, 1, 4, FAKE, FAKE, big,
                                   None) == status
    assert lib.fastnn_attend_workspace_size(s, 5, 2 * heads, 3, 0) == 0
    assert lib.fastnn_select_workspace_size(s, 5, 2 * heads, 3) == 0


def test_append_refusals(lib):
    def call(s=None, k=FAKE, ks=128, v=FAKE, vs=128, n=5, m=3, r=None, ws=FAKE, nb=256):
        return lib.fastnn_store_append(s or _desc(), k, ks, v, vs, n, m, r, ws, nb, None)
    assert lib.fastnn_store_append(None, FAKE, 128, FAKE, 128, 5, 3, None, FAKE, 256, None) == -1
    assert call(n=0, k=None, v=None, ws=None) == 0  # nothing to do
    assert call(n=-1) == -1 and call(n=1 << 31) == -1 and call(m=0) == -1 and call(m=6) == -1
    assert call(k=None) == -1 and call(v=None) == -1 and call(k=FAKE + 8) == -1 and call(v=FAKE + 2) == -1
    assert call(ks=120) == -1 and call(ks=132) == -1 and call(vs=64) == -1
    assert call(ws=FAKE + 16) == -1 and call(nb=255) == -3
    for name in ("k_pages", "v_pages", "page_table", "lens", "cu"):
        assert call(_desc(**{name: None})) == -1, name
    assert call(_desc(k_pages=FAKE + 8)) == -1 and call(_desc(k_mean=FAKE + 8)) == -1
    for change, status in ((dict(axes=0), -1), (dict(axes=3), -1), (dict(rot=65), -1), (dict(rot=66), -1),
                           (dict(rot=-2), -1), (dict(axes=2, rot=6), -1), (dict(layout=2), -2),
                           (dict(pos=None), -1), (dict(freq=None), -1), (dict(scale=float("nan")), -1),
                           (dict(scale=float("inf")), -1)):
        assert call(r=_rot(**change)) == status, change


def test_rotary_refusals(lib):
    def call(x=FAKE, xs=128, n=5, heads=2, d=64, dt=fnn.FASTNN_F16, r=None, out=FAKE, os=128):
        return lib.fastnn_rotary(x, xs, n, heads, d, dt, r or _rot(), 0, out, os, None)
    assert call(n=0, x=None, out=None) == 0
    assert call(dt=fnn.FASTNN_I8) == -2 and call(d=0) == -2 and call(d=1025) == -2
    assert call(n=-1) == -1 and call(heads=0) == -1 and call(xs=127) == -1 and call(os=100) == -1
    assert call(x=None) == -1 and call(out=None) == -1 and call(x=FAKE + 1) == -1
    assert call(os=136) == -1  # in place with another stride
    assert call(r=_rot(rot=0)) == -1 and call(r=_rot(rot=66)) == -1 and call(r=_rot(layout=7)) == -2
    assert lib.fastnn_rotary(FAKE, 128, 5, 2, 64, fnn.FASTNN_F16, None, 0, FAKE, 128, None) == -1


def test_attend_refusals(lib):
    big = 1 << 40

    def call(s=None, q=FAKE, qs=256, n=5, hq=4, m=3, scale=1.0, pages=None, sel=0, out=FAKE, ws=FAKE,
             nb=big, lse=FAKE):
        return lib.fastnn_attend(s or _desc(), q, qs, n, hq, m, 1, scale, pages, sel, out, lse, ws, nb, None)
    assert call(n=0, q=None, out=None, ws=None) == 0
    assert call(hq=3) == -1 and call(hq=0) == -1 and call(m=0) == -1 and call(m=6) == -1 and call(n=-2) == -1
    assert call(q=None) == -1 and call(q=FAKE + 4) == -1 and call(qs=200) == -1 and call(qs=260) == -1
    assert call(out=None) == -1 and call(out=FAKE + 8) == -1 and call(lse=FAKE + 2) == -1
    assert call(ws=FAKE + 128) == -1 and call(nb=64) == -3
    assert call(_desc(table_width=4096), ws=None) == -1  # splits need their scratch
    assert call(scale=float("nan")) == -1 and call(scale=float("inf")) == -1
    assert call(pages=FAKE) == -1 and call(sel=4) == -1 and call(pages=FAKE, sel=-1) == -1
    for name in ("k_pages", "v_pages", "page_table", "lens", "cu"):
        assert call(_desc(**{name: None})) == -1, name


def test_select_refusals(lib):
    def call(s=None, q=FAKE, qs=256, n=5, hq=4, m=3, first=0, last=1, sel=4, out=FAKE, ws=FAKE, nb=1 << 40):
        return lib.fastnn_select_pages(s or _desc(), q, qs, n, hq, m, 1, first, last, sel, out, ws, nb, None)
    assert call(n=0, q=None, out=None, ws=None) == 0
    assert call(sel=0) == -1 and call(sel=257) == -1 and call(last=0) == -1 and call(first=-1) == -1
    assert call(first=4) == -1 and call(first=2, last=3) == -1 and call(hq=5) == -1
    assert call(out=None) == -1 and call(q=None) == -1 and call(nb=0) == -3
    assert call(_desc(table_width=513), m=1, ws=None) == -1 and call(m=2, ws=None) == -1
    assert call(_desc(k_mean=None)) == -1
    need = lib.fastnn_select_workspace_size(_desc(table_width=1 << 20), 5, 4, 3)  # a key of 8 bytes a page
    assert need >= 2 * 3 * 2 * (1 << 20) * 8 and call(_desc(table_width=1 << 20), nb=need - 1) == -3


def test_workspace_sizes(lib):
    size = lambda n, m, sel=0, **kw: lib.fastnn_attend_workspace_size(_desc(**kw), n, 4, m, sel)  # noqa: E731
    assert size(0, 0) == 256
    assert size(5, 3) % 256 == 0 and size(5, 3) >= 256
    # a long table: partial outputs of several splits, 4 bytes an element and a sum a row
    assert size(2, 1, table_width=4096, heads=1) >= 256 + 2 * 2 * 4 * (64 + 1) * 4
    assert size(5, 3, sel=-1) == 0 and size(5, 9) == 0
    assert lib.fastnn_attend_workspace_size(_desc(), 5, 3, 3, 0) == 0
    assert fnn.fastnn_attend_workspace_size(5, 4, 2, 64, 64, 2, 3, 4, 16) == size(5, 3)
    assert fnn.fastnn_attend_workspace_size(5, 4, 2, 64, 64, 2, 3, 4, 16, dtype=torch.float32) == 0


def test_tensors_must_be_16_bit_and_on_a_gpu():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    store = z(4, 2, 16, 64), z(4, 2, 16, 64), i(2, 3), i(2), i(3)
    freq = torch.zeros(4, dtype=torch.float64)
    for dtype, error in ((torch.float32, TypeError), (torch.int8, TypeError), (torch.bfloat16, ValueError)):
        with pytest.raises(error):
            fnn.fastnn_attend(z(5, 4, 64, dtype=dtype), *store, 3)
        with pytest.raises(error):
            fnn.fastnn_rotary(z(5, 4, 64, dtype=dtype), i(5), freq)
        with pytest.raises(error):
            fnn.fastnn_store_append(z(5, 2, 64, dtype=dtype), z(5, 2, 64), *store, 3)
        with pytest.raises(error):
            fnn.fastnn_select_pages(z(5, 4, 64, dtype=dtype), z(4, 2, 64), *store[2:], 3, 16, 2)
    with pytest.raises(ValueError):
        fnn.fastnn_rotary_frequencies(10, axes=2)


def test_rotary_frequencies():
    f = fnn.fastnn_rotary_frequencies(8, base=16.0, stretch=2.0, device="cpu")
    assert f.dtype == torch.float64 and f.tolist() == [0.5, 0.25, 0.125, 0.0625]
    assert fnn.fastnn_rotary_frequencies(8, base=16.0, axes=2, device="cpu").tolist() == [1.0, 0.25]
    assert fnn.fastnn_rotary_frequencies(8, long_base=81.0, device="cpu")[1].item() == pytest.approx(1 / 3)


class _Side:
    """Stands for a stream other than the current one."""
    device = torch.device("cuda", 0)
    cuda_stream = 77


@pytest.fixture
def marshalled(lib, monkeypatch):
    """Runs the binding on CPU tensors up to the launch. Yields the launches: for each the tensors
    that the call has made, as (alive at the launch, stream whose memory it is, shape, streams that
    its memory is kept for)."""
    home, current, made, launches = object(), [], [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    real = torch.Tensor.new_empty

    def new_empty(self, *args, **kw):
        t = real(self, *args, **kw)
        made.append([weakref.ref(t), current[-1] if current else home, tuple(t.shape), []])
        return t

    def record_stream(self, stream):
        for m in made:
            if m[0]() is self:
                m[3].append(stream)

    def launch(what, dev, stream, *args):
        launches.append([(ref() is not None, where, shape, tuple(kept)) for ref, where, shape, kept in made])
        made.clear()

    monkeypatch.setattr(_store, "_device", lambda t: -1)  # a CPU tensor's get_device()
    monkeypatch.setattr(_store, "_launch", launch)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: current[-1] if current else home)
    monkeypatch.setattr(torch.Tensor, "new_empty", new_empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", record_stream)
    return home, launches


@pytest.mark.parametrize("stream", [None, _Side()], ids=["current", "side"])
def test_memory_of_a_call_belongs_to_its_stream_and_is_held_until_the_launch(marshalled, stream):
    """Scratch that goes back to the allocator before the launch, or that comes from the memory of
    another stream than the launch's, may be in use by another kernel at the same time."""
    home, launches = marshalled
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    store = z(9, 2, 16, 64), z(9, 2, 16, 64), i(2, 4096), i(2), i(3)
    for new in (1, 70):  # partial outputs of splits, of the tensor-core kernel
        q = z(2 * new, 4, 64)
        out, lse = fnn.fastnn_attend(q, *store, new, stream=stream)
        pages = fnn.fastnn_select_pages(q, z(9, 2, 64), *store[2:], new, 16, 4, stream=stream)
        fnn.fastnn_attend(q, *store, new, pages=pages, stream=stream)
        fnn.fastnn_attend(q, *store, new, out=out, lse=lse, stream=stream)
        fnn.fastnn_rotary(q, i(2 * new), torch.zeros(4, dtype=torch.float64), stream=stream)
    counts = [3, 2, 2, 1, 1] * 2  # outputs and scratch
    assert [len(made) for made in launches] == counts
    for made in launches:
        for alive, where, shape, kept in made:
            assert alive, shape
            assert where is (home if stream is None else stream), shape
            if stream is not None and len(shape) > 1:  # an output: read on the current stream next
                assert kept == (home,), shape


def test_batches_beyond_what_the_kernels_count_are_refused(lib):
    """Tokens and rows are counted in 32 bits, tiles of them rounded up: every kernel's path refuses
    what does not fit, before anything is launched."""
    big, top = 1 << 60, 1 << 30

    def attend(n, hq, m, scale=1.0, pages=None, sel=0, **kw):
        s = _desc(**kw)
        return (lib.fastnn_attend(s, FAKE, 1 << 20, n, hq, m, 1, scale, pages, sel, FAKE, FAKE, FAKE, big, None),
                lib.fastnn_attend_workspace_size(s, n, hq, m, sel))
    for scale in (1.0, -1.0):  # the tensor-core kernel's calls, the other's
        for pages, sel in ((None, 0), (FAKE, 4)):
            for n, hq, m in ((top + 1, 2, 1), (top + 1, 2, top + 1), ((1 << 31) - 1, 2, (1 << 31) - 1),
                             (top, 4, top), (1 << 29, 8, 1 << 29), ((1 << 31) // 6, 12, (1 << 31) // 6)):
                assert attend(n, hq, m, scale, pages, sel) == (-1, 0), (n, hq, m)
    s = _desc()
    for n, m in ((top + 1, 1), (top + 1, top + 1), ((1 << 31) - 1, (1 << 31) - 1)):
        assert lib.fastnn_select_pages(s, FAKE, 1 << 20, n, 2, m, 1, 0, 1, 4, FAKE, FAKE, big, None) == -1
        assert lib.fastnn_select_workspace_size(s, n, 2, m) == 0
        assert lib.fastnn_store_append(s, FAKE, 8192, FAKE, 8192, n, m, None, FAKE, 256, None) == -1
    # the largest that are taken
    assert lib.fastnn_attend_workspace_size(s, top, 2, top, 0) > 0
    assert lib.fastnn_attend_workspace_size(s, top, 4, top - 9, 0) > 0
    assert lib.fastnn_select_workspace_size(s, top, 2, top) > 0


def test_index_arrays_must_be_aligned(lib):
    """An address that is no multiple of its element's size would fault on the device."""
    big = 1 << 40
    for name in ("page_table", "lens", "cu"):
        for off in (1, 2):
            s = _desc(**{name: FAKE + off})
            assert lib.fastnn_store_append(s, FAKE, 128, FAKE, 128, 5, 3, None, FAKE, 256, None) == -1, name
            assert lib.fastnn_attend(s, FAKE, 256, 5, 4, 3, 1, 1.0, None, 0, FAKE, FAKE, FAKE, big, None) == -1, name
            assert lib.fastnn_select_pages(s, FAKE, 256, 5, 4, 3, 1, 0, 1, 4, FAKE, FAKE, big, None) == -1, name
    assert lib.fastnn_attend(_desc(), FAKE, 256, 5, 4, 3, 1, 1.0, FAKE + 2, 4, FAKE, FAKE, FAKE, big, None) == -1
    for r in (_rot(pos=FAKE + 2), _rot(freq=FAKE + 4)):
        assert lib.fastnn_rotary(FAKE, 128, 5, 2, 64, fnn.FASTNN_F16, r, 0, FAKE, 128, None) == -1
        assert lib.fastnn_store_append(_desc(), FAKE, 128, FAKE, 128, 5, 3, r, FAKE, 256, None) == -1
