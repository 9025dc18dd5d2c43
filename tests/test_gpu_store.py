"""The token store on the GPU: rotary positions, append, attention, page selection, against the
plain 64-bit forms of tests/_store.py at the sizes and masks where they can go wrong."""

from __future__ import annotations

import math
import threading

import pytest
import torch

import reciprocal_nearest_neighbours_b200 as fnn
from tests import _store as ref
from tests._dev import require_cuda

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


def _randn(*shape, dtype=BF16, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# ---- rotary ------------------------------------------------------------------------------------

@pytest.mark.parametrize("n,heads,d,rot,axes,layout,dtype", [
    (1, 1, 128, 128, 1, "half", BF16),
    (5, 3, 64, 64, 2, "interleaved", F16),
    (33, 4, 24, 24, 1, "half", BF16),
    (7, 2, 24, 8, 2, "interleaved", BF16),
    (19, 5, 80, 40, 1, "interleaved", F16),
    (300, 2, 128, 64, 1, "half", BF16),
    (9, 1, 20, 12, 2, "half", F16),
    (9, 3, 7, 2, 1, "interleaved", BF16),
    (11, 2, 15, 4, 2, "half", BF16),
    (2, 1, 1024, 1024, 1, "half", F16),
    (700, 16, 64, 64, 2, "half", BF16),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(n, heads, d, rot, axes, layout, dtype, inverse):
    x = _randn(n, heads, d, dtype=dtype, seed=n + d)
    pos = torch.randint(-50, 1 << 20, (n, axes), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(d)).cuda()
    freq = fnn.fastnn_rotary_frequencies(rot, axes=axes, stretch=1.5)
    got = fnn.fastnn_rotary(x, pos, freq, layout=layout, scale=0.75, inverse=inverse)
    ref.check_rotary(got, x, pos, freq, layout, 0.75, inverse)


def test_rotary_far_positions_keep_their_angle():
    x = _randn(6, 2, 32)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32).cuda()
    freq = torch.tensor([1.0, 0.3, 1e-3, 7.0] * 4, dtype=torch.float64).cuda()
    # the reference's own angle (fp64 product, radians up to 1.5e10) is good to 2e-6 only at the
    # far end: 1.5e10 * 2^-53 = 1.7e-6, below half a step of bf16
    want, mass = ref.rotary(x.cpu(), pos.cpu(), freq.cpu())
    got = fnn.fastnn_rotary(x, pos, freq)
    tol = 2.0 ** -8 * want.abs() + 1e-5 * mass
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


def test_rotary_in_place_and_strided():
    fused = _randn(40, 3 * 8, 64, seed=3)  # queries, keys and values side by side
    pos = torch.arange(40, dtype=torch.int32).cuda()
    freq = fnn.fastnn_rotary_frequencies(48)
    before = fused.clone()
    part = fused[:, 8:16]
    got = fnn.fastnn_rotary(part, pos, freq)
    ref.check_rotary(got, before[:, 8:16], pos, freq)
    fnn.fastnn_rotary(part, pos, freq, out=part)
    assert torch.equal(part, got)
    assert torch.equal(fused[:, :8], before[:, :8]) and torch.equal(fused[:, 16:], before[:, 16:])
    # rows at an address that is no multiple of 16 bytes
    odd = torch.empty(40 * 8 * 64 + 1, dtype=BF16, device="cuda")[1:].view(40, 8, 64)
    odd.copy_(before[:, 8:16])
    assert torch.equal(fnn.fastnn_rotary(odd, pos, freq), got)


def test_rotary_inverse_is_the_gradient():
    x = _randn(12, 2, 40, seed=1)
    pos = torch.randint(0, 500, (12, 2), dtype=torch.int32).cuda()
    freq = fnn.fastnn_rotary_frequencies(32, axes=2)
    dy = _randn(12, 2, 40, seed=2)
    dx = fnn.fastnn_rotary(dy, pos, freq, layout="interleaved", scale=1.25, inverse=True).cpu().double()
    # differences of <R x, dy> in 64 bits; R is linear, so any step will do
    f = lambda z: float((ref.rotary(z, pos.cpu(), freq.cpu(), "interleaved", 1.25)[0] * dy.cpu().double()).sum())  # noqa: E731
    base = x.cpu().double()
    _, mass = ref.rotary(dy.cpu(), pos.cpu(), freq.cpu(), "interleaved", 1.25, True)
    for at in [(0, 0, 0), (3, 1, 1), (5, 0, 17), (11, 1, 31), (7, 1, 35), (2, 0, 39)]:
        up, down = base.clone(), base.clone()
        up[at] += 1.0
        down[at] -= 1.0
        want = (f(up) - f(down)) / 2
        assert abs(float(dx[at]) - want) <= 2.0 ** -8 * abs(want) + 1e-5 * float(mass[at]) + 1e-9
    assert torch.equal(fnn.fastnn_rotary(x[:0], pos[:0], freq), x[:0])


# ---- append ------------------------------------------------------------------------------------

def _append(st, rot=0, axes=1, layout="half", scale=1.0, mean=True):
    kp, vp, km, k, v, table, before, cu = st.cuda("k_pages", "v_pages", "k_mean", "k", "v", "table",
                                                  "before", "cu")
    ws = torch.full((256,), 7, dtype=torch.uint8, device="cuda")
    pos = freq = None
    if rot:
        pos = torch.randint(0, 5000, (st.n, axes), dtype=torch.int32,
                            generator=torch.Generator().manual_seed(1)).cuda()
        freq = fnn.fastnn_rotary_frequencies(rot, axes=axes)
    fnn.fastnn_store_append(k, v, kp, vp, table, before, cu, st.max_new, k_mean=km if mean else None,
                            pos=pos, freq=freq, layout=layout, scale=scale, workspace=ws)
    return kp.cpu(), vp.cpu(), km.cpu(), pos, freq, fnn.fastnn_device_status(ws)


@pytest.mark.parametrize("lens,news,page,heads,d,dv,dtype,rot,axes,layout", [
    ([0], [1], 16, 1, 8, 8, BF16, 8, 1, "half"),
    ([0, 5, 16, 31], [1, 1, 1, 1], 16, 2, 64, 64, F16, 64, 1, "interleaved"),
    ([3, 0, 130, 64], [70, 0, 129, 1], 64, 3, 128, 128, BF16, 64, 1, "half"),
    ([127, 0], [300, 17], 128, 1, 24, 8, BF16, 24, 2, "half"),
    ([33, 12], [40, 100], 32, 2, 72, 16, F16, 20, 1, "half"),
    ([9, 64, 0], [55, 64, 2], 64, 2, 40, 128, BF16, 0, 1, "half"),
    ([1, 2], [31, 33], 16, 2, 128, 64, F16, 12, 2, "interleaved"),
])
def test_append(lens, news, page, heads, d, dv, dtype, rot, axes, layout):
    st = ref.Store(lens, news, page, heads, d, dv, dtype, seed=sum(news), tail=3)
    kp, vp, km, pos, freq, status = _append(st, rot, axes, layout, scale=1.5)
    assert status == 0
    placed = torch.zeros(st.n_pages, page, dtype=torch.bool)
    touched = {}
    for s in range(len(lens)):
        a = int(st.cu[s])
        for i in range(news[s]):
            p = lens[s] + i
            ph, row = int(st.table[s, p // page]), p % page
            placed[ph, row] = True
            touched[ph] = row + 1  # rows are filled in order
            assert torch.equal(vp[ph, :, row], st.v[a + i])
            if not rot:
                assert torch.equal(kp[ph, :, row], st.k[a + i])
            else:
                ref.check_rotary(kp[ph, :, row][None], st.k[a + i][None], pos[a + i][None], freq,
                                 layout, 1.5)
    away = ~placed[:, None, :].expand(-1, heads, -1)
    assert torch.equal(kp[away], st.k_pages[away]) and torch.equal(vp[away], st.v_pages[away])
    for ph in range(st.n_pages):
        if ph not in touched:
            assert torch.equal(km[ph], st.k_mean[ph])
            continue
        held = kp[ph, :, :touched[ph]].double()  # a sum of up to 128 fp32 terms, a quotient, a rounding
        want, mass = held.mean(1), held.abs().mean(1)
        tol = ref.U[dtype] * want.abs() + 130 * ref.U32 * mass + ref.TINY[dtype]
        assert bool(((km[ph].double() - want).abs() <= tol).all())


def test_append_without_mean_and_from_a_fused_projection():
    st = ref.Store([10, 3], [20, 5], 16, 2, 64, 64, BF16, seed=4)
    fused = torch.randn(st.n, 6, 64).to(BF16)
    st.k, st.v = fused[:, 2:4], fused[:, 4:6]
    gpu = fused.cuda()
    kp, vp, km, table, before, cu = st.cuda("k_pages", "v_pages", "k_mean", "table", "before", "cu")
    fnn.fastnn_store_append(gpu[:, 2:4], gpu[:, 4:6], kp, vp, table, before, cu, st.max_new)
    st.k, st.v = st.k.contiguous(), st.v.contiguous()
    kq, vq, kn, _, _, status = _append(st, mean=False)
    assert status == 0
    assert torch.equal(kp.cpu(), kq) and torch.equal(vp.cpu(), vq) and torch.equal(kn, st.k_mean)


@pytest.mark.parametrize("fault", ["hole", "table", "max_new", "negative", "id"])
def test_append_reports_tokens_without_a_place(fault):
    st = ref.Store([10, 30, 0], [10, 10, 40], 16, 1, 16, 16, BF16, seed=5)
    lost = {}
    if fault == "hole":
        st.table[1, 2] = -1
        lost = {1: range(2, 10)}      # positions 32 .. 39
    elif fault == "id":
        st.table[1, 2] = st.n_pages
        lost = {1: range(2, 10)}
    elif fault == "table":
        st.before[2] = 20             # 60 positions in a table of 3 pages
        st.table[2] = torch.tensor([int(x) for x in st.table[2]])
        lost = {2: range(28, 40)}
    elif fault == "max_new":
        st.max_new = 20
        lost = {2: range(20, 40)}
    else:
        st.before[0] = -4
        lost = {0: range(0, 10)}
    kp, vp, _, _, _, status = _append(st)
    assert status == -1
    for s in range(3):
        a = int(st.cu[s])
        for i in range(int(st.cu[s + 1]) - a):
            if i in lost.get(s, ()):
                continue
            p = int(st.before[s]) + i
            ph = int(st.table[s, p // 16])
            assert torch.equal(kp[ph, :, p % 16], st.k[a + i]), (s, i)
    st2 = ref.Store([10, 30, 0], [10, 10, 40], 16, 1, 16, 16, BF16, seed=5)
    assert _append(st2)[5] == 0  # the word is written anew by every call
    changed = int((kp != st.k_pages).any(-1).any(1).sum())
    assert changed <= 60 - sum(len(r) for r in lost.values())


# ---- attention ---------------------------------------------------------------------------------

def _attend(st, causal=True, scale=None, pages=None):
    q, kp, vp, table, lens, cu = st.cuda("q", "k_pages", "v_pages", "table", "lens", "cu")
    out = torch.full((st.n, st.heads * st.group, st.dv), 9.0, dtype=st.dtype, device="cuda")
    lse = torch.full((st.n, st.heads * st.group), 9.0, device="cuda")
    select = 0 if pages is None else pages.shape[2]
    need = fnn.fastnn_attend_workspace_size(st.n, st.heads * st.group, st.heads, st.d, st.dv, len(st.lens),
                                            st.max_new, st.width, st.page, select)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = fnn.fastnn_attend(q, kp, vp, table, lens, cu, st.max_new, causal=causal, scale=scale,
                            pages=None if pages is None else pages.cuda(), out=out, lse=lse,
                            workspace=ws)
    assert got[0] is out and got[1] is lse
    assert fnn.fastnn_device_status(ws) == 0
    end = int(st.cu[-1])
    assert bool((out[end:] == 9).all()) and bool((lse[end:] == 9).all())  # behind the last sequence
    return out, lse


ATTEND = [
    # lens before, new, page, heads, group, d, dv, dtype
    ([0], [1], 16, 1, 1, 8, 8, BF16),
    ([37], [1], 16, 2, 4, 64, 64, F16),
    ([0, 200, 15, 16], [1, 1, 1, 1], 32, 2, 8, 128, 128, BF16),
    ([100, 0, 7], [1, 0, 30], 16, 1, 7, 24, 8, BF16),
    ([64, 3], [40, 70], 64, 3, 1, 64, 64, F16),
    ([130], [129], 128, 1, 2, 72, 40, BF16),
    ([5, 300], [33, 3], 64, 2, 16, 96, 128, F16),
    ([20], [20], 16, 1, 33, 16, 24, BF16),
    ([0], [150], 64, 1, 1, 128, 128, BF16),
    ([0], [300], 32, 1, 2, 32, 32, F16),
    ([70], [257], 64, 1, 1, 40, 128, F16),
    ([10, 500, 0, 90], [130, 128, 1, 255], 16, 2, 1, 64, 64, BF16),
]


@pytest.mark.parametrize("lens,news,page,heads,group,d,dv,dtype", ATTEND)
@pytest.mark.parametrize("causal", [True, False])
def test_attend(lens, news, page, heads, group, d, dv, dtype, causal):
    st = ref.Store(lens, news, page, heads, d, dv, dtype, seed=d + group, group=group, tail=2)
    out, lse = _attend(st, causal)
    ref.check_attend(out, lse, st, causal)


@pytest.mark.parametrize("lens,news,group,d,dtype", [
    ([5000, 200], [70, 66], 1, 64, BF16),      # lone query tiles, many key tiles, divided between blocks
    ([9000], [128], 1, 128, F16),
    ([300, 130, 0, 60], [100, 64, 128, 80], 1, 128, BF16),
    ([2000, 126], [200, 129], 1, 64, F16),     # a pair, and a lone tile of a few rows
    ([700, 3000], [40, 33], 2, 32, BF16),
])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_few_query_tiles_many_keys(lens, news, group, d, dtype, causal):
    st = ref.Store(lens, news, 64, 2, d, d, dtype, seed=d + group, group=group, tail=1)
    out, lse = _attend(st, causal)
    ref.check_attend(out, lse, st, causal)
    again = _attend(st, causal)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("news", [[1, 1], [60, 200]])
def test_attend_rows_that_see_nothing(news):
    """Sequences of no length, and a batch that claims more new tokens than the store holds."""
    st = ref.Store([0, 0], news, 16, 2, 64, 64, BF16, group=2, seed=1)
    st.lens = torch.tensor([0, max(0, news[1] - 20)], dtype=torch.int32)
    out, lse = _attend(st)
    ref.check_attend(out, lse, st)
    out, lse = _attend(st, causal=False)
    ref.check_attend(out, lse, st, causal=False)
    st.lens = torch.tensor([-5, -2 ** 31], dtype=torch.int32)
    out, lse = _attend(st)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("news", [[1, 1, 1], [40, 3, 140]])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attend_ignores_what_lies_behind_the_length(news, dtype):
    """NaN and infinities in every row of the pages that no token sees, and in spare pages."""
    st = ref.Store([10, 64, 33], news, 64, 2, 64, 64, dtype, seed=2, group=2)
    used = torch.zeros(st.n_pages, st.page, dtype=torch.bool)
    for s in range(3):
        for ph, r in st.positions(s, upto=int(st.lens[s])):
            used[ph, r] = True
    bad = ~used[:, None, :].expand(-1, 2, -1)
    st.k_pages[bad] = float("nan")
    st.v_pages[bad] = float("inf")
    out, lse = _attend(st)
    ref.check_attend(out, lse, st)


def test_attend_holes_and_short_tables():
    st = ref.Store([100, 50], [3, 140], 16, 1, 64, 64, BF16, seed=3, group=2)
    st.table[0, 2] = -1
    st.table[0, 5] = st.n_pages + 100
    st.table[1, 0] = -7
    out, lse = _attend(st)
    ref.check_attend(out, lse, st)
    st.table[1, :] = -1  # a sequence of holes only
    out, lse = _attend(st)
    ref.check_attend(out, lse, st)
    short = ref.Store([100], [30], 16, 1, 64, 64, BF16, seed=3, width=3)  # 48 of 130 positions exist
    out, lse = _attend(short)
    ref.check_attend(out, lse, short)


def test_attend_scores_of_any_size():
    """Large scores (one weight is 1), scale 0 (a plain mean), a negative scale."""
    for scale in (30.0, 0.0, -1.0, 1e-3):
        for news in ([1, 5], [130, 140]):
            st = ref.Store([150, 20], news, 32, 1, 64, 64, BF16, seed=8, group=2)
            out, lse = _attend(st, scale=scale)
            ref.check_attend(out, lse, st, scale=scale)


def test_attend_takes_max_new_tokens():
    st = ref.Store([9, 9], [30, 4], 16, 1, 32, 32, F16, seed=6)
    st.max_new = 8
    q, kp, vp, table, lens, cu = st.cuda("q", "k_pages", "v_pages", "table", "lens", "cu")
    out = torch.full((st.n, 1, 32), 9.0, dtype=F16, device="cuda")
    fnn.fastnn_attend(q, kp, vp, table, lens, cu, 8, out=out)
    assert bool((out[8:30] == 9).all()) and not bool((out[:8] == 9).all(-1).any())
    assert not bool((out[30:] == 9).all(-1).any())


@pytest.mark.parametrize("dtype,group", [(BF16, 4), (F16, 1)])
def test_attend_long_ragged_steps_split(dtype, group):
    """Lengths over many splits, from one position to a split's border and one past it."""
    lens = [0, 255, 256, 257, 511, 2000, 2047, 2999]
    st = ref.Store(lens, [1] * 8, 64, 1, 64, 64, dtype, seed=11, group=group)
    out, lse = _attend(st)
    ref.check_attend(out, lse, st)
    again = _attend(st)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # the same bits


# ---- selected pages ----------------------------------------------------------------------------

SELECT = [
    # lens, news, page, heads, group, d, dtype, select, first, last
    ([40], [1], 16, 1, 1, 64, BF16, 2, 0, 1),
    ([1000, 3, 0, 700], [1, 1, 1, 1], 16, 2, 4, 128, BF16, 8, 1, 2),
    ([200, 90], [20, 33], 16, 2, 3, 24, F16, 4, 0, 1),
    ([900], [150], 32, 1, 16, 64, F16, 16, 2, 3),
    ([100], [5], 64, 1, 20, 40, BF16, 7, 7, 0 + 1),
]


@pytest.mark.parametrize("lens,news,page,heads,group,d,dtype,select,first,last", SELECT)
@pytest.mark.parametrize("causal", [True, False])
def test_select_and_attend(lens, news, page, heads, group, d, dtype, select, first, last, causal):
    first = min(first, select - last)
    st = ref.Store(lens, news, page, heads, d, d, dtype, seed=select, group=group, tail=1)
    q, km, table, ln, cu = st.cuda("q", "k_mean", "table", "lens", "cu")
    pages = torch.full((st.n, heads, select), -9, dtype=torch.int32, device="cuda")
    fnn.fastnn_select_pages(q, km, table, ln, cu, st.max_new, page, select, keep_first=first,
                            keep_last=last, causal=causal, out=pages)
    want = ref.select_pages(st, st.k_mean, select, first, last, causal)
    assert torch.equal(pages.cpu(), want)
    out, lse = _attend(st, causal, pages=pages)
    ref.check_attend(out, lse, st, causal, pages=want)


def test_select_ties_holes_and_nan():
    st = ref.Store([400], [60], 16, 2, 16, 16, BF16, seed=9, group=2)
    for p in range(0, 26, 3):
        st.k_mean[st.table[0, p].item()] = st.k_mean[st.table[0, 0].item()]  # equal scores
    st.k_mean[st.table[0, 4].item(), 0, 3] = float("nan")
    st.k_mean[st.table[0, 5].item(), 1] = float("inf")
    st.table[0, 7] = -1
    st.table[0, 8] = st.n_pages
    q, km, table, ln, cu = st.cuda("q", "k_mean", "table", "lens", "cu")
    for select, first, last in ((6, 0, 1), (3, 1, 1), (28, 0, 1), (40, 2, 2), (1, 0, 1)):
        got = fnn.fastnn_select_pages(q, km, table, ln, cu, st.max_new, 16, select,
                                      keep_first=first, keep_last=last)
        assert torch.equal(got.cpu(), ref.select_pages(st, st.k_mean, select, first, last)), select


def test_select_zero_queries_take_the_lowest_pages():
    st = ref.Store([320], [4], 16, 1, 32, 32, F16, seed=1)
    st.q.zero_()
    q, km, table, ln, cu = st.cuda("q", "k_mean", "table", "lens", "cu")
    got = fnn.fastnn_select_pages(q, km, table, ln, cu, 4, 16, 5)
    assert got[:, 0].tolist() == [[0, 1, 2, 3, 20]] * 4


def test_attend_listed_pages_twice_out_of_range_and_none():
    st = ref.Store([100, 40], [3, 2], 16, 1, 64, 64, BF16, seed=7, group=3)
    pages = torch.tensor([[0, 0, 2], [-1, 6, 99], [3, -5, 3], [1, 2, 2 ** 30], [-1, -1, -1]],
                         dtype=torch.int32)[:, None]
    st.table[1, 2] = -1
    out, lse = _attend(st, pages=pages)
    ref.check_attend(out, lse, st, pages=pages)


def test_attend_all_pages_listed_is_attention():
    st = ref.Store([300], [20], 32, 2, 64, 64, F16, seed=12, group=2)
    every = torch.arange(10, dtype=torch.int32).expand(20, 2, 10).contiguous()
    out, lse = _attend(st, pages=every)
    ref.check_attend(out, lse, st, pages=every)
    ref.check_attend(out, lse, st)


# ---- together ----------------------------------------------------------------------------------

def test_stream_of_images():
    """Images of two streams come one after another: queries and keys rotated by the pixels' x and
    y, keys appended, every new token matched with all its stream holds, then with chosen pages."""
    heads, group, d, page, dtype = 2, 2, 32, 16, BF16
    shapes = [[(4, 6), (3, 5)], [(4, 6), (1, 1)], [(5, 5), (7, 3)]]
    st = ref.Store([0, 0], [sum(h * w for h, w in (a[0] for a in shapes)),
                            sum(h * w for h, w in (a[1] for a in shapes))], page, heads, d, d, dtype)
    kp, vp, km = (torch.zeros_like(t).cuda() for t in (st.k_pages, st.v_pages, st.k_mean))
    table = st.table.cuda()
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    freq = fnn.fastnn_rotary_frequencies(32, base=100.0, axes=2)
    history = [[], []]
    for r, (one, two) in enumerate(shapes):
        news = [one[0] * one[1], two[0] * two[1]]
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32).cuda()
        pos = torch.cat([torch.cartesian_prod(torch.arange(w), torch.arange(h)) for h, w in (one, two)])
        pos = pos.to(torch.int32).cuda()
        n = sum(news)
        q, k, v = (_randn(n, hh, d, seed=10 * r + i) for i, hh in enumerate((heads * group, heads, heads)))
        qr = fnn.fastnn_rotary(q, pos, freq)
        fnn.fastnn_store_append(k, v, kp, vp, table, lens, cu, max(news), k_mean=km, pos=pos, freq=freq)
        lens += cu[1:] - cu[:-1]
        out, lse = fnn.fastnn_attend(qr, kp, vp, table, lens, cu, max(news), causal=False)
        pages = fnn.fastnn_select_pages(qr, km, table, lens, cu, max(news), page, 2, causal=False)
        sparse = fnn.fastnn_attend(qr, kp, vp, table, lens, cu, max(news), causal=False, pages=pages)
        # the store as the reference sees it, and the rotated queries
        ref.check_rotary(qr, q, pos, freq)
        st.q, st.n, st.group = qr.cpu(), n, group
        st.k_pages, st.v_pages, st.lens, st.cu = kp.cpu(), vp.cpu(), lens.cpu(), cu.cpu()
        ref.check_attend(out, lse, st, causal=False)
        want = ref.select_pages(st, km.cpu(), 2, 0, 1, causal=False)
        assert torch.equal(pages.cpu(), want)
        ref.check_attend(sparse[0], sparse[1], st, causal=False, pages=want)
        for s in range(2):
            history[s].append((k[cu[s]:cu[s + 1]], v[cu[s]:cu[s + 1]], pos[cu[s]:cu[s + 1]]))
            keys = torch.cat([h[0] for h in history[s]])
            ps = torch.cat([h[2] for h in history[s]])
            at = st.positions(s, upto=int(lens[s]))
            held = torch.stack([st.k_pages[ph, :, row] for ph, row in at])
            ref.check_rotary(held, keys, ps, freq)
            vals = torch.cat([h[1] for h in history[s]]).cpu()
            assert torch.equal(torch.stack([st.v_pages[ph, :, row] for ph, row in at]), vals)


@pytest.mark.parametrize("news", [[1, 1], [200, 130]])
def test_captured_step_follows_the_store(news):
    """A captured graph of rotary, append, select and attend reads lengths, tables and tokens anew
    at every replay; two graphs with workspaces of their own run on two streams at once."""
    st = ref.Store([700, 30], news, 16, 2, 64, 64, BF16, seed=21, group=2)
    freq = fnn.fastnn_rotary_frequencies(64)

    class Step:
        def __init__(self):
            (self.q, self.kp, self.vp, self.km, self.table, self.before, self.cu, self.k, self.v) = \
                st.cuda("q", "k_pages", "v_pages", "k_mean", "table", "before", "cu", "k", "v")
            need = fnn.fastnn_attend_workspace_size(st.n, 4, 2, 64, 64, 2, st.max_new, st.width, 16)
            self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            self.lens = torch.zeros_like(self.before)
            self.pos = torch.zeros(st.n, dtype=torch.int32, device="cuda")
            self.out = torch.zeros(st.n, 4, 64, dtype=BF16, device="cuda")
            self.lse = torch.zeros(st.n, 4, device="cuda")

        def run(self):
            self.qr = fnn.fastnn_rotary(self.q, self.pos, freq)
            fnn.fastnn_store_append(self.k, self.v, self.kp, self.vp, self.table, self.before, self.cu,
                                    st.max_new, k_mean=self.km, pos=self.pos, freq=freq)
            torch.add(self.before, self.cu[1:] - self.cu[:-1], out=self.lens)
            self.pages = fnn.fastnn_select_pages(self.qr, self.km, self.table, self.lens, self.cu,
                                                 st.max_new, 16, 6)
            self.sparse = fnn.fastnn_attend(self.qr, self.kp, self.vp, self.table, self.lens, self.cu,
                                            st.max_new, pages=self.pages)
            fnn.fastnn_attend(self.qr, self.kp, self.vp, self.table, self.lens, self.cu, st.max_new,
                              out=self.out, lse=self.lse, workspace=self.ws)

    steps, graphs, streams = [Step(), Step()], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, stream in zip(steps, streams):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            x.run()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            x.run()
        graphs.append(g)
    for r, before in enumerate(([700, 30], [3, 400], [0, 0])):
        for i, x in enumerate(steps):
            x.before.copy_(torch.tensor(before if i == 0 else before[::-1], dtype=torch.int32))
            x.pos.copy_(torch.randint(0, 999, (st.n,), dtype=torch.int32))
            x.q.copy_(_randn(st.n, 4, 64, seed=50 + 2 * r + i))
            if i == 1:
                x.table.copy_(st.table.flip(0))
        torch.cuda.synchronize()
        for stream, g in zip(streams, graphs):
            with torch.cuda.stream(stream):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(steps):
            have = ref.Store([0, 0], news, 16, 2, 64, 64, BF16, group=2)
            have.n_pages, have.width, have.table = st.n_pages, st.width, x.table.cpu()
            have.k_pages, have.v_pages, have.q = x.kp.cpu(), x.vp.cpu(), x.qr.cpu()
            have.lens, have.n = x.lens.cpu(), st.n
            assert have.lens.tolist() == [a + b for a, b in zip(x.before.tolist(), news)]
            ref.check_attend(x.out, x.lse, have)
            want = ref.select_pages(have, x.km.cpu(), 6, 0, 1)
            assert torch.equal(x.pages.cpu(), want)
            ref.check_attend(x.sparse[0], x.sparse[1], have, pages=want)


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """The tensor-core kernel's bounded waits, with a limit far below the call's duration: the call
    ends, its status says so, and the next one on the same workspace is right."""
    st = ref.Store([300, 0], [140, 200], 64, 2, 64, 64, BF16, seed=31, group=2)
    q, kp, vp, table, lens, cu = st.cuda("q", "k_pages", "v_pages", "table", "lens", "cu")
    need = fnn.fastnn_attend_workspace_size(st.n, 4, 2, 64, 64, 2, st.max_new, st.width, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    fnn.fastnn_set_wait_timeout_ns(200)
    try:
        fnn.fastnn_attend(q, kp, vp, table, lens, cu, st.max_new, workspace=ws)
        assert fnn.fastnn_device_status(ws) == -5
    finally:
        fnn.fastnn_set_wait_timeout_ns(0)
    out, lse = fnn.fastnn_attend(q, kp, vp, table, lens, cu, st.max_new, workspace=ws)
    assert fnn.fastnn_device_status(ws) == 0
    ref.check_attend(out, lse, st)


@pytest.mark.parametrize("news", [[1, 1], [90, 200]])
def test_queries_as_part_of_a_fused_projection(news):
    st = ref.Store([77, 5], news, 32, 2, 64, 64, F16, seed=32, group=2)
    fused = torch.zeros(st.n, 8, 64, dtype=F16, device="cuda")
    fused[:, 2:6] = st.q.cuda()
    fused[:, :2] = fused[:, 6:] = float("nan")
    kp, vp, km, table, lens, cu = st.cuda("k_pages", "v_pages", "k_mean", "table", "lens", "cu")
    out, lse = fnn.fastnn_attend(fused[:, 2:6], kp, vp, table, lens, cu, st.max_new)
    ref.check_attend(out, lse, st)
    pages = fnn.fastnn_select_pages(fused[:, 2:6], km, table, lens, cu, st.max_new, 32, 3)
    assert torch.equal(pages.cpu(), ref.select_pages(st, st.k_mean, 3, 0, 1))
    again = fnn.fastnn_attend(fused[:, 2:6], kp, vp, table, lens, cu, st.max_new)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # the same bits


def test_no_new_tokens():
    """Calls without a token do nothing, and batches whose sequences all lack one."""
    st = ref.Store([40, 3], [20, 5], 16, 2, 64, 64, BF16, seed=35, group=2)
    q, k, v, kp, vp, km, table, before, lens = st.cuda("q", "k", "v", "k_pages", "v_pages", "k_mean", "table",
                                                       "before", "lens")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    fnn.fastnn_store_append(k[:0], v[:0], kp, vp, table, before, zero, 0, k_mean=km)
    out, lse = fnn.fastnn_attend(q[:0], kp, vp, table, lens, zero, 0)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert fnn.fastnn_select_pages(q[:0], km, table, lens, zero, 0, 16, 3).shape == (0, 2, 3)
    for new in (1, 20):  # rows of no sequence stay as they are, in every kernel
        fnn.fastnn_store_append(k, v, kp, vp, table, before, zero, new, k_mean=km)
        out = torch.full((25, 4, 64), 9.0, dtype=BF16, device="cuda")
        fnn.fastnn_attend(q, kp, vp, table, lens, zero, new, out=out)
        pages = torch.full((25, 2, 3), -9, dtype=torch.int32, device="cuda")
        fnn.fastnn_select_pages(q, km, table, lens, zero, new, 16, 3, out=pages)
        listed = torch.zeros(25, 2, 3, dtype=torch.int32, device="cuda")
        fnn.fastnn_attend(q, kp, vp, table, lens, zero, new, out=out, pages=listed)
        assert bool((out == 9).all()) and bool((pages == -9).all())
    assert torch.equal(kp.cpu(), st.k_pages) and torch.equal(vp.cpu(), st.v_pages) and torch.equal(km.cpu(), st.k_mean)


def test_index_arrays_that_make_no_sense_are_survived():
    """Decreasing and negative offsets, offsets past the batch, lengths past the table: nothing is
    read or written out of range, and the well-formed sequence is answered."""
    for new in (2, 40):
        st = ref.Store([30, 20, 10], [new] * 3, 16, 1, 64, 64, BF16, seed=36, group=2)
        q, k, v, kp, vp, km, table = st.cuda("q", "k", "v", "k_pages", "v_pages", "k_mean", "table")
        for cu in ([0, new, -5, 3 * new], [0, new, new, 10 ** 9], [0, new, 2 ** 31 - 1, -2 ** 31],
                   [0, new, 3 * new + 7, 3 * new + 9]):
            bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
            lens = torch.tensor([30 + new, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
            out, lse = fnn.fastnn_attend(q, kp, vp, table, lens, bad, new)
            pages = fnn.fastnn_select_pages(q, km, table, lens, bad, new, 16, 3)
            listed = fnn.fastnn_attend(q, kp, vp, table, lens, bad, new, pages=pages)
            torch.cuda.synchronize()
            good = ref.Store([30], [new], 16, 1, 64, 64, BF16, group=2)
            good.table, good.width, good.n_pages = st.table[:1], st.width, st.n_pages
            good.k_pages, good.v_pages, good.q = st.k_pages, st.v_pages, st.q[:new]
            ref.check_attend(out[:new], lse[:new], good)
            want = ref.select_pages(good, st.k_mean, 3, 0, 1)
            assert torch.equal(pages[:new].cpu(), want)
            ref.check_attend(listed[0][:new], listed[1][:new], good, pages=want)
            ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
            fnn.fastnn_store_append(k, v, kp.clone(), vp.clone(), table, lens, bad, new, k_mean=km.clone(), workspace=ws)
            assert fnn.fastnn_device_status(ws) == -1


def test_many_sequences_at_once():
    """More sequences than one launch of the tensor-core kernel plans for, most without a token."""
    seqs = 700
    news = [(70 if s % 101 == 0 else 0) for s in range(seqs)]
    lens = [s % 50 for s in range(seqs)]
    st = ref.Store(lens, news, 16, 1, 16, 16, BF16, seed=33)
    out, lse = _attend(st)
    ref.check_attend(out, lse, st)
    one = ref.Store(lens, [1] * seqs, 16, 1, 16, 16, BF16, seed=34)
    out, lse = _attend(one)
    ref.check_attend(out, lse, one)
    q, km, table, ln, cu = one.cuda("q", "k_mean", "table", "lens", "cu")
    got = fnn.fastnn_select_pages(q, km, table, ln, cu, 1, 16, 2)
    assert torch.equal(got.cpu(), ref.select_pages(one, one.k_mean, 2, 0, 1))


def test_select_over_many_pages():
    """Tables wider than a block's registers (4096 pages), and between the kernels' borders."""
    for width, news, dtype in ((4200, [1], BF16), (4200, [9], F16), (1100, [3], BF16), (513, [12], F16),
                               (512, [7], BF16)):
        st = ref.Store([width * 16 - 40], news, 16, 1, 16, 16, dtype, seed=width, group=2)
        q, km, table, ln, cu = st.cuda("q", "k_mean", "table", "lens", "cu")
        got = fnn.fastnn_select_pages(q, km, table, ln, cu, news[0], 16, 200, keep_first=2, keep_last=3)
        assert torch.equal(got.cpu(), ref.select_pages(st, st.k_mean, 200, 2, 3)), width


def test_another_stream_than_the_current_one():
    st = ref.Store([500], [30], 16, 1, 64, 64, F16, seed=22, group=2)
    q, kp, vp, table, lens, cu = st.cuda("q", "k_pages", "v_pages", "table", "lens", "cu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = fnn.fastnn_attend(q, kp, vp, table, lens, cu, 30)
    got = fnn.fastnn_attend(q, kp, vp, table, lens, cu, 30, stream=side)
    for _ in range(8):  # memory that the call's own workspace must not share
        torch.full((1 << 20,), 5, dtype=torch.uint8, device="cuda")
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_pages_far_apart_in_a_large_store():
    """Page ids whose element offsets pass 32 bits: 2^31 elements and more."""
    page, heads, d = 128, 8, 128
    n_pages = (1 << 31) // (page * heads * d) + 64
    st = ref.Store([300], [40], page, 1, d, d, BF16, seed=23)
    kp = torch.zeros(n_pages, heads, page, d, dtype=BF16, device="cuda")
    vp = torch.zeros(n_pages, heads, page, d, dtype=BF16, device="cuda")
    far = torch.tensor([[n_pages - 1, n_pages - 7, n_pages - 3]], dtype=torch.int32)
    for p in range(3):
        for h in (0, 7):
            kp[int(far[0, p]), h] = st.k_pages[int(st.table[0, p]), 0].cuda()
            vp[int(far[0, p]), h] = st.v_pages[int(st.table[0, p]), 0].cuda()
    k = torch.zeros(40, heads, d, dtype=BF16)
    v = torch.zeros(40, heads, d, dtype=BF16)
    q = torch.zeros(40, heads, d, dtype=BF16)
    for h in (0, 7):
        k[:, h], v[:, h], q[:, h] = st.k[:, 0], st.v[:, 0], st.q[:, 0]
    before, cu, lens = st.cuda("before", "cu", "lens")
    fnn.fastnn_store_append(k.cuda(), v.cuda(), kp, vp, far.cuda(), before, cu, 40)
    out, lse = fnn.fastnn_attend(q.cuda(), kp, vp, far.cuda(), lens, cu, 40)
    for i in range(40):
        ph, row = int(st.table[0, (300 + i) // page]), (300 + i) % page
        st.k_pages[ph, 0, row], st.v_pages[ph, 0, row] = st.k[i, 0], st.v[i, 0]
    for h in (0, 7):
        ref.check_attend(out[:, h:h + 1], lse[:, h:h + 1], st)


def test_refusals_of_shapes_types_and_devices():
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    kp, vp, table, lens, cu = z(4, 2, 16, 64), z(4, 2, 16, 64), i(2, 3), i(2), i(3)
    q, freq = z(5, 4, 64), torch.zeros(4, dtype=torch.float64, device="cuda")
    for args in ((q, kp.half(), vp, table, lens, cu), (q, kp, vp.half(), table, lens, cu)):
        with pytest.raises(TypeError):
            fnn.fastnn_attend(*args, 3)
    for args in ((z(5, 3, 64), kp, vp, table, lens, cu), (q, kp, z(4, 2, 32, 64), table, lens, cu),
                 (q, kp, vp, table.long(), lens, cu), (q, kp, vp, table, i(3), cu), (q, kp, vp, table, lens, i(4)),
                 (q, kp, vp, table.cpu(), lens, cu), (q, kp.cpu(), vp, table, lens, cu),
                 (z(5, 4, 128)[:, :, ::2], kp, vp, table, lens, cu),
                 (z(5, 64, 4).transpose(1, 2), kp, vp, table, lens, cu),
                 (q, kp[:, :, :, :32], vp, table, lens, cu), (q, kp, vp, table[:, ::2], lens, cu)):
        with pytest.raises(ValueError):
            fnn.fastnn_attend(*args, 3)
    for kw in (dict(pages=i(5, 4, 2)), dict(pages=i(5, 2, 2).long()), dict(out=z(5, 4, 32)), dict(lse=z(5, 4)),
               dict(out=z(5, 64, 4).transpose(1, 2)), dict(workspace=torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            fnn.fastnn_attend(q, kp, vp, table, lens, cu, 3, **kw)
    for new in (0, 6):
        with pytest.raises(fnn.FastNNError):
            fnn.fastnn_attend(q, kp, vp, table, lens, cu, new)
    with pytest.raises(fnn.FastNNError):  # a workspace too small
        fnn.fastnn_attend(q, kp, vp, table, lens, cu, 3, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fnn.FastNNError):  # rows at an address that is no multiple of 16 bytes
        fnn.fastnn_attend(z(5 * 4 * 64 + 1)[1:].view(5, 4, 64), kp, vp, table, lens, cu, 3)
    for kw in (dict(pos=i(4), freq=freq), dict(pos=i(5, 3), freq=freq), dict(pos=i(5), freq=freq.float()),
               dict(pos=i(5), freq=freq, layout="quarter"), dict(pos=i(5).long(), freq=freq)):
        with pytest.raises(ValueError):
            fnn.fastnn_rotary(q, **kw)
    with pytest.raises(ValueError):
        fnn.fastnn_store_append(z(5, 2, 64), z(5, 2, 64), kp, vp, table, lens, cu, 3, pos=i(5))
    with pytest.raises(ValueError):
        fnn.fastnn_store_append(z(5, 2, 64), z(4, 2, 64), kp, vp, table, lens, cu, 3)
    with pytest.raises(ValueError):
        fnn.fastnn_store_append(z(5, 2, 64), z(5, 2, 64), kp, vp, table, lens, cu, 3, k_mean=z(4, 2, 32))
    with pytest.raises(fnn.FastNNError):
        fnn.fastnn_select_pages(q, z(4, 2, 64), table, lens, cu, 3, 16, 2, keep_first=2)
    with pytest.raises(ValueError):
        fnn.fastnn_select_pages(q, z(4, 3, 64), table, lens, cu, 3, 16, 2)


# ---- calls at the same time --------------------------------------------------------------------

def _twins(lens, news, seed):
    """Two stores of the same sizes with other contents, on the GPU, and what each call on them
    answers by itself (attention, chosen pages, attention over them)."""
    both = []
    for i in range(2):
        st = ref.Store(lens, news, 16, 2, 64, 64, BF16, seed=seed + i, group=2)
        args = st.cuda("q", "k_pages", "v_pages", "table", "lens", "cu")
        km = st.k_mean.cuda()

        def calls(stream=None, args=args, km=km, st=st):
            q, kp, vp, table, ln, cu = args
            pages = fnn.fastnn_select_pages(q, km, table, ln, cu, st.max_new, 16, 6, stream=stream)
            return (*fnn.fastnn_attend(*args, st.max_new, stream=stream), pages,
                    *fnn.fastnn_attend(*args, st.max_new, pages=pages, stream=stream))
        want = calls()
        ref.check_attend(want[0], want[1], st)
        assert torch.equal(want[2].cpu(), ref.select_pages(st, st.k_mean, 6, 0, 1))
        both.append((calls, want))
    torch.cuda.synchronize()
    return both


BATCHES = [([9000, 3000], [1, 1]), ([700, 300], [130, 70])]  # partial outputs of splits, of shares


@pytest.mark.parametrize("lens,news", BATCHES)
def test_a_call_on_another_stream_right_after_one_on_the_current(lens, news):
    (here, want_here), (there, want_there) = _twins(lens, news, 41)
    side = torch.cuda.Stream()
    busy = torch.randn(2048, 2048, device="cuda")
    size = max(1 << 20, fnn.fastnn_attend_workspace_size(sum(news), 4, 2, 64, 64, 2, max(news),
                                                         -(-(max(lens) + max(news)) // 16), 16))
    torch.cuda.synchronize()
    for turn in range(24):
        if turn % 2:  # the side stream is late: what it uses must still be there
            with torch.cuda.stream(side):
                for _ in range(4):
                    torch.mm(busy, busy)
        got_here = here()
        got_there = there(stream=side)
        fills = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        fills += [torch.full_like(x, 3) for x in want_here for _ in range(2)]
        del fills
        torch.cuda.current_stream().wait_stream(side)
        for got, want in zip((*got_here, *got_there), (*want_here, *want_there)):
            assert torch.equal(got, want), turn


@pytest.mark.parametrize("lens,news", BATCHES)
def test_calls_from_two_threads_on_one_stream(lens, news):
    both = _twins(lens, news, 51)
    wrong = []

    def many(calls, want):
        for turn in range(40):
            for got, w in zip(calls(), want):
                if not torch.equal(got, w):
                    wrong.append(turn)

    threads = [threading.Thread(target=many, args=x) for x in both]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---- scores far above those before -------------------------------------------------------------

@pytest.mark.parametrize("gap", [100, 127.5, 128.2, 129, 150, 200, 255, 300, 384, 400, 520, 3000])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (64, F16), (128, BF16), (128, F16)])
def test_attend_one_key_far_above_all_others(gap, d, dtype):
    """All keys zero but one, which scores ``gap`` (base 2) with every query: it has the weight, at
    every place that the kernels treat in a way of its own, in the key tiles without a mask too."""
    st = ref.Store([192], [64], 64, 1, d, d, dtype, seed=int(gap), group=1)
    st.q.zero_()
    st.q[:, :, 0] = 16.0
    q, vp, table, lens, cu = st.cuda("q", "v_pages", "table", "lens", "cu")
    scale = gap * math.log(2.0) / 256
    for at in [*range(9), 31, 32, 33, 66, 96, 127, 128, 160]:
        st.k_pages.zero_()
        st.k_pages[int(st.table[0, at // 64]), 0, at % 64, 0] = 16.0
        for causal in (False, True):
            out, lse = fnn.fastnn_attend(q, st.k_pages.cuda(), vp, table, lens, cu, 64, causal=causal, scale=scale)
            # every token sees the key; the others' weights, 2^-gap each, are below half a step
            want = st.v_pages[int(st.table[0, at // 64]), 0, at % 64]
            assert bool((out.cpu() == want).all()), (at, causal)
            # the product is exact; scale, its product with log2 e, the score, its way back to nats
            # and the result are rounded to fp32 once each, the exponential of 0 and log2 are good to 2^-21
            off = (lse.cpu().double() - gap * math.log(2.0)).abs().max()
            assert float(off) <= 6 * 2.0 ** -24 * gap + 2.0 ** -21, (at, causal)


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_attend_a_few_scores_far_above_all_others(d, dtype):
    """Keys of ordinary size and, for a few rows of a few warps, one far larger: over several tiles."""
    for seed, (scale, at) in enumerate(((2.0, 0), (6.0, 2), (20.0, 129), (40.0, 33), (3.0, 256))):
        st = ref.Store([500], [70], 64, 1, d, d, dtype, seed=60 + seed, group=2)
        st.k_pages *= 0.05
        ph = int(st.table[0, at // 64])
        st.k_pages[ph, 0, at % 64] = 0
        st.k_pages[ph, 0, at % 64, 0] = 8.0
        st.q[:, :, 0] = 0
        st.q[::9, :, 0] = 8.0  # one row in nine
        out, lse = _attend(st, causal=bool(seed & 1), scale=scale)
        ref.check_attend(out, lse, st, bool(seed & 1), scale=scale)


# ---- queries that are no numbers ---------------------------------------------------------------

@pytest.mark.parametrize("lens,news,group,d", [
    ([40], [70], 2, 64),           # chunks: one tile, several, divided between blocks
    ([700, 300], [130, 66], 1, 128),
    ([9000, 20], [66, 70], 1, 64),
    ([9000], [64], 1, 128),
    ([40, 7], [1, 1], 4, 64),      # single tokens: one split, several
    ([9000, 3000], [1, 1], 2, 64),
    ([2999, 40], [1, 3], 4, 128),
])
@pytest.mark.parametrize("causal", [True, False])
def test_nan_in_a_query_is_the_answer_of_its_row_alone(lens, news, group, d, causal):
    st = ref.Store(lens, news, 64, 2, d, d, BF16, seed=70, group=group)
    clean, lse_clean = _attend(st, causal)
    ref.check_attend(clean, lse_clean, st, causal)
    whole = st.q.clone()
    bad = torch.zeros(st.n, 2 * group, dtype=torch.bool)
    bad[0, 0] = bad[st.n // 2, -1] = bad[st.n - 1, group] = True
    st.q[bad] = float("nan")
    out, lse = _attend(st, causal)
    gone = bad.cuda()
    assert bool(out[gone].isnan().all()) and bool(lse[gone].isnan().all())
    out[gone], lse[gone] = clean[gone], lse_clean[gone]
    st.q = whole
    ref.check_attend(out, lse, st, causal)


def test_nan_in_a_query_that_sees_nothing():
    for news in ([1, 1], [70, 3]):
        st = ref.Store([0, 0], news, 16, 1, 64, 64, F16, seed=3)
        st.q[:] = float("nan")
        st.lens = torch.tensor([0, -3], dtype=torch.int32)
        out, lse = _attend(st, causal=False)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("news,select", [([1, 1], 2), ([1, 3], 24), ([90, 5], 6)])
def test_nan_in_a_query_over_listed_pages(news, select):
    """The lowest pages are taken, all scores being NaN; splits in one block and in clusters."""
    st = ref.Store([2000, 300], news, 64, 2, 64, 64, F16, seed=71, group=4)
    q, km, table, lens, cu = st.cuda("q", "k_mean", "table", "lens", "cu")
    q[0] = float("nan")
    pages = fnn.fastnn_select_pages(q, km, table, lens, cu, st.max_new, 64, select)
    st.q = q.cpu()
    want = ref.select_pages(st, st.k_mean, select, 0, 1)
    assert torch.equal(pages.cpu(), want)
    out, lse = _attend(st, pages=pages)
    assert bool(out[0].isnan().all()) and bool(lse[0].isnan().all())
    st.q[0] = 0  # the others' answers
    clean, lse_clean = _attend(st, pages=pages)
    out[0], lse[0] = clean[0], lse_clean[0]
    ref.check_attend(out, lse, st, pages=want)


# ---- what earlier kernels leave in shared memory -----------------------------------------------

@pytest.mark.parametrize("group", [3, 5, 7, 48])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_the_same_bits_whatever_ran_before(group, d):
    """Groups that do not divide a tile of 128 rows leave rows of it unfilled: what an earlier call
    left there has no part in how the others are computed."""
    before = ref.Store([64] * 8, [300] * 8, 64, 8, d, d, BF16, seed=80)  # every SM, whole tiles
    fill = before.cuda("q", "k_pages", "v_pages", "table", "lens", "cu")
    st = ref.Store([900, 300], [130, 60], 64, 2, d, d, BF16, seed=81, group=group)
    args = st.cuda("q", "k_pages", "v_pages", "table", "lens", "cu")
    got = []
    for x in (0.0, float("nan"), 300.0, -300.0):
        fill[0].fill_(x)
        fnn.fastnn_attend(*fill, before.max_new, causal=False)
        got.append(fnn.fastnn_attend(*args, st.max_new, causal=False))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert not bool(got[0][1].isnan().any())
