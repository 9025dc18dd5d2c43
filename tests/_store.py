"""Plain 64-bit forms of the token store calls, and the bounds their kernels are held to.

Everything here is NumPy / torch float64 on the CPU, token by token.
"""

from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half a step of subnormals
U32 = 2.0 ** -24


def rotary(x, pos, freq, layout="half", scale=1.0, inverse=False):
    """x [n, heads, d] -> float64 result and, per element, |u| + |w| of its pair."""
    x, pos = x.double(), pos.reshape(x.shape[0], -1)
    out, mass = x.clone(), torch.zeros_like(x)
    axes, nf = pos.shape[1], freq.shape[0]
    for a in range(axes):
        for j in range(nf):
            t = pos[:, a].double() * freq[j].double()
            cos, sin = torch.cos(t)[:, None] * scale, torch.sin(t)[:, None] * scale
            if inverse:
                sin = -sin
            base = a * 2 * nf
            i1, i2 = (base + j, base + j + nf) if layout == "half" else \
                (base + 2 * j, base + 2 * j + 1)
            u, w = x[:, :, i1], x[:, :, i2]
            out[:, :, i1], out[:, :, i2] = u * cos - w * sin, w * cos + u * sin
            mass[:, :, i1] = mass[:, :, i2] = (u.abs() + w.abs()) * abs(scale)
    return out, mass


def check_rotary(got, x, pos, freq, layout="half", scale=1.0, inverse=False):
    """One rounding to 16 bits (half a step), and before it fp32: the sine and cosine are of an
    angle rounded to fp32 within half a turn (at most pi * 2^-25) and within 2 steps of 2^-24
    themselves, times scale; two products and a sum: below 8 * 2^-24 of |u| + |w|."""
    want, mass = rotary(x.cpu(), pos.cpu(), freq.cpu(), layout, scale, inverse)
    fine = 8 * U32 * mass
    tol = U[got.dtype] * (want.abs() + fine) + fine + TINY[got.dtype]
    rot = 2 * freq.shape[0] * (1 if pos.dim() == 1 else pos.shape[1])
    tol[:, :, rot:] = 0  # copied
    off = (got.cpu().double() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


class Store:
    """A paged store with shuffled pages, on the CPU, and its batch of new tokens."""

    def __init__(self, lens, news, page, heads, d, dv, dtype, seed=0, group=1, spare=2, width=None,
                 tail=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.heads, self.d, self.dv, self.dtype, self.group = page, heads, d, dv, dtype, group
        need = [max(1, -(-(a + b) // page)) for a, b in zip(lens, news)]
        self.width = max(need) if width is None else width
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        for s, c in enumerate(need):
            for p in range(min(c, self.width)):
                self.table[s, p] = order.pop()
        cu = [0]
        for b in news:
            cu.append(cu[-1] + b)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.before = torch.tensor(lens, dtype=torch.int32)
        self.lens = self.before + self.cu[1:] - self.cu[:-1]  # after the append
        self.n = cu[-1] + tail  # tokens behind the last sequence
        self.max_new = max(1, max(news))
        r = lambda *shape: torch.randn(shape, generator=g).to(dtype)  # noqa: E731
        self.k_pages, self.v_pages = r(self.n_pages, heads, page, d), r(self.n_pages, heads, page, dv)
        self.k_mean = r(self.n_pages, heads, d)
        self.k, self.v = r(self.n, heads, d), r(self.n, heads, dv)
        self.q = r(self.n, heads * group, d)

    def cuda(self, *names):
        return [getattr(self, n).cuda() for n in names]

    def visible(self, s, i, causal):
        m = int(self.cu[s + 1] - self.cu[s])
        v = int(self.lens[s]) - m + i + 1 if causal else int(self.lens[s])
        return max(0, min(v, self.width * self.page))

    def positions(self, s, pages=None, upto=0):
        """(page id, row) of the positions below `upto` that exist, in order; of the listed
        logical pages only, where a list is given."""
        every = range(-(-upto // self.page)) if pages is None else pages
        got = []
        for p in every:
            if not 0 <= p < self.width:
                continue
            ph = int(self.table[s, p])
            if 0 <= ph < self.n_pages:
                got += [(ph, r) for r in range(self.page) if p * self.page + r < upto]
        return got


def attend(st: Store, causal=True, scale=None, pages=None):
    """Yields (token, head, out, lse, sum w |v|, largest |product|, count) in float64."""
    scale = 1 / math.sqrt(st.d) if scale is None else scale
    kp, vp, q = st.k_pages.double(), st.v_pages.double(), st.q.double()
    for s in range(len(st.lens)):
        a, b = int(st.cu[s]), int(st.cu[s + 1])
        for t in range(a, b):
            for g in range(st.heads):
                at = st.positions(s, None if pages is None else pages[t, g].tolist(),
                                  st.visible(s, t - a, causal))
                for h in range(g * st.group, (g + 1) * st.group):
                    if not at:
                        yield t, h, torch.zeros(st.dv).double(), -math.inf, torch.zeros(st.dv).double(), 0.0, 0
                        continue
                    ids, rows = torch.tensor([x[0] for x in at]), torch.tensor([x[1] for x in at])
                    keys, vals = kp[ids, g, rows], vp[ids, g, rows]
                    x = keys @ q[t, h] * scale
                    z = torch.logsumexp(x, 0)
                    w = torch.exp(x - z)
                    big = float((keys.abs() @ q[t, h].abs()).max() * abs(scale))
                    yield t, h, w @ vals, float(z), w @ vals.abs(), big, len(at)


def check_attend(out, lse, st: Store, causal=True, scale=None, pages=None):
    """The bound, with u = half a step of the 16-bit type:
      u |out|                     the result's rounding
      u A, A = sum w |v|          the weights' rounding before the second product
      (2 e + N 2^-24) A           the fp32 part: a score of d products is off by at most
                                  e = (d + 4) 2^-24 max sum |q k| (absolute, so relative in its
                                  weight; twice, for the sum of the weights), exp2 by 2^-21 of
                                  its value, the sums of N terms by N 2^-24 at most
      N 2^-25 max |v| (fp16)      weights below the normal range
    and for lse the score's, exponential's and sums' parts, and two roundings of its value."""
    out, lse = out.cpu().double(), lse.cpu().double()
    u, top = U[st.dtype], float(st.v_pages.double().nan_to_num(0, 0, 0).abs().max())
    for t, h, want, z, mass, big, count in attend(st, causal, scale, pages):
        if count == 0:
            assert bool((out[t, h] == 0).all()) and float(lse[t, h]) == -math.inf, (t, h)
            continue
        e = (st.d + 4) * U32 * big + 2.0 ** -21
        fine = (2 * e + count * U32) * mass
        if st.dtype == torch.float16:
            fine = fine + count * 2.0 ** -25 * top
        tol = (u * want.abs() + u * mass + fine) * (1 + 2 * u) + TINY[st.dtype]
        off = (out[t, h] - want).abs()
        assert bool((off <= tol).all()), (t, h, float((off / tol).max()))
        ztol = e + count * U32 + 4 * U32 * (abs(z) + 1)
        assert abs(float(lse[t, h]) - z) <= ztol, (t, h, float(lse[t, h]), z, ztol)


def select_pages(st: Store, k_mean, select, keep_first, keep_last, causal=True):
    """int32 [n, heads, select] by the definition, -9 in the rows of no sequence."""
    want = torch.full((st.n, st.heads, select), -9, dtype=torch.int32)
    mean, q = k_mean.double(), st.q.double()
    for s in range(len(st.lens)):
        a, b = int(st.cu[s]), int(st.cu[s + 1])
        for t in range(a, b):
            seen = -(-st.visible(s, t - a, causal) // st.page)
            for g in range(st.heads):
                qs = q[t, g * st.group:(g + 1) * st.group].sum(0)
                rank = []
                for p in range(seen):
                    ph = int(st.table[s, p])
                    if not 0 <= ph < st.n_pages:
                        continue
                    x = float(qs @ mean[ph, g])
                    forced = p < keep_first or p >= seen - keep_last
                    rank.append((0 if forced else 1 if x == x else 2, -x if x == x else 0.0, p))
                kept = sorted(p for _, _, p in sorted(rank)[:select])
                want[t, g] = torch.tensor(kept + [-1] * (select - len(kept)), dtype=torch.int32)
    return want
