"""The cases by which the token-store operators are measured.

Four operators that belong together, for a stream of images whose tokens (descriptors,
patch features) stay in a paged store and are matched softly by the tokens of the next one:

  rotary   position rotation of query or key rows (and its inverse, the gradient)
  append   new keys (rotated on the way) and values into the paged store, with the mean key of
           every page that the call touches
  attend   softmax-weighted mean of the stored values under the dot products of the queries
           with the stored keys: chunks of new tokens, and single tokens
  sparse   the same over the pages that score best for each query by their mean key

With ``own`` false each runs in elementary torch operations, with ``own`` true through the
package's entry points.
"""

from __future__ import annotations

import math

import torch

own = False

# Spread of ragged sizes: fractions of the golden ratio fill [0, 1) evenly, whatever the count.
_PHI = 0.6180339887498949


def _ragged(lo: int, hi: int, count: int) -> list:
    return [lo + int((hi - lo) * (((i + 1) * _PHI) % 1.0) + 0.5) for i in range(count)]


def _news(c) -> list:
    return _ragged(c["new_lo"], c["new_hi"], c["seqs"])


def _helds(c) -> list:
    return _ragged(c["held_lo"], c["held_hi"], c["seqs"])


def listed():
    att = dict(op="attend")
    sel = dict(op="sparse", first=1, last=2)
    return [
        # one new token of each of 64 live streams, before a single-token step; half layout
        dict(name="rotary_step_64", op="rotary", tokens=64, heads=32, d=128, rot=128, axes=1,
             layout="half", inverse=False, base=10000.0, stretch=1.0, far=65536, type="bf16"),
        # gradient of the rotation of 16 image pairs' patch tokens (512x384 in 16-px patches), two axes
        dict(name="rotary_grad_2d", op="rotary", tokens=16 * 2 * 768, heads=16, d=64, rot=64,
             axes=2, layout="interleaved", inverse=True, base=100.0, stretch=1.0, far=32, type="f16"),
        # one new token of each of 256 streams into the store
        dict(name="append_step_256", op="append", seqs=256, new_lo=1, new_hi=1, held_lo=1, held_hi=4000,
             heads=8, d=128, dv=128, page=64, rot=128, axes=1, layout="half", base=500000.0,
             stretch=8.0, type="bf16"),
        # prompts of very different lengths, part of the head rotated
        dict(name="append_prompts", op="append", seqs=12, new_lo=1, new_hi=4097, held_lo=0, held_hi=900,
             heads=8, d=128, dv=128, page=64, rot=64, axes=1, layout="interleaved", base=10000.0,
             stretch=1.0, type="bf16"),
        # one token for each of 3 long streams: few rows, long axes
        dict(name="attend_step_long", seqs=3, new_lo=1, new_hi=1, held_lo=30001, held_hi=65535,
             hq=32, hk=8, d=128, dv=128, page=64, causal=True, type="bf16", **att),
        # one token for each of 96 streams of very different lengths
        dict(name="attend_step_96", seqs=96, new_lo=1, new_hi=1, held_lo=17, held_hi=8191,
             hq=32, hk=8, d=128, dv=128, page=16, causal=True, type="bf16", **att),
        # a new 512x288 image in 16-px patches (576 tokens) against the images of its stream
        dict(name="attend_image_8", seqs=8, new_lo=576, new_hi=576, held_lo=576, held_hi=9216,
             hq=12, hk=12, d=64, dv=64, page=32, causal=False, type="f16", **att),
        # a chunk of a long prompt
        dict(name="attend_chunk_2k_16k", seqs=1, new_lo=2048, new_hi=2048, held_lo=14336, held_hi=14336,
             hq=32, hk=8, d=128, dv=128, page=64, causal=True, type="bf16", **att),
        # soft matching: the 4-px grid of a 512x384 map against every pixel of the other map,
        # descriptors of 24, values of 8 (a 3D point and its confidence, padded)
        dict(name="attend_map_d24", seqs=1, new_lo=12288, new_hi=12288, held_lo=184320, held_hi=184320,
             hq=1, hk=1, d=24, dv=8, page=128, causal=False, type="bf16", **att),
        # one token for each of 4 short streams: the shortest selection
        dict(name="sparse_step_4", seqs=4, new_lo=1, new_hi=1, held_lo=1500, held_hi=4000, hq=16, hk=4,
             d=64, dv=64, page=32, causal=True, select=16, type="f16", **sel),
        # one token for each of 16 long streams
        dict(name="sparse_step_16_long", seqs=16, new_lo=1, new_hi=1, held_lo=32768, held_hi=65535,
             hq=32, hk=4, d=128, dv=128, page=64, causal=True, select=32, type="bf16", **sel),
        # a chunk of a long prompt, every token with pages of its own
        dict(name="sparse_chunk_2k_16k", seqs=1, new_lo=2048, new_hi=2048, held_lo=14336, held_hi=14336,
             hq=32, hk=4, d=128, dv=128, page=64, causal=True, select=16, type="bf16", **sel),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "attend", "sparse", "sparse"])
    typ = rng.choice(["bf16", "f16"])
    d = rng.choice([16, 24, 32, 40, 64, 64, 72, 96, 128, 128, 128])
    axes = rng.choice([1, 1, 2])
    rots = [r for r in range(4 * axes, d + 1, 4 * axes)]
    rotation = dict(rot=rng.choice([rots[-1], rng.choice(rots)]), axes=axes,
                    layout=rng.choice(["half", "interleaved"]),
                    base=rng.choice([100.0, 10000.0, 500000.0]), stretch=rng.choice([1.0, 4.0, 8.0]))
    if op == "rotary":
        heads = rng.choice([1, 4, 8, 12, 16, 32])
        return dict(op=op, tokens=_log_int(rng, 1, 50331648 // (heads * d)) if heads * d > 1024
                    else _log_int(rng, 1, 32768), heads=heads, d=d,
                    inverse=rng.random() < 0.5, far=_log_int(rng, 32, 1 << 20), type=typ, **rotation)
    if op == "append":
        dv = rng.choice([d, d, 8, 64])
        seqs = _log_int(rng, 1, 256)
        return dict(op=op, seqs=seqs, new_lo=1, new_hi=_log_int(rng, 1, 40000 // seqs),
                    held_lo=0, held_hi=_log_int(rng, 1, min(8192, 200000 // seqs)),
                    heads=rng.choice([1, 2, 4, 8]), d=d, dv=dv, page=rng.choice([16, 32, 64, 128]),
                    type=typ, **rotation)
    hk = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8])
    dv = rng.choice([d, d, d, 8, 64]) if op == "attend" else d
    c = dict(op=op, hq=hk * group, hk=hk, d=d, dv=dv, page=rng.choice([16, 32, 64, 128]),
             causal=rng.random() < 0.7, type=typ)
    if op == "sparse":
        c.update(first=rng.randint(0, 2), last=rng.randint(1, 3), select=rng.choice([8, 16, 24, 32]))
    kind = rng.choice(["step", "chunk", "chunk"])
    if kind == "step":
        seqs = _log_int(rng, 1, 96)
        top = _log_int(rng, 64, min(65535, 400000 // seqs))
        c.update(seqs=seqs, new_lo=1, new_hi=1, held_lo=rng.randint(0, top // 2), held_hi=top)
        return c
    # a chunk: rows x keys over all heads stay below half of the largest listed case's
    seqs = _log_int(rng, 1, 16)
    pairs = (5.0e8 if op == "attend" else 1.5e8) / (seqs * hk * group)
    new = _log_int(rng, 2, min(4096, int(math.sqrt(pairs))))
    keys = _log_int(rng, 16, max(17, min(40000, int(pairs / new) - new)))
    c.update(seqs=seqs, new_lo=max(1, new // 3), new_hi=new, held_lo=keys // 3, held_hi=keys)
    return c


_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _frequencies(c):
    n = c["rot"] // (2 * c["axes"])
    i = torch.arange(n, dtype=torch.float64)
    return (c["base"] ** (-i / n) / c["stretch"]).cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[c["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    st = dict(case=c)
    if c["op"] == "rotary":
        st.update(x=normal(c["tokens"], c["heads"], c["d"]), pos=whole(0, c["far"], c["tokens"], c["axes"]),
                  freq=_frequencies(c))
        return st
    news, helds = _news(c), _helds(c)
    totals = [a + b for a, b in zip(news, helds)]
    n, page, seqs = sum(news), c["page"], c["seqs"]
    cu = [0]
    for v in news:
        cu.append(cu[-1] + v)
    need = [-(-v // page) for v in totals]
    width, pages = max(need), sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(seqs, width, dtype=torch.int32)
    at, first = 0, []
    for v in need:
        first.append(at)
        at += v
    rows = torch.arange(width)[None, :]
    index = torch.tensor(first)[:, None] + rows
    held = rows < torch.tensor(need)[:, None]
    table = torch.where(held.cuda(), order[(index * held).cuda()], torch.full((), -1, dtype=torch.int32, device="cuda"))
    hk = c["heads"] if c["op"] == "append" else c["hk"]
    st.update(table=table.contiguous(), cu=torch.tensor(cu, dtype=torch.int32).cuda(), max_new=max(news),
              k_pages=normal(pages, hk, page, c["d"]), v_pages=normal(pages, hk, page, c["dv"]))
    if c["op"] == "append":
        st.update(lens=torch.tensor(helds, dtype=torch.int32).cuda(), k=normal(n, hk, c["d"]),
                  v=normal(n, hk, c["dv"]), k_mean=normal(pages, hk, c["d"]), freq=_frequencies(c))
        own_pos = torch.cat([torch.arange(b, b + a, dtype=torch.int32) for a, b in zip(news, helds)])
        st.update(pos=torch.stack([own_pos] * c["axes"], 1).contiguous().cuda())
        return st
    st.update(lens=torch.tensor(totals, dtype=torch.int32).cuda(), q=normal(n, c["hq"], c["d"]))
    if c["op"] == "sparse":
        # keys of one page have a direction in common, as those of neighbouring tokens do
        lean = torch.randn((pages, hk, 1, c["d"]), generator=g, device="cuda") * 0.5
        st["k_pages"] = (st["k_pages"].float() + lean).to(t)
        fill = torch.zeros(pages, dtype=torch.int64, device="cuda")
        part = (torch.tensor(totals)[:, None] - rows * page).clamp(0, page)
        fill[table.long()[held.cuda()]] = part[held].cuda()
        seen = torch.arange(page, device="cuda")[None, :] < fill[:, None]
        total = (st["k_pages"].double() * seen[:, None, :, None]).sum(2)
        st["k_mean"] = (total / fill.clamp(min=1)[:, None, None]).to(t)
    return st


def run(state):
    return _RUN[state["case"]["op"]](state)


# ---- rotary ------------------------------------------------------------------------------------


def _turn(x, pos, freq, c, inverse):
    """x [n, heads, d] with its first c["rot"] elements rotated by pos * freq, in 32 bits."""
    n, heads, d = x.shape
    a = pos.double()[:, :, None] * freq[None, None, :]  # far positions: angles in 64 bits
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    if inverse:
        sin = -sin
    part = x[:, :, :c["rot"]].float().reshape(n, heads, c["axes"], c["rot"] // c["axes"])
    if c["layout"] == "half":
        u, w = part.chunk(2, dim=3)
    else:
        u, w = part[..., 0::2], part[..., 1::2]
    u, w = u * cos - w * sin, w * cos + u * sin
    part = torch.cat([u, w], 3) if c["layout"] == "half" else torch.stack([u, w], 4)
    return torch.cat([part.reshape(n, heads, c["rot"]), x[:, :, c["rot"]:].float()], 2)


def _run_rotary(st):
    c = st["case"]
    if own:
        import reciprocal_nearest_neighbours_b200 as fnn
        return fnn.fastnn_rotary(st["x"], st["pos"], st["freq"], layout=c["layout"], inverse=c["inverse"])
    return _turn(st["x"], st["pos"], st["freq"], c, c["inverse"]).to(st["x"].dtype)


# ---- append ------------------------------------------------------------------------------------


def _run_append(st):
    c = st["case"]
    if own:
        import reciprocal_nearest_neighbours_b200 as fnn
        fnn.fastnn_store_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                st["cu"], st["max_new"], k_mean=st["k_mean"], pos=st["pos"],
                                freq=st["freq"], layout=c["layout"])
        return st["k_pages"], st["v_pages"], st["k_mean"]
    page, cu, lens, table = c["page"], st["cu"].long(), st["lens"].long(), st["table"].long()
    k = _turn(st["k"], st["pos"], st["freq"], c, False).to(st["k"].dtype)
    tok = torch.arange(k.shape[0], device="cuda")
    seq = torch.searchsorted(cu, tok, right=True) - 1
    at = lens[seq] + tok - cu[seq]
    phys, slot = table[seq, at // page], at % page
    st["k_pages"][phys, :, slot] = k
    st["v_pages"][phys, :, slot] = st["v"]
    total = lens + cu[1:] - cu[:-1]
    p = torch.arange(table.shape[1], device="cuda")[None, :]
    s, p = torch.nonzero((p >= (lens // page)[:, None]) & (p * page < total[:, None]), as_tuple=True)
    fill = (total[s] - p * page).clamp(max=page)
    rows = st["k_pages"][table[s, p]].float()
    seen = torch.arange(page, device="cuda")[None, :] < fill[:, None]
    total = torch.where(seen[:, None, :, None], rows, torch.zeros((), device="cuda")).sum(2)
    st["k_mean"][table[s, p]] = (total / fill[:, None, None].float()).to(st["k_mean"].dtype)
    return st["k_pages"], st["v_pages"], st["k_mean"]


# ---- attend and sparse -------------------------------------------------------------------------


def _padded(st):
    """Keys and values [seqs, hk, keys, .] and queries [seqs, hk, group, new, d] in 32 bits, the
    visible length of each new token, and which padded tokens there are."""
    c = st["case"]
    cu, lens, t = st["cu"].long(), st["lens"].long(), st["table"].long().clamp(min=0)
    seqs, width = t.shape
    keys = st["k_pages"][t].float().transpose(1, 2).reshape(seqs, c["hk"], width * c["page"], c["d"])
    vals = st["v_pages"][t].float().transpose(1, 2).reshape(seqs, c["hk"], width * c["page"], c["dv"])
    i = torch.arange(st["max_new"], device="cuda")[None, :]
    new = (cu[1:] - cu[:-1])[:, None]
    there = i < new
    tok = torch.where(there, cu[:-1, None] + i, 0)
    q = st["q"][tok].float().reshape(seqs, st["max_new"], c["hk"], c["hq"] // c["hk"], c["d"])
    sees = lens[:, None] - new + i + 1 if c["causal"] else lens[:, None].expand(seqs, st["max_new"])
    return q.permute(0, 2, 3, 1, 4), keys, vals, sees, there, tok


def _softly(st, padded, mask):
    """Softmax over the keys that `mask` (broadcast to [seqs, hk, group, new, keys]) lets through."""
    c = st["case"]
    q, keys, vals, sees, there, tok = padded
    seqs, hk, group, new, d = q.shape
    s = torch.matmul(q.reshape(seqs, hk, group * new, d) * (d ** -0.5), keys.transpose(2, 3))
    s = s.view(seqs, hk, group, new, -1).masked_fill_(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(seqs, hk, group * new, -1), vals).view(seqs, hk, group, new, -1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total))[..., 0]
    out = torch.empty(st["q"].shape[0], c["hq"], c["dv"], device="cuda", dtype=st["q"].dtype)
    out[tok[there]] = o.permute(0, 3, 1, 2, 4).reshape(seqs, new, c["hq"], c["dv"])[there].to(out.dtype)
    back = torch.empty(st["q"].shape[0], c["hq"], device="cuda")
    back[tok[there]] = lse.permute(0, 3, 1, 2).reshape(seqs, new, c["hq"])[there]
    return out, back


def _run_attend(st):
    c = st["case"]
    if own:
        import reciprocal_nearest_neighbours_b200 as fnn
        return fnn.fastnn_attend(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["cu"],
                                 st["max_new"], causal=c["causal"])
    padded = _padded(st)
    keys, sees = padded[1], padded[3]
    mask = torch.arange(keys.shape[2], device="cuda") < sees[:, None, None, :, None]
    return _softly(st, padded, mask)


def _run_sparse(st):
    c = st["case"]
    if own:
        import reciprocal_nearest_neighbours_b200 as fnn
        pages = fnn.fastnn_select_pages(st["q"], st["k_mean"], st["table"], st["lens"], st["cu"],
                                        st["max_new"], c["page"], c["select"], keep_first=c["first"],
                                        keep_last=c["last"], causal=c["causal"])
        out, lse = fnn.fastnn_attend(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                     st["cu"], st["max_new"], causal=c["causal"], pages=pages)
        return pages, out, lse
    padded = _padded(st)
    q, keys, _, sees, there, tok = padded
    width, select, page = st["table"].shape[1], c["select"], c["page"]
    means = st["k_mean"][st["table"].long().clamp(min=0)].double().transpose(1, 2)  # [seqs, hk, width, d]
    # values next to a border: the scores that decide are held in 64 bits
    score = torch.matmul(q.double().sum(2), means.transpose(2, 3))  # [seqs, hk, new, width]
    p = torch.arange(width, device="cuda")
    seen = ((sees.clamp(min=0) + page - 1) // page)[:, None, :, None]  # visible pages
    score = score.masked_fill((p < c["first"]) | (p >= seen - c["last"]), math.inf)
    score = score.masked_fill(p >= seen, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(score, dtype=torch.bool).scatter_(3, order[..., :select], True) & (p < seen)
    mask = kept.repeat_interleave(page, 3)[:, :, None]
    mask = mask & (torch.arange(keys.shape[2], device="cuda") < sees[:, None, None, :, None])
    out, lse = _softly(st, padded, mask)
    named = torch.where(kept, p, width)
    if width < select:
        named = torch.cat([named, named.new_full((*named.shape[:3], select - width), width)], 3)
    named = named.sort(dim=-1).values[..., :select]
    named = torch.where(named < width, named, -1).to(torch.int32).transpose(1, 2)
    back = torch.empty(st["q"].shape[0], c["hk"], select, dtype=torch.int32, device="cuda")
    back[tok[there]] = named[there]
    return back, out, lse


_RUN = {"rotary": _run_rotary, "append": _run_append, "attend": _run_attend, "sparse": _run_sparse}


# ---- what a pass cannot do without -------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["tokens"] * c["heads"] * c["d"]
        return dict(bytes=4.0 * n + 4.0 * c["tokens"] * c["axes"], flops=3.0 * n)
    news, helds = _news(c), _helds(c)
    n, page = sum(news), c["page"]
    if c["op"] == "append":
        rows = n * c["heads"] * (c["d"] + c["dv"])
        old = sum((h % page) for h in helds) * c["heads"] * c["d"]  # keys that a touched page held
        touched = sum(-(-(h + m) // page) - h // page for h, m in zip(helds, news))
        return dict(bytes=4.0 * rows + 2.0 * old + 2.0 * touched * c["heads"] * c["d"] + 4.0 * n * c["axes"],
                    flops=4.0 * n * c["heads"] * c["d"])
    wide = c["d"] + c["dv"]
    if c["op"] == "attend":
        keys = sum(h + m for h, m in zip(helds, news))
        pairs = sum(m * (h + m) - (m * (m - 1) / 2 if c["causal"] else 0) for h, m in zip(helds, news))
        return dict(bytes=2.0 * keys * c["hk"] * wide + 2.0 * n * c["hq"] * wide + 4.0 * n * c["hq"],
                    flops=2.0 * pairs * c["hq"] * wide)
    pairs = touched = scored = whole = 0.0
    for h, m in zip(helds, news):
        mean_seen = h + (m + 1) / 2 if c["causal"] else h + m
        seen = min(mean_seen, c["select"] * page)
        pairs += m * seen
        touched += min(h + m, m * seen)  # each key at most once
        scored += m * mean_seen / page
        whole += (h + m) / page
    return dict(bytes=2.0 * touched * c["hk"] * wide + 2.0 * whole * c["hk"] * c["d"] + 2.0 * n * c["hq"] * wide
                + 4.0 * n * (c["hq"] + c["hk"] * c["select"]),
                flops=2.0 * pairs * c["hq"] * wide + 2.0 * scored * c["hk"] * c["d"])


# ---- the definitions in 64 bits ----------------------------------------------------------------


def _rotated64(row, pos, c, freq, inverse):
    """row [n, heads, d] in 64 bits: each pair is one complex number, turned by its angle."""
    out = row.double().clone()
    per = c["rot"] // c["axes"]
    for a in range(c["axes"]):
        angle = pos[:, a].double()[:, None] * freq[None, :]
        turn = torch.polar(torch.ones_like(angle), -angle if inverse else angle)[:, None, :]
        at = torch.arange(per // 2, device="cuda")
        if c["layout"] == "half":
            re, im = a * per + at, a * per + per // 2 + at
        else:
            re, im = a * per + 2 * at, a * per + 2 * at + 1
        z = torch.complex(row[:, :, re].double(), row[:, :, im].double()) * turn
        out[:, :, re], out[:, :, im] = z.real, z.imag
    return out


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "rotary":
        return _rotated64(st["x"], st["pos"], c, st["freq"], c["inverse"])
    page, table, cu, lens = c["page"], st["table"].tolist(), st["cu"].tolist(), st["lens"].tolist()
    if c["op"] == "append":
        k = _rotated64(st["k"], st["pos"], c, st["freq"], False)
        kp, vp, km = st["k_pages"].double(), st["v_pages"].double(), st["k_mean"].double()
        held = st["k_pages"].dtype
        for s in range(c["seqs"]):
            done, i, end = lens[s], cu[s], cu[s + 1]
            while i < end:  # page by page
                at = done % page
                m = min(page - at, end - i)
                ph = table[s][done // page]
                kp[ph, :, at:at + m] = k[i:i + m].transpose(0, 1)
                vp[ph, :, at:at + m] = st["v"][i:i + m].double().transpose(0, 1)
                # the mean is that of the keys as the store holds them
                km[ph] = kp[ph, :, :at + m].to(held).double().mean(1)
                done, i = done + m, i + m
        return kp, vp, km
    group = c["hq"] // c["hk"]
    n = st["q"].shape[0]
    out = torch.zeros(n, c["hq"], c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((n, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for s in range(c["seqs"]):
        a, b, length = cu[s], cu[s + 1], lens[s]
        ids = torch.tensor(table[s][:-(-length // page)], dtype=torch.int64, device="cuda")
        for h in range(c["hk"]):
            keys = st["k_pages"][ids, h].reshape(-1, c["d"])[:length].double()
            vals = st["v_pages"][ids, h].reshape(-1, c["dv"])[:length].double()
            for r in range(a, b, 512):
                e = min(b, r + 512)
                q = st["q"][r:e, h * group:(h + 1) * group].double()
                sees = length - (b - torch.arange(r, e, device="cuda")) + 1
                if not c["causal"]:
                    sees = torch.full_like(sees, length)
                hidden = torch.arange(length, device="cuda")[None, :] >= sees[:, None]
                if c["op"] == "sparse":
                    hidden = hidden | ~_kept64(c, st, q.sum(1), ids, h, sees, length)
                x = torch.einsum("tgd,kd->tgk", q, keys) / math.sqrt(c["d"])
                x = x.masked_fill(hidden[:, None, :], -math.inf)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
                out[r:e, h * group:(h + 1) * group] = torch.einsum("tgk,kv->tgv", w, vals)
                lse[r:e, h * group:(h + 1) * group] = z
    return (None, out, lse) if c["op"] == "sparse" else (out, lse)


def _kept64(c, st, q, ids, h, sees, length):
    """Which keys each token's pages hold, by counting the pages that come before each."""
    page, total = c["page"], len(ids)
    score = torch.einsum("td,pd->tp", q, st["k_mean"][ids, h].double())
    p = torch.arange(total, device="cuda")
    seen = ((sees.clamp(min=0) + page - 1) // page)[:, None]
    score[(p[None, :] < c["first"]) | (p[None, :] >= seen - c["last"])] = math.inf
    score[p[None, :] >= seen] = -math.inf
    level = torch.sort(score, dim=1, descending=True).values[:, min(c["select"], total) - 1, None]
    above = score > level
    room = min(c["select"], total) - above.sum(1, keepdim=True)
    tied = (score == level) & (torch.cumsum(score == level, 1) <= room)
    kept = (above | tied) & (p[None, :] < seen)
    return kept.repeat_interleave(page, 1)[:, :length]
