"""A server's token step around the paged KV cache: cases, inputs, plain forms.

Four operators, in the order in which a step calls them:

* ``rope``    rotary positions of query and key rows (halves or pairs, part of the head, scaled);
* ``place``   the new rows' keys, rotated at their tokens' places, and values go to the pages; queries rotated with them;
* ``prefix``  attention of one new token per sequence, where groups of sequences share their first pages;
* ``sample``  a token per row of logits by temperature, top-k, top-p and min-p from a given number, and its confidence.

With ``own`` false ``run`` computes them by elementary torch operations; with ``own`` true it makes the
framework's calls.  ``exact`` computes the same from the definitions in 64 bits, row by row or sequence by sequence.

Rotation: the first ``rot`` elements of a head turn in pairs (i, i + rot / 2) ("half") or (2 i, 2 i + 1) ("pairs") by
position * f_i, f_i = theta^(-2 i / rot), scaled: "linear" f / s; "base" f s^(-2 i / (rot - 2)); "bands" g f + (1 - g) f / s
with g = clamp((trained f / 2 pi - slow) / (fast - slow), 0, 1).  Cosines and sines are multiplied by ``magnitude``.

Sampling of a row: of the tokens with a logit above -inf, the top_k of largest logit (ties: lowest index); of those, by their
softmax at the temperature, the shortest run from the largest on whose weight reaches top_p; of those, the ones with at
least min_p of the largest one's weight.  The token is the first one, in index order, up to which more than u of the
weight lies; a weight below 2^-44 of the largest counts as 0.  Temperature 0 is the first largest.  The confidence is the
token's softmax probability at temperature 1, nothing left out.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the fp32 model's sequence (96 positions, 4 query and 4 key heads of 64): latency
        dict(name="rope_fp32_96", op="rope", rows=96, heads=8, values=4, head_dim=64, dtype="fp32", far=96, rot=64, layout="half",
             theta=10000.0, scaling="none", mix=1),
        # one block of 64 positions, 32 query and 32 key heads, half of each head rotated, neighbours paired
        dict(name="rope_block_64_pairs", op="rope", rows=64, heads=64, values=32, head_dim=128, dtype="bf16", far=1536, rot=64,
             layout="pairs", theta=10000.0, scaling="linear", factor=4.0, mix=2),
        # a long prompt, 8704 rows of 16 query and 16 key heads, frequencies scaled in bands for a longer context
        dict(name="rope_prompt_8704", op="rope", rows=8704, heads=32, values=16, head_dim=128, dtype="bf16", far=140000, rot=128,
             layout="half", theta=500000.0, scaling="bands", factor=8.0, trained=8192, slow=1.0, fast=4.0, magnitude=1.2, mix=3),
        # one token of each of 64 running sequences, 32 query heads on 8: the smallest call of a serving step
        dict(name="place_step_b64", op="place", n=64, lo=40, hi=1536, rows=1, kv_heads=8, heads=32, head_dim=128, page=16,
             order="token", dtype="bf16", rot=128, layout="half", theta=10000.0, scaling="none", mix=4),
        # a prompt of 8704 rows, 16 heads, one layer
        dict(name="place_prompt_8704", op="place", n=1, lo=8704, hi=8704, rows=8704, kv_heads=16, heads=16, head_dim=128, page=32,
             order="token", dtype="bf16", rot=128, layout="half", theta=10000.0, scaling="base", factor=2.0, mix=5),
        # four short sequences of the fp32 model that begin alike: latency
        dict(name="prefix_fp32_b4", op="prefix", groups=1, n=4, prefix=64, lo=1, hi=32, heads=4, kv_heads=4, head_dim=64, page=16,
             order="token", dtype="fp32", mix=6),
        # 64 continuations of one long prompt, 32 query heads on 8
        dict(name="prefix_b64_8192", op="prefix", groups=1, n=64, prefix=8192, lo=1, hi=1024, heads=32, kv_heads=8, head_dim=128,
             page=16, order="token", dtype="bf16", mix=7),
        # 32 answers of 512 tokens to the long-context workload's prompt, 16 heads on 16
        dict(name="prefix_b32_heads16", op="prefix", groups=1, n=32, prefix=8192, lo=512, hi=512, heads=16, kv_heads=16,
             head_dim=128, page=32, order="token", dtype="bf16", mix=8),
        # three system prompts of different lengths, 96 ragged conversations: heads of 64, one key head per 8
        dict(name="prefix_groups_b96", op="prefix", groups=3, n=96, prefix=24000, lo=16, hi=2000, heads=64, kv_heads=8, head_dim=64,
             page=64, order="head", dtype="bf16", mix=9),
        # one row of logits, top-p: the latency of a single sequence's step
        dict(name="sample_b1_top_p", op="sample", rows=1, vocab=126464, dtype="fp32", kind="top_p", mix=10),
        # the 64 positions of a block, temperature alone: every token of the vocabulary takes part
        dict(name="sample_block_64", op="sample", rows=64, vocab=157184, dtype="fp32", kind="temperature", mix=11),
        # 512 rows (16 sequences' blocks of 32) in bf16, every row with settings of its own
        dict(name="sample_b512_mixed", op="sample", rows=512, vocab=126464, dtype="bf16", kind="mixed", mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _turn(rng, head_dim):
    """A rotation's settings."""
    scaling = rng.choice(("none", "linear", "base", "bands"))
    c = dict(rot=rng.choice((head_dim, head_dim, head_dim // 2, head_dim // 4)), layout=rng.choice(("half", "pairs")),
             theta=rng.choice((10000.0, 500000.0, 1000000.0)), scaling=scaling)
    if scaling != "none":
        c["factor"] = rng.choice((2.0, 4.0, 8.0, 32.0))
    if scaling == "bands":
        c.update(trained=rng.choice((4096, 8192, 32768)), slow=1.0, fast=rng.choice((4.0, 32.0)), magnitude=rng.choice((1.0, 1.2)))
    return c


def _one(rng):
    op = rng.choice(("rope", "place", "prefix", "prefix", "sample", "sample"))
    dtype = "fp32" if rng.random() < 0.3 else "bf16"
    mix = rng.randrange(1 << 20)
    if op == "sample":
        return dict(op=op, rows=_log(rng, 1, 512), vocab=_log(rng, 1000, 200000), dtype=rng.choice(("fp32", "fp32", "bf16")),
                    kind=rng.choice(("temperature", "top_k", "top_p", "mixed")), mix=mix)
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8))
    base = dict(op=op, head_dim=head_dim, dtype=dtype, mix=mix)
    if op == "rope":
        return dict(base, rows=_log(rng, 1, 8704), heads=heads + kv_heads, values=kv_heads, far=_log(rng, 100, 1000000), **_turn(rng, head_dim))
    base.update(heads=heads, kv_heads=kv_heads, page=rng.choice((8, 16, 24, 32, 64, 128)), order=rng.choice(("token", "head")))
    if op == "place":
        hi = _log(rng, 16, 8704)
        return dict(base, n=_log(rng, 1, 96), lo=max(1, hi // rng.choice((1, 3, 10))), hi=hi,
                    rows=rng.choice((1, 1, _log(rng, 1, 8704))), **_turn(rng, head_dim))
    groups = rng.choice((1, 1, 2, 3, 5))
    hi = _log(rng, 1, 2000)
    return dict(base, groups=groups, n=max(groups, _log(rng, 2, 128)), prefix=_log(rng, 16, 24000), lo=max(1, hi // rng.choice((1, 5, 50))), hi=hi)


def draw(rng):
    """A case of the same ranges: no more work than the largest listed one, nor more memory in its plain form."""
    while True:
        c = _one(rng)
        w = work(c)
        if w["bytes"] > 1.4e8 or w["flops"] > 2.8e10 or w["bytes"] < 2e3:
            continue
        if c["op"] == "prefix":
            if sum(_lens(c)) * max(c["heads"], 8) * c["head_dim"] > 6e9:
                continue  # the plain form's scores and gathered keys
        return c


def _lens(case):
    """The sequences' lengths, spread over the logarithm from lo to hi, both ends among them; behind a prefix their sum with it."""
    r = random.Random(case["mix"])
    lens = [_log(r, case["lo"], case["hi"]) for _ in range(case["n"])]
    lens[0] = case["hi"]
    if len(lens) > 1:
        lens[-1] = case["lo"]
    if case["op"] == "prefix":
        bounds, prefix = _groups(case)
        for g, p in enumerate(prefix):
            for i in range(bounds[g], bounds[g + 1]):
                lens[i] += p
    return lens


def _groups(case):
    """First sequence of each group (and their number), tokens that each group shares: the first one the most."""
    r = random.Random(case["mix"] + 99)
    g, n = case["groups"], case["n"]
    cuts = sorted(r.sample(range(1, n), g - 1)) if g > 1 else []
    prefix = [case["prefix"]] + [_log(r, max(1, case["prefix"] // 40), case["prefix"]) for _ in range(g - 1)]
    return [0] + cuts + [n], prefix


def _rows(case):
    return [min(case["rows"], x) for x in _lens(case)]


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    if case["op"] == "rope":
        elems = case["rows"] * case["heads"] * case["head_dim"]
        return {"bytes": 2 * elems * _size(case) + 4 * case["rows"], "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    if case["op"] == "place":
        rows = sum(_rows(case))
        heads = case["heads"] + case["kv_heads"]
        return {"bytes": 2 * rows * (heads + case["kv_heads"]) * case["head_dim"] * _size(case) + 12 * case["n"],
                "flops": 3 * rows * heads * case["rot"]}
    if case["op"] == "prefix":
        bounds, prefix = _groups(case)
        lens = _lens(case)
        shared = [p // case["page"] * case["page"] for p in prefix]  # whole pages are shared
        keys = sum(shared) + sum(x - shared[g] for g in range(len(prefix)) for x in lens[bounds[g]:bounds[g + 1]])
        ends = 2 * case["n"] * case["heads"] * case["head_dim"] * _size(case)
        return {"bytes": 2 * keys * case["kv_heads"] * case["head_dim"] * _size(case) + ends + 4 * -(-keys // case["page"]),
                "flops": 4 * sum(lens) * case["heads"] * case["head_dim"]}
    return {"bytes": case["rows"] * (case["vocab"] * _size(case) + 28), "flops": 4 * case["rows"] * case["vocab"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    return _ints([0] + list(np.cumsum(v)))


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _store(case, pages, g):
    """One of the two cache tensors of one layer, viewed as [1, pages, page_size, kv_heads, head_dim]."""
    dt = _TYPES[case["dtype"]]
    if case["order"] == "token":
        return _normal((1, pages, case["page"], case["kv_heads"], case["head_dim"]), g, dt)
    return _normal((1, pages, case["kv_heads"], case["page"], case["head_dim"]), g, dt).transpose(2, 3)


def _tables(case, lens):
    """Scattered pages for the sequences; those of a group hold the same ones for the full pages of what they share."""
    page = case["page"]
    held = [-(-x // page) for x in lens]
    alike = [0] * len(lens)
    first = list(range(len(lens)))
    if case["op"] == "prefix":
        bounds, prefix = _groups(case)
        for g, p in enumerate(prefix):
            for i in range(bounds[g], bounds[g + 1]):
                alike[i], first[i] = p // page, bounds[g]
    pages = sum(h - (a if f != i else 0) for i, (h, a, f) in enumerate(zip(held, alike, first))) + 2
    at = np.random.RandomState((case["mix"] + 17) % (1 << 31)).permutation(pages)
    table = np.full((len(lens), max(held)), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    used = 0
    for s, h in enumerate(held):
        a = alike[s] if first[s] != s else 0
        table[s, :a] = table[first[s], :a]
        table[s, a:h] = at[used:used + h - a]
        used += h - a
        refs[table[s, :h]] += 1
    return table, refs


def _settings(case):
    """temperature, top_k, top_p, min_p of every row (None: off), by the case alone."""
    r = random.Random(case["mix"] + 5)
    n, kind = case["rows"], case["kind"]
    temperature = [r.choice((0.7, 1.0, 1.3)) for _ in range(n)]
    if kind == "temperature":
        return temperature, None, None, None
    if kind == "top_k":
        return temperature, [r.choice((1, 20, 50, 1000)) for _ in range(n)], None, None
    if kind == "top_p":
        return temperature, None, [r.choice((0.5, 0.9, 0.95)) for _ in range(n)], None
    temperature = [r.choice((0.0, 0.3, 0.7, 1.0, 1.3)) for _ in range(n)]
    return (temperature, [r.choice((0, 0, 20, 50, 1000)) for _ in range(n)], [r.choice((1.0, 0.5, 0.9, 0.95)) for _ in range(n)],
            [r.choice((0.0, 0.0, 0.05, 0.1)) for _ in range(n)])


def _frequencies(case):
    """Turns of pair i per position, in radians: 64 bits."""
    r, s = case["rot"], case.get("factor", 1.0)
    i = torch.arange(r // 2, dtype=torch.float64)
    f = case["theta"] ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "base":
        f = f * s ** (-2.0 * i / (r - 2))
    if case["scaling"] == "bands":
        g = ((case["trained"] * f / (2 * math.pi) - case["slow"]) / (case["fast"] - case["slow"])).clamp(0, 1)
        f = g * f + (1 - g) * f / s
    return f.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    st = {"case": case, "op": case["op"]}
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        spread = 1.0 + 2.0 * torch.rand((rows, 1), generator=g, device="cuda")
        x = torch.randn((rows, vocab), generator=g, device="cuda") * spread
        for _ in range(12):  # the few tokens that the model would like
            at = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
            x.scatter_add_(1, at, 12.0 * torch.rand((rows, 1), generator=g, device="cuda"))
        x[:, vocab - 1] = -math.inf  # the mask token, which is never chosen
        u = torch.rand(rows, generator=g, device="cuda")
        t, k, p, m = (None if v is None else torch.tensor(v, dtype=torch.int32 if j == 1 else torch.float32, device="cuda")
                      for j, v in enumerate(_settings(case)))
        st.update(logits=x.to(_TYPES[case["dtype"]]), u=u, temperature=t, top_k=k, top_p=p, min_p=m)
    else:
        dt, hd = _TYPES[case["dtype"]], case["head_dim"]
        if case["op"] != "prefix":
            st["f"] = _frequencies(case)
        if case["op"] == "rope":  # queries and keys of one projection's output, which holds values too
            x = _normal((case["rows"], (case["heads"] + case["values"]) * hd), g, dt)
            st.update(x=x[:, :case["heads"] * hd].unflatten(1, (-1, hd)),
                      positions=torch.randint(0, case["far"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32))
        else:
            lens = _lens(case)
            table, refs = _tables(case, lens)
            st.update(k=_store(case, len(refs), g), v=_store(case, len(refs), g), table=_ints(table), lens=_ints(lens), refs=_ints(refs))
            rows = _rows(case) if case["op"] == "place" else [1] * case["n"]
            x = _normal((sum(rows), (case["heads"] + 2 * case["kv_heads"]) * hd), g, dt).unflatten(1, (-1, hd))
            st.update(q=x[:, :case["heads"]])
            if case["op"] == "place":
                st.update(new_k=x[:, case["heads"]:-case["kv_heads"]], new_v=x[:, -case["kv_heads"]:],
                          rows=_cum(rows) if case["rows"] > 1 else None)
            else:
                bounds, prefix = _groups(case)
                st.update(groups=_ints(bounds), prefix=_ints(prefix), most=max(lens), scale=1.0 / math.sqrt(hd))
    if own:
        from block_denoising_gb300 import dinfer
        st["ops"] = dinfer
        if "f" in st:
            st["rope"] = dinfer.Rope(case["rot"], theta=case["theta"], layout=case["layout"], scaling=case["scaling"],
                                     factor=case.get("factor", 1.0), trained=case.get("trained", 0), slow=case.get("slow", 0.0),
                                     fast=case.get("fast", 0.0), magnitude=case.get("magnitude", 1.0))
        if "table" in st:
            st["kv"] = dinfer.PagedKV(st["k"], st["v"], st["table"], st["lens"], st["refs"])
        if case["op"] == "prefix":
            st["ws"] = dinfer.OpWorkspace()
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return _own(st) if own else _PLAIN[st["op"]](st)


def _own(st):
    op = st["op"]
    if op == "rope":
        return st["ops"].op_rope(st["x"], st["rope"], positions=st["positions"])
    if op == "place":
        q = st["kv"].append_rope(0, st["rope"], st["new_k"], st["new_v"], q=st["q"], rows=st["rows"])
        return {"q": q, "k": st["k"], "v": st["v"]}
    if op == "prefix":
        return st["kv"].prefix_attention(0, st["q"], st["ws"], prefix=st["prefix"], groups=st["groups"], scale=st["scale"])
    return st["ops"].op_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                               min_p=st["min_p"])


def _rotate(x, positions, st):
    """x [rows, heads, head_dim] at positions [rows]: angles in 64 bits, the rest in 32."""
    case = st["case"]
    rot, m = case["rot"], case.get("magnitude", 1.0)
    angle = positions.double()[:, None, None] * st["f"]
    c, s = (torch.cos(angle) * m).float(), (torch.sin(angle) * m).float()
    y = x.float().clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a] = xa * c - xb * s
    y[..., b] = xa * s + xb * c
    return y.to(x.dtype)


def _plain_rope(st):
    return _rotate(st["x"], st["positions"], st)


def _plain_place(st):
    lens, page = st["lens"].long(), st["case"]["page"]
    n = len(lens)
    rows = torch.ones_like(lens) if st["rows"] is None else (st["rows"][1:] - st["rows"][:-1]).long()
    start = torch.cumsum(rows, 0) - rows
    total = st["new_k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), rows, output_size=total)
    pos = (lens - rows - start)[seq] + torch.arange(total, device="cuda")
    at = st["table"][seq, pos // page].long(), pos % page
    st["k"][0][at] = _rotate(st["new_k"], pos, st)
    st["v"][0][at] = st["new_v"]
    return {"q": _rotate(st["q"], pos, st), "k": st["k"], "v": st["v"]}


def _plain_prefix(st):
    q, lens, page = st["q"], st["lens"], st["case"]["page"]
    n, heads, hd = q.shape
    pos = torch.arange(st["most"], device="cuda")
    out = torch.empty((n, heads, hd), dtype=q.dtype, device="cuda")
    for a in range(0, n, 32):  # a few sequences at a time: their keys side by side
        b = min(n, a + 32)
        seen = pos < lens[a:b, None]
        at = st["table"][a:b, pos // page].clamp(min=0).long(), (pos % page).expand(b - a, -1)
        wipe = ~seen[:, :, None, None]
        k = st["k"][0][at].float().masked_fill(wipe, 0.0).transpose(1, 2)  # [n, kv_heads, keys, head_dim]
        v = st["v"][0][at].float().masked_fill(wipe, 0.0).transpose(1, 2)
        s = (q[a:b].float().reshape(b - a, k.shape[1], -1, hd) @ k.transpose(-1, -2)) * st["scale"]
        s = torch.where(seen[:, None, None], s, -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        out[a:b] = ((p @ v) / p.sum(-1, keepdim=True)).reshape(b - a, heads, hd).to(q.dtype)
    return out


def _plain_sample(st):
    x = st["logits"].float()
    rows, vocab = x.shape
    top = x.amax(1, keepdim=True)
    best = torch.argmax((x == top).to(torch.int32), 1)
    t = st["temperature"][:, None]
    w = torch.exp((x - top).double() / torch.where(t > 0, t, 1.0).double())
    w = torch.where((x > -math.inf) & (w >= 2.0 ** -44), w, 0.0)
    if st["top_k"] is not None or st["top_p"] is not None or st["min_p"] is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        sorted_w = w.gather(1, order)
        keep = torch.ones_like(sorted_w, dtype=torch.bool)
        if st["top_k"] is not None:
            k = st["top_k"].long()[:, None]
            keep &= (torch.arange(vocab, device="cuda") < k) | (k <= 0)
        sorted_w = torch.where(keep, sorted_w, 0.0)
        if st["top_p"] is not None:
            p = st["top_p"].double()[:, None]
            before = torch.cumsum(sorted_w, 1) - sorted_w
            keep &= (before < p * sorted_w.sum(1, keepdim=True)) | (p >= 1)
        if st["min_p"] is not None:
            keep &= sorted_w >= st["min_p"].double()[:, None] * sorted_w[:, :1]
        w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, sorted_w, 0.0))
    up = torch.cumsum(w, 1)
    tok = torch.searchsorted(up, st["u"].double()[:, None] * up[:, -1:], right=True)[:, 0].clamp(max=vocab - 1)
    tok = torch.where(st["temperature"] > 0, tok, best)
    conf = torch.exp(x.gather(1, tok[:, None]) - top) / torch.exp(x - top).sum(1, keepdim=True)
    return tok.to(torch.int32), conf[:, 0]


_PLAIN = {"rope": _plain_rope, "place": _plain_place, "prefix": _plain_prefix, "sample": _plain_sample}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "place": _exact_place, "prefix": _exact_prefix, "sample": _exact_sample}[case["op"]](case, st)


def _turned(x, positions, case):
    """Pairs as complex numbers, each multiplied by magnitude * e^(i angle)."""
    rot = case["rot"]
    x = x.double()
    pairs = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else x[..., :rot].unflatten(-1, (-1, 2))
    s = case.get("factor", 1.0)
    f = []
    for i in range(rot // 2):
        w = math.exp(-2.0 * i / rot * math.log(case["theta"]))
        if case["scaling"] == "linear":
            w /= s
        elif case["scaling"] == "base":
            w = math.exp(-2.0 * i / rot * (math.log(case["theta"]) + math.log(s) * rot / (rot - 2)))
        elif case["scaling"] == "bands":
            part = (case["trained"] * w / (2 * math.pi) - case["slow"]) / (case["fast"] - case["slow"])
            part = min(1.0, max(0.0, part))
            w = w * part + w / s * (1 - part)
        f.append(w)
    angle = positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, case.get("magnitude", 1.0)), angle)[:, None]
    z = torch.view_as_real(z)
    z = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else z.flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def _exact_rope(case, st):
    return _turned(st["x"], st["positions"], case)


def _exact_place(case, st):
    """Sequence by sequence, its pages looked up on the host."""
    k, v, page, table = st["k"].double(), st["v"].double(), case["page"], st["table"].cpu().numpy()
    q = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    a = 0
    for s, (n, r) in enumerate(zip(_lens(case), _rows(case))):
        p = np.arange(n - r, n)
        at, slot = torch.from_numpy(table[s, p // page].astype(np.int64)).cuda(), torch.from_numpy(p % page).cuda()
        where = torch.from_numpy(p).cuda()
        k[0, at, slot] = _turned(st["new_k"][a:a + r], where, case)
        v[0, at, slot] = st["new_v"][a:a + r].double()
        q[a:a + r] = _turned(st["q"][a:a + r], where, case)
        a += r
    return {"q": q, "k": k, "v": v}


def _exact_prefix(case, st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    group, table, page = case["heads"] // case["kv_heads"], st["table"].cpu().numpy(), case["page"]
    for s, n in enumerate(_lens(case)):
        pages = torch.from_numpy(table[s, :-(-n // page)].astype(np.int64)).cuda()
        k = st["k"][0, pages].flatten(0, 1)[:n].double().transpose(0, 1)  # [kv_heads, keys, head_dim]
        v = st["v"][0, pages].flatten(0, 1)[:n].double().transpose(0, 1)
        w = torch.softmax(torch.bmm(st["q"][s].double().unflatten(0, (-1, group)), k.transpose(1, 2)) * st["scale"], -1)
        out[s] = torch.bmm(w, v).flatten(0, 1)
    return out


def _exact_sample(case, st):
    """Row by row: the kept tokens as a list, in the order of their indices."""
    settings = _settings(case)
    toks, confs = [], []
    u = st["u"].tolist()
    for r in range(case["rows"]):
        x = st["logits"][r].double()
        t, k, p, m = (None if v is None else v[r] for v in settings)
        t, p, m = (None if v is None else float(np.float32(v)) for v in (t, p, m))
        top = float(x.max())
        if t > 0:
            at = torch.nonzero(x > max(-1e300, top - 44 * math.log(2) * t))[:, 0]
            if k is not None or p is not None or m is not None:
                at = at[torch.argsort(x[at], descending=True, stable=True)]
                if k is not None and k > 0:
                    at = at[:k]
                w = torch.exp((x[at] - top) / t)
                if p is not None and p < 1:
                    share = torch.cumsum(w, 0)
                    at = at[:int(torch.searchsorted(share, p * share[-1])) + 1]
                    w = w[:len(at)]
                if m is not None:
                    at = at[w >= m]
                at = at.sort().values
            share = torch.cumsum(torch.exp((x[at] - top) / t), 0)
            pick = int(torch.searchsorted(share, u[r] * share[-1], right=True))
            tok = int(at[min(pick, len(at) - 1)])
        else:
            tok = int(torch.nonzero(x == top)[0, 0])
        toks.append(tok)
        confs.append(float(torch.exp(x[tok] - top) / torch.exp(x - top).sum()))
    return torch.tensor(toks, dtype=torch.int32), torch.tensor(confs, dtype=torch.float64)
