"""The paged KV cache's operators and windowed prompt attention: cases, inputs, plain forms.

Four operators, as a serving loop uses them:

* ``append``  the new rows' keys and values go to their sequences' pages;
* ``pages``   sequences are freed, forked (sharing full pages, or copied) and the cache is compacted;
* ``decode``  attention of one new token per sequence over its pages, with a window and sinks;
* ``prompt``  attention of many rows with a sliding window and sinks, over ragged sequences.

With ``own`` false ``run`` computes them by elementary torch operations in 32 bits; with ``own`` true it makes
the framework's calls.  ``exact`` computes the same from the definitions in 64 bits, sequence by sequence.

Layouts: a cache tensor is [layers, pages, page_size, kv_heads, head_dim], stored in that order ("token") or
with the heads outside the slots ("head"); ``table`` [max_seqs, max_pages] holds a sequence's pages in order
(-1: none), ``lens`` its tokens, ``refs`` how many sequences hold each page.  A row at position p sees key j if
j <= p + right and (j < sinks or j >= p - left); -1 is an open side.  A row that sees nothing gives zeros.
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
        # one token of each of 64 running sequences is stored, one layer: the smallest call of a serving step
        dict(name="append_step_b64", op="append", n=64, lo=40, hi=1536, rows=1, kv_heads=8, heads=32, head_dim=128,
             page=16, order="token", dtype="bf16", mix=3),
        # the keys and values of a long prompt (16 heads of 128, 8704 rows) are stored, one layer
        dict(name="append_prompt_8704", op="append", n=1, lo=8704, hi=8704, rows=8704, kv_heads=16, heads=16,
             head_dim=128, page=32, order="token", dtype="bf16", mix=1),
        # eight continuations of one 1000-token prompt dropped and forked again; their last, partly filled page is copied
        dict(name="fork_share_8", op="pages", kind="fork", share=True, n=8, sources=1, lo=1000, hi=1000, layers=16,
             kv_heads=16, head_dim=128, page=16, order="token", dtype="bf16", mix=5),
        # four sequences of a 32-head model copied whole (block decoding rewrites its slots, so nothing can be shared)
        dict(name="fork_copy_4x1536", op="pages", kind="fork", share=False, n=4, sources=4, lo=1400, hi=1536, layers=8,
             kv_heads=32, head_dim=128, page=64, order="token", dtype="bf16", mix=6),
        # half of a 2 GB cache is free, scattered: the live pages are packed to the front
        dict(name="compact_half", op="pages", kind="compact", n=40, lo=100, hi=800, shared=3, layers=16, kv_heads=8,
             head_dim=128, page=16, order="head", dtype="bf16", fill=0.5, mix=7),
        # one token of the fp32 model (4 heads of 64, 96 positions), a batch of 4: latency
        dict(name="decode_fp32_b4", op="decode", n=4, lo=33, hi=96, heads=4, kv_heads=4, head_dim=64, page=16,
             order="token", dtype="fp32", window=-1, sinks=0, mix=8),
        # one sequence of the long-context workload (8192 + 512 positions, 16 heads): split over its length
        dict(name="decode_b1_8704", op="decode", n=1, lo=8704, hi=8704, heads=16, kv_heads=16, head_dim=128, page=32,
             order="token", dtype="bf16", window=-1, sinks=0, mix=9),
        # 64 sequences of very different lengths, 32 query heads on 8 key-value heads
        dict(name="decode_b64_ragged", op="decode", n=64, lo=1, hi=8192, heads=32, kv_heads=8, head_dim=128, page=16,
             order="token", dtype="bf16", window=-1, sinks=0, mix=10),
        # long sequences of which a token sees 4 first tokens and the last 4096: heads of 64, one key head per 8
        dict(name="decode_b16_window", op="decode", n=16, lo=5000, hi=60000, heads=64, kv_heads=8, head_dim=64, page=64,
             order="head", dtype="bf16", window=4095, sinks=4, mix=11),
        # a causal prompt of 8704 rows, 16 heads: a window of 4096 and 4 sinks
        dict(name="prompt_8704_causal", op="prompt", n=1, lo=8704, hi=8704, past=0, heads=16, kv_heads=16, head_dim=128,
             dtype="bf16", left=4095, right=0, sinks=4, mix=12),
        # ragged prompts seen on both sides (a vicinity of 256), grouped heads
        dict(name="prompt_ragged_both", op="prompt", n=8, lo=70, hi=2048, past=0, heads=32, kv_heads=8, head_dim=128,
             dtype="bf16", left=256, right=256, sinks=16, mix=13),
        # the fp32 model's sequence (96 positions, 4 heads of 64): latency
        dict(name="prompt_fp32_96", op="prompt", n=1, lo=96, hi=96, past=0, heads=4, kv_heads=4, head_dim=64,
             dtype="fp32", left=31, right=31, sinks=2, mix=14),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _one(rng):
    op = rng.choice(("append", "pages", "decode", "decode", "prompt", "prompt"))
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    group = rng.choice((1, 2, 3, 4, 7, 8))
    page = rng.choice((8, 16, 24, 32, 64, 128))
    mix = rng.randrange(1 << 20)
    order = rng.choice(("token", "head"))
    base = dict(op=op, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, mix=mix)
    if op == "append":
        n = _log(rng, 1, 96)
        hi = _log(rng, 16, 8704)
        return dict(base, n=n, lo=max(1, hi // rng.choice((1, 3, 10))), hi=hi, heads=kv_heads * group, page=page, order=order,
                    rows=rng.choice((1, 1, _log(rng, 1, 8704))))
    if op == "pages":
        hi = _log(rng, 10, 3000)
        layers = rng.choice((1, 2, 4, 8, 16))
        if rng.random() < 0.5:
            n = _log(rng, 1, 32)
            return dict(base, kind="fork", share=rng.random() < 0.5, n=n, sources=rng.randint(1, n), lo=max(1, hi // 4), hi=hi,
                        layers=layers, page=page, order=order)
        return dict(base, kind="compact", n=_log(rng, 1, 64), lo=max(1, hi // 4), hi=hi, shared=rng.randint(0, 3), layers=layers,
                    page=page, order=order, fill=round(rng.uniform(0.3, 0.9), 2))
    if op == "decode":
        hi = _log(rng, 1, 60000)
        window = rng.choice((-1, -1, 0, _log(rng, 1, 8192)))
        return dict(base, n=_log(rng, 1, 96), lo=max(1, hi // rng.choice((1, 5, 50))), hi=hi, heads=kv_heads * group, page=page,
                    order=order, window=window, sinks=0 if window < 0 else rng.choice((0, 1, 4, 37)))
    hi = _log(rng, 1, 8704 if dtype == "bf16" else 1500)
    left, right = rng.choice(((-1, 0), (-1, -1), (_log(rng, 1, 4096), 0), (_log(rng, 1, 1024), _log(rng, 1, 1024))))
    return dict(base, n=_log(rng, 1, 12), lo=max(1, hi // rng.choice((1, 3, 20))), hi=hi, past=rng.choice((0, 0, _log(rng, 1, 2000))),
                heads=kv_heads * group, left=left, right=right, sinks=rng.choice((0, 4, 130)))


def draw(rng):
    """A case of the same ranges: no more work than the largest listed one, nor more memory in its plain form."""
    while True:
        c = _one(rng)
        w = work(c)
        if w["bytes"] > 1.5e9 or w["flops"] > 2.5e11 or w["bytes"] < 2e3:
            continue
        lens = _lens(c)
        if c["op"] == "prompt" and len(lens) * c["heads"] * max(lens) * (max(lens) + c["past"]) > 1.3e9:
            continue  # the plain form's scores
        if c["op"] == "decode" and len(lens) * max(lens) * c["heads"] * c["head_dim"] > 1.5e9:
            continue  # the plain form's gathered keys
        if c["op"] in ("append", "pages") and (sum(lens) + max(lens) * c["n"]) * c.get("layers", 1) * c["kv_heads"] * c["head_dim"] > 6e8:
            continue  # the cache
        return c


def _lens(case):
    """The sequences' lengths: spread over the logarithm from lo to hi, both ends among them."""
    r = random.Random(case["mix"])
    n = case["sources"] if case.get("kind") == "fork" else case["n"]
    lens = [_log(r, case["lo"], case["hi"]) for _ in range(n)]
    lens[0] = case["hi"]
    if n > 1:
        lens[-1] = case["lo"]
    return lens


def _rows(case):
    return [min(case["rows"], x) for x in _lens(case)]


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    lens = _lens(case)
    row = case["kv_heads"] * case["head_dim"] * _size(case) * 2  # keys and values of one token, one layer
    if case["op"] == "append":
        rows = sum(_rows(case))
        return {"bytes": 2 * rows * row + 4 * (rows + 3 * case["n"]), "flops": 0}
    if case["op"] == "pages":
        page, layers = case["page"], case["layers"]
        held = [-(-x // page) for x in lens]
        if case["kind"] == "fork":
            src = [lens[i % len(lens)] for i in range(case["n"])]
            tokens = sum(x % page if case["share"] else x for x in src)
            return {"bytes": 2 * tokens * row * layers + 8 * sum(-(-x // page) for x in src), "flops": 0}
        pages, live, moved = _compact_plan(case)
        return {"bytes": 2 * moved * page * row * layers + 4 * (pages + 2 * sum(held)), "flops": 0}
    if case["op"] == "decode":
        seen = sum(int(_seen(np.array([x - 1]), x, case["window"], 0, case["sinks"])[0]) for x in lens)
        ends = 2 * len(lens) * case["heads"] * case["head_dim"] * _size(case)
        return {"bytes": seen * row + ends + 4 * sum(-(-x // case["page"]) for x in lens), "flops": 4 * seen * case["heads"] * case["head_dim"]}
    seen = sum(int(_seen(np.arange(x) + case["past"], x + case["past"], case["left"], case["right"], case["sinks"]).sum()) for x in lens)
    ends = 2 * sum(lens) * case["heads"] * case["head_dim"] * _size(case)
    return {"bytes": ends + (sum(lens) + case["past"] * len(lens)) * row, "flops": 4 * seen * case["heads"] * case["head_dim"]}


def _seen(p, keys, left, right, sinks):
    """How many of `keys` keys each position p sees."""
    hi = np.full_like(p, keys - 1) if right < 0 else np.minimum(keys - 1, p + right)
    lo = np.zeros_like(p) if left < 0 else np.maximum(0, p - left)
    both = np.maximum(0, hi - lo + 1)
    return both + np.maximum(0, np.minimum(np.minimum(sinks, lo), hi + 1))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    return _ints([0] + list(np.cumsum(v)))


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype) if math.prod(shape) < 1 << 28 else \
        torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _store(case, layers, pages, g):
    """One of the two cache tensors, viewed as [layers, pages, page_size, kv_heads, head_dim]."""
    dt = _TYPES[case["dtype"]]
    if case["order"] == "token":
        return _normal((layers, pages, case["page"], case["kv_heads"], case["head_dim"]), g, dt)
    return _normal((layers, pages, case["kv_heads"], case["page"], case["head_dim"]), g, dt).transpose(2, 3)


def _compact_plan(case):
    """Pages of the cache, how many are live and how many of those lie behind the live count: by the case alone."""
    first, table, refs = _compact_tables(case)
    live = int((refs > 0).sum())
    return len(refs), live, int((refs[live:] > 0).sum())


def _compact_tables(case):
    lens, page = _lens(case), case["page"]
    held = [-(-x // page) for x in lens]
    shared = min([case["shared"]] + [x // page for x in lens])
    live = shared + sum(h - shared for h in held)
    pages = max(live + 1, int(live / case["fill"]))
    at = np.random.RandomState(case["mix"] % (1 << 31)).permutation(pages)[:live]
    table = np.full((len(lens), max(held)), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    used = shared
    for s, h in enumerate(held):
        table[s, :shared] = at[:shared]
        table[s, shared:h] = at[used:used + h - shared]
        used += h - shared
        refs[table[s, :h]] += 1
    return lens, table, refs


def _tables(case, lens, spare, seqs):
    """Scattered pages for the sequences: (table, refs) with `spare` more pages and `seqs` rows in all."""
    page = case["page"]
    held = [-(-x // page) for x in lens]
    pages = sum(held) + spare
    at = np.random.RandomState((case["mix"] + 17) % (1 << 31)).permutation(pages)
    table = np.full((seqs, max(held)), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    used = 0
    for s, h in enumerate(held):
        table[s, :h] = at[used:used + h]
        refs[at[used:used + h]] = 1
        used += h
    return table, refs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    dt = _TYPES[case["dtype"]]
    lens, hd = _lens(case), case["head_dim"]
    st = {"case": case, "op": case["op"], "page": case.get("page", 0), "scale": 1.0 / math.sqrt(hd)}
    if case["op"] == "prompt":
        total, keys = sum(lens), sum(lens) + case["past"] * len(lens)
        q_of, k_of = case["heads"] * hd, case["kv_heads"] * hd
        if case["past"]:
            q = _normal((total, case["heads"], hd), g, dt)
            k, v = (_normal((keys, case["kv_heads"], hd), g, dt) for _ in range(2))
        else:  # the three parts of one projection's output
            x = _normal((total, q_of + 2 * k_of), g, dt)
            q = x[:, :q_of].unflatten(1, (-1, hd))
            k = x[:, q_of:q_of + k_of].unflatten(1, (-1, hd))
            v = x[:, q_of + k_of:].unflatten(1, (-1, hd))
        st.update(q=q, k=k, v=v, cu_q=_cum(lens), cu_k=_cum([x + case["past"] for x in lens]), left=case["left"],
                  right=case["right"], sinks=case["sinks"], most_q=max(lens), most_k=max(lens) + case["past"])
    else:
        if case["op"] == "pages" and case["kind"] == "compact":
            _, table, refs = _compact_tables(case)
            st.update(table0=_ints(table), refs0=_ints(refs), lens0=_ints(lens))
        elif case["op"] == "pages":
            need = [-(-lens[i % len(lens)] // case["page"]) for i in range(case["n"])]
            table, refs = _tables(case, lens, sum(need) + 3, len(lens) + case["n"])
            st.update(src=_ints([i % len(lens) for i in range(case["n"])]), dst=_ints(range(len(lens), len(lens) + case["n"])),
                      share=case["share"])
            lens = lens + [0] * case["n"]
        else:
            table, refs = _tables(case, lens, 2, len(lens))
        layers = case.get("layers", 1)
        st.update(k=_store(case, layers, len(refs), g), v=_store(case, layers, len(refs), g), table=_ints(table), lens=_ints(lens),
                  refs=_ints(refs))
        if case["op"] == "append":
            rows = _rows(case)
            q_of, k_of = case["heads"] * hd, case["kv_heads"] * hd
            x = _normal((sum(rows), q_of + 2 * k_of), g, dt)
            st.update(new_k=x[:, q_of:q_of + k_of].unflatten(1, (-1, hd)), new_v=x[:, q_of + k_of:].unflatten(1, (-1, hd)),
                      rows=_cum(rows) if case["rows"] > 1 else None)
        if case["op"] == "decode":
            x = _normal((case["n"], (case["heads"] + 2 * case["kv_heads"]) * hd), g, dt)
            st.update(q=x[:, :case["heads"] * hd].unflatten(1, (-1, hd)), window=case["window"], sinks=case["sinks"],
                      most=max(lens))
    if own:
        from block_denoising_gb300 import dinfer
        st["ops"] = dinfer
        if case["op"] in ("decode", "prompt"):
            st["ws"] = dinfer.OpWorkspace()
        if case["op"] != "prompt":
            st["kv"] = dinfer.PagedKV(st["k"], st["v"], st["table"], st["lens"], st["refs"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    return _own(st) if own else _PLAIN[st["op"]](st)


def _own(st):
    op = st["op"]
    if op == "prompt":
        return st["ops"].op_window_attention(st["q"], st["k"], st["v"], st["ws"], cu_q=st["cu_q"], cu_k=st["cu_k"], left=st["left"],
                                             right=st["right"], sinks=st["sinks"], scale=st["scale"])
    kv = st["kv"]
    if op == "decode":
        return kv.attention(0, st["q"], st["ws"], window=st["window"], sinks=st["sinks"], scale=st["scale"])
    if op == "append":
        kv.append(0, st["new_k"], st["new_v"], rows=st["rows"])
        return {"k": st["k"], "v": st["v"]}
    if "src" in st:
        kv.free(st["dst"])
        kv.fork(st["src"], st["dst"], share=st["share"])
    else:
        kv.set_tables(st["table0"], st["lens0"], st["refs0"])
        kv.compact()
    return {n: st[n] for n in ("k", "v", "table", "lens", "refs")}


def _plain_append(st):
    lens, page = st["lens"].long(), st["page"]
    n = len(lens)
    rows = torch.ones_like(lens) if st["rows"] is None else (st["rows"][1:] - st["rows"][:-1]).long()
    start = torch.cumsum(rows, 0) - rows
    total = st["new_k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), rows, output_size=total)
    pos = (lens - rows - start)[seq] + torch.arange(total, device="cuda")
    at = st["table"][seq, pos // page].long(), pos % page
    st["k"][0][at] = st["new_k"]
    st["v"][0][at] = st["new_v"]
    return {"k": st["k"], "v": st["v"]}


def _plain_pages(st):
    page, table, lens, refs = st["page"], st["table"], st["lens"], st["refs"]
    k, v = st["k"], st["v"]
    slots = torch.arange(table.shape[1], device="cuda")
    if "src" not in st:
        table.copy_(st["table0"])
        lens.copy_(st["lens0"])
        refs.copy_(st["refs0"])
        live = refs > 0
        count = int(live.sum())
        index = torch.arange(len(refs), device="cuda")
        src, dst = index[live & (index >= count)], index[~live & (index < count)]
        k[:, dst], v[:, dst] = k[:, src], v[:, src]
        refs[dst] = refs[src]
        refs[src] = 0
        to = index.to(torch.int32)
        to[src] = dst.to(torch.int32)
        table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    else:
        src, dst = st["src"].long(), st["dst"].long()
        held = (lens[dst] + page - 1) // page  # freed
        old = table[dst][slots < held[:, None]].long()
        refs.index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
        table[dst] = -1
        lens[dst] = 0
        size = lens[src]  # forked
        held = (size + page - 1) // page
        kept = size // page if st["share"] else torch.zeros_like(size)
        shared, fresh = slots < kept[:, None], (slots >= kept[:, None]) & (slots < held[:, None])
        pages = table[src]
        old = pages[shared].long()
        refs.index_add_(0, old, torch.ones_like(old, dtype=torch.int32))
        was = pages[fresh].long()
        now = torch.nonzero(refs == 0)[:len(was), 0]
        refs[now] = 1
        pages[fresh] = now.to(torch.int32)
        table[dst] = torch.where(slots < held[:, None], pages, -1)
        lens[dst] = size
        which, nth = torch.nonzero(fresh, as_tuple=True)  # the tokens of each copied page
        pair, slot = torch.nonzero(torch.arange(page, device="cuda") < (size[which] - nth * page)[:, None], as_tuple=True)
        k[:, now[pair], slot], v[:, now[pair], slot] = k[:, was[pair], slot], v[:, was[pair], slot]
    return {n: st[n] for n in ("k", "v", "table", "lens", "refs")}


def _attend(q, k, v, seen, scale):
    """softmax(scale q k^T) v over the keys that `seen` names; q, k, v [..., rows or keys, head_dim] in 32 bits."""
    s = torch.where(seen, (q @ k.transpose(-1, -2)) * scale, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, (p @ v) / total, 0.0)


def _plain_decode(st):
    q, lens, page = st["q"], st["lens"], st["page"]
    n, heads, hd = q.shape
    pos = torch.arange(st["most"], device="cuda")
    seen = pos < lens[:, None]
    if st["window"] >= 0:
        seen = seen & ((pos >= lens[:, None] - 1 - st["window"]) | (pos < st["sinks"]))
    at = st["table"][:, pos // page].clamp(min=0).long(), (pos % page).expand(n, -1)
    wipe = ~seen[:, :, None, None]
    k = st["k"][0][at].float().masked_fill(wipe, 0.0).transpose(1, 2)  # [n, kv_heads, keys, head_dim]
    v = st["v"][0][at].float().masked_fill(wipe, 0.0).transpose(1, 2)
    o = _attend(q.float().reshape(n, k.shape[1], -1, hd), k, v, seen[:, None, None], st["scale"])
    return o.reshape(n, heads, hd).to(q.dtype)


def _plain_prompt(st):
    q, cu_q, cu_k = st["q"], st["cu_q"].long(), st["cu_k"].long()
    rows, heads, hd = q.shape
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(st["most_q"], device="cuda"), torch.arange(st["most_k"], device="cuda")
    at_q = (cu_q[:-1, None] + i).clamp(max=rows - 1)
    at_k = (cu_k[:-1, None] + j).clamp(max=st["k"].shape[0] - 1)
    p = (nk - nq)[:, None, None] + i[:, None]  # positions
    seen = (j < nk[:, None, None]) & (i < nq[:, None])[:, :, None]
    if st["right"] >= 0:
        seen = seen & (j <= p + st["right"])
    if st["left"] >= 0:
        seen = seen & ((j >= p - st["left"]) | (j < st["sinks"]))
    group = heads // st["k"].shape[1]
    k = st["k"][at_k].float().transpose(1, 2).repeat_interleave(group, 1)
    v = st["v"][at_k].float().transpose(1, 2).repeat_interleave(group, 1)
    o = _attend(q[at_q].float().transpose(1, 2), k, v, seen[:, None], st["scale"]).transpose(1, 2).to(q.dtype)
    return o[(i < nq[:, None])]


_PLAIN = {"append": _plain_append, "pages": _plain_pages, "decode": _plain_decode, "prompt": _plain_prompt}


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
    lens = _lens(case)
    if case["op"] == "prompt":
        return _exact_prompt(case, st, lens)
    if case["op"] == "decode":
        return _exact_decode(case, st, lens)
    return _exact_moves(case, st, lens)


def _exact_rows(q, k, v, lo, hi, sinks, scale):
    """Rows q [rows, hd] over keys lo[r] .. hi[r] and the first `sinks` up to hi[r]: sums of 64-bit weights."""
    j = torch.arange(k.shape[0], device="cuda")
    out = ((j >= lo[:, None]) | (j < sinks)).logical_and_(j <= hi[:, None]).logical_not_()
    w = torch.matmul(q.double(), k.double().T).mul_(scale).masked_fill_(out, -math.inf)
    top = w.max(dim=1, keepdim=True).values
    w.sub_(top.nan_to_num(neginf=0.0)).exp_()
    return torch.matmul(w, v.double()) / w.sum(1, keepdim=True).clamp(min=1e-300)


def _exact_prompt(case, st, lens):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    a = b = 0
    for n in lens:
        m = n + case["past"]
        p = torch.arange(n, device="cuda") + case["past"]
        hi = torch.full_like(p, m - 1) if case["right"] < 0 else torch.clamp(p + case["right"], max=m - 1)
        lo = torch.zeros_like(p) if case["left"] < 0 else torch.clamp(p - case["left"], min=0)
        for h in range(case["heads"]):
            out[a:a + n, h] = _exact_rows(st["q"][a:a + n, h], st["k"][b:b + m, h // group], st["v"][b:b + m, h // group], lo, hi,
                                          case["sinks"], st["scale"])
        a, b = a + n, b + m
    return out


def _exact_decode(case, st, lens):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    group, table, page = case["heads"] // case["kv_heads"], st["table"].cpu().numpy(), case["page"]
    for s, n in enumerate(lens):
        pages = torch.from_numpy(table[s, :-(-n // page)].astype(np.int64)).cuda()
        k = st["k"][0, pages].flatten(0, 1)[:n]
        v = st["v"][0, pages].flatten(0, 1)[:n]
        first = 0 if case["window"] < 0 else max(0, n - 1 - case["window"])
        keep = list(range(min(case["sinks"], first))) + list(range(first, n))
        keep = torch.tensor(keep, device="cuda")
        k, v = k[keep], v[keep]
        lo, hi = (torch.full((group,), x, device="cuda") for x in (0, len(keep) - 1))
        for h in range(case["kv_heads"]):
            out[s, h * group:(h + 1) * group] = _exact_rows(st["q"][s, h * group:(h + 1) * group], k[:, h], v[:, h], lo, hi, 0, st["scale"])
    return out


def _exact_moves(case, st, lens):
    """Tables by plain Python on the host; the cache's values are only moved."""
    k, v, page = st["k"].double(), st["v"].double(), case["page"]
    table, refs, size = (st[n].cpu().numpy().copy() for n in ("table", "refs", "lens"))
    if case["op"] == "append":
        a = 0
        for s, r in enumerate(_rows(case)):
            p = np.arange(lens[s] - r, lens[s])
            at, slot = torch.from_numpy(table[s, p // page].astype(np.int64)).cuda(), torch.from_numpy(p % page).cuda()
            k[0, at, slot] = st["new_k"][a:a + r].double()
            v[0, at, slot] = st["new_v"][a:a + r].double()
            a += r
        return {"k": k, "v": v}
    if case["kind"] == "compact":
        live = [p for p in range(len(refs)) if refs[p]]
        holes = [p for p in range(len(live)) if not refs[p]]
        for old, new in zip([p for p in live if p >= len(live)], holes):
            k[:, new] = k[:, old]
            v[:, new] = v[:, old]
            refs[new], refs[old] = refs[old], 0
            table[table == old] = new
    else:
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            size[d] = size[s]
            for i in range(-(-int(size[s]) // page)):
                there = min(page, int(size[s]) - i * page)
                if case["share"] and there == page:
                    table[d, i] = table[s, i]
                    refs[table[s, i]] += 1
                    continue
                new = int(np.flatnonzero(refs == 0)[0])
                table[d, i], refs[new] = new, 1
                k[:, new, :there] = k[:, int(table[s, i]), :there]
                v[:, new, :there] = v[:, int(table[s, i]), :there]
    return {"k": k, "v": v, "table": torch.from_numpy(table), "lens": torch.from_numpy(size), "refs": torch.from_numpy(refs)}
