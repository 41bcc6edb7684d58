"""Measured cases of the decoder-layer operators between two weight products: rotary positions with the append to a
paged key / value cache, attention of new tokens over that cache, and the management of its pages.

``own`` False computes each operator in its plain form (elementary torch operations in 32 bits, rounded once at the
end); ``own`` True makes the library calls a user makes.  ``exact`` gives the same results from the definition in 64
bits.  Everything about a case, its ragged lengths included, follows from its dict alone; only the values of the
inputs come from the seed.
"""
import collections
import itertools
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "f16": 1, "bf16": 2}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases ---------------------------------------------------------------------------------------------------------

def _rotary(name, batch, q, kv, hq, hkv, d, rot, layout, dtype, page, order, ragged=False, lens_seed=1):
    return {"name": name, "op": "append", "batch": batch, "q": q, "kv": kv, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "layout": layout, "dtype": dtype, "page": page, "order": order, "ragged": ragged, "lens_seed": lens_seed}


def _attend(name, batch, q, kv, hq, hkv, d, dtype, page, order, window=0, ragged=False, lens_seed=1):
    return {"name": name, "op": "attend", "batch": batch, "q": q, "kv": kv, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "page": page, "order": order, "window": window, "ragged": ragged, "lens_seed": lens_seed}


def listed():
    return [
        # one token of one sequence between the QKV product and its attention: latency counts
        _rotary("append_1_token", 1, 1, 1500, 32, 8, 128, 128, "half", "bf16", 16, "hnd"),
        # three prompts of different lengths, packed into one call
        _rotary("append_prompts", 3, 5000, 5000, 32, 8, 128, 128, "half", "bf16", 64, "hnd", True, 5),
        # the gradient of a partial interleaved rotation, on heads that are a slice of a wider row
        {"name": "rotary_gradient", "op": "rotate", "tokens": 4999, "heads": 18, "d": 96, "rot": 64, "n_pos": 16384,
         "layout": "interleaved", "dtype": "f32", "inverse": True, "pad_heads": 5},
        # the next token of one conversation
        _attend("decode_1x777", 1, 1, 777, 32, 8, 128, "bf16", 16, "hnd"),
        # the next token of a full serving batch, contexts of very different lengths
        _attend("decode_64_ragged", 64, 1, 8192, 32, 8, 128, "bf16", 16, "hnd", 0, True, 7),
        # the next token at the end of one very long document
        _attend("decode_1x131001", 1, 1, 131001, 64, 8, 128, "f16", 64, "nhd"),
        # a few drafted tokens per sequence, checked at once under a sliding window
        _attend("draft_16x8_window", 16, 8, 4000, 16, 4, 64, "f16", 32, "nhd", 1024, True, 9),
        # two whole prompts
        _attend("prompt_2x4096", 2, 4096, 4096, 32, 8, 128, "bf16", 64, "hnd"),
        # one chunk of a long prompt that is fed in pieces
        _attend("chunk_500_of_32000", 1, 500, 32000, 32, 8, 128, "bf16", 16, "hnd"),
        # pages moved by a given list, over the keys and values of all layers
        {"name": "pages_copy", "op": "copy", "planes": 32, "pages": 2500, "page_elems": 16384, "n": 700,
         "lens_seed": 3},
        # samples of one prompt: each shares its pages and gets its own copy of the last one when it grows
        {"name": "fan_out_12", "op": "fan", "planes": 48, "pages": 900, "page_elems": 8192, "page": 16, "seqs": 13,
         "prompt": 1003, "n": 12, "grow": 5, "lens_seed": 4},
        # a cache with holes is pressed together
        {"name": "compact_40pc", "op": "compact", "planes": 32, "pages": 3000, "page_elems": 8192, "page": 16,
         "seqs": 60, "live": 0.6, "lens_seed": 6},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rotate", "attend", "attend", "attend", "copy", "fan", "compact"])
    seed = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    page, order = rng.choice([16, 32, 64, 128]), rng.choice(["hnd", "nhd"])
    if op == "append":
        c = _rotary("", _log_int(rng, 1, 40), 1, 1, 1, rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 256]), 0,
                    rng.choice(["half", "interleaved"]), rng.choice(["bf16", "f16", "f32"]), page, order,
                    rng.random() < 0.7, seed)
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 5, 7, 8])
        c["rot"] = rng.choice([c["d"], c["d"] // 2])
        c["q"] = 1 if rng.random() < 0.3 else _log_int(rng, 1, max(2, 40_000_000 // (c["batch"] * c["hq"] * c["d"] * ESIZE[c["dtype"]])))
        c["q"] = min(c["q"], 5000)
        c["kv"] = c["q"] + (0 if rng.random() < 0.5 else _log_int(rng, 1, 3000))
        c.pop("name")
        return c
    if op == "rotate":
        d = rng.choice([64, 80, 96, 128, 256])
        heads = rng.randint(1, 40)
        return {"op": op, "tokens": _log_int(rng, 1, max(2, 30_000_000 // (heads * d * 4))), "heads": heads, "d": d,
                "rot": rng.choice([d, d // 2]), "n_pos": rng.choice([4096, 32768]), "layout": rng.choice(["half", "interleaved"]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "inverse": rng.random() < 0.4, "pad_heads": rng.choice([0, 1, 8])}
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
        d = rng.choice([64, 80, 96, 128, 128, 128, 256])
        q = rng.choice([1, 1, _log_int(rng, 1, 64), _log_int(rng, 16, 2048)])
        batch = _log_int(rng, 1, 64 if q <= 64 else 8)
        # no more than about half of the largest listed traffic and arithmetic, padded to the longest
        most = min(300e6 / (batch * hkv * d * 4), 120e9 / (4.0 * d * hq * q * batch), 70000)
        kv = max(q, _log_int(rng, 1, max(2, most)))
        window = 0 if rng.random() < 0.7 else _log_int(rng, 1, 2000)
        c = _attend("", batch, q, kv, hq, hkv, d, dtype, page, order, window, batch > 1 and rng.random() < 0.7, seed)
        c.pop("name")
        while work(c)["flops"] > 200e9 and c["q"] > 1:
            c["q"], c["kv"] = c["q"] // 2, max(c["q"] // 2, c["kv"] // 2)
        return c
    planes = rng.choice([2, 16, 33, 48])
    elems = page * rng.choice([64, 256, 512])
    if op == "copy":
        n = _log_int(rng, 1, max(2, min(2000, 350_000_000 // (planes * elems))))
        return {"op": op, "planes": planes, "pages": 2 * n + rng.randint(1, 50), "page_elems": elems, "n": n, "lens_seed": seed}
    if op == "fan":
        n, prompt, grow = _log_int(rng, 1, 40), _log_int(rng, 1, 3000), rng.randint(1, 20)
        need = -(-prompt // page) + n * (-(-grow // page) + 1)
        return {"op": op, "planes": planes, "pages": need + rng.randint(0, 100), "page_elems": elems, "page": page, "seqs": n + 1 + rng.randint(0, 5),
                "prompt": prompt, "n": n, "grow": grow, "lens_seed": seed}
    return {"op": op, "planes": planes, "pages": _log_int(rng, 20, max(40, min(4000, 700_000_000 // (planes * elems)))), "page_elems": elems,
            "page": page, "seqs": rng.randint(1, 100), "live": rng.choice([0.1, 0.4, 0.7, 0.95]), "lens_seed": seed}


def _lengths(case):
    """(new tokens, keys with the new ones) of each sequence of the call."""
    r = random.Random(case["lens_seed"])
    more = case["batch"] - 1
    if not case["ragged"]:
        return [case["q"]] * (more + 1), [case["kv"]] * (more + 1)
    q_lens = [r.randint(1, case["q"]) for _ in range(more)]
    kv_lens = [max(n, int(case["kv"] * math.exp(-2.5 * r.random()))) for n in q_lens]
    return [case["q"]] + q_lens, [case["kv"]] + kv_lens


def _visible(case):
    """(rows times visible keys, keys that some row sees), over the sequences."""

    def one(nq, nk):
        w = case["window"] or nk
        first = nk - nq  # position of the first new token
        full = max(0, min(nq, w - first - 1))  # rows that see fewer than w keys
        return full * (first + 1) + full * (full - 1) // 2 + (nq - full) * w, nk - max(0, first - w + 1)

    seen = [one(*n) for n in zip(*_lengths(case))]
    return sum(n for n, _ in seen), sum(n for _, n in seen)


def _holes(case):
    """The compacted cache: rows of pages (one per sequence), its reference counts and lengths, as lists."""
    r = random.Random(case["lens_seed"])
    order = list(range(case["pages"]))
    r.shuffle(order)
    live = max(1, int(case["live"] * case["pages"]))
    seqs = case["seqs"]
    tables = [order[live * i // seqs:live * (i + 1) // seqs] for i in range(seqs)]
    if seqs > 1:  # the last sequence shares the start of the first one
        tables[-1] = tables[0][:len(tables[0]) // 2] + tables[-1]
    held = collections.Counter(p for row in tables for p in row)
    refs = [held[p] for p in range(case["pages"])]
    lens = [max(0, len(row) * case["page"] - (i % case["page"])) for i, row in enumerate(tables)]
    return tables, refs, lens


def work(case):
    op = case["op"]
    if op == "rotate":
        e = ESIZE[case["dtype"]]
        n = case["tokens"] * case["heads"] * case["d"]
        rows = min(case["tokens"], case["n_pos"])
        return {"bytes": 2 * n * e + rows * case["rot"] * 4 + case["tokens"] * 4, "flops": 3 * n * case["rot"] / case["d"]}
    if op == "append":
        q_lens, kv_lens = _lengths(case)
        t, e = sum(q_lens), ESIZE[case["dtype"]]
        n = t * (case["hq"] + 2 * case["hkv"]) * case["d"]
        rows = len({p for a, b in zip(q_lens, kv_lens) for p in range(b - a, b)})
        return {"bytes": 2 * n * e + rows * case["rot"] * 4, "flops": 3 * t * (case["hq"] + case["hkv"]) * case["rot"]}
    if op == "attend":
        pairs, keys = _visible(case)
        t, e = sum(_lengths(case)[0]), ESIZE[case["dtype"]]
        return {"bytes": 2 * keys * case["hkv"] * case["d"] * e + 2 * t * case["hq"] * case["d"] * e + 4 * t * case["hq"] + 4 * keys // case["page"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    page_bytes = 2 * case["page_elems"] * case["planes"]
    if op == "copy":
        return {"bytes": 2 * case["n"] * page_bytes + 8 * case["n"], "flops": 0}
    if op == "fan":
        n, ps = case["n"], case["page"]
        held = -(-case["prompt"] // ps)
        copies = n if case["prompt"] % ps else 0
        return {"bytes": 2 * copies * page_bytes + 8 * n * held + 4 * case["pages"], "flops": 0}
    tables, refs, _ = _holes(case)
    live = sum(1 for x in refs if x)
    moved = sum(1 for x in refs[live:] if x)
    return {"bytes": 2 * moved * page_bytes + 8 * case["pages"] + 8 * sum(len(t) for t in tables), "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------------------------

def _normal(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(DT[dtype])


def _angles(n_pos, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    t = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return t.cos().float(), t.sin().float()


def _paged(case, s, gen):
    """Pages of keys and values in a shuffled order, with the tables and lengths of the call's sequences."""
    q_lens, kv_lens = _lengths(case)
    ps, hkv, d = case["page"], case["hkv"], case["d"]
    held = [-(-n // ps) for n in kv_lens]
    total = sum(held) + 3
    shape = (total, hkv, ps, d) if case["order"] == "hnd" else (total, ps, hkv, d)
    s["k_pages"] = _normal(shape, case["dtype"], gen)
    s["v_pages"] = _normal(shape, case["dtype"], gen)
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(max(held), device="cuda")
    n = torch.tensor(held, device="cuda")[:, None]
    s["tables"] = torch.where(col < n, perm[((torch.cumsum(n, 0) - n) + col).clamp(max=total - 1)], -1).to(torch.int32)
    starts = list(itertools.accumulate(q_lens, initial=0))
    s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["tokens"], s["max_q"], s["max_kv"] = starts[-1], max(q_lens), max(kv_lens)
    s["q_lens"], s["kv_list"] = q_lens, kv_lens


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "rotate":
        t, h, d = case["tokens"], case["heads"], case["d"]
        s["cos"], s["sin"] = _angles(case["n_pos"], case["rot"])
        s["x"] = _normal((t, h + case["pad_heads"], d), case["dtype"], gen)[:, :h]
        s["positions"] = torch.randint(0, case["n_pos"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        s["y"] = torch.empty((t, h, d), dtype=DT[case["dtype"]], device="cuda")
    elif op == "append":
        _paged(case, s, gen)
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        s["n_pos"] = s["max_kv"]
        s["cos"], s["sin"] = _angles(s["n_pos"], case["rot"])
        qkv = _normal((s["tokens"], hq + 2 * hkv, d), case["dtype"], gen)  # one row of the QKV product per token
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["y"] = torch.empty((s["tokens"], hq, d), dtype=DT[case["dtype"]], device="cuda")
    elif op == "attend":
        _paged(case, s, gen)
        # rotated queries of norm 2 sqrt(d): scores of deviation 2, as of a head that looks at some keys more than at others
        s["q"] = _normal((s["tokens"], case["hq"], case["d"]), case["dtype"], gen, 2.0)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((s["tokens"], case["hq"]), dtype=torch.float32, device="cuda")
        s["scale"] = case["d"] ** -0.5
    else:
        # the bits of 16-bit keys and values: they are moved, never computed with
        s["pool"] = _normal((case["planes"], case["pages"], case["page_elems"]), "bf16", gen).view(torch.int16)
        if op == "copy":
            perm = torch.randperm(case["pages"], generator=gen, device="cuda").to(torch.int32)
            s["src"], s["dst"] = perm[:case["n"]].contiguous(), perm[case["n"]:2 * case["n"]].contiguous()
        elif op == "fan":
            held = -(-case["prompt"] // case["page"])
            width = held + -(-case["grow"] // case["page"])
            pages = torch.randperm(case["pages"], generator=gen, device="cuda")[:held].to(torch.int32)
            s["tables"] = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")
            s["tables"][0, :held] = pages
            s["refs"] = torch.zeros(case["pages"], dtype=torch.int32, device="cuda")
            s["refs"][pages.long()] = 1
            s["lens"] = torch.zeros(case["seqs"], dtype=torch.int32, device="cuda")
            s["lens"][0] = case["prompt"]
            s["src"] = torch.zeros(case["n"], dtype=torch.int32, device="cuda")
            s["dst"] = torch.arange(1, case["n"] + 1, dtype=torch.int32, device="cuda")
            s["new_lens"] = torch.full((case["n"],), case["prompt"] + case["grow"], dtype=torch.int32, device="cuda")
        else:
            tables, refs, lens = _holes(case)
            width = max(1, max(len(t) for t in tables))
            s["tables"] = torch.tensor([t + [-1] * (width - len(t)) for t in tables], dtype=torch.int32, device="cuda")
            s["refs"] = torch.tensor(refs, dtype=torch.int32, device="cuda")
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
            s["refs_out"], s["tables_out"] = torch.empty_like(s["refs"]), torch.empty_like(s["tables"])
            s["counts"] = torch.empty(2, dtype=torch.int32, device="cuda")
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _rotated(x, cos, sin, rot, layout):
    """x [T, H, D] in 32 bits, cos and sin [T, 1, rot / 2]."""
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _rows(s):
    """Sequence and position of each token of the call."""
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
    start, end = s["q_start"].long()[seq], s["q_start"].long()[seq + 1]
    return t, seq, t - start, s["kv_lens"].long()[seq] - (end - start) + (t - start)


def _plain_append(s):
    c = s["case"]
    _, seq, _, pos = _rows(s)
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    k = _rotated(s["k"].float(), cos, sin, c["rot"], c["layout"]).to(s["k_pages"].dtype)
    page, row = s["tables"][seq, pos // c["page"]].long(), pos % c["page"]
    if c["order"] == "hnd":
        s["k_pages"][page, :, row] = k
        s["v_pages"][page, :, row] = s["v"]
    else:
        s["k_pages"][page, row] = k
        s["v_pages"][page, row] = s["v"]
    return _rotated(s["q"].float(), cos, sin, c["rot"], c["layout"]).to(s["q"].dtype)


def _plain_attend(s):
    c = s["case"]
    b, hq, hkv, d, nq = c["batch"], c["hq"], c["hkv"], c["d"], s["max_q"]
    t, seq, i, pos = _rows(s)
    held = s["tables"].clamp(min=0).long()
    nk = held.shape[1] * c["page"]
    there = torch.arange(nk, device="cuda") < s["kv_lens"][:, None]  # [B, keys]

    def gathered(pages):
        x = pages[held].float()
        x = x.permute(0, 2, 1, 3, 4) if c["order"] == "hnd" else x.permute(0, 3, 1, 2, 4)
        return x.reshape(b, hkv, nk, d)

    q = torch.zeros((b, nq, hq, d), device="cuda")
    q[seq, i] = s["q"].float()
    at = torch.full((b, nq), -1, device="cuda", dtype=torch.long)
    at[seq, i] = pos
    q = q.view(b, nq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    scores = (torch.matmul(q, gathered(s["k_pages"]).transpose(2, 3)) * s["scale"]).view(b, hkv, hq // hkv, nq, nk)
    j = torch.arange(nk, device="cuda")
    seen = (j <= at[..., None]) & there[:, None]
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = gathered(s["v_pages"]).masked_fill_(~there[:, None, :, None], 0.0)
    o = torch.matmul(p.view(b, hkv, -1, nk), v).view(b, hkv, -1, nq, d) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, nq, hq, d)[seq, i].to(s["q"].dtype)
    return o, lse.permute(0, 3, 1, 2).reshape(b, nq, hq)[seq, i]


def _count(refs, pages, ok, sign):
    refs.index_add_(0, pages[ok].long(), torch.full_like(pages[ok], sign))


def _plain_fork(s):
    width, ps = s["tables"].shape[1], s["case"]["page"]
    col = torch.arange(width, device="cuda")
    src, dst = s["src"].long(), s["dst"].long()
    rows, lens = s["tables"][src], s["lens"][src]
    mine = s["tables"][dst]
    _count(s["refs"], rows, col < ((lens + ps - 1) // ps)[:, None], 1)
    _count(s["refs"], mine, col < ((s["lens"][dst] + ps - 1) // ps)[:, None], -1)
    s["tables"][dst] = torch.where(col < ((lens + ps - 1) // ps)[:, None], rows, -1)
    s["lens"][dst] = lens


def _plain_resize(s):
    """Sequences s["dst"] grow to s["new_lens"]."""
    ps = s["case"]["page"]
    seqs, new = s["dst"].long(), s["new_lens"]
    old = s["lens"][seqs]
    had, want = (old + ps - 1) // ps, (new + ps - 1) // ps
    last = s["tables"][seqs, (had - 1).clamp(min=0).long()]
    split = (old % ps != 0) & (new > old) & (s["refs"][last.clamp(min=0).long()] > 1)
    need = (want - had).clamp(min=0) + split.int()
    first = torch.cumsum(need, 0) - need
    free = torch.nonzero(s["refs"] == 0).squeeze(1).int()
    col = torch.arange(s["tables"].shape[1], device="cuda", dtype=torch.int32)
    start = had - split.int()  # first column that gets a page
    fresh = (col >= start[:, None]) & (col < want[:, None]) & (need > 0)[:, None]
    at = (first[:, None] + col - start[:, None])[fresh].long()
    old_pages, new_pages = last[split].long(), free[first[split].long()].long()
    s["pool"][:, new_pages] = s["pool"][:, old_pages]
    s["refs"].index_add_(0, old_pages, torch.full_like(last[split], -1))
    s["refs"][free[at].long()] = 1
    rows = s["tables"][seqs]
    rows[fresh] = free[at]
    s["tables"][seqs] = rows
    s["lens"][seqs] = new


def _plain_compact(s):
    refs = s["refs"]
    used = refs > 0
    live = used.sum()
    page = torch.arange(refs.numel(), device="cuda")
    src, dst = torch.nonzero(used & (page >= live)).squeeze(1), torch.nonzero(~used & (page < live)).squeeze(1)
    s["pool"][:, dst] = s["pool"][:, src]
    name = page.clone()
    name[src] = dst
    col = torch.arange(s["tables"].shape[1], device="cuda")
    held = col < ((s["lens"] + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    tables = torch.where(held, name[s["tables"].clamp(min=0).long()].int(), s["tables"])
    refs_out = torch.where(page < live, refs, 0)
    refs_out[dst] = refs[src]
    return tables, refs_out, torch.stack([live, torch.tensor(src.numel(), device="cuda")]).int()


# ---- one pass ------------------------------------------------------------------------------------------------------

def _kept(s, make):
    """The handles and workspaces that a program keeps beside its buffers."""
    if "kept" not in s:
        s["kept"] = make()
    return s["kept"]


def _scratch(nbytes):
    return torch.empty(max(256, nbytes), dtype=torch.uint8, device="cuda")


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "rotate":
            pos = s["positions"].long()
            sin = s["sin"][pos][:, None]
            return _rotated(s["x"].float(), s["cos"][pos][:, None], -sin if c["inverse"] else sin, c["rot"], c["layout"]).to(s["x"].dtype)
        if op == "append":
            return {"q": _plain_append(s), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if op == "attend":
            o, lse = _plain_attend(s)
            return {"o": o, "lse": lse}
        if op == "copy":
            s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
            return {"pool": s["pool"]}
        if op == "fan":
            _plain_fork(s)
            _plain_resize(s)
            return {"pool": s["pool"], "refs": s["refs"], "tables": s["tables"], "lens": s["lens"]}
        tables, refs, counts = _plain_compact(s)
        return {"pool": s["pool"], "refs": refs, "tables": tables, "counts": counts}

    import block_quantized_weight_matmulnbits_gb300 as mnb
    if op == "rotate":
        flags = (mnb.MNB_ROTARY_INTERLEAVED if c["layout"] == "interleaved" else 0) | (mnb.MNB_ROTARY_INVERSE if c["inverse"] else 0)
        mnb.mnb_rotary(s["x"], s["y"], s["positions"], s["cos"], s["sin"], CODE[c["dtype"]], flags=flags)
        return s["y"]
    if op == "append":
        cache = _kept(s, lambda: mnb.kv_cache(s["k_pages"], s["v_pages"], s["tables"], s["kv_lens"], c["order"], CODE[c["dtype"]]))
        mnb.mnb_rotary_append(s["q"], s["y"], s["k"], s["v"], s["cos"], s["sin"], cache, s["q_start"],
                              flags=mnb.MNB_ROTARY_INTERLEAVED if c["layout"] == "interleaved" else 0)
        return {"q": s["y"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "attend":
        cache, ws = _kept(s, lambda: (
            mnb.kv_cache(s["k_pages"], s["v_pages"], s["tables"], s["kv_lens"], c["order"], CODE[c["dtype"]]),
            _scratch(mnb.mnb_attention_workspace_size(c["batch"], s["tokens"], c["hq"], c["hkv"], c["d"], s["max_q"], s["max_kv"], CODE[c["dtype"]]))))
        mnb.mnb_paged_attention(s["q"], s["o"], cache, s["q_start"], s["max_q"], s["max_kv"], s["scale"], lse=s["lse"],
                                window=c["window"], workspace=ws)
        return {"o": s["o"], "lse": s["lse"]}
    if op == "copy":
        planes = _kept(s, lambda: mnb.page_planes(s["pool"]))
        mnb.mnb_pages_copy(planes, s["src"], s["dst"])
        return {"pool": s["pool"]}
    planes, state, ws = _kept(s, lambda: (
        mnb.page_planes(s["pool"]), mnb.cache_state(s["refs"], s["tables"], s["lens"], c["page"]),
        _scratch(mnb.mnb_cache_workspace_size(c["pages"], c["seqs"], s["tables"].shape[1]))))
    if op == "fan":
        mnb.mnb_cache_fork(state, s["src"], s["dst"], workspace=ws)
        mnb.mnb_cache_resize(state, planes, s["dst"], s["new_lens"], workspace=ws)
        return {"pool": s["pool"], "refs": s["refs"], "tables": s["tables"], "lens": s["lens"]}
    mnb.mnb_cache_compact(state, planes, s["refs_out"], s["tables_out"], s["counts"], workspace=ws)
    return {"pool": s["pool"], "refs": s["refs_out"], "tables": s["tables_out"], "counts": s["counts"]}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _turn64(x, pos, cos, sin, rot, layout, sign):
    """Each pair as a complex number, times the table's cos + i sin (or its conjugate)."""
    z = torch.complex(cos.double()[pos], sign * sin.double()[pos])
    y = x.double().clone()
    first, second = (range(0, rot // 2), range(rot // 2, rot)) if layout == "half" else (range(0, rot, 2), range(1, rot, 2))
    first, second = torch.tensor(list(first), device="cuda"), torch.tensor(list(second), device="cuda")
    w = torch.complex(y[..., first], y[..., second]) * z[:, None]
    y[..., first], y[..., second] = w.real, w.imag
    return y


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "rotate":
        return _turn64(s["x"], s["positions"].long(), s["cos"], s["sin"], case["rot"], case["layout"], -1.0 if case["inverse"] else 1.0)
    if op == "append":
        pos = torch.cat([torch.arange(n - m, n) for m, n in zip(s["q_lens"], s["kv_list"])]).cuda()
        q = _turn64(s["q"], pos, s["cos"], s["sin"], case["rot"], case["layout"], 1.0)
        k = _turn64(s["k"], pos, s["cos"], s["sin"], case["rot"], case["layout"], 1.0)
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        t = 0
        for b, (m, n) in enumerate(zip(s["q_lens"], s["kv_list"])):
            p = torch.arange(n - m, n, device="cuda")
            pages, rows = s["tables"][b].long()[p // case["page"]], p % case["page"]
            for to, x in ((kp, k), (vp, s["v"].double())):
                view = to if case["order"] == "nhd" else to.transpose(1, 2)
                view[pages, rows] = x[t:t + m]
            t += m
        return {"q": q, "k_pages": kp, "v_pages": vp}
    if op == "attend":
        if _visible(case)[0] * case["hq"] * case["d"] > 4e11:
            return None
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        t, g = 0, case["hq"] // case["hkv"]
        for b, (m, n) in enumerate(zip(s["q_lens"], s["kv_list"])):
            pages = s["tables"][b, :-(-n // case["page"])].long()
            for h in range(case["hkv"]):
                pick = (lambda x: x[pages, h]) if case["order"] == "hnd" else (lambda x: x[pages, :, h])
                k, v = (pick(x).reshape(-1, case["d"])[:n].double() for x in (s["k_pages"], s["v_pages"]))
                where = torch.arange(n - m, n, device="cuda")[:, None] - torch.arange(n, device="cuda")
                hidden = (where < 0) | (where >= (case["window"] or n + 1))
                for a in range(h * g, h * g + g):
                    z = (s["q"][t:t + m, a].double() @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
                    lse[t:t + m, a] = torch.logsumexp(z, 1)
                    o[t:t + m, a] = torch.softmax(z, 1) @ v
            t += m
        return {"o": o, "lse": lse}
    return None  # the management of pages moves values and computes none
