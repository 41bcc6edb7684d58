"""Measured cases of what follows the attention in a decoder's step: the root-mean-square norm with the residual's
addition (and int8 codes with block scales, the activations of accuracy level 4), a mixture-of-experts layer over
block-quantised weights for a few tokens, and the draw of the next tokens.

``own`` False computes each operator in its plain form (elementary torch operations in 32 bits, in 64 where sums of many
small weights decide a token, rounded once at the end); ``own`` True makes the library calls a user makes.  ``exact``
gives the same results from the definition in 64 bits.  Everything about a case, the experts its tokens pick included,
follows from its dict alone; only the values of the inputs come from the seed.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "f16": 1, "bf16": 2}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases ---------------------------------------------------------------------------------------------------------

def _norm(name, rows, width, dtype, residual, out, block=32, offset=False, pad=0):
    """out: "y" (values of dtype), "codes" (int8 and a scale for each block of a row)."""
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "residual": residual, "out": out,
            "block": block, "offset": offset, "pad": pad}


def _moe(name, tokens, top_k, experts, hidden, inner, bits, bs, dtype, scale_dtype, zp, scoring="softmax", lens_seed=1):
    return {"name": name, "op": "moe", "tokens": tokens, "top_k": top_k, "experts": experts, "hidden": hidden,
            "inner": inner, "bits": bits, "bs": bs, "dtype": dtype, "scale_dtype": scale_dtype, "zp": zp,
            "scoring": scoring, "lens_seed": lens_seed}


def _sample(name, rows, vocab, dtype, cuts, masked=0.0, lens_seed=1):
    """cuts: "all" (top-k, top-p and min-p), "top_p", "none", or "mixed" (each row its own, greedy ones among them)."""
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "cuts": cuts, "masked": masked,
            "lens_seed": lens_seed}


def listed():
    return [
        # one token between the output product and the next int8-activation product: latency counts
        _norm("norm_1_codes", 1, 4096, "bf16", True, "codes"),
        # a full serving batch
        _norm("norm_64", 64, 8192, "bf16", True, "y"),
        # a packed batch of prompts, rows that are a slice of a wider buffer, gain 1 + w
        _norm("norm_4999_odd", 4999, 5120, "f16", True, "y", offset=True, pad=24),
        # a long prompt ahead of an int8-activation product
        _norm("norm_16384_codes", 16384, 4096, "bf16", True, "codes"),
        # the next token of one conversation through many small experts
        _moe("moe_1_of_64", 1, 8, 64, 2048, 1024, 4, 32, "bf16", "f16", True),
        # four tokens through few large experts
        _moe("moe_4_of_8", 4, 2, 8, 4096, 14336, 4, 32, "bf16", "f16", True, lens_seed=2),
        # a small serving batch: most experts have a token or two
        _moe("moe_16_of_64", 16, 8, 64, 2048, 1408, 4, 64, "f16", "bf16", False, "sigmoid", 3),
        # odd sizes, 8-bit codes
        _moe("moe_3_odd", 3, 3, 10, 1000, 616, 8, 16, "bf16", "f32", True, "sigmoid", 4),
        # the next token of one conversation
        _sample("sample_1", 1, 128000, "bf16", "all"),
        # a serving batch whose requests set what they like
        _sample("sample_64_mixed", 64, 128000, "f32", "mixed", 0.0, 5),
        # many short-vocabulary rows, a nucleus only, some rows under a grammar's mask
        _sample("sample_256_top_p", 256, 50257, "f16", "top_p", 0.25, 6),
        # plain draws at the full width
        _sample("sample_16_plain", 16, 200003, "f32", "none", 0.0, 7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "moe", "sample"])
    seed = rng.randrange(1 << 20)
    if op == "norm":
        width = rng.choice([1024, 2048, 4096, 5120, 7168, 8192, _log_int(rng, 64, 16384)])
        dtype, out = rng.choice([("bf16", "y"), ("bf16", "codes"), ("f16", "y"), ("f16", "codes"), ("f32", "y")])
        c = _norm("", _log_int(rng, 1, max(2, min(16384, 60_000_000 // width))), width, dtype, rng.random() < 0.8, out,
                  rng.choice([16, 32, 64, 128, 256]), rng.random() < 0.3, rng.choice([0, 0, 8, 40]))
    elif op == "moe":
        experts = rng.choice([4, 8, 16, 60, 64, 128])
        top_k = rng.randint(1, min(8, experts))
        hidden = rng.choice([512, 1024, 2048, 4096, _log_int(rng, 128, 4096)])
        inner = rng.choice([768, 1024, 1408, 2816, _log_int(rng, 64, 4096)])
        inner = max(64, min(inner, 400_000_000 // (experts * hidden)))
        c = _moe("", _log_int(rng, 1, 16), top_k, experts, hidden, inner, rng.choice([4, 4, 4, 8, 2]),
                 rng.choice([16, 32, 32, 64, 128]), rng.choice(["bf16", "bf16", "f16"]), rng.choice(["f16", "bf16", "f32"]),
                 rng.random() < 0.6, rng.choice(["softmax", "sigmoid"]), seed)
    else:
        vocab = rng.choice([32000, 50257, 128000, _log_int(rng, 1000, 200000)])
        c = _sample("", _log_int(rng, 1, max(2, min(256, 12_000_000 // vocab))), vocab, rng.choice(["bf16", "f16", "f32"]),
                    rng.choice(["all", "top_p", "none", "mixed"]), rng.choice([0.0, 0.0, 0.3]), seed)
    c.pop("name")
    return c


def _routes(case):
    """The experts that each token's logits favour: some experts are more popular than others."""
    r = random.Random(case["lens_seed"])
    popular = [math.exp(r.gauss(0.0, 0.7)) for _ in range(case["experts"])]
    rows = []
    for _ in range(case["tokens"]):
        keys = sorted(range(case["experts"]), key=lambda e: -(r.random() ** (1.0 / popular[e])))
        rows.append(keys[:case["top_k"]])
    return rows


def _params(case):
    """Temperature, top-k, top-p and min-p of each row (0, 0, 1 and 0 turn the last three off)."""
    r = random.Random(case["lens_seed"])
    rows = []
    for _ in range(case["rows"]):
        t, k, p, m = r.uniform(0.6, 1.2), 0, 1.0, 0.0
        kind = r.choice(["all", "top_p", "none", "greedy", "min_p", "top_k"]) if case["cuts"] == "mixed" else case["cuts"]
        if kind == "all":
            k, p, m = r.randint(20, 100), r.uniform(0.8, 0.98), r.choice([0.0, 0.05])
        elif kind == "top_p":
            p = r.uniform(0.7, 0.99)
        elif kind == "greedy":
            t = 0.0
        elif kind == "min_p":
            m = r.uniform(0.01, 0.2)
        elif kind == "top_k":
            k = _log_int(r, 2, case["vocab"])
        rows.append((t, k, p, m))
    return rows


def work(case):
    if case["op"] == "norm":
        n, e = case["rows"] * case["width"], ESIZE[case["dtype"]]
        out = e * n if case["out"] == "y" else n + 4 * case["rows"] * -(-case["width"] // case["block"])
        return {"bytes": n * e * (3 if case["residual"] else 1) + out + 4 * case["width"], "flops": 6 * n}
    if case["op"] == "moe":
        k, i, t, s = case["hidden"], case["inner"], case["tokens"], case["top_k"]
        active = len({e for row in _routes(case) for e in row})

        def weight(n, d):
            kb = -(-d // case["bs"])
            zp = n * -(-kb * case["bits"] // 8) if case["zp"] else 0
            return n * kb * (case["bs"] * case["bits"] // 8 + ESIZE[case["scale_dtype"]]) + zp

        return {"bytes": active * (2 * weight(i, k) + weight(k, i)) + 2 * t * k * ESIZE[case["dtype"]] + t * case["experts"] * 4 + 8 * t * s,
                "flops": 6 * t * s * k * i}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * ESIZE[case["dtype"]] + 24 * case["rows"], "flops": 8 * n}


# ---- inputs --------------------------------------------------------------------------------------------------------

def _normal(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(DT[dtype])


def _scratch(nbytes):
    raw = torch.empty(max(256, nbytes) + 256, dtype=torch.uint8, device="cuda")
    off = (-raw.data_ptr()) % 256
    return raw[off:off + max(256, nbytes)]


def _experts(case, n, k, gen):
    """Codes of [experts, n, k] weights in the operator's storage, with scales that give outputs of order 1."""
    e, bits, bs = case["experts"], case["bits"], case["bs"]
    kb = -(-k // bs)
    w = {"n": n, "k": k}
    w["codes"] = torch.randint(0, 256, (e, n, kb, bs * bits // 8), generator=gen, device="cuda", dtype=torch.uint8)
    deviation = 2 ** bits / math.sqrt(12.0)
    base = torch.rand((e, n, kb), generator=gen, device="cuda") + 0.5
    w["scales"] = base.mul_(k ** -0.5 / deviation).to(DT[case["scale_dtype"]])
    w["zp"] = None
    if case["zp"]:
        w["zp"] = torch.zeros((e, n, -(-kb * bits // 8)), dtype=torch.uint8, device="cuda")
        mid = 2 ** (bits - 1)
        z = torch.randint(mid - mid // 4 - 1, mid + mid // 4 + 1, (e, n, w["zp"].shape[2] * (8 // bits)), generator=gen, device="cuda")
        for j in range(8 // bits):
            w["zp"] |= (z[..., j::8 // bits] << (j * bits)).to(torch.uint8)
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        t, h = case["rows"], case["width"]
        s["x"] = _normal((t, h + case["pad"]), case["dtype"], gen)[:, :h]
        # the residual stream: wider than what a layer adds, with a few large channels
        s["residual"] = None
        if case["residual"]:
            channel = torch.exp(0.8 * torch.randn(h, generator=gen, device="cuda"))
            s["residual"] = (torch.randn((t, h), generator=gen, device="cuda") * channel * 3.0).to(DT[case["dtype"]])
            s["sum"] = torch.empty_like(s["residual"])
        s["weight"] = (1.0 + 0.2 * torch.randn(h, generator=gen, device="cuda")).to(DT[case["dtype"]])
        if case["offset"]:
            s["weight"] = s["weight"] - 1
        s["eps"] = 1e-6
        if case["out"] == "y":
            s["y"] = torch.empty((t, h), dtype=DT[case["dtype"]], device="cuda")
        else:
            kb = -(-h // case["block"])
            s["codes"] = torch.empty((t, kb * case["block"]), dtype=torch.int8, device="cuda")
            s["scales"] = torch.empty((t, kb), dtype=torch.float32, device="cuda")
            s["values"] = torch.empty((t, kb, case["block"]), dtype=DT[case["dtype"]], device="cuda")
        return s
    if case["op"] == "moe":
        t, e, k = case["tokens"], case["experts"], case["hidden"]
        s["x"] = _normal((t, k), case["dtype"], gen)
        logits = torch.randn((t, e), generator=gen, device="cuda").clamp_(-2.0, 2.0)
        for row, picked in enumerate(_routes(case)):
            logits[row, picked] += 4.5
        s["logits"] = logits
        s["bias"] = None
        if case["scoring"] == "sigmoid":  # a selection bias that evens the load out, too small to move these picks
            s["bias"] = 0.001 * torch.randn(e, generator=gen, device="cuda")
        s["gate"], s["up"] = (_experts(case, case["inner"], k, gen) for _ in range(2))
        s["down"] = _experts(case, k, case["inner"], gen)
        s["y"] = torch.empty((t, k), dtype=DT[case["dtype"]], device="cuda")
        s["ids"] = torch.empty((t, case["top_k"]), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((t, case["top_k"]), dtype=torch.float32, device="cuda")
        if own:  # weights are laid out once, when a model is loaded
            import block_quantized_weight_matmulnbits_gb300 as mnb
            for w in (s["gate"], s["up"], s["down"]):
                nbytes = mnb.mnb_packed_size(w["n"], w["k"], case["bits"], case["bs"])
                packed = _scratch(nbytes * e)
                for i in range(e):
                    mnb.mnb_pack_weights(w["codes"][i], packed[i * nbytes:(i + 1) * nbytes], w["n"], w["k"], case["bits"], case["bs"])
                w["handle"] = mnb.expert_weights(packed, w["scales"], w["zp"], e, w["n"], w["k"], case["bits"], case["bs"])
            s["workspace"] = _scratch(mnb.mnb_moe_workspace_size(t, case["top_k"], e, k, case["inner"]))
        return s
    b, v = case["rows"], case["vocab"]
    # logits of a language model: a wide bulk, and a few dozen likely tokens above it
    x = torch.randn((b, v), generator=gen, device="cuda").mul_(2.0)
    likely = torch.randint(0, v, (b, 40), generator=gen, device="cuda")
    x.scatter_reduce_(1, likely, 6.0 + 2.5 * torch.randn((b, 40), generator=gen, device="cuda"), "amax")
    if case["masked"]:
        r = random.Random(case["lens_seed"] + 1)
        rows = [i for i in range(b) if r.random() < case["masked"]]
        keep = torch.rand((len(rows), v), generator=gen, device="cuda") < 0.02
        keep[:, 0] = True
        x[rows] = x[rows].masked_fill(~keep, -math.inf)
    s["logits"] = x.to(DT[case["dtype"]])
    t, k, p, m = zip(*_params(case))
    s["temperature"] = torch.tensor(t, dtype=torch.float32, device="cuda")
    s["top_k"] = torch.tensor(k, dtype=torch.int32, device="cuda")
    s["top_p"] = torch.tensor(p, dtype=torch.float32, device="cuda")
    s["min_p"] = torch.tensor(m, dtype=torch.float32, device="cuda")
    s["u"] = torch.rand(b, generator=gen, device="cuda")
    s["tokens"] = torch.empty(b, dtype=torch.int32, device="cuda")
    s["probs"] = torch.empty(b, dtype=torch.float32, device="cuda")
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if c["residual"]:
        x = x + s["residual"].float()
    gain = s["weight"].float() + (1.0 if c["offset"] else 0.0)
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + s["eps"]) * gain
    out = {"sum": x.to(s["x"].dtype)} if c["residual"] else {}
    if c["out"] == "y":
        out["y"] = y.to(s["x"].dtype)
        return out
    kb = -(-c["width"] // c["block"])
    y = torch.cat([y, y.new_zeros((c["rows"], kb * c["block"] - c["width"]))], 1).view(c["rows"], kb, c["block"])
    scale = y.abs().amax(2, keepdim=True) / 127.0
    q = torch.where(scale > 0, y / scale, torch.zeros_like(y))
    q = (torch.sign(q) * torch.floor(q.abs() + 0.5)).clamp(-127, 127)
    out["scales"], out["values"] = scale.squeeze(2), (q * scale).to(s["x"].dtype)
    return out


def _dense(case, w, e, dtype):
    """Weights [n, k] of expert e from their codes."""
    bits, bs, n, k = case["bits"], case["bs"], w["n"], w["k"]
    per, mask = 8 // bits, 2 ** bits - 1
    shift = torch.arange(per, device="cuda", dtype=torch.int32) * bits
    kb = w["scales"].shape[2]
    q = ((w["codes"][e].to(torch.int32)[..., None] >> shift) & mask).view(n, kb, bs)
    if w["zp"] is None:
        z = 2 ** (bits - 1)
    else:
        z = ((w["zp"][e].to(torch.int32)[..., None] >> shift) & mask).view(n, -1)[:, :kb, None]
    return ((q - z).to(dtype) * w["scales"][e].to(dtype)[..., None]).view(n, -1)[:, :k]


def _plain_route(s):
    c = s["case"]
    if c["scoring"] == "softmax":
        score = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
        ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    else:
        score = 1.0 / (1.0 + torch.exp(-s["logits"]))
        ids = torch.sort(score + s["bias"], dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = torch.gather(score, 1, ids)
    return ids, w / w.sum(1, keepdim=True)


def _plain_moe(s):
    c = s["case"]
    ids, weights = _plain_route(s)
    x = s["x"].float()
    y = torch.zeros((c["tokens"], c["hidden"]), device="cuda")
    for e in sorted({e for row in _routes(c) for e in row}):
        hit = ids == e
        gate = torch.matmul(x, _dense(c, s["gate"], e, torch.float32).T)
        up = torch.matmul(x, _dense(c, s["up"], e, torch.float32).T)
        h = gate / (1.0 + torch.exp(-gate)) * up
        y += (weights * hit).sum(1, keepdim=True) * torch.matmul(h, _dense(c, s["down"], e, torch.float32).T)
    return {"y": y.to(s["x"].dtype), "ids": ids.to(torch.int32), "weights": weights}


def _plain_sample(s):
    c = s["case"]
    v = c["vocab"]
    x, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    greedy = s["temperature"] == 0
    t = torch.where(greedy, 1.0, s["temperature"]).double()
    w = torch.exp((x - x[:, :1]) / t[:, None])
    rank = torch.arange(v, device="cuda")
    k = torch.where(greedy, 1, torch.where(s["top_k"] > 0, s["top_k"], v)).clamp(max=v)
    w = torch.where(rank < k[:, None], w, 0.0)
    before = torch.cumsum(w, 1) - w
    p = s["top_p"].double()
    keep = (before < (p * w.sum(1))[:, None]) | (p >= 1)[:, None] | (rank == 0)
    keep &= w >= s["min_p"].double()[:, None]
    w = torch.where(keep, w, 0.0)
    upto = torch.cumsum(w, 1)
    total = upto[:, -1:]
    at = (upto <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=v - 1)
    token = torch.gather(order, 1, at).squeeze(1)
    return {"tokens": token.to(torch.int32), "probs": (torch.gather(w, 1, at) / total).squeeze(1).float()}


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "moe": _plain_moe, "sample": _plain_sample}[c["op"]](s)
    import block_quantized_weight_matmulnbits_gb300 as mnb
    if c["op"] == "norm":
        flags = mnb.MNB_NORM_UNIT_OFFSET if c["offset"] else 0
        out = {}
        if c["residual"]:
            out["sum"] = s["sum"]
        if c["out"] == "y":
            mnb.mnb_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"], residual_out=out.get("sum"), y=s["y"], flags=flags)
            out["y"] = s["y"]
        else:
            mnb.mnb_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"], residual_out=out.get("sum"), codes=s["codes"],
                             scales=s["scales"], block_size=c["block"], flags=flags)
            out["scales"] = s["scales"]
            # what the codes stand for, in the activations' type
            out["values"] = torch.mul(s["codes"].view(c["rows"], -1, c["block"]), s["scales"][:, :, None], out=s["values"])
        return out
    if c["op"] == "moe":
        scoring = mnb.MNB_MOE_SOFTMAX if c["scoring"] == "softmax" else mnb.MNB_MOE_SIGMOID
        mnb.mnb_moe(s["x"], s["logits"], s["gate"]["handle"], s["up"]["handle"], s["down"]["handle"], s["y"], c["top_k"],
                    ids=s["ids"], weights=s["weights"], bias=s["bias"], scoring=scoring, workspace=s["workspace"])
        return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}
    mnb.mnb_sample(s["logits"], s["u"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                   min_p=s["min_p"], probs=s["probs"])
    return {"tokens": s["tokens"], "probs": s["probs"]}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _exact_norm(case, s):
    out = {}
    h = s["x"].double()
    if case["residual"]:
        h += s["residual"].double()
        out["sum"] = h.clone()
    norm = torch.linalg.vector_norm(h, dim=1, keepdim=True)
    h *= (norm.square() / case["width"] + s["eps"]).pow(-0.5)
    w = s["weight"].double()
    h *= w + 1.0 if case["offset"] else w
    if case["out"] == "y":
        out["y"] = h
        return out
    bs = case["block"]
    values = h.new_zeros((case["rows"], -(-case["width"] // bs) * bs))
    values[:, :case["width"]] = h
    blocks = values.unflatten(1, (-1, bs))
    scale = blocks.abs().max(2).values / 127.0
    steps = torch.nan_to_num(blocks / scale[..., None])
    out["scales"] = scale
    out["values"] = torch.copysign(torch.trunc(steps.abs() + 0.5), steps) * scale[..., None]
    return out


def _exact_moe(case, s):
    picked = _routes(case)
    logits = s["logits"].double()
    y = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
    ids, weights, cache = [], [], {}
    for t in range(case["tokens"]):
        score = torch.softmax(logits[t], 0) if case["scoring"] == "softmax" else torch.sigmoid(logits[t])
        rank = (logits[t] if case["scoring"] == "softmax" else score + s["bias"].double()).tolist()
        row = sorted(picked[t], key=lambda e: (-rank[e], e))
        w = score[row]
        ids.append(row)
        weights.append(w / w.sum())
    for t in range(case["tokens"]):
        for e, w in zip(ids[t], weights[t]):
            if e not in cache:
                if len(cache) >= 4:  # dense 64-bit weights of a large expert take a gigabyte
                    cache.pop(next(iter(cache)))
                cache[e] = [_dense(case, s[n], e, torch.float64) for n in ("gate", "up", "down")]
            gate, up, down = cache[e]
            a = gate @ s["x"][t].double()
            y[t] += w * (down @ (a * torch.sigmoid(a) * (up @ s["x"][t].double())))
    return {"y": y, "ids": torch.tensor(ids, dtype=torch.int32, device="cuda"), "weights": torch.stack(weights)}


def _exact_sample(case, s):
    tokens, probs = [], []
    for b, (t, k, p, m) in enumerate(_params(case)):
        x = s["logits"][b].double()
        order = torch.argsort(-x, stable=True)
        if t == 0.0:
            tokens.append(order[0])
            probs.append(torch.ones((), dtype=torch.float64, device="cuda"))
            continue
        t, p, m = float(s["temperature"][b]), float(s["top_p"][b]), float(s["min_p"][b])
        order = order[:k] if k else order
        q = torch.softmax(x[order] / t, 0)
        if p < 1.0:  # the shortest start that holds p
            q = q[:int(torch.searchsorted(torch.cumsum(q, 0), p)) + 1]
        if m > 0.0:
            q = q[q >= m * q[0]]
        upto = torch.cumsum(q, 0)
        at = min(int(torch.searchsorted(upto, float(s["u"][b]) * float(upto[-1]), right=True)), q.numel() - 1)
        tokens.append(order[at])
        probs.append(q[at] / upto[-1])
    return {"tokens": torch.stack(tokens).to(torch.int32), "probs": torch.stack(probs)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "moe": _exact_moe, "sample": _exact_sample}[case["op"]](case, s)
