"""Cases, plain forms and 64-bit values of the operators that take a chunk of tokens through an attention layer and to
the sampler: rotating queries and keys by their positions and appending keys and values to a paged cache; attention of
the new tokens over that cache; penalties, biases and grammar masks on the head's logits.

`own` chooses between the plain form (elementary torch operations in 32 bits, angles in 64, rounded once at the end)
and the library's kernels. The lengths of a ragged batch follow from the case alone, the values from the seed.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # one user's decode step: the f32 outputs of one fused int8 projection, a quarter of the head rotated
        dict(name="append 1 token", op="append", rows=1, tokens=1, shortest=1, idle=0, cached=699, heads=16, kv_heads=2,
             dim=256, rot=64, interleaved=False, scaling="none", source="f32", dtype="f16", page=64, pad=0, mix=1),
        # a full server's decode step, idle slots, a batch padded to 256 rows
        dict(name="append 250 tokens", op="append", rows=256, tokens=1, shortest=1, idle=6, cached=2000, heads=16,
             kv_heads=2, dim=256, rot=64, interleaved=False, scaling="none", source="f32", dtype="bf16", page=64, pad=6,
             mix=2),
        # ragged prompts of a batch, whole heads rotated in neighbouring pairs, scaled for a long context
        dict(name="append 19 prompts", op="append", rows=19, tokens=1500, shortest=3, idle=2, cached=9000, heads=20,
             kv_heads=4, dim=128, rot=128, interleaved=True, scaling="yarn", source="bf16", dtype="bf16", page=16, pad=0,
             mix=3),
        # a long document's chunk
        dict(name="append 32000 tokens", op="append", rows=1, tokens=32000, shortest=32000, idle=0, cached=100000,
             heads=16, kv_heads=2, dim=256, rot=64, interleaved=False, scaling="linear", source="f32", dtype="f16",
             page=64, pad=0, mix=4),
        # one user, four speculated tokens checked at once
        dict(name="chunk 4 over 700", op="chunk", rows=1, tokens=4, shortest=4, idle=0, cached=696, heads=16, kv_heads=2,
             dim=256, page=64, dtype="f16", pad=0, mix=5),
        # speculated tokens of a busy server over ragged caches, idle slots
        dict(name="chunk 24 x 8 over 16k", op="chunk", rows=24, tokens=8, shortest=2, idle=2, cached=16000, heads=16,
             kv_heads=2, dim=256, page=64, dtype="bf16", pad=5, mix=6),
        # a prompt's first chunk, of the MoE block's prefill size
        dict(name="chunk 2048", op="chunk", rows=1, tokens=2048, shortest=2048, idle=0, cached=0, heads=16, kv_heads=2,
             dim=256, page=64, dtype="f16", pad=0, mix=7),
        # ragged prompts, some over cached prefixes, small pages, an odd group of heads
        dict(name="chunk 19 prompts", op="chunk", rows=19, tokens=1500, shortest=3, idle=2, cached=9000, heads=20,
             kv_heads=4, dim=128, page=16, dtype="bf16", pad=0, mix=8),
        # a late chunk of a long document
        dict(name="chunk 2048 over 64k", op="chunk", rows=1, tokens=2048, shortest=2048, idle=0, cached=63488, heads=16,
             kv_heads=2, dim=256, page=64, dtype="bf16", pad=0, mix=9),
        # one user's penalties and a few biases
        dict(name="logits 1 x 152064", op="logits", rows=1, vocab=152064, history=900, bias=20, grammars=0, dtype="f32",
             in_place=True, mix=10),
        # a decode step over the larger vocabulary, half of it under grammars, the raw logits kept
        dict(name="logits 61 x 248320", op="logits", rows=61, vocab=248320, history=4000, bias=5, grammars=30,
             dtype="f32", in_place=False, mix=11),
        # a full server, long histories, every row under a grammar
        dict(name="logits 256 x 152064", op="logits", rows=256, vocab=152064, history=8000, bias=50, grammars=256,
             dtype="f32", in_place=True, mix=12),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "logits"])
    mix = rng.randrange(1 << 20)
    if op == "logits":
        vocab = _log(rng, 20, 260000)
        rows = _log(rng, 1, max(2, min(2000, 256 * 152064 // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, history=rng.choice([0, _log(rng, 1, 8000), _log(rng, 1, 8000)]),
                    bias=rng.choice([0, 1, _log(rng, 1, 300)]), grammars=rng.choice([0, rows, rng.randrange(rows + 1)]),
                    dtype=rng.choice(["f16", "bf16", "f32", "f32"]), in_place=rng.random() < 0.6, mix=mix)
    kv = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128, 256])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 11, 16])
    rows = _log(rng, 1, 200)
    # of the largest listed cases: products of a chunk, values of an append; keys in the caches
    products, values, keys = 2048 * 65536 * 16 * 256, 32000 * 20 * 256, 80_000_000 // (kv * dim)
    token = kv * group * dim
    longest = math.isqrt(products // (rows * token)) if op == "chunk" else values // (rows * (token + 2 * kv * dim))
    longest = max(1, min(4096, 20000 // rows, longest))
    tokens = min(longest, rng.choice([1, 2, 4])) if rng.random() < 0.3 else _log(rng, 1, longest)
    most = max(1, min(65536 - tokens, keys // rows))
    if op == "chunk":
        most = max(1, min(most, products // (2 * rows * tokens * token)))
    case = dict(op=op, rows=rows, tokens=tokens, shortest=_log(rng, 1, tokens), idle=rng.randrange(0, 1 + rows // 4),
                cached=rng.choice([0, _log(rng, 1, most), _log(rng, 1, most)]), heads=kv * group, kv_heads=kv, dim=dim,
                dtype=rng.choice(["f16", "bf16"]), page=rng.choice([1, 16, 17, 32, 48, 64, 128, 256]),
                pad=rng.choice([0, 0, rng.randrange(1, 20)]), mix=mix)
    if op == "append":
        case.update(rot=16 * rng.randrange(0, dim // 16 + 1), interleaved=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "yarn"]), source=rng.choice(["f32", case["dtype"]]))
    return case


def _batch(case):
    """(new tokens, cached tokens) of each sequence, log-uniform, one of each longest, `idle` sequences of none."""
    rng = random.Random(case["mix"])
    n = case["rows"] - case["idle"]
    new = [case["tokens"]] + [_log(rng, case["shortest"], case["tokens"]) for _ in range(n - 1)]
    old = [case["cached"]] + [_log(rng, 1, case["cached"] + 1) - 1 for _ in range(n - 1)]
    both = list(zip(new, old)) + [(0, 0)] * case["idle"]
    rng.shuffle(both)
    return [a for a, _ in both], [b for _, b in both]


def _lists(case):
    """(ids, of these the prompt's, biases) of each row of logits."""
    rng = random.Random(case["mix"])
    most = case["history"]
    ids = [most] + [_log(rng, 1, most + 1) - 1 for _ in range(case["rows"] - 1)]
    prompt = [rng.randrange(0, n + 1) for n in ids]
    bias = [min(case["vocab"], case["bias"])] + [rng.randrange(0, min(case["vocab"], case["bias"]) + 1)
                                                for _ in range(case["rows"] - 1)]
    return ids, prompt, bias


def work(case):
    if case["op"] == "logits":
        ids, _, bias = _lists(case)
        size, v, m = SIZE[case["dtype"]], case["vocab"], case["rows"]
        listed_bytes = 4 * sum(ids) + 8 * sum(bias) + case["grammars"] * 4 * -(-v // 32)
        # in place, only the touched logits: banned ones (seven of eight under a grammar) are written; else all of them
        touched = m * v * size * 2 if not case["in_place"] else case["grammars"] * v * size * 7 // 8
        return {"bytes": listed_bytes + touched, "flops": 4 * sum(ids) + sum(bias)}
    new, old = _batch(case)
    t, h, kv, d = sum(new), case["heads"], case["kv_heads"], case["dim"]
    size = SIZE[case["dtype"]]
    if case["op"] == "append":
        return {"bytes": t * (h + 2 * kv) * d * (SIZE[case["source"]] + size), "flops": 3 * t * (h + kv) * case["rot"]}
    keys = sum(a + b for a, b in zip(new, old))
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
    return {"bytes": 2 * keys * kv * d * size + 2 * t * h * d * size + 4 * t * h, "flops": 4 * pairs * h * d}


def _rotary(case):
    """Arguments of the frequencies, as a model's configuration has them."""
    scaling = {"none": None, "linear": {"type": "linear", "factor": 4.0},
               "yarn": {"type": "yarn", "factor": 4.0, "original": 32768}}[case["scaling"]]
    return dict(rot=case["rot"], base=1e6, interleaved=case["interleaved"], scaling=scaling)


def _frequencies(case):
    """(frequencies in 64 bits, factor of cosine and sine)."""
    rot, base = case["rot"], 1e6
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    if case["scaling"] == "none" or rot == 0:
        return f, 1.0
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    # frequencies that turn more than 32 times within the original length stay, those below one turn are divided, a ramp
    # over their index lies between
    index = [rot * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    low, high = max(math.floor(index[0]), 0), min(math.ceil(index[1]), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64, device="cuda") - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    if case["op"] == "logits":
        ids, prompt, bias = _lists(case)
        m, v = case["rows"], case["vocab"]
        # a history repeats its tokens: low numbers are frequent ones
        u = torch.rand(sum(ids), generator=gen, device="cuda", dtype=torch.float64)
        words, r = -(-v // 32), case["grammars"]
        s = {"logits": normal(m, v, dtype=dt) * 2.5, "ids": (u ** 3 * v).int().clamp(max=v - 1),
             "at": whole([0] + ids).cumsum(0).int(), "prompt": whole(prompt),
             "repetition": 1.0 + 0.3 * torch.rand(m, generator=gen, device="cuda"),
             "frequency": 0.5 * torch.rand(m, generator=gen, device="cuda"),
             "presence": torch.rand(m, generator=gen, device="cuda") - 0.2,
             "bias_at": whole([0] + bias).cumsum(0).int(), "bias": 4 * normal(sum(bias)),
             "bias_ids": torch.cat([torch.randperm(v, generator=gen, device="cuda")[:n] for n in bias]).int(),
             "allowed": None, "allowed_rows": None}
        if r:
            # one bit of eight, as after an opened bracket; rows without a grammar say -1
            bits = torch.randint(-2 ** 31, 2 ** 31, (3, r, words), generator=gen, device="cuda", dtype=torch.int64)
            s["allowed"] = (bits[0] & bits[1] & bits[2]).int()
            order = torch.randperm(m, generator=gen, device="cuda").int()
            s["allowed_rows"] = torch.where(order < r, order, torch.full_like(order, -1))
        return {"case": case, **s}
    new, old = _batch(case)
    ps, kv, h, d = case["page"], case["kv_heads"], case["heads"], case["dim"]
    lens = [a + b for a, b in zip(new, old)]
    need = [-(-n // ps) for n in lens]
    n_pages, width = sum(need) + 7, max(need) + 1
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    count = torch.tensor(need, device="cuda")
    first = torch.cumsum(count, 0) - count
    col = torch.arange(width, device="cuda")
    table = torch.where(col < count[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
    t = sum(new) + case["pad"]
    s = {"k": normal(n_pages, kv, ps, d, dtype=dt), "v": normal(n_pages, kv, ps, d, dtype=dt), "table": table,
         "at": whole([0] + new).cumsum(0).int(), "lens": whole(lens), "new": new, "old": old}
    if case["op"] == "chunk":
        return {"case": case, **s, "q": normal(t, h, d).to(dt) * 2, "scale": 1.0 / math.sqrt(d), "longest": max(lens)}
    # one fused projection's output: a token's query, key and value heads side by side
    fused = normal(t, h + 2 * kv, d).to(DT[case["source"]])
    s.update(q_in=fused[:, :h], k_in=fused[:, h:h + kv], v_in=fused[:, h + kv:])
    if own and case["rot"]:
        from bit_trellis_quantized_gb300 import native

        s["rotary"] = native.Rotary(**_rotary(case), device="cuda")
    return {"case": case, **s}


# ---- plain forms --------------------------------------------------------------------------------------------


def _places(s):
    """(sequence, position) of every token that belongs to a sequence."""
    new, at, lens = s["at"][1:] - s["at"][:-1], s["at"].long(), s["lens"].long()
    seq = torch.repeat_interleave(torch.arange(len(new), device=at.device), new.long(), output_size=sum(s["new"]))
    t = torch.arange(seq.shape[0], device=at.device)
    return seq, lens[seq] - new.long()[seq] + t - at[seq]


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    if rot == 0:
        return x
    turned, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, rest], -1)


def _append_in(s, dt):
    """Rotated queries, keys and the values in type `dt`, and their places in the cache."""
    case = s["case"]
    seq, pos = _places(s)
    t = seq.shape[0]
    f, factor = _frequencies(case)
    angle = pos.double()[:, None, None] * f
    cos, sin = (torch.cos(angle) * factor).to(dt), (torch.sin(angle) * factor).to(dt)
    q = _rotate(s["q_in"][:t].to(dt), cos, sin, case["interleaved"])
    k = _rotate(s["k_in"][:t].to(dt), cos, sin, case["interleaved"])
    page = s["table"][seq, pos // case["page"]].long()
    return q, k, s["v_in"][:t].to(dt), page, pos % case["page"]


def _append(s):
    q, k, v, page, slot = _append_in(s, torch.float32)
    s["k"][page, :, slot] = k.to(s["k"].dtype)
    s["v"][page, :, slot] = v.to(s["v"].dtype)
    return {"q": q.to(s["k"].dtype), "k": s["k"], "v": s["v"]}


def _attend(s, dt, budget):
    """Sequence by sequence, in blocks of tokens whose scores are at most `budget` numbers."""
    case, q = s["case"], s["q"]
    kv, h, d, ps = case["kv_heads"], case["heads"], case["dim"], case["page"]
    t, group, first = sum(s["new"]), h // kv, 0
    out = torch.zeros((t, h, d), dtype=dt, device=q.device)
    lse = torch.full((t, h), -math.inf, dtype=dt, device=q.device)
    for b, (n, old) in enumerate(zip(s["new"], s["old"])):
        length = n + old
        if n == 0:
            continue
        pages = s["table"][b, :-(-length // ps)].long()
        keys = s["k"][pages].transpose(0, 1).reshape(kv, -1, d)[:, :length].to(dt)
        values = s["v"][pages].transpose(0, 1).reshape(kv, -1, d)[:, :length].to(dt)
        step = max(1, budget // (h * length))
        for a in range(0, n, step):
            e = min(n, a + step)
            there = old + e  # keys that the block's last token sees
            rows = q[first + a:first + e].to(dt).reshape(e - a, kv, group, d).permute(1, 2, 0, 3).reshape(kv, -1, d)
            x = torch.matmul(rows, keys[:, :there].transpose(1, 2)).mul_(s["scale"]).reshape(kv, group, e - a, there)
            late = torch.arange(there, device=q.device) > torch.arange(old + a, old + e, device=q.device)[:, None]
            x.masked_fill_(late, -math.inf)
            top = x.amax(-1, keepdim=True)
            x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            y = torch.matmul(x.reshape(kv, -1, there), values[:, :there]).reshape(kv, group, e - a, d) / total
            out[first + a:first + e] = y.permute(2, 0, 1, 3).reshape(e - a, h, d)
            lse[first + a:first + e] = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(e - a, h)
        first += n
    return out, lse


def _chunk(s):
    out, lse = _attend(s, torch.float32, 1 << 29)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _adjust(s, dt):
    x, v = s["logits"].to(dt), s["case"]["vocab"]
    row = torch.arange(x.shape[0], device=x.device)
    ids, at = s["ids"].long(), s["at"].long()
    of = torch.repeat_interleave(row, at[1:] - at[:-1], output_size=ids.shape[0])
    late = (torch.arange(ids.shape[0], device=x.device) - at[of]) >= s["prompt"][of]
    # occurrences behind the prompt, and 2^40 for any at all
    seen = torch.zeros(x.shape, dtype=torch.int64, device=x.device)
    seen.view(-1).scatter_add_(0, of * v + ids, late.long() + (1 << 40))
    count = (seen & ((1 << 40) - 1)).to(dt)
    rep = s["repetition"].to(dt)[:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - (s["frequency"].to(dt)[:, None] * count + s["presence"].to(dt)[:, None] * (count > 0).to(dt))
    bias_at = s["bias_at"].long()
    of = torch.repeat_interleave(row, bias_at[1:] - bias_at[:-1], output_size=s["bias"].shape[0])
    x.view(-1).index_add_(0, of * v + s["bias_ids"].long(), s["bias"].to(dt))
    if s["allowed"] is not None:
        token = torch.arange(v, device=x.device)
        bits = (s["allowed"].long()[s["allowed_rows"].clamp(min=0).long()][:, token // 32] >> (token % 32)) & 1
        x = x.masked_fill((bits == 0) & (s["allowed_rows"] >= 0)[:, None], -math.inf)
    return x


def _logits(s):
    x = _adjust(s, torch.float32).to(s["logits"].dtype)
    if not s["case"]["in_place"]:
        return {"logits": x}
    s["logits"].copy_(x)
    return {"logits": s["logits"]}


def _call(s):
    from bit_trellis_quantized_gb300 import native

    case = s["case"]
    if case["op"] == "append":
        q = native.rotary_append(s["q_in"], s["k_in"], s["v_in"], s["k"], s["v"], s["table"], s["at"], s["lens"],
                                 rotary=s.get("rotary"))
        return {"q": q[:sum(s["new"])], "k": s["k"], "v": s["v"]}
    if case["op"] == "chunk":
        out, lse = native.chunk_attention(s["q"], s["k"], s["v"], s["table"], s["at"], s["lens"], scale=s["scale"],
                                          max_len=s["longest"])
        return {"out": out[:sum(s["new"])], "lse": lse[:sum(s["new"])]}
    x = native.adjust_logits(s["logits"], s["ids"], s["at"], prompt=s["prompt"], repetition=s["repetition"],
                             frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"],
                             bias_at=s["bias_at"], allowed=s["allowed"], allowed_rows=s["allowed_rows"],
                             out=s["logits"] if case["in_place"] else None)
    return {"logits": x}


def run(state):
    if own:
        return _call(state)
    return {"append": _append, "chunk": _chunk, "logits": _logits}[state["case"]["op"]](state)


# ---- the definitions in 64 bits ------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        # every token by itself: a pair is a complex number, turned by its angle
        k, v = s["k"].double(), s["v"].double()
        f, factor = _frequencies(case)
        half, rot = case["rot"] // 2, case["rot"]
        even = torch.arange(half, device="cuda")
        one, two = (2 * even, 2 * even + 1) if case["interleaved"] else (even, even + half)
        first, parts = 0, []
        for b, (n, old) in enumerate(zip(s["new"], s["old"])):
            if n == 0:
                continue
            pos = torch.arange(old, old + n, device="cuda")
            turn = torch.polar(torch.full((n, 1, half), factor, dtype=torch.float64, device="cuda"),
                               (pos.double()[:, None] * f)[:, None])

            def turned(x):
                x = x[first:first + n].double()
                z = torch.complex(x[..., one], x[..., two]) * turn
                y = x.clone()
                y[..., one], y[..., two] = z.real, z.imag
                return y

            parts.append(turned(s["q_in"]))
            page, slot = s["table"][b].long()[pos // case["page"]], pos % case["page"]
            k[page, :, slot] = turned(s["k_in"])
            v[page, :, slot] = s["v_in"][first:first + n].double()
            first += n
        return {"q": torch.cat(parts), "k": k, "v": v}
    if case["op"] == "chunk":
        if work(case)["flops"] > 8e12:  # 64-bit products run at about a teraflop a second
            return None
        q, kv, ps, first = s["q"], case["kv_heads"], case["page"], 0
        group, outs, lses = case["heads"] // kv, [], []
        for b, (n, old) in enumerate(zip(s["new"], s["old"])):
            if n == 0:
                continue
            pages = s["table"][b, :-(-(n + old) // ps)].long()
            out = torch.empty(n, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
            lse = torch.empty(n, case["heads"], dtype=torch.float64, device="cuda")
            for i in range(kv):
                keys = s["k"][pages, i].reshape(-1, case["dim"])[:n + old].double()
                values = s["v"][pages, i].reshape(-1, case["dim"])[:n + old].double()
                for a in range(0, n, 256):
                    e = min(n, a + 256)
                    x = torch.einsum("thd,kd->thk", q[first + a:first + e, i * group:(i + 1) * group].double(),
                                     keys[:old + e]) * s["scale"]
                    seen = torch.ones(e - a, old + e, dtype=torch.bool, device="cuda").tril(old + a)
                    x = torch.where(seen[:, None], x, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                    out[a:e, i * group:(i + 1) * group] = torch.einsum("thk,kd->thd", torch.softmax(x, 2),
                                                                       values[:old + e])
                    lse[a:e, i * group:(i + 1) * group] = torch.logsumexp(x, 2)
            outs.append(out)
            lses.append(lse)
            first += n
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    x, at, bias_at, v = s["logits"].double(), s["at"].tolist(), s["bias_at"].tolist(), case["vocab"]
    for r, prompt in enumerate(s["prompt"].tolist()):
        ids = s["ids"][at[r]:at[r + 1]].long()
        some = torch.unique(ids)
        rep = s["repetition"][r].double()
        x[r, some] = torch.where(x[r, some] > 0, x[r, some] / rep, x[r, some] * rep)
        count = torch.bincount(ids[prompt:], minlength=v).double()
        x[r] -= s["frequency"][r].double() * count + s["presence"][r].double() * (count > 0)
        x[r, s["bias_ids"][bias_at[r]:bias_at[r + 1]].long()] += s["bias"][bias_at[r]:bias_at[r + 1]].double()
        if s["allowed"] is not None and int(s["allowed_rows"][r]) >= 0:
            words = s["allowed"][s["allowed_rows"][r].long()].long()
            bits = ((words[:, None] >> torch.arange(32, device="cuda")) & 1).flatten()[:v]
            x[r, bits == 0] = -math.inf
    return {"logits": x}
