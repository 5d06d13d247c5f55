"""Cases, plain forms and 64-bit values of the operators around the MoE block: what a token mixer reads and keeps
(attention of one new token over a paged key-value cache; the gated delta rule, one token at a time or over prompts)
and what comes after the head (log probabilities of given tokens with entropy and top alternatives).

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once at the end) and the
library's kernels. The lengths of a ragged batch follow from the case alone, the values from the seed.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
CHUNK = 64  # tokens of one step of the plain chunked delta rule


def listed():
    return [
        # one user's conversation, its first answer: latency of a single short sequence
        dict(name="attention 1 x 700", op="attention", rows=1, longest=700, shortest=700, idle=0, heads=16, kv_heads=2,
             dim=256, page=64, dtype="f16", mix=1),
        # a small server's decode step: ragged lengths, small pages, odd group of heads
        dict(name="attention 31 to 8k", op="attention", rows=31, longest=8000, shortest=130, idle=2, heads=20,
             kv_heads=4, dim=128, page=16, dtype="bf16", mix=2),
        # one very long document
        dict(name="attention 1 x 131071", op="attention", rows=1, longest=131071, shortest=131071, idle=0, heads=16,
             kv_heads=2, dim=256, page=64, dtype="bf16", mix=3),
        # a full server's decode step, some slots idle
        dict(name="attention 192 to 16k", op="attention", rows=192, longest=16384, shortest=500, idle=5, heads=16,
             kv_heads=2, dim=256, page=64, dtype="f16", mix=4),
        # one user's decode step: 16 key heads and 32 value heads, as wide as the 2048 -> 4096 projections
        dict(name="delta step 1", op="delta", rows=1, tokens=1, shortest=1, idle=0, k_heads=16, v_heads=32, k_dim=128,
             v_dim=128, dtype="f16", mix=5),
        # a full server's decode step, every slot's state read and written
        dict(name="delta step 250", op="delta", rows=256, tokens=1, shortest=1, idle=6, k_heads=16, v_heads=32,
             k_dim=128, v_dim=128, dtype="bf16", mix=6),
        # one chunk of a prompt, as the MoE block's prefill chunk
        dict(name="delta prompt 2048", op="delta", rows=1, tokens=2048, shortest=2048, idle=0, k_heads=16, v_heads=32,
             k_dim=128, v_dim=128, dtype="f16", mix=7),
        # several prompts of a batch, ragged, keys narrower than values
        dict(name="delta prompts 19", op="delta", rows=19, tokens=1500, shortest=3, idle=3, k_heads=6, v_heads=12,
             k_dim=64, v_dim=128, dtype="bf16", mix=8),
        # a long document through one layer
        dict(name="delta prompt 32000", op="delta", rows=1, tokens=32000, shortest=32000, idle=0, k_heads=16,
             v_heads=32, k_dim=128, v_dim=128, dtype="bf16", mix=9),
        # the sampled token's log probability and 20 alternatives, one user
        dict(name="logprobs 1 x 152064", op="logprobs", rows=1, vocab=152064, given=1, top=20, banned=0, dtype="f32"),
        # a decode step of a server over the larger vocabulary, banned tokens among them
        dict(name="logprobs 61 x 248320", op="logprobs", rows=61, vocab=248320, given=1, top=5, banned=300,
             dtype="f32"),
        # a prompt's tokens scored against the head's f32 logits
        dict(name="logprobs 2048 x 152064", op="logprobs", rows=2048, vocab=152064, given=1, top=8, banned=0,
             dtype="f32"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["attention", "delta", "delta", "logprobs"])
    mix = rng.randrange(1 << 20)
    if op == "attention":
        kv = rng.choice([1, 2, 3, 4, 8])
        dim = rng.choice([64, 128, 256])
        rows = _log(rng, 1, 200)
        most = min(131071, 190 * 16384 * 512 // (rows * kv * dim))
        longest = _log(rng, 1, most)
        return dict(op=op, rows=rows, longest=longest, shortest=min(longest, _log(rng, 1, longest + 1)),
                    idle=rng.randrange(0, 1 + rows // 4), heads=kv * rng.choice([1, 2, 3, 4, 5, 6, 8, 11, 16]),
                    kv_heads=kv, dim=dim, page=rng.choice([1, 16, 17, 32, 48, 64, 128, 256]),
                    dtype=rng.choice(["f16", "bf16"]), mix=mix)
    if op == "delta":
        hk = rng.choice([1, 2, 4, 5, 8, 16])
        hv = hk * rng.choice([1, 2, 3])
        dk, dv = rng.choice([64, 128]), rng.choice([32, 64, 96, 128, 256])
        rows = _log(rng, 1, 300)
        if rng.random() < 0.4:
            longest = rng.choice([1, 1, 1, 2, 3, 5])
        else:
            longest = _log(rng, 6, max(7, min(16000, 60000 // rows)))
        return dict(op=op, rows=rows, tokens=longest, shortest=min(longest, _log(rng, 1, longest + 1)),
                    idle=rng.randrange(0, 1 + rows // 4), k_heads=hk, v_heads=hv, k_dim=dk, v_dim=dv,
                    dtype=rng.choice(["f16", "bf16"]), mix=mix)
    vocab = _log(rng, 20, 260000)
    rows = _log(rng, 1, max(2, min(4096, 300_000_000 // vocab)))
    return dict(op=op, rows=rows, vocab=vocab, given=rng.choice([0, 1, 1, 2, 7]), top=min(vocab, rng.randrange(0, 33)),
                banned=rng.choice([0, 0, vocab // 50]), dtype=rng.choice(["f16", "bf16", "f32", "f32"]))


def _lens(case):
    """The batch's lengths: log-uniform from shortest to longest, one of each end, `idle` rows of none."""
    rng = random.Random(case["mix"])
    n, a, b = case["rows"] - case["idle"], case["shortest"], case["longest" if case["op"] == "attention" else "tokens"]
    lens = [b] + [_log(rng, a, b) for _ in range(n - 1)]
    lens += [0] * case["idle"]
    rng.shuffle(lens)
    return lens


def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "attention":
        lens, d, h, kv = _lens(case), case["dim"], case["heads"], case["kv_heads"]
        keys, live = sum(lens), sum(n > 0 for n in lens)
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * keys * kv * d * size + 2 * len(lens) * h * d * size + 4 * len(lens) * h + 4 * pages
                + 2 * live * kv * d * size, "flops": 4 * keys * h * d}
    if case["op"] == "delta":
        lens, hv, hk, dk, dv = _lens(case), case["v_heads"], case["k_heads"], case["k_dim"], case["v_dim"]
        t, live = sum(lens), sum(n > 0 for n in lens)
        return {"bytes": t * (2 * hk * dk * size + 2 * hv * dv * size + 8 * hv) + 2 * live * hv * dk * dv * 4,
                "flops": 6 * t * hv * dk * dv}
    m, v = case["rows"], case["vocab"]
    return {"bytes": m * v * size + m * (8 * case["given"] + 8 + 8 * case["top"]), "flops": 4 * m * v}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    if case["op"] == "attention":
        lens, ps = _lens(case), case["page"]
        need = [-(-n // ps) for n in lens]
        n_pages, width = sum(need) + 7, max(need) + 1
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        at = torch.tensor(need, device="cuda")
        first = torch.cumsum(at, 0) - at
        col = torch.arange(width, device="cuda")
        table = torch.where(col < at[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)],
                            torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
        shape = (n_pages, case["kv_heads"], ps, case["dim"])
        s = {"k": normal(*shape, dtype=dt), "v": normal(*shape, dtype=dt),
             "q": normal(len(lens), case["heads"], case["dim"]).to(dt) * 2,
             "k_new": normal(len(lens), case["kv_heads"], case["dim"]).to(dt),
             "v_new": normal(len(lens), case["kv_heads"], case["dim"]).to(dt),
             "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "scale": 1.0 / math.sqrt(case["dim"])}
        return {"case": case, "longest": max(lens), "rows": [b for b, n in enumerate(lens) if n], **s}
    if case["op"] == "delta":
        lens, hk, hv, dk, dv = _lens(case), case["k_heads"], case["v_heads"], case["k_dim"], case["v_dim"]
        t = sum(lens)
        at = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        # log decays of a head: from nearly none to a few tokens' memory
        rate = torch.exp(normal(hv) * 1.5 - 2.5)
        g = -rate * torch.log1p(torch.exp(normal(t, hv)))
        return {"case": case, "q": normal(t, hk, dk).to(dt), "k": normal(t, hk, dk).to(dt),
                "v": normal(t, hv, dv).to(dt), "g": g, "beta": torch.sigmoid(normal(t, hv)),
                "state": normal(len(lens), hv, dk, dv) * 0.2, "at": at, "longest": max(lens),
                "scale": 1.0 / math.sqrt(dk)}
    m, v = case["rows"], case["vocab"]
    logits = (normal(m, v, dtype=dt) * 2.5)
    if case["banned"]:
        logits[:, torch.randperm(v, generator=gen, device="cuda")[:case["banned"]]] = -math.inf
    ids = torch.randint(0, v, (m, case["given"]), generator=gen, device="cuda", dtype=torch.int32)
    return {"case": case, "logits": logits, "ids": ids}


# ---- plain forms --------------------------------------------------------------------------------------------


def _attention(s):
    k, v, q, table, lens = s["k"], s["v"], s["q"], s["table"], s["lens"].long()
    n, ps = q.shape[0], k.shape[2]
    # the new token's key and value go to the last position of each live row
    rows = torch.nonzero(lens).flatten()
    last = lens[rows] - 1
    page = table[rows, last // ps].long()
    k[page, :, last % ps] = s["k_new"][rows]
    v[page, :, last % ps] = s["v_new"][rows]
    width = -(-s["longest"] // ps)
    pages = table[:, :width].clamp(min=0).long()
    live = (torch.arange(width * ps, device=q.device) < lens[:, None])[:, None]  # [n][1][keys]
    keys = k[pages].permute(0, 2, 1, 3, 4).reshape(n, k.shape[1], width * ps, -1).float()
    values = v[pages].permute(0, 2, 1, 3, 4).reshape(n, k.shape[1], width * ps, -1).float()
    values = torch.where(live[..., None], values, torch.zeros((), device=q.device))
    x = torch.matmul(q.float().reshape(n, k.shape[1], -1, q.shape[2]), keys.transpose(2, 3)) * s["scale"]
    x = torch.where(live[:, :, None], x, torch.full((), -math.inf, device=q.device))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.where(total == 0, torch.full_like(total, -math.inf), top + torch.log(total))
    return {"out": out.reshape(q.shape).to(q.dtype), "lse": lse.reshape(q.shape[:2]), "k": k, "v": v}


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _delta(s):
    case, state = s["case"], s["state"]
    n, hv, dk, dv = state.shape
    rep = hv // s["k"].shape[1]
    at = s["at"].long()
    lens = at[1:] - at[:-1]
    c = 1 if s["longest"] == 1 else CHUNK
    nc = -(-s["longest"] // c)
    step = torch.arange(nc * c, device=state.device)
    there = step < lens[:, None]  # [n][tokens]
    row = (at[:-1, None] + step).clamp(max=max(0, s["v"].shape[0] - 1))

    def padded(x, w):  # [t][h][w] -> [chunk][n][h][c][w]
        y = torch.where(there[:, :, None, None], x[row], torch.zeros((), device=x.device, dtype=x.dtype))
        return y.reshape(n, nc, c, -1, w).permute(1, 0, 3, 2, 4)

    q = padded(_unit(s["q"].float()).repeat_interleave(rep, 1), dk) * s["scale"]
    k = padded(_unit(s["k"].float()).repeat_interleave(rep, 1), dk)
    v = padded(s["v"].float(), dv)
    beta = padded(s["beta"][..., None], 1)
    # sums of log decays in 64 bits: their differences are what counts
    run_g = padded(s["g"].double()[..., None], 1).cumsum(3)
    one = torch.ones(c, c, device=state.device, dtype=torch.bool)
    zero = torch.zeros((), device=state.device)
    decay = torch.exp((run_g - run_g.transpose(3, 4)).masked_fill(~one.tril(), -math.inf)).float()
    fall, rest = torch.exp(run_g).float(), torch.exp(run_g[:, :, :, -1:] - run_g).float()
    a = torch.where(one.tril(-1), beta * decay * torch.matmul(k, k.transpose(3, 4)), zero)
    inv, power, reach = torch.eye(c, device=state.device) - a, a, 1
    while 2 * reach < c:  # (1 + a)^-1 = (1 - a)(1 + a^2)(1 + a^4) ..., as a^c = 0
        power = torch.matmul(power, power)
        inv, reach = inv + torch.matmul(inv, power), 2 * reach
    p = torch.matmul(q, k.transpose(3, 4)) * decay
    x, outs = state, []
    for i in range(nc):
        u = torch.matmul(inv[i], beta[i] * (v[i] - fall[i] * torch.matmul(k[i], x)))
        outs.append(fall[i] * torch.matmul(q[i], x) + torch.matmul(p[i], u))
        x = fall[i][:, :, -1:] * x + torch.matmul((rest[i] * k[i]).transpose(2, 3), u)
    state.copy_(x)
    o = torch.stack(outs).permute(1, 0, 3, 2, 4).reshape(n, nc * c, hv, dv)[there]
    return {"out": o.to(s["v"].dtype), "state": state}


def _logprobs(s):
    x, ids, top = s["logits"].float(), s["ids"].long(), s["case"]["top"]
    most = x.amax(1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(1, keepdim=True)
    lse = most + torch.log(total)
    p = e / total
    entropy = lse[:, 0] - torch.where(p == 0, torch.zeros_like(p), p * x).sum(1)
    # the order of (value, lower index first) as one whole number
    bits = x.view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = order * (1 << 20) + ((1 << 20) - 1 - torch.arange(x.shape[1], device=x.device))
    best = torch.topk(key, top, 1).values
    top_ids = (1 << 20) - 1 - (best & ((1 << 20) - 1))
    return {"logprobs": torch.gather(x, 1, ids) - lse, "entropy": entropy, "lse": lse[:, 0],
            "top_ids": top_ids.int(), "top_logprobs": torch.gather(x, 1, top_ids) - lse}


def _call(s):
    from bit_trellis_quantized_gb300 import native

    op = s["case"]["op"]
    if op == "attention":
        out, lse = native.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], k_new=s["k_new"],
                                          v_new=s["v_new"], scale=s["scale"], max_len=s["longest"])
        return {"out": out, "lse": lse, "k": s["k"], "v": s["v"]}
    if op == "delta":
        out = native.delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["at"], scale=s["scale"],
                                norm_eps=1e-6, max_len=s["longest"])
        return {"out": out, "state": s["state"]}
    r = native.token_logprobs(s["logits"], s["ids"], top=s["case"]["top"])
    return {"logprobs": r["logprobs"], "entropy": r["entropy"], "lse": r["lse"], "top_ids": r["top_ids"],
            "top_logprobs": r["top_logprobs"]}


def run(state):
    if own:
        return _call(state)
    return {"attention": _attention, "delta": _delta, "logprobs": _logprobs}[state["case"]["op"]](state)


# ---- the definitions in 64 bits ------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        q, lens = s["q"].double(), s["lens"].tolist()
        h, kv, ps = case["heads"], case["kv_heads"], case["page"]
        out = torch.zeros_like(q)
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pages = s["table"][b, :-(-n // ps)].long()
            s["k"][pages[-1], :, (n - 1) % ps] = s["k_new"][b]
            s["v"][pages[-1], :, (n - 1) % ps] = s["v_new"][b]
            for i in range(kv):
                keys = s["k"][pages, i].reshape(-1, case["dim"])[:n].double()
                values = s["v"][pages, i].reshape(-1, case["dim"])[:n].double()
                mine = slice(i * (h // kv), (i + 1) * (h // kv))
                x = (q[b, mine] @ keys.T) * s["scale"]
                out[b, mine] = torch.softmax(x, 1) @ values
                lse[b, mine] = torch.logsumexp(x, 1)
        return {"out": out, "lse": lse, "k": s["k"].double(), "v": s["v"].double()}
    if case["op"] == "delta":
        rep = case["v_heads"] // case["k_heads"]
        unit = lambda x: x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)  # noqa: E731
        q = unit(s["q"].double()).repeat_interleave(rep, 1) * s["scale"]
        k = unit(s["k"].double()).repeat_interleave(rep, 1)
        v, keep, beta = s["v"].double(), torch.exp(s["g"].double()), s["beta"].double()
        state, out, at = s["state"].double(), torch.zeros_like(v), s["at"].tolist()
        lens = [b - a for a, b in zip(at, at[1:])]
        for i in range(max(lens)):  # token i of every sequence that has one
            on = [b for b, n in enumerate(lens) if n > i]
            every = len(on) == len(lens)
            rows = torch.tensor([at[b] + i for b in on], device="cuda")
            where = torch.tensor(on, device="cuda")
            x = (state if every else state[where]) * keep[rows][:, :, None, None]
            ki = k[rows]
            u = beta[rows][..., None] * (v[rows] - torch.einsum("bhij,bhi->bhj", x, ki))
            x = x + ki[..., None] * u[:, :, None]
            out[rows] = torch.einsum("bhij,bhi->bhj", x, q[rows])
            if every:
                state = x
            else:
                state[where] = x
        return {"out": out, "state": state}
    x, ids = s["logits"], s["ids"].long()
    r = {"logprobs": [], "entropy": [], "lse": [], "top_ids": None, "top_logprobs": []}
    for a in range(0, case["rows"], 64):
        y = x[a:a + 64].double()
        lp = y - torch.logsumexp(y, 1, keepdim=True)
        r["lse"].append(torch.logsumexp(y, 1))
        r["entropy"].append(-torch.xlogy(torch.exp(lp), torch.exp(lp)).sum(1))
        r["logprobs"].append(torch.gather(lp, 1, ids[a:a + 64]))
        r["top_logprobs"].append(torch.sort(lp, 1, descending=True).values[:, :case["top"]])
    return {k: None if v is None else torch.cat(v) for k, v in r.items()}
