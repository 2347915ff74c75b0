"""The operators that a decode step of a served batch needs between its products: the cases that
are timed, their inputs, their plain forms, and their values in 64 bits.

  norm     a block's output normed, gated and scaled onto the residual stream, and the norm of the
           next block's input (block_norm)
  prefix   R rows of new tokens of sequences that share prompts, over the paged cache
           (prefix_attention)
  sample   a token per row of logits with temperature, top-k, top-p and min-p from given uniforms
           (sample)

Plain forms use elementary torch operations in 32 bits and round once; the draw of tokens, where
masses are compared with borders, is in 64. `exact` computes the same from the definitions in 64
bits.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # One verify step of one sequence between two blocks. The smallest call, latency counts.
        dict(name="norm step 6 x 4096", op="norm", tokens=6, hidden=4096, residual="bf16",
             post=False, gate="none", offset=0.0, x_scale=1.0, y_scale=1.0),
        # 64 sequences of 6 verify rows, residual stream in 32 bits, norms before and after.
        dict(name="norm 384 x 5000 fp32", op="norm", tokens=384, hidden=5000, residual="fp32",
             post=True, gate="none", offset=1.0, x_scale=1.0, y_scale=0.22),
        # A prompt in one piece, with a gate per channel.
        dict(name="norm prompt 16384 x 4096", op="norm", tokens=16384, hidden=4096,
             residual="bf16", post=True, gate="channel", offset=0.0, x_scale=1.0, y_scale=1.0),
        # A prompt's tokens with a gate per token and channel.
        dict(name="norm prompt 4099 x 2048 gated", op="norm", tokens=4099, hidden=2048,
             residual="fp32", post=True, gate="token", offset=0.0, x_scale=0.9, y_scale=1.0),
        # Four samples of a short prompt, one token each.
        dict(name="prefix 4 x 1 after 1000", op="prefix", prompts=1, samples=4, rows=1, heads=16,
             kv_heads=2, dim=128, page=16, prefix=1000, context=100, cache="bf16"),
        # A batch behind a long system prompt, cache in 8 bits, verify steps of 6 rows.
        dict(name="prefix 64 x 6 after 8192 q8", op="prefix", prompts=1, samples=64, rows=6,
             heads=32, kv_heads=8, dim=128, page=64, prefix=8192, context=512, cache="q8"),
        # 16 sequences that go on from a document of 100k tokens, all heads on one key head.
        dict(name="prefix 16 x 1 after 100k", op="prefix", prompts=1, samples=16, rows=1, heads=16,
             kv_heads=1, dim=128, page=64, prefix=100_003, context=256, cache="bf16"),
        # Three prompts with eight samples each, of which the lengths differ.
        dict(name="prefix 3 of 8 x 2 after 3001", op="prefix", prompts=3, samples=8, rows=2,
             heads=20, kv_heads=4, dim=64, page=32, prefix=3001, context=700, cache="bf16"),
        # The largest: a batch of verify steps behind 16k tokens.
        dict(name="prefix 64 x 6 after 16384", op="prefix", prompts=1, samples=64, rows=6,
             heads=32, kv_heads=8, dim=128, page=64, prefix=16384, context=512, cache="bf16"),
        # One sequence's token from the product over the vocabulary, in bf16.
        dict(name="sample 1 x 129280 top-k", op="sample", rows=1, vocab=129280, logits="bf16",
             temperature=0.8, top_k=50, top_p=0.95, min_p=0.0),
        # A batch's tokens, nucleus and min-p.
        dict(name="sample 64 x 129280 top-p", op="sample", rows=64, vocab=129280, logits="fp32",
             temperature=1.0, top_k=0, top_p=0.9, min_p=0.02),
        # Draft tokens of many rows over an odd vocabulary, temperature alone.
        dict(name="sample 200 x 32003", op="sample", rows=200, vocab=32003, logits="bf16",
             temperature=1.0, top_k=0, top_p=1.0, min_p=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "prefix", "sample"])
    if op == "norm":
        hidden = 8 * _log(rng, 8, 2048)
        return dict(op=op, tokens=_log(rng, 1, min(32768, 40_000_000 // hidden)), hidden=hidden,
                    residual=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token"]), offset=rng.choice([0.0, 1.0]),
                    x_scale=rng.choice([1.0, 0.9]), y_scale=rng.choice([1.0, 0.22]))
    if op == "sample":
        vocab = _log(rng, 500, 200_000)
        return dict(op=op, rows=_log(rng, 1, min(512, 8_273_920 // vocab)), vocab=vocab,
                    logits=rng.choice(["bf16", "fp32"]), temperature=rng.uniform(0.4, 1.4),
                    top_k=rng.choice([0, 0, 1, _log(rng, 2, 2000)]),
                    top_p=rng.choice([1.0, rng.uniform(0.5, 0.99)]),
                    min_p=rng.choice([0.0, rng.uniform(0.01, 0.2)]))
    kv = rng.choice([1, 2, 4, 8])
    rows = rng.randint(1, 8)
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16) if g * rows <= 128])
    prompts = rng.choice([1, 1, 1, 2, 3])
    samples = _log(rng, 1, 64)
    most = 64 * 6 * 32 * 16384 // (prompts * samples * rows * kv * group)
    prefix = _log(rng, 1, min(100_000, most, 1_000_000 // (prompts * kv)))
    context = _log(rng, 1, max(1, min(1024, most - prefix, 300_000 // (prompts * samples * kv))))
    return dict(op=op, prompts=prompts, samples=samples, rows=rows, heads=kv * group, kv_heads=kv,
                dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]), prefix=prefix,
                context=context, cache=rng.choice(["bf16", "q8"]))


# --------------------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _own_lengths(case):
    """Own tokens of each sequence, the new ones among them."""
    c, R = case["context"], case["rows"]
    n = case["prompts"] * case["samples"]
    return [max(R, c * (1 + (7 * b + 15) % 16) // 16) for b in range(n)]


def _prefix_lengths(case):
    return [max(1, case["prefix"] * (4 - p) // 4) for p in range(case["prompts"])]


def _tables(g, lens, page, order, at):
    """Page tables of these lengths from the pages order[at:], -1 behind them."""
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, at


def _prepare_prefix(case, g, st):
    page, D, kv = case["page"], case["dim"], case["kv_heads"]
    first, later = _prefix_lengths(case), _own_lengths(case)
    pages = sum(-(-n // page) for n in first + later) + 3
    shape = (pages, kv, page, D)
    pool = {}
    for side in ("k", "v"):
        if case["cache"] == "bf16":
            pool[side] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        else:
            pool[side] = torch.randint(-127, 128, shape, generator=g, device="cuda",
                                       dtype=torch.int8)
            pool[side + "_scale"] = torch.rand(shape[:3], generator=g, device="cuda") * 0.02 + 0.005
    st["cache"] = pool
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    st["prefix_table"], at = _tables(g, first, page, order, 0)
    st["table"], at = _tables(g, later, page, order, at)
    st["prefix_lengths"] = torch.tensor(first, dtype=torch.int32, device="cuda")
    st["lengths"] = torch.tensor(later, dtype=torch.int32, device="cuda")
    st["q"] = (_normal(g, len(later), case["rows"], case["heads"], D) * 1.5).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = {"case": case}
    if case["op"] == "prefix":
        _prepare_prefix(case, g, st)
    elif case["op"] == "norm":
        T, H = case["tokens"], case["hidden"]
        channel = torch.exp(0.5 * _normal(g, H))
        x = _normal(g, T, H) * channel * 4
        st["x"] = x if case["residual"] == "fp32" else x.to(torch.bfloat16)
        st["y"] = (_normal(g, T, H) * channel).to(torch.bfloat16)
        about = 1 - case["offset"]
        st["weight"] = (about + 0.1 * _normal(g, H)).to(torch.bfloat16)
        st["post_weight"] = None
        if case["post"]:
            st["post_weight"] = (about + 0.1 * _normal(g, H)).to(torch.bfloat16)
        st["gate"] = None
        if case["gate"] != "none":
            shape = (H,) if case["gate"] == "channel" else (T, H)
            st["gate"] = torch.sigmoid(_normal(g, *shape)).to(torch.bfloat16)
    else:
        B, V = case["rows"], case["vocab"]
        # a few likely tokens over a broad rest
        z = _normal(g, B, V) * 2 + 3 * torch.relu(_normal(g, B, V) - 2)
        st["logits"] = z.to(torch.bfloat16) if case["logits"] == "bf16" else z
        st["u"] = torch.rand(B, generator=g, device="cuda", dtype=torch.float64)
        # each row has its own settings, as the requests of a batch do
        row = torch.arange(B, device="cuda")
        st["temperature"] = (case["temperature"] * (1 + 0.1 * (row % 3))).to(torch.float32)
        st["top_k"] = (case["top_k"] * (1 + row % 2)).to(torch.int32)
        st["top_p"] = (case["top_p"] - 0.05 * (row % 2) * (case["top_p"] < 1)).to(torch.float32)
        st["min_p"] = (case["min_p"] * (1 + 0.5 * (row % 2))).to(torch.float32)
    return st


# -------------------------------------------------------------------------- the plain forms
def _norm(st):
    case = st["case"]
    x, y, o = st["x"].float(), st["y"].float(), case["offset"]
    if case["post"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (st["post_weight"].float() + o)
    if st["gate"] is not None:
        y = y * st["gate"].float()
    x = x * case["x_scale"] + y * case["y_scale"]
    h = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (st["weight"].float() + o)
    return [x.to(st["x"].dtype), h.to(torch.bfloat16)]


def _tokens(st, side, table):
    """The tokens of these pages, [sequences, kv_heads, tokens, D] in 32 bits."""
    pool, case = st["cache"], st["case"]
    table = table.long().clamp(min=0)
    x = pool[side][table].float()                          # [n, pages, kv, page, D]
    if case["cache"] == "q8":
        x = x * pool[side + "_scale"][table][..., None]
    return x.transpose(1, 2).reshape(table.shape[0], case["kv_heads"], -1, case["dim"])


def _prefix(st):
    case = st["case"]
    P, n, R = case["prompts"], case["samples"], case["rows"]
    H, kv, D = case["heads"], case["kv_heads"], case["dim"]
    B, G = P * n, case["heads"] // case["kv_heads"]
    q = st["q"].float().view(B, R, kv, G, D).permute(0, 2, 1, 3, 4).reshape(B, kv, R * G, D)
    # a prompt's sequences side by side, as rows of one product with its tokens
    qp = q.view(P, n, kv, R * G, D).transpose(1, 2).reshape(P, kv, n * R * G, D)
    sp = torch.matmul(qp, _tokens(st, "k", st["prefix_table"]).transpose(2, 3))
    seen = torch.arange(sp.shape[-1], device="cuda") < st["prefix_lengths"].long()[:, None]
    sp = sp.mul_(D ** -0.5).masked_fill_(~seen[:, None, None], float("-inf"))
    so = torch.matmul(q, _tokens(st, "k", st["table"]).transpose(2, 3)) * D ** -0.5
    r = torch.arange(R, device="cuda").repeat_interleave(G)
    last = st["lengths"].long()[:, None] - (R - 1 - r)      # visible: t < last
    seen = torch.arange(so.shape[-1], device="cuda") < last[..., None]
    so = so.masked_fill(~seen[:, None], float("-inf"))

    def by_prompt(x):     # [B, kv, R G, ...] as rows of the prompts
        return x.view(P, n, kv, R * G, -1).transpose(1, 2).reshape(P, kv, n * R * G, -1)

    def by_sequence(x):
        return x.view(P, kv, n, R * G, -1).transpose(1, 2).reshape(B, kv, R * G, -1)

    top = torch.maximum(sp.amax(-1, keepdim=True), by_prompt(so.amax(-1, keepdim=True)))
    sp = sp.sub_(top).exp_()
    so = torch.exp(so - by_sequence(top))
    total = by_sequence(sp.sum(-1, keepdim=True)) + so.sum(-1, keepdim=True)
    o = by_sequence(torch.matmul(sp, _tokens(st, "v", st["prefix_table"])))
    o = (o + torch.matmul(so, _tokens(st, "v", st["table"]))) / total
    return [o.view(B, kv, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, H, D).to(torch.bfloat16)]


def _sample(st):
    z = st["logits"].double()
    B, V = z.shape
    top = z.amax(-1, keepdim=True)
    T = st["temperature"].double()[:, None]
    near = z - top
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices   # ties: lowest first
    w = torch.exp(near / T)
    sw = w.gather(1, order)
    place = torch.arange(V, device=z.device)
    k = st["top_k"].long()[:, None]
    keep = (place < k) | (k <= 0)
    sw = torch.where(keep, sw, torch.zeros_like(sw))
    upto = sw.cumsum(-1)
    p = st["top_p"].double()[:, None]
    keep &= ((upto - sw) < p * upto[:, -1:]) | (p >= 1) | (place == 0)
    keep &= near.gather(1, order) >= T * torch.log(st["min_p"].double()[:, None])
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    w = torch.where(kept, w, torch.zeros_like(w))
    upto = w.cumsum(-1)
    total = upto[:, -1:]
    token = (upto <= st["u"][:, None] * total).sum(-1, keepdim=True).clamp(max=V - 1)
    prob = w.gather(1, token) / total
    return [token[:, 0].to(torch.int32), prob[:, 0].float()]


# ---------------------------------------------------------------------- the framework's calls
def _own(st):
    import q4_moe_speculative_gb300 as dsm
    case = st["case"]
    if case["op"] == "norm":
        return list(dsm.block_norm(st["x"], st["y"], weight=st["weight"],
                                   post_weight=st["post_weight"], gate=st["gate"], eps=EPS,
                                   weight_offset=case["offset"], x_scale=case["x_scale"],
                                   y_scale=case["y_scale"]))
    if case["op"] == "prefix":
        return [dsm.prefix_attention(st["q"], dsm.PagedCache(**st["cache"]), st["prefix_table"],
                                     st["prefix_lengths"], st["table"], st["lengths"])]
    return list(dsm.sample(st["logits"], st["u"], temperature=st["temperature"],
                           top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"]))


def _plain(st):
    return {"norm": _norm, "prefix": _prefix, "sample": _sample}[st["case"]["op"]](st)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "norm":
        T, H = case["tokens"], case["hidden"]
        x = 4 if case["residual"] == "fp32" else 2
        gate = {"none": 0, "channel": 2.0 * H, "token": 2.0 * T * H}[case["gate"]]
        return {"bytes": T * H * (2 * x + 2 + 2.0) + gate + 2.0 * H * (1 + case["post"]),
                "flops": T * H * (6.0 + 3 * case["post"])}
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2.0 if case["logits"] == "bf16" else 4.0), "flops": 4.0 * n}
    kept = case["dim"] * 2 if case["cache"] == "bf16" else case["dim"] + 4
    first, later = _prefix_lengths(case), _own_lengths(case)
    per = case["rows"] * case["heads"] * case["dim"]        # values of a sequence's queries
    pairs = case["samples"] * sum(first) + sum(later)       # (sequence, token)
    return {"bytes": 2.0 * (sum(first) + sum(later)) * case["kv_heads"] * kept + 4.0 * len(later) * per,
            "flops": 4.0 * pairs * per}


# ------------------------------------------------------------------------------------ exact
def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "prefix": _exact_prefix, "sample": _exact_sample}[case["op"]](st)


def _exact_norm(st):
    case = st["case"]

    def normed(t, w):
        t = t.double()
        rms = torch.sqrt(torch.sum(t ** 2, -1, keepdim=True) / t.shape[-1] + EPS)
        return t / rms * (w.double() + case["offset"])

    block = normed(st["y"], st["post_weight"]) if case["post"] else st["y"].double()
    factor = case["y_scale"] if st["gate"] is None else case["y_scale"] * st["gate"].double()
    x = case["x_scale"] * st["x"].double() + factor * block
    return [x, normed(x, st["weight"])]


def _exact_side(st, side, row, n):
    """The first n tokens behind a row of a page table, [kv_heads, n, D]."""
    page = st["case"]["page"]
    pages = row[:-(-n // page)].long()
    x = st["cache"][side][pages].double()
    if st["case"]["cache"] == "q8":
        x = x * st["cache"][side + "_scale"][pages].double().unsqueeze(-1)
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_prefix(st):
    case = st["case"]
    kv, R, G = case["kv_heads"], case["rows"], case["heads"] // case["kv_heads"]
    first, later = _prefix_lengths(case), _own_lengths(case)
    q = st["q"].double()
    out = torch.zeros_like(q)
    for p, np_ in enumerate(first):
        pk, pv = (_exact_side(st, s, st["prefix_table"][p], np_) for s in ("k", "v"))
        for b in range(p * case["samples"], (p + 1) * case["samples"]):
            k, v = (torch.cat((shared, _exact_side(st, s, st["table"][b], later[b])), 1)
                    for s, shared in (("k", pk), ("v", pv)))
            see = np_ + later[b] - (R - 1 - torch.arange(R, device="cuda"))
            qb = q[b].view(R, kv, G, -1)
            s = torch.einsum("rhgd,htd->hrgt", qb, k) / math.sqrt(case["dim"])
            hidden = torch.arange(k.shape[1], device="cuda") >= see[:, None]
            s = s.masked_fill(hidden[None, :, None], -math.inf)
            out[b] = torch.einsum("hrgt,htd->rhgd", torch.softmax(s, -1), v).reshape(q[b].shape)
    return [out]


def _exact_sample(st):
    """Row by row: the kept set from the sorted tokens, then the draw in token order."""
    tokens, probs = [], []
    for b in range(st["logits"].shape[0]):
        z = st["logits"][b].double()
        T = st["temperature"][b].double()
        logp = torch.log_softmax(z / T, 0)
        by_id = torch.argsort(-z, stable=True)
        k = int(st["top_k"][b])
        if k > 0:
            by_id = by_id[:k]
        mass = torch.exp(logp[by_id])
        if float(st["top_p"][b]) < 1:
            before = torch.cat((mass.new_zeros(1), torch.cumsum(mass, 0)[:-1]))
            by_id = by_id[:max(1, int((before < st["top_p"][b].double() * mass.sum()).sum()))]
        if float(st["min_p"][b]) > 0:
            by_id = by_id[z[by_id] - z.max() >= T * math.log(float(st["min_p"][b]))]
        ids = torch.sort(by_id).values
        mass = torch.exp(logp[ids])
        upto = torch.cumsum(mass, 0)
        at = min(int((upto <= st["u"][b] * upto[-1]).sum()), len(ids) - 1)
        tokens.append(ids[at])
        probs.append(mass[at] / upto[-1])
    return [torch.stack(tokens).to(torch.int32), torch.stack(probs)]
