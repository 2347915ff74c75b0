"""The serving operators around the paged key-value cache and the Q4 projection: the cases that
are timed, their inputs, their plain forms, and their values in 64 bits.

  rotate   norms of queries and keys per head with the position rotation (qk_norm_rope)
  admit    the same pass with the keys and values going to the paged cache (qk_norm_rope_write)
  write    keys and values into the paged cache (cache_write); a Q8 cache is read back as well
  read     tokens of the cache back as bf16 (cache_read)
  attend   R rows of new tokens over the paged cache (paged_attention)
  q4       R rows through one tile-major Q4 matrix (q4_project)

Plain forms use elementary torch operations in 32 bits (64 for the angles of far positions) and
round once; `exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0
FIRST_POSITION = 200_000    # tokens of a long context: far positions


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # One verify step of one sequence: 6 rows, 16 query heads on one shared key head (the
        # head layout of the sparse attention). The smallest call, latency counts.
        dict(name="rotate step 6 rows", op="rotate", tokens=6, heads=16, kv_heads=1, dim=128,
             rotary=128, interleaved=False),
        # A prompt in one piece.
        dict(name="rotate prompt 16384", op="rotate", tokens=16384, heads=16, kv_heads=4, dim=128,
             rotary=64, interleaved=True),
        # 64 sequences of 6 verify rows, keys and values kept in 8 bits, read back to be compared.
        dict(name="admit 64 steps q8", op="admit", tokens=384, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, page=64, cache="q8"),
        # A prompt's tokens on their way into a bf16 cache.
        dict(name="admit prompt 4099 bf16", op="admit", tokens=4099, heads=16, kv_heads=4, dim=64,
             rotary=32, interleaved=True, page=16, cache="bf16"),
        # The new tokens of a few sequences.
        dict(name="write step 48 bf16", op="write", tokens=48, kv_heads=4, dim=128, page=32,
             cache="bf16"),
        # A long prompt's keys and values quantised, and read back.
        dict(name="write prompt 32768 q8", op="write", tokens=32768, kv_heads=8, dim=128, page=64,
             cache="q8"),
        # A shared prefix read back for the prompts that go on from it.
        dict(name="read prefix 8192 q8", op="read", tokens=8192, kv_heads=4, dim=128, page=64,
             cache="q8"),
        # One new token after a short context.
        dict(name="attend 1 x 1 at 500", op="attend", seqs=1, rows=1, heads=16, kv_heads=2,
             dim=128, page=16, context=500, ragged=False, cache="bf16"),
        # A batch of verify steps at ragged contexts of up to 8k tokens, cache in 8 bits.
        dict(name="attend 32 x 6 at 8k q8", op="attend", seqs=32, rows=6, heads=32, kv_heads=8,
             dim=128, page=64, context=8192, ragged=True, cache="q8"),
        # One sequence's verify step at 300k tokens, all heads on one key head.
        dict(name="attend 1 x 6 at 300k", op="attend", seqs=1, rows=6, heads=16, kv_heads=1,
             dim=128, page=64, context=300_000, ragged=False, cache="bf16"),
        # A square projection of the hidden size for one row.
        dict(name="q4 4096 x 4096 R1", op="q4", rows=4096, K=4096, R=1),
        # The product over the vocabulary for one verify step.
        dict(name="q4 129280 x 4096 R6", op="q4", rows=129280, K=4096, R=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "admit", "write", "read", "attend", "attend", "q4"])
    if op == "q4":
        K = 64 * _log(rng, 1, 192)
        most = 129280 * 4096 // K // 16
        return dict(op=op, rows=16 * _log(rng, 1, min(most, 8080)), K=K, R=rng.randint(1, 8))
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "q8"])
    if op == "attend":
        rows = rng.randint(1, 8)
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16) if g * rows <= 128])
        seqs = _log(rng, 1, 64)
        context = _log(rng, 1, min(300_000, 700_000 // (seqs * kv),
                                   28_800_000 // (seqs * kv * rows * group)))
        return dict(op=op, seqs=seqs, rows=rows, heads=kv * group, kv_heads=kv, dim=dim, page=page,
                    context=context, ragged=rng.random() < 0.7, cache=cache)
    if op in ("write", "read"):
        return dict(op=op, tokens=_log(rng, 1, 32768 * 8 // kv // 2), kv_heads=kv, dim=dim,
                    page=page, cache=cache)
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    case = dict(op=op, tokens=_log(rng, 1, 16384 * 24 // (heads + 2 * kv)), heads=heads,
                kv_heads=kv, dim=dim, rotary=rng.choice([dim, dim // 2, 16, 0]),
                interleaved=rng.random() < 0.5)
    if op == "admit":
        case.update(page=page, cache=cache)
    return case


# --------------------------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens of each sequence (the new ones among them)."""
    n, c = case["seqs"], case["context"]
    if not case["ragged"]:
        return [c] * n
    return [max(1, c * (1 + (7 * b + 15) % 16) // 16) for b in range(n)]


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pool(g, case, pages):
    """Pages of a cache in use: keys and values of every slot."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    pool = {}
    for side in ("k", "v"):
        if case["cache"] == "bf16":
            pool[side] = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        else:
            pool[side] = torch.randint(-127, 128, shape, generator=g, device="cuda",
                                       dtype=torch.int8)
            pool[side + "_scale"] = torch.rand(shape[:3], generator=g, device="cuda") * 0.02 + 0.005
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, st = case["op"], {"case": case}
    if op == "q4":
        U, Tk = case["rows"] // 16, case["K"] // 64
        tiles = torch.randint(0, 256, (U, Tk, 576), generator=g, device="cuda", dtype=torch.uint8)
        scales = (_normal(g, U, Tk, 32) * 0.02).abs().to(torch.float16)
        tiles[..., 512:] = scales.view(torch.uint8)
        st["tiles"] = tiles
        st["x"] = _normal(g, case["R"], case["K"]).to(torch.bfloat16)
        return st
    D, kv = case["dim"], case["kv_heads"]
    if op == "attend":
        lens, page = _lengths(case), case["page"]
        need = [-(-n // page) for n in lens]
        st["cache"] = _pool(g, case, sum(need) + 3)
        order = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["seqs"], max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        st["table"] = table
        st["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q"] = (_normal(g, case["seqs"], case["rows"], case["heads"], D) * 1.5).to(torch.bfloat16)
        return st
    T = case["tokens"]
    if op in ("rotate", "admit"):
        # one projection's output holds a token's queries, keys and values side by side
        h = case["heads"]
        channel = torch.exp(0.5 * _normal(g, h + 2 * kv, D))
        qkv = (_normal(g, T, h + 2 * kv, D) * channel).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        st["q_weight"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16)
        st["k_weight"] = (1 + 0.1 * _normal(g, D)).to(torch.bfloat16)
        st["positions"] = (torch.arange(T, device="cuda") + FIRST_POSITION).to(torch.int32)
        n = case["rotary"]
        f = BASE ** (-torch.arange(0, n, 2, dtype=torch.float64, device="cuda") / max(n, 1))
        st["inv_freq"] = f
        st["freqs"] = torch.round(f / (2 * math.pi) * 2.0 ** 64).to(torch.int64)
    elif op == "write":
        kv_new = (_normal(g, T, 2, kv, D) * torch.exp(0.5 * _normal(g, 2, kv, D))).to(torch.bfloat16)
        st["k"], st["v"] = kv_new[:, 0], kv_new[:, 1]
    if op != "rotate":
        pages = -(-T * 9 // 8 // case["page"]) + 2
        st["cache"] = _pool(g, case, pages)
        slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * case["page"]
        slots = (slots + torch.arange(case["page"], device="cuda")).reshape(-1)[:T]
        st["slots"] = slots.to(torch.int32).contiguous()
    return st


# -------------------------------------------------------------------------- the plain forms
def _turned(x, weight, st):
    """Norm per head and rotation of x [T, heads, D], in 32 bits."""
    case = st["case"]
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    n = case["rotary"]
    if n == 0:
        return x
    a = st["positions"].double()[:, None] * st["inv_freq"]
    c, s = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    if case["interleaved"]:
        u, w = x[..., 0:n:2], x[..., 1:n:2]
        r = torch.stack((u * c - w * s, w * c + u * s), -1).flatten(-2)
    else:
        u, w = x[..., :n // 2], x[..., n // 2:n]
        r = torch.cat((u * c - w * s, w * c + u * s), -1)
    return torch.cat((r, x[..., n:]), -1)


def _put(st, side, x):
    """Rows x [T, kv_heads, D] into the cache's slots."""
    case, pool = st["case"], st["cache"]
    page, off = st["slots"].long() // case["page"], st["slots"].long() % case["page"]
    if case["cache"] == "bf16":
        pool[side][page, :, off] = x.to(torch.bfloat16)
        return
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    full = torch.full_like(top, 127.0)
    codes = torch.where(top > 0, torch.round(x * 127.0 / top), torch.zeros_like(x))
    pool[side][page, :, off] = codes.to(torch.int8)
    pool[side + "_scale"][page, :, off] = (top / full)[..., 0]


def _get(st, side):
    case, pool = st["case"], st["cache"]
    page, off = st["slots"].long() // case["page"], st["slots"].long() % case["page"]
    x = pool[side][page, :, off]
    if case["cache"] == "q8":
        x = (x.float() * pool[side + "_scale"][page, :, off][..., None]).to(torch.bfloat16)
    return x


def _kept(st):
    """What the cache holds after a write, as the values it stands for."""
    if st["case"]["cache"] == "bf16":
        return [st["cache"]["k"], st["cache"]["v"]]
    return [_get(st, "k"), _get(st, "v")]


def _attend(st):
    case, pool = st["case"], st["cache"]
    B, R, H, kv, D = case["seqs"], case["rows"], case["heads"], case["kv_heads"], case["dim"]
    table = st["table"].long().clamp(min=0)

    def tokens(side):
        x = pool[side][table].float()                      # [B, pages, kv, page, D]
        if case["cache"] == "q8":
            x = x * pool[side + "_scale"][table][..., None]
        return x.transpose(1, 2).reshape(B, kv, -1, D)

    q = st["q"].float().view(B, R, kv, H // kv, D).permute(0, 2, 1, 3, 4).reshape(B, kv, -1, D)
    s = torch.matmul(q, tokens("k").transpose(2, 3)) * D ** -0.5
    r = torch.arange(R, device="cuda").repeat_interleave(H // kv)
    last = st["lengths"].long()[:, None] - (R - 1 - r)      # visible: t < last
    seen = torch.arange(s.shape[-1], device="cuda") < last[..., None]
    s = s.masked_fill(~seen[:, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    o = torch.matmul(p, tokens("v")) / p.sum(-1, keepdim=True)
    o = torch.where((last > 0)[:, None, :, None], o, torch.zeros_like(o))
    return o.view(B, kv, R, H // kv, D).permute(0, 2, 1, 3, 4).reshape(B, R, H, D).to(torch.bfloat16)


def _q4(st):
    U, Tk = st["tiles"].shape[:2]
    n = st["tiles"][..., :512].view(U, Tk, 8, 4, 2, 2, 4)   # row, word, block, half, byte
    n = torch.stack((n & 15, n >> 4), -1)
    s = st["tiles"][..., 512:].view(torch.float16).view(U, Tk, 8, 2, 2).float()
    w = (n.float() - 8.0) * s[:, :, :, None, :, :, None, None]
    w = w.permute(0, 5, 2, 1, 4, 3, 6, 7).reshape(U * 16, Tk * 64)
    return torch.matmul(st["x"].float(), w.t()).to(torch.bfloat16)


def _plain(st):
    op = st["case"]["op"]
    if op == "rotate":
        return [_turned(st["q"], st["q_weight"], st).to(torch.bfloat16),
                _turned(st["k"], st["k_weight"], st).to(torch.bfloat16)]
    if op == "admit":
        q = _turned(st["q"], st["q_weight"], st).to(torch.bfloat16)
        _put(st, "k", _turned(st["k"], st["k_weight"], st))
        _put(st, "v", st["v"])
        return [q] + _kept(st)
    if op == "write":
        _put(st, "k", st["k"])
        _put(st, "v", st["v"])
        return _kept(st)
    if op == "read":
        return [_get(st, "k"), _get(st, "v")]
    return [_attend(st) if op == "attend" else _q4(st)]


# ---------------------------------------------------------------------- the framework's calls
def _own(st):
    import q4_moe_speculative_gb300 as dsm
    op = st["case"]["op"]
    if op == "q4":
        return [dsm.q4_project(st["tiles"], st["x"])]
    if op == "rotate":
        return list(dsm.qk_norm_rope(st["q"], st["k"], st["positions"], st["freqs"],
                                     q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                                     interleaved=st["case"]["interleaved"]))
    cache = dsm.PagedCache(**st["cache"])
    if op == "attend":
        return [dsm.paged_attention(st["q"], cache, st["table"], st["lengths"])]
    if op == "read":
        return list(dsm.cache_read(cache, st["slots"]))
    head = []
    if op == "admit":
        head = [dsm.qk_norm_rope_write(st["q"], st["k"], st["v"], st["positions"], st["freqs"],
                                       cache, st["slots"], q_weight=st["q_weight"],
                                       k_weight=st["k_weight"], eps=EPS,
                                       interleaved=st["case"]["interleaved"])]
    else:
        dsm.cache_write(cache, st["k"], st["v"], st["slots"])
    if st["case"]["cache"] == "bf16":
        return head + [cache.k, cache.v]
    return head + list(dsm.cache_read(cache, st["slots"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "q4":
        return {"bytes": case["rows"] * case["K"] * 9 / 16 + 2 * case["R"] * (case["rows"] + case["K"]),
                "flops": 2.0 * case["R"] * case["rows"] * case["K"]}
    D, kv = case["dim"], case["kv_heads"]
    kept = D * 2 if case.get("cache") == "bf16" else D + 4      # bytes of one row in the cache
    if op == "attend":
        n, per = sum(_lengths(case)), case["rows"] * case["heads"] * D
        return {"bytes": 2 * n * kv * kept + 4.0 * case["seqs"] * per, "flops": 4.0 * n * per}
    T = case["tokens"]
    back = 0 if case.get("cache") == "bf16" else 2 * T * kv * (kept + 2 * D)   # reading it back
    if op == "rotate":
        return {"bytes": 4.0 * T * (case["heads"] + kv) * D, "flops": 8.0 * T * (case["heads"] + kv) * D}
    if op == "admit":
        return {"bytes": 4.0 * T * case["heads"] * D + 2 * T * kv * (2 * D + kept) + back,
                "flops": 8.0 * T * (case["heads"] + kv) * D}
    if op == "write":
        return {"bytes": 2.0 * T * kv * (2 * D + kept) + back, "flops": 2.0 * T * kv * D}
    return {"bytes": 2.0 * T * kv * (kept + 2 * D), "flops": 2.0 * T * kv * D}


# ------------------------------------------------------------------------------------ exact
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "q4":
        return [_exact_q4(st)]
    if op == "attend":
        return [_exact_attend(st)]
    if op == "read":
        return [_exact_cached(st, "k"), _exact_cached(st, "v")]
    out = []
    if op in ("rotate", "admit"):
        k = _exact_turn(st, st["k"], st["k_weight"])
        out.append(_exact_turn(st, st["q"], st["q_weight"]))
        if op == "rotate":
            return out + [k]
    else:
        k = st["k"].double()
    for side, x in (("k", k), ("v", st["v"].double())):
        if case["cache"] == "bf16":
            whole = st["cache"][side].double()
            flat = whole.transpose(1, 2).reshape(-1, *whole.shape[1::2])   # by slot
            flat[st["slots"].long()] = x
            out.append(flat.view(whole.shape[0], case["page"], case["kv_heads"], -1).transpose(1, 2)
                       .contiguous())
        else:
            unit = x.abs().max(dim=-1, keepdim=True).values / 127.0
            out.append(torch.where(unit > 0, torch.round(x / unit) * unit, torch.zeros_like(x)))
    return out


def _exact_turn(st, x, weight):
    n, D = st["case"]["rotary"], st["case"]["dim"]
    x = x.double()
    x = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / D + EPS) * weight.double()
    if n == 0:
        return x
    i = torch.arange(n // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if st["case"]["interleaved"] else (i, i + n // 2)
    angle = st["positions"].double()[:, None, None] * torch.pow(
        torch.tensor(BASE, dtype=torch.float64, device="cuda"), -2.0 * i.double() / n)
    z = torch.polar(torch.ones_like(angle), angle) * torch.complex(x[..., first], x[..., second])
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_cached(st, side):
    slots, page = st["slots"].long(), st["case"]["page"]
    rows = st["cache"][side].transpose(1, 2).flatten(0, 1).double()
    if st["case"]["cache"] == "q8":
        rows = rows * st["cache"][side + "_scale"].transpose(1, 2).reshape(-1, rows.shape[1], 1).double()
    assert rows.shape[0] % page == 0
    return rows[slots]


def _exact_attend(st):
    case = st["case"]
    kv, page, R = case["kv_heads"], case["page"], case["rows"]
    q = st["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // kv
    for b, n in enumerate(_lengths(case)):
        pages = st["table"][b, :-(-n // page)].long()
        kvs = {}
        for side in ("k", "v"):
            x = st["cache"][side][pages].double()
            if case["cache"] == "q8":
                x = x * st["cache"][side + "_scale"][pages].double().unsqueeze(-1)
            kvs[side] = x.transpose(0, 1).flatten(1, 2)[:, :n]     # [kv, n, D]
        for r in range(R):
            see = n - (R - 1 - r)
            if see <= 0:
                continue
            qr = q[b, r].reshape(kv, group, -1)
            s = torch.einsum("hgd,htd->hgt", qr, kvs["k"][:, :see]) / math.sqrt(case["dim"])
            out[b, r] = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1),
                                     kvs["v"][:, :see]).reshape(-1, case["dim"])
    return out


def _exact_q4(st):
    """Row by row from the format's byte positions."""
    rows, K = st["case"]["rows"], st["case"]["K"]
    k = torch.arange(K, device="cuda")
    tile_k, in_tile = k // 64, k % 64
    block, value = in_tile // 32, in_tile % 32
    x = st["x"].double()
    y = torch.empty((x.shape[0], rows), dtype=torch.float64, device="cuda")
    flat = st["tiles"].view(-1)
    halves = st["tiles"].view(-1).view(torch.float16)
    for at in range(0, rows, 4096):
        i = torch.arange(at, min(rows, at + 4096), device="cuda")[:, None]
        tile = (i // 16) * (K // 64) + tile_k
        g, low = i % 8, (i % 16) // 8
        byte = tile * 576 + 16 * (4 * g + value // 8) + 4 * (2 * block + low) + (value % 8) // 2
        code = (flat[byte].long() >> (4 * (value % 2))) % 16 - 8
        scale = halves[tile * 288 + 256 + 4 * g + 2 * block + low].double()
        y[:, at:at + 4096] = x @ (code.double() * scale).t()
    return y
