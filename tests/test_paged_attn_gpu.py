"""Attention over the paged cache (ds_paged_attention) against a plain implementation in 64
bits, tolerances as derived in paged_ref.check_attention; and the operators of a decode step
run together.

The kernel is chosen by the query rows per key head and by the tokens that the page table has
room for: `wide` tables have room for more than 200,000 tokens, most of it unused, so that
more than 32 rows (24 at head_dim 128) take the tensor-memory kernel at short lengths too."""
import pytest
import torch

import paged_ref as ref
import synth
import q4_moe_speculative_gb300 as dsm

pytestmark = pytest.mark.gpu

DEV = "cuda"


def problem(lens, R, Hq, kv, D, page, q8, seed, strided=False, sigma=1.0, spare=2, wide=False):
    g = torch.Generator()
    g.manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + spare
    shape = (pages, 2, kv, page, D)
    if q8:
        pool = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).to(DEV)
        sc = (torch.rand(shape[:4], generator=g) * 0.02 + 0.002).to(DEV)
        parts = [pool[:, 0], pool[:, 1], sc[:, 0], sc[:, 1]]
    else:
        pool = torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)
        parts = [pool[:, 0], pool[:, 1]]
    cache = dsm.PagedCache(*(p if strided else p.contiguous() for p in parts))
    order = torch.randperm(pages, generator=g).to(torch.int32)
    columns = max(1, max(need))
    if wide:
        columns = max(columns, 200_000 // (page * len(lens) * kv) + 1)
    table = torch.full((len(lens), columns), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = (torch.randn((len(lens), R, Hq, D), generator=g) * sigma).to(torch.bfloat16)
    return q.to(DEV), cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def check(q, cache, table, lengths, scale=None, got=None):
    D = q.shape[-1]
    if got is None:
        got = dsm.paged_attention(q, cache, table, lengths, scale=scale)
    want = ref.attention(q, cache, table, lengths, D ** -0.5 if scale is None else scale)
    ref.check_attention(got, want, max(1, int(lengths.max())), D)
    return got


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,R,Hq,kv,D,page", [
    ([1], 1, 1, 1, 128, 16),                       # one token, one head
    ([1], 1, 8, 8, 64, 16),
    ([16, 17, 63, 64, 65, 127, 1, 3], 1, 4, 2, 128, 16),
    ([500], 1, 16, 2, 128, 16),
    ([300, 7], 6, 16, 1, 128, 64),                 # M = 96
    ([257], 8, 16, 1, 64, 32),                     # M = 128
    ([190, 191, 64, 66], 8, 16, 2, 128, 32),       # M = 64
    ([1, 0, 129, 2, 256, 640, 127], 5, 16, 2, 128, 16),   # M = 40
    ([400, 3, 128, 257], 7, 14, 2, 64, 64),        # M = 49
    ([1000, 128, 5], 5, 16, 1, 128, 128),          # M = 80
    ([130, 5, 70], 3, 6, 2, 64, 128),              # M = 9
    ([77, 200], 4, 14, 2, 128, 16),                # M = 28
    ([2, 0, 1, 5, 0], 8, 2, 1, 128, 16),           # rows that see nothing, empty sequences
    ([0, 0, 0], 2, 2, 2, 64, 64),                  # nothing at all
    ([3000], 1, 5, 1, 128, 64),
    ([5000, 40], 2, 4, 2, 64, 128),
    ([1 + 13 * i % 150 for i in range(70)], 2, 3, 3, 64, 16),
])
def test_attention_matches_64_bits(lens, R, Hq, kv, D, page, q8, wide):
    check(*problem(lens, R, Hq, kv, D, page, q8, seed=sum(lens) + R + D, strided=R % 2 == 0,
                   wide=wide))


@pytest.mark.parametrize("M", [1, 15, 16, 17, 31, 32, 33, 48, 64, 65, 80, 96, 97, 112, 127, 128])
@pytest.mark.parametrize("D,q8", [(128, False), (64, True), (128, True), (64, False)])
def test_every_count_of_rows(M, D, q8):
    R = 1 if M % 2 else (8 if M % 8 == 0 and M <= 64 else 2)
    check(*problem([150, 65], R, M // R, 1, D, 32, q8, seed=M))
    if 24 < M:
        check(*problem([150, 65], R, M // R, 1, D, 32, q8, seed=M, wide=True))


@pytest.mark.parametrize("Hq,wide", [(4, False), (8, False), (8, True), (10, False), (10, True), (30, True)])
@pytest.mark.parametrize("q8", [False, True])
def test_peaked_and_rising_scores(q8, Hq, wide):
    # scores of hundreds, growing along the length: the reference of every row moves again
    # and again
    q, cache, table, lengths = problem([700, 333], 4, Hq, 1, 128, 16, q8, seed=3, sigma=12.0,
                                       wide=wide)
    check(q, cache, table, lengths)
    ramp = torch.linspace(0.01, 4, 700)
    slots = table[0].cpu().long()[torch.arange(700) // 16] * 16 + torch.arange(700) % 16
    rows = q[0, 3, 0].float().cpu()[None] * ramp[:, None] / 12
    if q8:
        codes, sc = ref.quantise(rows.to(torch.bfloat16)[:, None])
        for i, s in enumerate(slots.tolist()):
            cache.k[s // 16, 0, s % 16] = torch.from_numpy(codes[i, 0]).to(DEV)
            cache.k_scale[s // 16, 0, s % 16] = float(sc[i, 0])
    else:
        for i, s in enumerate(slots.tolist()):
            cache.k[s // 16, 0, s % 16] = rows[i].to(torch.bfloat16).to(DEV)
    check(q, cache, table, lengths)


def test_scale_argument():
    p = problem([100, 30], 2, 4, 2, 64, 16, False, seed=5)
    for scale in (0.0, 1.0, -0.3):
        check(*p, scale=scale)


@pytest.mark.parametrize("Hq,wide", [(4, False), (16, False), (16, True), (20, False), (20, True), (60, True)])
@pytest.mark.parametrize("q8", [False, True])
def test_what_is_not_visible_does_not_matter(q8, Hq, wide):
    # everything behind the lengths, in other pages, and in new tokens that a row does not
    # see holds infinities and NaN
    lens, R, page = [37, 64, 129, 6, 3], 4, 16
    q, cache, table, lengths = problem(lens, R, Hq, 2, 128, page, q8, seed=8, wide=wide)
    clean = dsm.paged_attention(q, cache, table, lengths)
    seen = torch.zeros(cache.k.shape[0] * page, dtype=torch.bool)
    for b, n in enumerate(lens):
        t = torch.arange(n - (R - 1) if n > R - 1 else 0)
        seen[table[b].cpu().long()[t // page] * page + t % page] = True
    one_q = q[:, :1].contiguous()
    for bad in (float("inf"), float("nan"), -float("inf")):
        parts = {}
        for n in ("k", "v", "k_scale", "v_scale"):
            t = getattr(cache, n)
            if t is None or (q8 and not n.endswith("scale")):
                parts[n] = t
                continue
            by_slot = ref.flat(t).clone()
            by_slot[~seen.to(DEV)] = bad
            parts[n] = by_slot.view(t.shape[0], page, *by_slot.shape[1:]).transpose(1, 2).contiguous()
        dirty = dsm.PagedCache(**parts)
        out = dsm.paged_attention(q, dirty, table, lengths)
        # row 0 sees only clean tokens; the others see a new one, and show it
        assert torch.equal(out[:, 0], clean[:, 0])
        # longer sequences in the cache than asked for: all rows clean when one fewer is new
        short = (lengths - (R - 1)).clamp(min=0)
        one = dsm.paged_attention(one_q, dirty, table, short)
        want = dsm.paged_attention(one_q, cache, table, short)
        assert torch.equal(one, want)
        assert bool(torch.isfinite(one).all())


@pytest.mark.parametrize("Hq,wide", [(4, False), (32, True), (40, False), (40, True), (100, True)])
@pytest.mark.parametrize("q8", [False, True])
def test_bad_pages_are_skipped(q8, Hq, wide):
    page = 16
    q, cache, table, lengths = problem([100, 64, 40], 2, Hq, 2, 128, page, q8, seed=9, wide=wide)
    table[0, 2], table[1, 0], table[1, 3], table[2, :] = -1, cache.k.shape[0], 2**31 - 1, -5
    out = check(q, cache, table, lengths)
    assert bool((out[2] == 0).all())


@pytest.mark.parametrize("Hq,wide", [(2, False), (40, False), (40, True)])
def test_lengths_are_clamped(Hq, wide):
    q, cache, table, lengths = problem([64, 64], 1, Hq, 1, 64, 16, True, seed=10, wide=wide)
    want = dsm.paged_attention(q, cache, table, lengths)
    odd = torch.tensor([2**31 - 1, -3], dtype=torch.int32, device=DEV)
    out = dsm.paged_attention(q, cache, table, odd)
    assert torch.equal(out[0], want[0]) and bool((out[1] == 0).all())


@pytest.mark.parametrize("Hq,wide", [(8, False), (32, False), (32, True)])
def test_shared_pages_and_repeated_rows(Hq, wide):
    # two sequences on the same pages give the same bytes, and so do two calls
    q, cache, table, lengths = problem([900, 900], 2, Hq, 1, 128, 32, True, seed=11, wide=wide)
    table[1], q[1] = table[0], q[0]
    out = dsm.paged_attention(q, cache, table, lengths)
    again = dsm.paged_attention(q, cache, table, lengths)
    assert torch.equal(out, again)
    check(q, cache, table, lengths, got=out)


def test_no_sequences():
    q, cache, _, _ = problem([5], 1, 2, 1, 64, 16, False, seed=1)
    none = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    out = dsm.paged_attention(q[:0], cache, none, none[:, 0].contiguous())
    assert out.shape == (0, 1, 2, 64)


@pytest.mark.parametrize("Hq", [1, 5, 10, 20, 40])
@pytest.mark.parametrize("q8", [False, True])
def test_a_long_context_over_every_cta(q8, Hq):
    # 70,000 tokens of one head: pieces on every CTA, joined; against fp64 on the device
    n, page = 70_001, 64
    q, cache, table, lengths = problem([n], 3, Hq, 1, 128, page, q8, seed=12, sigma=2.0,
                                       wide=Hq in (20, 40))
    out = dsm.paged_attention(q, cache, table, lengths)
    t = torch.arange(n, device=DEV)
    slots = table[0].long()[t // page] * page + t % page
    kv = []
    for side in ("k", "v"):
        x = ref.flat(getattr(cache, side))[slots, 0].double()
        if q8:
            x = x * ref.flat(getattr(cache, side + "_scale"))[slots, 0].double()[:, None]
        kv.append(x)
    s = torch.einsum("rhd,td->rht", q[0].double(), kv[0]) * 128 ** -0.5
    last = n - (2 - torch.arange(3, device=DEV))
    s = s.masked_fill(t >= last[:, None, None], float("-inf"))
    p = torch.softmax(s, -1)
    top = float((q[0].double().abs().flatten(0, 1) @ kv[0].abs().t()).max() * 128 ** -0.5)
    want = (torch.einsum("rht,td->rhd", p, kv[1])[None].cpu(),
            torch.einsum("rht,td->rhd", p, kv[1].abs())[None].cpu(),
            torch.einsum("rht,td->rhd", p * p, kv[1] ** 2).sqrt()[None].cpu(), top)
    # (a CTA sums its own tiles, 70,001 / 152 tokens at most, then the pieces)
    ref.check_attention(out, want, n // 64, 128)


# --------------------------------------------------------------------- the operators together
def decode_step(st, cache):
    """The attention side of a layer's verify step: norms, rotation and cache write of the new
    tokens, attention, and the output projection."""
    T, R = st["qkv"].shape[0], st["R"]
    Hq, kv = st["Hq"], st["kv"]
    qkv = st["qkv"]
    q = dsm.qk_norm_rope_write(qkv[:, :Hq], qkv[:, Hq:Hq + kv], qkv[:, Hq + kv:], st["pos"],
                               st["freqs"], cache, st["slots"], q_weight=st["qw"],
                               k_weight=st["kw"])
    o = dsm.paged_attention(q.view(T // R, R, Hq, -1), cache, st["table"], st["lengths"])
    y = [dsm.q4_project(st["tiles"], o[b].reshape(R, -1)) for b in range(T // R)]
    return q, o, torch.stack(y)


def step_inputs(B, R, Hq, kv, D, page, steps, H, seed):
    total = R * steps
    per = -(-total // page)
    table = torch.randperm(B * per, generator=torch.Generator().manual_seed(seed))
    table = table.view(B, per).to(torch.int32)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    qs, sc = synth.q4_matrix((), H, Hq * D, g, DEV)
    st = {"R": R, "Hq": Hq, "kv": kv, "table": table.to(DEV), "freqs": dsm.rope_frequencies(D),
          "qw": (1 + ref.normal(D, seed=1, sigma=0.1).float()).to(torch.bfloat16).to(DEV),
          "kw": (1 + ref.normal(D, seed=2, sigma=0.1).float()).to(torch.bfloat16).to(DEV),
          "tiles": dsm.q4_tile(qs, sc)}
    return st, table, B * per


def step_at(table, i, B, R, Hq, kv, D, page, seed):
    pos = torch.arange(R)[None] + i * R + torch.zeros(B, 1, dtype=torch.long)
    slots = torch.gather(table.long(), 1, pos // page) * page + pos % page
    return {"qkv": ref.normal(B * R, Hq + 2 * kv, D, seed=seed + i).to(DEV),
            "pos": pos.flatten().to(torch.int32).to(DEV),
            "slots": slots.flatten().to(torch.int32).to(DEV),
            "lengths": torch.full((B,), (i + 1) * R, dtype=torch.int32, device=DEV)}


@pytest.mark.parametrize("q8", [False, True])
def test_decode_steps_eager_and_captured(q8):
    B, R, Hq, kv, D, page, steps, H = 3, 4, 8, 2, 128, 16, 9, 256
    st, table, pages = step_inputs(B, R, Hq, kv, D, page, steps, H, seed=31)
    eager = dsm.PagedCache.zeros(pages, kv, page, D, q8=q8)
    wants = []
    W = ref.q4_weights(st["tiles"])
    for i in range(steps):
        st.update(step_at(table, i, B, R, Hq, kv, D, page, seed=50))
        q, o, y = decode_step(st, eager)
        wants.append((q.clone(), o.clone(), y.clone()))
        # every operator against its own formula on what the one before it gave
        f, _ = ref.turn_steps(D)
        x = st["qkv"].cpu()
        qref, both = ref.norm_rope(x[:, :Hq], st["qw"].cpu(), st["pos"].cpu(), f, 1e-6, False)
        err = (q.cpu().double() - qref).abs()
        assert bool((err <= ref.HALF_BF16 * qref.abs() + 2.0 ** -19 * both * 1.01).all())
        check(q.view(B, R, Hq, D), eager, st["table"], st["lengths"], got=o)
        for b in range(B):
            xb = o[b].reshape(R, -1).cpu().double()
            tol = ref.HALF_BF16 * (xb @ W.t()).abs() + 100 * 2 * ref.U32 * (xb.abs() @ W.abs().t())
            assert bool(((y[b].cpu().double() - xb @ W.t()).abs() <= tol).all())
    # the same steps as replays of one captured graph
    cache = dsm.PagedCache.zeros(pages, kv, page, D, q8=q8)
    st.update({k: v.clone() for k, v in step_at(table, 0, B, R, Hq, kv, D, page, 50).items()})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode_step(st, cache)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = decode_step(st, cache)
    for i in range(steps):
        for k, v in step_at(table, i, B, R, Hq, kv, D, page, seed=50).items():
            st[k].copy_(v)
        graph.replay()
        for got, want in zip(outs, wants[i]):
            assert torch.equal(got, want), i
    for n in ("k", "v", "k_scale", "v_scale"):
        if getattr(cache, n) is not None:
            assert torch.equal(getattr(cache, n), getattr(eager, n)), n


@pytest.mark.parametrize("Hq,q8", [(8, True), (40, False)])
def test_two_streams_at_once(Hq, q8):
    # two calls in flight, each with its own workspace (allocated on its own stream)
    ps = [problem([4000, 100], 2, Hq, 2, 128, 32, q8, seed=40 + i, wide=Hq > 8)
          for i in range(2)]
    wants = [dsm.paged_attention(*p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [[] for _ in ps]
    for _ in range(20):
        for i, (p, s) in enumerate(zip(ps, streams)):
            outs[i].append(dsm.paged_attention(*p, stream=s))
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        for o in got:
            assert torch.equal(o, want)


@pytest.mark.parametrize("Hq,lens,wide", [(8, [2000], False), (8, [2000], True), (3, [2000], False),
                                          (4, [700, 90, 333] * 4, False)])
def test_given_workspace_and_output(Hq, lens, wide):
    # whatever the workspace holds
    q, cache, table, lengths = problem(lens, 6, Hq, 1, 128, 64, False, seed=44, wide=wide)
    want = dsm.paged_attention(q, cache, table, lengths)
    out = torch.empty_like(q)
    for fill in (0xA5, 0x00, 0x01, 0xFF):
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device=DEV)
        assert dsm.paged_attention(q, cache, table, lengths, out=out, workspace=ws) is out
        assert torch.equal(out, want)
        assert dsm.workspace_status(ws) == 0
    with pytest.raises(dsm.DsmoeError) as e:
        dsm.paged_attention(q, cache, table, lengths, workspace=ws[:256])
    assert e.value.status == 3


@pytest.mark.parametrize("Hq,q8,wide", [(3, True, False), (4, False, False), (10, False, False),
                                        (10, True, True)])
def test_replays_with_other_lengths(Hq, q8, wide):
    # one captured call (the first of its sizes in this process or not) whose lengths, table and
    # queries change between replays; the workspace keeps what the longer calls left in it
    q, cache, table, lengths = problem([900, 130, 64, 700], 4, Hq, 1, 64, 32, q8, seed=21,
                                       wide=wide)
    out = torch.empty_like(q)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsm.paged_attention(q, cache, table, lengths, out=out, workspace=ws)
    for lens in ([900, 130, 64, 700], [1, 0, 64, 3], [0, 0, 0, 0], [64, 130, 2, 512], [900, 130, 0, 1]):
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(q.flip(0))
        g.replay()
        check(q, cache, table, lengths, got=out)


@pytest.mark.parametrize("q8", [False, True])
def test_caches_beyond_32_bits(q8):
    # pages more than 2^32 bytes and 2^31 values apart give what the same pages side by side give
    page, kv, D, R, lens = 64, 8, 128, 5, [250, 129]
    n = 70_000 if q8 else 40_000
    big = dsm.PagedCache.zeros(1, kv, page, D, q8=q8)
    big = dsm.PagedCache(*(torch.empty((n, *t.shape[1:]), dtype=t.dtype, device=DEV)
                           for t in (big.k, big.v, big.k_scale, big.v_scale) if t is not None))
    small = dsm.PagedCache.zeros(8, kv, page, D, q8=q8)
    near = torch.arange(8, dtype=torch.int32).view(2, 4)
    pages = torch.tensor([n - 1, 0, n - 2, 1, n // 2, n - 3, 3, n - 4], dtype=torch.int32)
    far = pages.view(2, 4)
    T = sum(lens)
    k, v = (ref.normal(T, kv, D, seed=50 + i).to(DEV) for i in range(2))
    at = {}
    for name, table, cache in (("near", near, small), ("far", far, big)):
        slots = torch.cat([table[b].long()[torch.arange(m) // page] * page + torch.arange(m) % page
                           for b, m in enumerate(lens)]).to(torch.int32).to(DEV)
        dsm.cache_write(cache, k, v, slots)
        at[name] = [dsm.cache_read(cache, slots)]
        for G, room in ((1, 4), (8, 4), (8, 12000)):
            q = ref.normal(2, R, G * kv, D, seed=60 + G).to(DEV)
            wide = torch.full((2, room), -1, dtype=torch.int32)
            wide[:, :4] = table
            at[name].append((dsm.paged_attention(
                q, cache, wide.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)),))
    for a, b in zip(at["near"], at["far"]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
