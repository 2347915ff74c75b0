"""Attention of sequences that share prefixes (ds_prefix_attention) against a plain implementation
in 64 bits, tolerances as derived in paged_ref.check_attention."""
import pytest
import torch

import paged_ref as ref
import q4_moe_speculative_gb300 as dsm

pytestmark = pytest.mark.gpu

DEV = "cuda"


def problem(prefixes, lens, R, Hq, kv, D, page, q8, seed, strided=False, sigma=1.0, room=0):
    """Queries, cache, prefix table and lengths, page table and lengths. `room`: unused entries of
    both tables."""
    g = torch.Generator()
    g.manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in list(prefixes) + list(lens)]
    pages = sum(need) + 2
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
    tables, at = [], 0
    for counts in (need[:len(prefixes)], need[len(prefixes):]):
        t = torch.full((len(counts), max(1, max(counts)) + room), -1, dtype=torch.int32)
        for b, n in enumerate(counts):
            t[b, :n] = order[at:at + n]
            at += n
        tables.append(t.to(DEV))
    q = (torch.randn((len(lens), R, Hq, D), generator=g) * sigma).to(torch.bfloat16).to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return q, cache, tables[0], i32(prefixes), tables[1], i32(lens)


def slots_of(table, n, page, pages):
    n = min(max(n, 0), table.numel() * page)
    t = torch.arange(n)
    pg = table[t // page].long()
    ok = (pg >= 0) & (pg < pages)
    return t[ok], (pg * page + t % page)[ok]


def reference(q, cache, ptable, plens, table, lengths, scale):
    """(result, sum p |v|, sqrt(sum p^2 v^2), largest sum |q k| scale) in fp64, from the header's
    formula."""
    q = q.cpu().double()
    B, R, H, D = q.shape
    pages, kv, page, _ = cache.k.shape
    k, v = ref.values(cache, "k"), ref.values(cache, "v")
    ptable, plens, table, lengths = (t.cpu() for t in (ptable, plens, table, lengths))
    out, mag, rss = (torch.zeros_like(q) for _ in range(3))
    top, per = 0.0, B // ptable.shape[0]
    for b in range(B):
        n = min(int(lengths[b]), table.shape[1] * page)
        if n < 0:
            continue
        _, shared = slots_of(ptable[b // per], int(plens[b // per]), page, pages)
        t, own = slots_of(table[b], n, page, pages)
        for r in range(R):
            sl = torch.cat((shared, own[t < n - (R - 1 - r)]))
            if not len(sl):
                continue
            kk = k[sl].repeat_interleave(H // kv, 1)           # [tokens, H, D]
            vv = v[sl].repeat_interleave(H // kv, 1)
            p = torch.softmax(torch.einsum("thd,hd->ht", kk, q[b, r]) * scale, -1)
            out[b, r] = torch.einsum("ht,thd->hd", p, vv)
            mag[b, r] = torch.einsum("ht,thd->hd", p, vv.abs())
            rss[b, r] = torch.sqrt(torch.einsum("ht,thd->hd", p * p, vv * vv))
            top = max(top, float(torch.einsum("thd,hd->ht", kk.abs(), q[b, r].abs()).max() * abs(scale)))
    return out, mag, rss, top


def check(q, cache, ptable, plens, table, lengths, scale=None, got=None):
    D = q.shape[-1]
    if got is None:
        got = dsm.prefix_attention(q, cache, ptable, plens, table, lengths, scale=scale)
    want = reference(q, cache, ptable, plens, table, lengths, D ** -0.5 if scale is None else scale)
    ref.check_attention(got, want, max(1, int(lengths.max()) + int(plens.max())), D)
    return got


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("prefixes,lens,R,Hq,kv,D,page", [
    ([1], [1], 1, 1, 1, 128, 16),                     # one token each
    ([1], [0], 1, 1, 1, 64, 16),                      # the prefix alone
    ([0], [3], 1, 2, 1, 128, 16),                     # no prefix
    ([128], [5, 1], 1, 8, 2, 128, 16),
    ([127], [5, 1, 3], 2, 8, 8, 64, 32),
    ([129], [7] * 4, 1, 16, 2, 128, 64),
    ([1000], [100, 50, 25, 1], 1, 16, 2, 128, 16),    # 32 rows: one row tile
    ([700], [70, 30, 20, 8], 8, 16, 2, 128, 16),      # 256 rows: two
    ([300], [9] * 17, 3, 8, 1, 64, 128),              # 408 rows: four, the last of 24
    ([513], [11] * 13, 3, 8, 1, 128, 32),             # 312 rows: three, so a pair and one
    ([2000, 40, 0], [6, 3, 200, 0, 1, 70], 4, 6, 2, 64, 64),   # three prefixes, one of them empty
    ([65, 1, 640], [2, 1, 0, 5, 9, 3, 0, 0, 1], 5, 10, 2, 128, 16),   # rows before their own tokens
    ([0, 0], [0, 0, 0, 0], 2, 2, 2, 64, 64),          # nothing at all
    ([300], [40, -1, 0, -7], 2, 4, 2, 128, 16),       # sequences that are not there
    ([4000], [33], 1, 5, 1, 128, 64),
    ([5], [300, 700], 8, 16, 1, 128, 16),             # own tokens in the tcgen05 kernel's range
    ([150] * 9, [1 + 13 * i % 50 for i in range(36)], 2, 3, 3, 64, 16),
])
def test_prefix_attention_matches_64_bits(prefixes, lens, R, Hq, kv, D, page, q8):
    check(*problem(prefixes, lens, R, Hq, kv, D, page, q8, seed=sum(lens) + R + D,
                   strided=R % 2 == 0))


@pytest.mark.parametrize("MP", [1, 31, 127, 128, 129, 255, 256, 257, 384, 385, 600])
@pytest.mark.parametrize("D,q8", [(128, False), (64, True), (128, True), (64, False)])
def test_every_count_of_rows(MP, D, q8):
    # one new token of MP sequences, or of MP / 5 with five heads
    heads = 5 if MP % 5 == 0 else 1
    check(*problem([260], [1 + i % 3 for i in range(MP // heads)], 1, heads, 1, D, 32, q8, seed=MP))


@pytest.mark.parametrize("q8", [False, True])
def test_peaked_and_rising_scores(q8):
    # scores of hundreds, growing along the prefix: every row's reference moves again and again
    p = problem([900], [30, 9], 4, 8, 1, 128, 16, q8, seed=3, sigma=12.0)
    check(*p)
    q, cache, ptable = p[:3]
    t = torch.arange(900)
    slots = ptable[0].cpu().long()[t // 16] * 16 + t % 16
    rows = q[0, 3, 0].float().cpu()[None] * torch.linspace(0.01, 4, 900)[:, None] / 12
    page, off = (slots // 16).to(DEV), (slots % 16).to(DEV)
    if q8:
        codes, sc = ref.quantise(rows.to(torch.bfloat16)[:, None])
        cache.k[page, 0, off] = torch.from_numpy(codes[:, 0]).to(DEV)
        cache.k_scale[page, 0, off] = torch.from_numpy(sc[:, 0]).to(DEV)
    else:
        cache.k[page, 0, off] = rows.to(torch.bfloat16).to(DEV)
    check(*p)


def test_scale_argument():
    p = problem([100], [30, 4], 2, 4, 2, 64, 16, False, seed=5)
    for scale in (0.0, 1.0, -0.3):
        check(*p, scale=scale)


@pytest.mark.parametrize("exp", [20, 34, 68, -26, -68])
def test_scores_of_any_size(exp):
    # two sizes of score per row, far apart: the mean of the values at the larger one, met in the
    # prefix and among the own tokens alike
    prefixes, lens, D, page = [1000], [130, 5], 128, 16
    q, cache, ptable, plens, table, lengths = problem(prefixes, lens, 1, 4, 1, D, page, False, seed=7)
    sign = 1.0 if exp > 0 else -1.0
    q.zero_()
    q[..., 0] = 2.0 ** (abs(exp) // 2)
    mag = 2.0 ** (abs(exp) - abs(exp) // 2)
    k = ref.flat(cache.k)
    big = torch.arange(k.shape[0], device=DEV) % 5 == 2
    key = torch.where(big, mag, mag / 2) if sign > 0 else -torch.where(big, mag / 2, mag)
    k = torch.zeros_like(k)
    k[:, 0, 0] = key.to(torch.bfloat16)
    cache.k.copy_(k.view(-1, page, 1, D).transpose(1, 2))
    got = dsm.prefix_attention(q, cache, ptable, plens, table, lengths).cpu().double()
    v = ref.values(cache, "v")
    for b in range(2):
        _, a = slots_of(ptable[0].cpu(), 1000, page, cache.k.shape[0])
        _, o = slots_of(table[b].cpu(), lens[b], page, cache.k.shape[0])
        sl = torch.cat((a, o))
        seen = v[sl[big.cpu()[sl]], 0]
        # fp32 sums of at most 300 values, the weights exact; rounded once
        tol = ref.HALF_BF16 * seen.mean(0).abs() + 300 * 2 * ref.U32 * seen.abs().mean(0)
        assert bool(((got[b, 0] - seen.mean(0)).abs() <= tol).all())


@pytest.mark.parametrize("q8", [False, True])
def test_what_is_not_visible_does_not_matter(q8):
    # behind the prefixes, behind the lengths, and in other pages there are infinities and NaN
    page = 16
    q, cache, ptable, plens, table, lengths = problem([200, 131], [37, 6, 3, 64], 1, 8, 2, 128, page,
                                                      q8, seed=8, room=2)
    clean = dsm.prefix_attention(q, cache, ptable, plens, table, lengths)
    pages = cache.k.shape[0]
    seen = torch.zeros(pages * page, dtype=torch.bool)
    for t, n in ((ptable, plens), (table, lengths)):
        for row, m in zip(t.cpu(), n.tolist()):
            seen[slots_of(row, m, page, pages)[1]] = True
    hidden = (~seen).to(DEV).view(pages, 1, page)
    for bad in (float("inf"), -float("inf"), float("nan")):
        parts = {}
        for n in ("k", "v", "k_scale", "v_scale"):
            t = getattr(cache, n)
            if t is not None and not (q8 and not n.endswith("scale")):
                m = hidden if t.dim() == 3 else hidden[..., None]
                t = torch.where(m, torch.full_like(t, bad), t)
            parts[n] = t
        assert torch.equal(dsm.prefix_attention(q, dsm.PagedCache(**parts), ptable, plens, table,
                                                lengths), clean)


def test_what_is_visible_and_not_finite_shows():
    q, cache, ptable, plens, table, lengths = problem([200], [5, 9], 1, 4, 1, 128, 16, False, seed=9)
    cache.v[int(ptable[0, 2]), 0, 3, 70] = float("nan")
    got = dsm.prefix_attention(q, cache, ptable, plens, table, lengths).isnan()
    assert bool(got[..., 70].all()) and int(got.sum()) == got[..., 70].numel()


@pytest.mark.parametrize("q8", [False, True])
def test_scores_of_minus_infinity_weigh_nothing(q8):
    # (a Q8 key's scale of infinity makes them; the bf16 keys hold them)
    q, cache, ptable, plens, table, lengths = problem([150], [4, 0], 1, 4, 1, 64, 16, q8, seed=10)
    q[..., 0] = q[..., 0].abs() + 0.5
    for i, t in enumerate((0, 5, 149)):
        at = int(ptable[0, t // 16]), 0, t % 16
        if q8:
            cache.k[at] = 0
            cache.k[at][0] = -1
            cache.k_scale[at] = float("inf")
            q[..., 1:] = 0       # 0 x code keeps the sum at one infinity
        else:
            cache.k[at][0] = -float("inf")
    got = dsm.prefix_attention(q, cache, ptable, plens, table, lengths)
    if q8:
        keep = cache.k_scale.isfinite()
        cache.k_scale[~keep] = 1e30      # as far from weighing anything
    else:
        cache.k[cache.k.isinf()] = -1e30
    check(q, cache, ptable, plens, table, lengths, got=got)


def test_bad_pages_are_skipped():
    q, cache, ptable, plens, table, lengths = problem([500, 90], [40, 70, 8, 3], 2, 8, 2, 128, 16,
                                                      False, seed=11)
    ptable[0, 3] = -1
    ptable[0, 30] = cache.k.shape[0]
    ptable[0, 8:16] = 2 ** 31 - 1        # a whole tile
    ptable[1, 0] = -(2 ** 31)
    table[1, 2] = 10 ** 6
    check(q, cache, ptable, plens, table, lengths)


def test_lengths_beyond_the_tables_and_empty_ones():
    q, cache, ptable, plens, table, lengths = problem([100, 64], [20, 30, 5, 9], 1, 4, 2, 64, 32,
                                                      False, seed=12)
    want = dsm.prefix_attention(q, cache, ptable[:, :3].contiguous(),
                                torch.tensor([96, 64], dtype=torch.int32, device=DEV), table, lengths)
    plens[0] = 2 ** 31 - 1
    got = dsm.prefix_attention(q, cache, ptable[:, :3].contiguous(), plens, table, lengths)
    assert torch.equal(got, want)
    plens[:] = -5                         # no prefix: the sequences' own tokens
    got = dsm.prefix_attention(q, cache, ptable, plens, table, lengths)
    check(q, cache, ptable, plens, table, lengths, got=got)


@pytest.mark.parametrize("q8", [False, True])
def test_the_same_as_without_sharing(q8):
    # page-aligned prefixes can be written into each sequence's own table
    q, cache, ptable, plens, table, lengths = problem([256], [33, 70, 128], 6, 16, 2, 128, 64, q8,
                                                      seed=13)
    whole = torch.cat((ptable.expand(3, -1), table), 1).contiguous()
    got = dsm.prefix_attention(q, cache, ptable, plens, table, lengths)
    ref.check_attention(got, ref.attention(q, cache, whole, lengths + 256, 128 ** -0.5), 400, 128)


def test_workspace_contents_streams_and_repeats():
    p = problem([700, 300], [30, 9, 61, 5], 3, 8, 2, 128, 32, False, seed=14)
    first = dsm.prefix_attention(*p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(p[0])
    torch.cuda.synchronize()
    for _ in range(3):
        dsm.prefix_attention(*p, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, first) and dsm.workspace_status(ws, s) == 0
    with pytest.raises(dsm.DsmoeError):
        dsm.prefix_attention(*p, workspace=ws[:4096])


@pytest.mark.parametrize("prefixes,per,R,Hq,D", [(300, 1, 1, 2, 64), (40, 3, 2, 4, 128),
                                                 (3, 33, 1, 8, 128), (2, 40, 2, 16, 64)])
def test_workspace_of_exactly_the_size(prefixes, per, R, Hq, D):
    p = problem([1 + 37 * i % 150 for i in range(prefixes)], [3 + i % 5 for i in range(prefixes * per)],
                R, Hq, 2, D, 16, False, seed=21)
    q, cache, ptable, plens, table, lengths = p
    lib, args = dsm.N.load(), dsm._paged_args(q, cache, table, lengths, None, None, None)
    args = dsm.N.DsPrefixAttnArgs(args, prefixes, ptable.shape[1], ptable.data_ptr(), plens.data_ptr())
    need = lib.ds_prefix_attn_workspace_size(args)
    ws = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device=DEV)
    got = check(*p, got=dsm.prefix_attention(*p, workspace=ws[:need]))
    assert bool((ws[need:] == 0x5A).all())
    assert torch.equal(got, dsm.prefix_attention(*p))


def test_captured_replays_with_other_lengths():
    q, cache, ptable, plens, table, lengths = problem([600, 600], [50] * 6, 2, 8, 2, 128, 32, False,
                                                      seed=15)
    out, ws = torch.empty_like(q), torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    dsm.prefix_attention(q, cache, ptable, plens, table, lengths, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsm.prefix_attention(q, cache, ptable, plens, table, lengths, out=out, workspace=ws)
    for a, b in (([600, 1], [50, 1, 0, 7, -1, 30]), ([0, 384], [2, 50, 50, 50, 3, 3]), ([77, 600], [50] * 6)):
        plens.copy_(torch.tensor(a, dtype=torch.int32))
        lengths.copy_(torch.tensor(b, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dsm.prefix_attention(q, cache, ptable, plens, table, lengths))
        check(q, cache, ptable, plens, table, lengths, got=out)


def test_a_long_prefix_on_many_heads():
    # 512 x 8 rows against 64 bits on a few of the heads and sequences: work on every SM, units cut by
    # CTAs, and results that repeat
    q, cache, ptable, plens, table, lengths = problem([6000], [20] * 48, 2, 32, 8, 128, 64, False,
                                                      seed=16)
    got = dsm.prefix_attention(q, cache, ptable, plens, table, lengths)
    assert torch.equal(got, dsm.prefix_attention(q, cache, ptable, plens, table, lengths))
    pick = [0, 17, 47]
    check(q[pick].contiguous(), cache, ptable, plens, table[pick].contiguous(), lengths[pick],
          got=got[pick])


@pytest.mark.parametrize("q8", [False, True])
def test_pages_beyond_32_bits(q8):
    # the same pages far apart in a cache of more than 2^32 values (8 bits: scales behind 2^26 too)
    R, Hq, kv, D, page = 3, 16, 8, 128, 64
    q, cache, ptable, plens, table, lens = problem([700], [90, 5, 64, 0], R, Hq, kv, D, page, q8, seed=7)
    want = dsm.prefix_attention(q, cache, ptable, plens, table, lens)
    pages = (1 << 32) // (kv * page * D) + cache.k.shape[0]
    at = torch.tensor([i if i % 2 else pages - 1 - i for i in range(cache.k.shape[0])], device=DEV)
    far = []
    for name in ("k", "v") + (("k_scale", "v_scale") if q8 else ()):
        t = getattr(cache, name)
        big = torch.empty((pages, *t.shape[1:]), dtype=t.dtype, device=DEV)
        big[at] = t
        far.append(big)
    move = lambda t: torch.where(t >= 0, at[t.clamp(min=0).long()], -1).to(torch.int32)  # noqa: E731
    got = dsm.prefix_attention(q, dsm.PagedCache(*far), move(ptable), plens, move(table), lens)
    assert torch.equal(got, want)


def test_inputs_written_right_before_the_call():
    # kernels that write queries, cache, tables and lengths, and the call behind them without a pause,
    # eager and captured in turn on one workspace: each sees what was written last
    problems = [problem([640, 90], [40, 3, 17, 64], 2, 8, 2, 128, 32, False, seed=s) for s in range(4)]
    want = [dsm.prefix_attention(*p) for p in problems]
    q, cache, *rest = problem([640, 90], [40, 3, 17, 64], 2, 8, 2, 128, 32, False, seed=9)
    ws, out = torch.empty(64 << 20, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    into = [q, cache.k, cache.v, *rest]
    graph = torch.cuda.CUDAGraph()
    call = lambda: dsm.prefix_attention(q, cache, *rest, out=out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    got = []
    for i in range(40):
        p = problems[i * 7 % 4]
        for to, x in zip(into, (p[0], p[1].k, p[1].v, *p[2:])):
            to.copy_(x)
        graph.replay() if i % 3 else call()
        got.append(out.clone())
    for i, x in enumerate(got):
        assert torch.equal(x, want[i * 7 % 4]), i
    assert dsm.workspace_status(ws) == 0 and not ws[8:16].any()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("scale", [None, 0.5, 1.0, 2.5, -1.0, 0.0])
def test_what_is_no_number_among_queries_and_keys_shows(scale, q8):
    # a row with a query that is NaN, and rows all of whose prefix's scores are, at scales on both sides of
    # where the smallest fp32 value times the factor is infinite
    def make():
        return problem([200, 150], [5, 9, 3, 4], 2, 4, 2, 128, 16, q8, seed=9)
    q, *rest = make()
    clean = dsm.prefix_attention(q, *rest, scale=scale)
    q[1, 0, 2, 17] = float("nan")
    got = dsm.prefix_attention(q, *rest, scale=scale)
    assert bool(got[1, 0, 2].isnan().all())
    got[1, 0, 2] = clean[1, 0, 2]
    assert torch.equal(got, clean)
    q, cache, ptable, *rest = make()
    for page in ptable[1, :10].tolist():
        (cache.k_scale if q8 else cache.k)[page, 1] = float("nan")     # one key head
    got = dsm.prefix_attention(q, cache, ptable, *rest, scale=scale)
    assert bool(got[2:, :, 2:].isnan().all())
    assert torch.equal(got[:2], clean[:2]) and torch.equal(got[2:, :, :2], clean[2:, :, :2])
