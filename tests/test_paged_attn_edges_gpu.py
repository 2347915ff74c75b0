"""Attention over the paged cache (ds_paged_attention) where its kernels take their rare paths:
scores of any finite size, weights in two parts, new tokens that only some rows see, and scores
of -infinity. `wide` tables (test_paged_attn_gpu.py) take the tensor-memory kernel, and so do
more than 24 or 32 rows whose tables have room for 39,000 tokens times key heads or more."""
import pytest
import torch

import paged_ref as ref
import q4_moe_speculative_gb300 as dsm
from test_paged_attn_gpu import problem

pytestmark = pytest.mark.gpu

DEV = "cuda"


def slots_of(table, page, b, n):
    t = torch.arange(n)
    return table[b].cpu().long()[t // page] * page + t % page


def put(cache, side, slots, rows, scales=None):
    """rows [tokens, kv, D] (bf16, or int8 with scales [tokens, kv]) at slots of the cache."""
    page = cache.k.shape[2]
    p, off = (slots // page).to(DEV), (slots % page).to(DEV)
    getattr(cache, side)[p, :, off] = rows.to(DEV)
    if scales is not None:
        getattr(cache, side + "_scale")[p, :, off] = scales.to(DEV)


# every kernel: up to 32 rows, more, and the tensor-memory one with each number of columns
KERNELS = [(1, False), (7, False), (20, False), (32, False), (40, False), (72, False), (128, False),
           (28, True), (48, True), (80, True), (128, True)]


# ------------------------------------------------------------------------ scores of any size
@pytest.mark.parametrize("M,wide", KERNELS)
@pytest.mark.parametrize("D,scale", [(64, 64 ** -0.5), (128, 0.7)])
@pytest.mark.parametrize("q8", [False, True])
def test_scores_of_any_size(q8, D, scale, M, wide):
    # All scores are one of two values per row, far apart, so the result is the mean of the
    # values at the larger one: that of n additions in fp32, rounded. The larger one is met
    # again and again along the length, and in the first tiles of some sequences not at all.
    # (8 heads of 4 sequences: several tiles on every CTA, and the kernel meant: see `wide`.)
    lens, page, kv = [1100, 1000, 700, 130], 128, 8
    if wide or M <= 24:
        lens = [5000, 4000, 900, 130]
    q, cache, table, lengths = problem(lens, 1, M * kv, kv, D, page, q8, seed=M + D, wide=wide)
    if q8:
        cache.v_scale.fill_(2.0 ** -7)
    v = ref.flat(cache.v).double()
    if q8:
        v = v * ref.flat(cache.v_scale).double()[..., None]
    for exp, more in ((20, 1.5), (26, 1.25), (34, 1.5), (68, 1.0), (112, 1.75),
                      (-20, 1.75), (-26, 1.5), (-34, 1.25), (-68, 1.5), (-112, 1.0)):
        sign = 1.0 if exp > 0 else -1.0
        q.zero_()
        q[..., 0] = 2.0 ** (abs(exp) // 2) * more
        q[:, :, ::3, 0] *= 4.0
        want = torch.zeros(len(lens), 1, M * kv, D, dtype=torch.float64)
        size = torch.zeros_like(want)
        for b, n in enumerate(lens):
            slots = slots_of(table, page, b, n)
            big = torch.arange(n) % 5 == 2
            if b < 2:
                big &= torch.arange(n) > n * 3 // 8
            # (the larger score is the one nearer to 0 where the scores are negative)
            mag = 2.0 ** (abs(exp) - abs(exp) // 2)
            key = torch.where(big, mag, mag / 2) if sign > 0 else -torch.where(big, mag / 2, mag)
            rows = torch.zeros(n, kv, D)
            if q8:
                rows[..., 0] = 64 * sign
                put(cache, "k", slots, rows.to(torch.int8),
                    (key / (64 * sign))[:, None].expand(n, kv))
            else:
                rows[..., 0] = key[:, None]
                put(cache, "k", slots, rows.to(torch.bfloat16))
            seen = v[slots[big].to(DEV)].cpu()
            want[b, 0] = seen.mean(0).repeat_interleave(M, 0)
            size[b, 0] = seen.abs().mean(0).repeat_interleave(M, 0)
        got = dsm.paged_attention(q, cache, table, lengths, scale=scale).cpu().double()
        err = (got - want).abs()
        tol = ref.HALF_BF16 * want.abs() + size * (2.0 ** -16 + max(lens) * 2 * ref.U32)
        assert bool((err <= tol).all()), (exp, float((err - tol).max()))


# -------------------------------------------------------------------------- weights in two parts
@pytest.mark.parametrize("M,wide", KERNELS + [(33, False), (64, False), (96, False), (64, True),
                                              (65, True), (96, True), (97, True)])
@pytest.mark.parametrize("D,q8", [(128, False), (64, True), (128, True), (64, False)])
def test_weights_have_two_parts(D, q8, M, wide):
    # Values chosen so that everything cancels at a weight of 0.75 + 2^-9, which lies half way
    # between two bf16 values: what is left of a result is 2^-9 of sum p |v| or less, and its
    # own rounding to bf16 is 2^-17 of it, so an error of the weight shows. A weight in two
    # bf16 parts is off by (2^-8)^2 relative; the score by fp32 (magnitudes below 1).
    n, page = 300, 16
    q, cache, table, lengths = problem([n, n], 1, M, 1, D, page, q8, seed=M, wide=wide)
    g = torch.Generator()
    g.manual_seed(M + D)
    weights = torch.tensor([0.75 + 2.0 ** -9, 0.75, 0.75 - 3 * 2.0 ** -10], dtype=torch.float64)
    pick = torch.randint(0, 3, (2, M), generator=g)
    # a query of two values whose sum reaches the wanted score closely: log(w) = q . (1, 1)
    s = torch.log(weights)[pick]
    hi = s.float().to(torch.bfloat16)
    q.zero_()
    q[:, 0, :, 0] = hi.to(DEV)
    q[:, 0, :, 1] = (s - hi.double()).float().to(torch.bfloat16).to(DEV)
    kind = torch.randint(0, 4, (n,), generator=g)          # 0, 1: weight w; 2: 1; 3: 1, the rest
    count = [int((kind <= 1).sum()), int((kind == 2).sum()), int((kind == 3).sum())]
    w0 = float(weights[0])
    keys = torch.zeros(n, 1, D)
    keys[kind <= 1, 0, :2] = 1.0
    vb = torch.rand(D, generator=g, dtype=torch.float64) + 0.5
    if q8:
        unit = [2.0 ** -6, 2.0 ** -5, 2.0 ** -12]
        code = torch.round(vb / unit[0])
        vb = code * unit[0]
        ca = torch.round(-count[0] * w0 * vb / count[1] / unit[1])
        va = ca * unit[1]
        cc = torch.round(-(count[0] * w0 * vb + count[1] * va) / count[2] / unit[2]).clamp(-127, 127)
        codes = torch.stack((code, ca, cc))
        assert float(codes.abs().max()) <= 127
        idx = (kind - 1).clamp(min=0)
        vals, scales = codes[idx][:, None], torch.tensor(unit, dtype=torch.float64)[idx][:, None]
    else:
        vb = vb.to(torch.bfloat16).double()
        va = (-count[0] * w0 * vb / count[1]).to(torch.bfloat16).double()
        vc = (-(count[0] * w0 * vb + count[1] * va) / count[2]).to(torch.bfloat16).double()
        vals, scales = torch.stack((vb, va, vc))[(kind - 1).clamp(min=0)][:, None], None
    for b in range(2):
        slots = slots_of(table, page, b, n)
        if q8:
            put(cache, "k", slots, keys.to(torch.int8), torch.ones(n, 1))
            put(cache, "v", slots, vals.to(torch.int8), scales.float())
        else:
            put(cache, "k", slots, keys.to(torch.bfloat16))
            put(cache, "v", slots, vals.to(torch.bfloat16))
    got = dsm.paged_attention(q, cache, table, lengths, scale=1.0).cpu().double()
    want, mag, _, top = ref.attention(q, cache, table, lengths, 1.0)
    assert float((want.abs() / mag).max()) < 2.0 ** -7
    tol = ref.HALF_BF16 * want.abs() + mag * (2.0 ** -16 + 2 * (top * 8 * ref.U32 + 2.0 ** -21) +
                                              n * 2 * ref.U32)
    err = (got - want).abs()
    assert bool((err <= tol).all()), float((err / mag).max())


# ------------------------------------------------------------ new tokens that only some rows see
def attention64(q, cache, table, lengths, scale):
    """What paged_ref.attention gives without its third part, in fp64 on the device."""
    B, R, H, D = q.shape
    kv, page = cache.k.shape[1:3]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    mag, top = torch.zeros_like(out), 0.0
    for b in range(B):
        n = int(lengths[b])
        slots = slots_of(table, page, b, n).to(DEV)
        k, v = (ref.flat(getattr(cache, s))[slots].double() for s in ("k", "v"))
        if cache.q8:
            k = k * ref.flat(cache.k_scale)[slots].double()[..., None]
            v = v * ref.flat(cache.v_scale)[slots].double()[..., None]
        for r in range(R):
            see = n - (R - 1 - r)
            if see <= 0:
                continue
            x = q[b, r].double().view(kv, H // kv, D)
            p = torch.softmax(torch.einsum("hgd,thd->hgt", x, k[:see]) * scale, -1)
            out[b, r] = torch.einsum("hgt,thd->hgd", p, v[:see]).reshape(H, D)
            mag[b, r] = torch.einsum("hgt,thd->hgd", p, v[:see].abs()).reshape(H, D)
            top = max(top, float(torch.einsum("hgd,thd->hgt", x.abs(), k[:see].abs()).max() * scale))
    return out, mag, top


def tolerance(out, mag, top, n, D):
    """Per element, as in paged_ref.check_attention, with weights of two bf16 parts: 2^-16. (A
    weight below 2^-126 of the largest may be taken as 0: n of them times values below 2^12 are
    far below 1e-30.)"""
    score = top * (D + 4) * 2 * ref.U32 + 2.0 ** -21
    return ref.HALF_BF16 * out.abs() + mag * (2.0 ** -16 + 2 * score + n * 2 * ref.U32) + 1e-30


@pytest.mark.parametrize("R,G,wide", [(8, 1, False), (4, 5, False), (8, 3, False), (5, 8, False),
                                      (8, 16, False), (7, 4, True), (5, 8, True), (5, 16, True),
                                      (8, 16, True)])
@pytest.mark.parametrize("D,q8", [(128, False), (64, False), (128, True), (64, True)])
@pytest.mark.parametrize("rising", [False, True])
def test_new_tokens_that_some_rows_see(R, G, wide, D, q8, rising):
    # One new token holds NaN in its keys, or infinities in a few of its values: rows before it
    # are those of the clean cache, rows from it on are NaN, or infinite in those values and
    # right in the others. Lengths put the new tokens on both sides of a tile's border (16, 64
    # and 128 tokens); 8 heads of these sequences give every CTA several tiles. rising: the last
    # tokens have scores that move every row's reference.
    kv, page = 8, 64
    lens = [5 * 128 + 1, 6 * 128 + 3, 8 * 128 + 5, R - 1]
    if wide or R * G <= 24:
        lens = [5 * 128 + 1, 6 * 128 + 3, 16 * 128 + 5, 17 * 128 + 2, 5000, R - 1]
    q, cache, table, lengths = problem(lens, R, G * kv, kv, D, page, q8, seed=R * G + D, wide=wide)
    if rising:
        q[..., 0] = q[..., 0].abs() + 1
        for b, n in enumerate(lens[:-1]):
            slots = slots_of(table, page, b, n)[-7:]
            p, off = (slots // page).to(DEV), (slots % page).to(DEV)
            step = torch.arange(1, 8, device=DEV)[:, None]
            if q8:   # (the scale of the row's other codes as well)
                cache.k[p, :, off, 0] = 127
                cache.k_scale[p, :, off] = 0.02 * step * (8 if D == 128 else 6)
            else:
                cache.k[p, :, off, 0] = (20 * step).to(torch.bfloat16).expand(7, kv)
    clean, mag, top = attention64(q, cache, table, lengths, D ** -0.5)
    tol = tolerance(clean, mag, top, max(lens), D)
    got = dsm.paged_attention(q, cache, table, lengths).double()
    assert bool(((got - clean).abs() <= tol).all()), float(((got - clean).abs() - tol).max())
    bad_dims = [3, D // 2 + 1, D - 1]
    fine_dims = [d for d in range(D) if d not in bad_dims]
    for u in sorted({0, (R - 1) // 2, R - 2}):            # seen by the rows after row u
        for side, what in (("k", float("nan")), ("v", float("inf")), ("v", -float("inf"))):
            if q8 and what == -float("inf"):
                continue
            dirty = dsm.PagedCache(*(None if t is None else t.clone() for t in (
                cache.k, cache.v, cache.k_scale, cache.v_scale)))
            for b, n in enumerate(lens):
                t = n - (R - 1) + u
                slot = int(slots_of(table, page, b, n)[t])
                at = getattr(dirty, side + "_scale" if q8 else side)
                if q8 or side == "k":
                    at[slot // page, :, slot % page] = what
                else:
                    at[slot // page, :, slot % page, bad_dims] = what
            out = dsm.paged_attention(q, dirty, table, lengths).double()
            blind, sees = list(range(u + 1)), list(range(u + 1, R))
            fine = (out - clean).abs() <= tol
            assert bool(fine[:, blind].all()), (u, side, what)
            if q8 or side == "k":
                assert not bool(torch.isfinite(out[:, sees]).any()), (u, side)
                continue
            assert bool((out[:, sees][..., bad_dims] == what).all()), (u, side, what)
            assert bool(fine[:, sees][..., fine_dims].all()), (u, side, what)


# ------------------------------------------------------------------------- scores of -infinity
@pytest.mark.parametrize("M,wide", KERNELS)
@pytest.mark.parametrize("q8", [False, True])
def test_scores_of_minus_infinity_weigh_nothing(q8, M, wide):
    # tokens whose score overflows to -infinity, among them all of the first tiles of one
    # sequence and all tokens of another
    lens, page, D = [400, 150, 90], 16, 128
    q, cache, table, lengths = problem(lens, 1, M, 1, D, page, q8, seed=M, wide=wide)
    q[..., 0] = 2.0 ** 20
    gone = [torch.arange(lens[0]) < 260, torch.arange(lens[1]) % 3 > 0, torch.ones(lens[2], dtype=torch.bool)]
    for b, n in enumerate(lens):
        slots = slots_of(table, page, b, n)
        low = slots[gone[b]]
        p, off = (slots // page).to(DEV), (slots % page).to(DEV)
        cache.k[p, :, off, 0] = 0
        p, off = (low // page).to(DEV), (low % page).to(DEV)
        if q8:
            cache.k[p, :, off] = 0
            cache.k[p, :, off, 0] = -127
            cache.k_scale[p, :, off] = 2.0 ** 120
        else:
            cache.k[p, :, off, 0] = -2.0 ** 126
    got = dsm.paged_attention(q, cache, table, lengths)
    assert bool((got[2] == 0).all())
    kept = [torch.nonzero(~g).flatten() for g in gone[:2]]
    # the same tokens without them
    for b in range(2):
        slots = slots_of(table, page, b, lens[b])[kept[b]]
        k, v = (ref.values(cache, s)[slots, 0] for s in ("k", "v"))
        s = q[b, 0].cpu().double() @ k.t() * D ** -0.5
        p = torch.softmax(s, -1)
        mag = p @ v.abs()
        # (the dimension of 2^20 adds nothing to a score: its keys are 0)
        x = q[b, 0].cpu().double().clone()
        x[:, 0] = 0
        top = float((x.abs() @ k.abs().t()).max() * D ** -0.5)
        tol = tolerance(p @ v, mag, top, lens[b], D)
        assert bool(((got[b, 0].cpu().double() - p @ v).abs() <= tol).all()), b


# ---------------------------------------------------------------------- large and small values
@pytest.mark.parametrize("M,wide", KERNELS)
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("exp", [92, -96])
def test_large_and_small_values(exp, q8, M, wide):
    # a power of two in front of the values (below 8 times it) is one in front of the results
    lens, page, D = [1500, 130], 64, 64
    q, cache, table, lengths = problem(lens, 1, M, 1, D, page, q8, seed=M, wide=wide)
    want = dsm.paged_attention(q, cache, table, lengths)
    if q8:
        cache.v_scale *= 2.0 ** exp
    else:
        cache.v *= 2.0 ** exp
    got = dsm.paged_attention(q, cache, table, lengths)
    assert bool(torch.isfinite(got).all())
    assert torch.equal(got.float(), want.float() * 2.0 ** exp)


# ------------------------------------------------------------------------------------ refusals
def test_arguments_that_are_refused():
    q, cache, table, lengths = problem([40], 1, 2, 1, 64, 16, False, seed=1)
    for bad in (5, [1], "ws"):
        with pytest.raises(TypeError):
            dsm.paged_attention(q, cache, table, lengths, workspace=bad)
    none = dsm.PagedCache.zeros(2, 1, 16, 0)               # no head_dim
    with pytest.raises(dsm.DsmoeError) as e:
        dsm.paged_attention(q[..., :0].contiguous(), none, table, lengths)
    assert e.value.status == 1


def test_sizes_beyond_32_bits_are_refused():
    # (what 32 bits keep of these sizes would be a call that is allowed)
    q, cache, table, lengths = problem([40], 1, 2, 1, 64, 16, False, seed=2)
    wide = torch.empty((1, 2 ** 32 + 4), dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    with pytest.raises(dsm.DsmoeError) as e:
        dsm.paged_attention(q, cache, wide, lengths)
    assert e.value.status == 1
    del wide
    tiles = torch.empty((1, 2 ** 26 + 1, 576), dtype=torch.uint8, device=DEV)
    x = torch.empty((1, 2 ** 32 + 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(dsm.DsmoeError) as e:
        dsm.q4_project(tiles, x)
    assert e.value.status == 1
    del tiles, x
    torch.cuda.empty_cache()
