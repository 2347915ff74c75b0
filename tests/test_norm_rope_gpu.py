"""Norms of queries and keys per head with the position rotation (ds_qk_norm_rope), and the
paged cache's writes and reads (ds_cache_write, ds_cache_read, ds_qk_norm_rope_write), against
plain implementations in 64 bits.

Tolerances, with u = 2^-24: the norm's sum of D squares is a chain of 8 and a tree of 4 (12 u
of the sum, 6 u of its root), the reciprocal root is good to 2 steps (4 u), three products
3 u; the angle is off by 2^-32 turns and half a step of fp32 (together below 4 u), sine and
cosine by 2 steps (4 u), and the rotation rounds twice: below 32 u = 2^-19 of |u| + |v|, the
two values a result is made from. Then half a step of bf16 of the result. What is copied or
quantised from bf16 is compared bit for bit."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import q4_moe_speculative_gb300 as dsm

pytestmark = pytest.mark.gpu

DEV = "cuda"


def tokens_of_a_projection(T, Hq, Hkv, D, seed, sigma=1.0):
    qkv = ref.normal(T, Hq + 2 * Hkv, D, seed=seed, sigma=sigma)
    return (qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]), qkv.to(DEV)


def on_device(qkv, Hq, Hkv):
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


def weights(D, seed):
    return tuple((1 + 0.2 * ref.normal(D, seed=seed + i).float()).to(torch.bfloat16)
                 for i in range(2))


def check_rows(got, x, w, pos, f, eps, inter):
    want, both = ref.norm_rope(x, w, pos, f, eps, inter)
    err = (got.cpu().double() - want).abs()
    tol = ref.HALF_BF16 * want.abs() + 2.0 ** -19 * both * (1 + ref.HALF_BF16)
    assert bool((err <= tol + 1e-38).all()), float((err - tol).max())


CASES = [
    # T, Hq, Hkv, D, rotary, interleaved, normed (q, k), first position
    (1, 1, 1, 128, 128, False, (True, True), 0),
    (6, 16, 1, 128, 128, False, (True, True), 299_994),
    (6, 16, 1, 128, 128, True, (True, False), 7),
    (5, 3, 2, 64, 64, False, (True, True), 1_000_003),
    (7, 5, 1, 64, 32, True, (False, True), 123),
    (33, 8, 4, 128, 64, False, (True, True), 2**31 - 40),
    (129, 7, 7, 128, 16, False, (False, False), -60),
    (131, 40, 8, 64, 16, True, (True, True), -(2**31)),
    (1025, 32, 8, 128, 96, False, (True, True), 50_000),
    (4099, 12, 3, 128, 0, False, (True, True), 0),
    (2500, 20, 4, 64, 48, True, (True, True), 90_000),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,normed,first", CASES)
def test_rows_match_64_bits(T, Hq, Hkv, D, rot, inter, normed, first):
    (q, k, _), qkv = tokens_of_a_projection(T, Hq, Hkv, D, seed=T + Hq)
    dq, dk, _ = on_device(qkv, Hq, Hkv)
    qw, kw = (w if on else None for w, on in zip(weights(D, seed=9), normed))
    pos = torch.arange(T, dtype=torch.int64) + first
    pos = pos.to(torch.int32)
    f, steps = ref.turn_steps(rot)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo, ko = dsm.qk_norm_rope(dq, dk, dev(pos), dev(steps), q_weight=dev(qw), k_weight=dev(kw),
                              eps=1e-5, interleaved=inter)
    check_rows(qo, q, qw, pos, f, 1e-5, inter)
    check_rows(ko, k, kw, pos, f, 1e-5, inter)
    assert torch.equal(qkv.cpu()[:, :Hq], q)     # the inputs stay


def test_frequencies_helper_gives_the_steps():
    for rot in (16, 64, 128):
        f, steps = ref.turn_steps(rot)
        assert torch.equal(dsm.rope_frequencies(rot).cpu(), steps)
        assert torch.equal(dsm.rope_frequencies(inv_freq=f).cpu(), steps)


def test_whole_turns_rotate_by_nothing():
    # a frequency of a quarter turn: every fourth position gives the values back exactly
    T, D = 9, 64
    x = ref.normal(T, 1, D, seed=4).to(DEV)
    f = torch.full((D // 2,), np.pi / 2, dtype=torch.float64)
    steps = torch.full((D // 2,), 1 << 62, dtype=torch.int64, device=DEV)
    assert torch.equal(dsm.rope_frequencies(inv_freq=f), steps)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 4
    q, k = dsm.qk_norm_rope(x, x, pos, steps)
    assert torch.equal(q, x) and torch.equal(k, x)
    q, _ = dsm.qk_norm_rope(x, x, pos + 1, steps)     # (u, v) -> (-v, u)
    assert torch.equal(q[..., :32], -x[..., 32:]) and torch.equal(q[..., 32:], x[..., :32])


def test_in_place_and_no_rotation_copy():
    x = ref.normal(70, 6, 128, seed=1).to(DEV)
    q, k = x.clone(), x[:, :2].contiguous()
    k0 = k.clone()
    pos = torch.arange(70, dtype=torch.int32, device=DEV)
    steps = dsm.rope_frequencies(128)
    want = dsm.qk_norm_rope(q, k, pos, steps)
    got = dsm.qk_norm_rope(q, k, pos, steps, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    same = dsm.qk_norm_rope(x, k0, None, None)        # neither norm nor rotation
    assert torch.equal(same[0], x) and torch.equal(same[1], k0)


def test_zero_rows_and_large_values():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    x[1] = 2.0 ** 60                                   # its square's sum is below 2^127
    x[2, 0, 5] = 2.0 ** -60                            # far below eps
    w = torch.ones(64, dtype=torch.bfloat16)
    q, _ = dsm.qk_norm_rope(x.to(DEV), x.to(DEV), None, None, q_weight=w.to(DEV), eps=1e-6)
    q = q.cpu()
    assert bool((q[0] == 0).all()) and bool((q[1] == 1).all())
    assert float(q[2, 0, 5]) == pytest.approx(2.0 ** -60 * 1e3, rel=2.0 ** -8)


def test_no_tokens():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    qo, ko = dsm.qk_norm_rope(q, k, none, dsm.rope_frequencies(64))
    assert qo.shape == q.shape and ko.shape == k.shape
    cache = dsm.PagedCache.zeros(2, 2, 16, 64, q8=True)
    dsm.cache_write(cache, k, k, none)
    assert dsm.cache_read(cache, none)[0].shape == (0, 2, 64)
    dsm.qk_norm_rope_write(q, k, k, none, dsm.rope_frequencies(64), cache, none)
    assert int(cache.k.count_nonzero()) == 0


# ------------------------------------------------------------------------------ the cache
def filled_cache(pages, kv, page, D, q8, strided, seed):
    """A cache whose every byte is set; strided: keys and values side by side in one pool."""
    g = torch.Generator()
    g.manual_seed(seed)
    if q8:
        pool = torch.randint(-127, 128, (pages, 2, kv, page, D), generator=g, dtype=torch.int8)
    else:
        pool = torch.randn((pages, 2, kv, page, D), generator=g).to(torch.bfloat16)
    pool = pool.to(DEV)
    k, v = (pool[:, 0], pool[:, 1]) if strided else (pool[:, 0].contiguous(),
                                                     pool[:, 1].contiguous())
    if not q8:
        return dsm.PagedCache(k, v)
    sc = (torch.rand((pages, 2, kv, page), generator=g) + 0.1).to(DEV)
    ks, vs = (sc[:, 0], sc[:, 1]) if strided else (sc[:, 0].contiguous(), sc[:, 1].contiguous())
    return dsm.PagedCache(k, v, ks, vs)


def snapshot(cache):
    return {n: getattr(cache, n).cpu().clone() for n in ("k", "v", "k_scale", "v_scale")
            if getattr(cache, n) is not None}


def slots_for(T, pages, page, seed, skipped=()):
    g = torch.Generator()
    g.manual_seed(seed)
    s = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    for i, bad in skipped:
        s[i] = bad
    return s


BAD = [-1, -(2**31), 2**31 - 1]


@pytest.mark.parametrize("T,kv,D,page,q8,strided", [
    (1, 1, 128, 16, False, False), (1, 1, 64, 16, True, False), (48, 4, 128, 32, False, True),
    (50, 3, 64, 128, True, True), (333, 8, 128, 64, True, False), (2049, 2, 128, 16, True, True),
    (1111, 5, 64, 32, False, False), (300, 1, 64, 64, True, False)])
def test_write_and_read_are_exact(T, kv, D, page, q8, strided):
    pages = T // page + 3
    cache = filled_cache(pages, kv, page, D, q8, strided, seed=T)
    before = snapshot(cache)
    (k, _, v), qkv = tokens_of_a_projection(T, kv, kv, D, seed=T + 1, sigma=3.0)
    if T > 4:
        k[2] = 0                                       # a row of zeros
        k[3, 0, 7] = float("inf")
        v[4, kv - 1, 1] = float("nan")
        qkv.copy_(torch.cat([k, qkv[:, kv:2 * kv].cpu(), v], 1))
    skip = list(zip(range(5, 8), BAD)) if T > 10 else []
    slots = slots_for(T, pages, page, seed=T + 2, skipped=skip)
    if T > 10:
        slots[8] = pages * page                        # one behind the last slot
    dsm.cache_write(cache, qkv[:, :kv], qkv[:, 2 * kv:], slots.to(DEV))
    after = snapshot(cache)
    kept = (slots >= 0) & (slots < pages * page)
    for side, x in (("k", k), ("v", v)):
        want = ref.flat(before[side]).clone()
        at = slots[kept].long()
        if q8:
            codes, scale = ref.quantise(x)
            want_s = ref.flat(before[side + "_scale"]).clone()
            want[at] = torch.from_numpy(codes)[kept]
            want_s[at] = torch.from_numpy(scale)[kept]
            got_s = ref.flat(after[side + "_scale"])
            assert torch.equal(torch.nan_to_num(got_s, -7), torch.nan_to_num(want_s, -7))
            assert torch.equal(got_s.isnan(), want_s.isnan())
            assert torch.equal(ref.flat(after[side]), want)
        else:
            want[at] = x[kept]
            got = ref.flat(after[side])
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(want, 9.0))
    # reading back, any order, repeats and slots outside
    ask = torch.cat([slots, slots.flip(0), torch.tensor(BAD + [pages * page], dtype=torch.int32)])
    outs = dsm.cache_read(cache, ask.to(DEV))
    inside = (ask >= 0) & (ask < pages * page)
    for side, got in zip(("k", "v"), outs):
        x = ref.flat(after[side])[ask.clamp(0, pages * page - 1).long()]
        if q8:
            sc = ref.flat(after[side + "_scale"])[ask.clamp(0, pages * page - 1).long()]
            x = (x.float() * sc[..., None]).to(torch.bfloat16)
        x[~inside] = 0
        got = got.cpu()
        assert torch.equal(got.isnan(), x.isnan())
        assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(x, 9.0))


def test_quantising_keeps_ties_and_extremes():
    # x / a of a half, a quarter ...: 63.5 and other ties go to even; and rows near both ends
    # of bf16's range
    rows = torch.zeros(8, 1, 64)
    rows[0, 0, :6] = torch.tensor([1.0, 0.5, -0.5, 0.25, 1.5 / 127, 0.0])
    rows[1, 0, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])
    rows[2, 0, :4] = torch.tensor([3.3e38, -1.0e38, 1.7e38, 1.0])
    rows[3, 0, :4] = torch.tensor([9.0e-41, 4.6e-41, -9.0e-41, 1e-41])
    rows[4, 0, :3] = torch.tensor([-254.0, 1.0, 3.0])
    rows[5] = torch.linspace(-3, 3, 64)
    rows[6, 0, 3] = -2.0 ** -126
    rows = rows.to(torch.bfloat16)
    cache = dsm.PagedCache.zeros(1, 1, 16, 64, q8=True)
    slots = torch.arange(8, dtype=torch.int32, device=DEV)
    dsm.cache_write(cache, rows.to(DEV), rows.to(DEV), slots)
    codes, scale = ref.quantise(rows)
    for side in ("k", "v"):
        assert np.array_equal(ref.flat(getattr(cache, side)).cpu().numpy()[:8], codes)
        assert np.array_equal(ref.flat(getattr(cache, side + "_scale")).cpu().numpy()[:8], scale)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,normed,first", CASES)
@pytest.mark.parametrize("q8", [False, True])
def test_fused_write(T, Hq, Hkv, D, rot, inter, normed, first, q8):
    page = 32
    pages = T // page + 2
    cache = filled_cache(pages, Hkv, page, D, q8, T % 2 == 1, seed=T)
    before = snapshot(cache)
    (q, k, v), qkv = tokens_of_a_projection(T, Hq, Hkv, D, seed=T + Hq)
    dq, dk, dv = on_device(qkv, Hq, Hkv)
    qw, kw = (w if on else None for w, on in zip(weights(D, seed=9), normed))
    pos = (torch.arange(T, dtype=torch.int64) + first).to(torch.int32)
    f, steps = ref.turn_steps(rot)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    slots = slots_for(T, pages, page, seed=5, skipped=[(T // 2, -1)] if T > 2 else [])
    args = dict(q_weight=dev(qw), k_weight=dev(kw), eps=1e-5, interleaved=inter)
    qo = dsm.qk_norm_rope_write(dq, dk, dv, dev(pos), dev(steps), cache, dev(slots), **args)
    q2, k2 = dsm.qk_norm_rope(dq, dk, dev(pos), dev(steps), **args)
    assert torch.equal(qo, q2)
    kept, after = slots >= 0, snapshot(cache)
    at = slots[kept].long()
    others = torch.ones(pages * page, dtype=torch.bool)
    others[at] = False
    for n in after:
        assert torch.equal(ref.flat(after[n])[others], ref.flat(before[n])[others]), n
    if not q8:
        assert torch.equal(ref.flat(after["k"])[at], k2.cpu()[kept])
        assert torch.equal(ref.flat(after["v"])[at], v[kept])
        return
    codes, scale = ref.quantise(v)
    assert torch.equal(ref.flat(after["v"])[at], torch.from_numpy(codes)[kept])
    assert torch.equal(ref.flat(after["v_scale"])[at], torch.from_numpy(scale)[kept])
    # keys: half a code step, and the row's own error (its largest value is off as well)
    want, both = ref.norm_rope(k, kw, pos, f, 1e-5, inter)
    want, both = want[kept], both[kept]
    sc = ref.flat(after["k_scale"]).double()[at][..., None]
    off = 2.0 ** -19 * both.amax(-1, keepdim=True)
    top = want.abs().amax(-1, keepdim=True) / 127
    assert bool(((sc - top).abs() <= off / 127 + 2 * ref.U32 * top).all())
    err = (ref.flat(after["k"]).double()[at] * sc - want).abs()
    assert bool((err <= sc * (0.5 + 2.0 ** -15) + 2 * off).all()), float((err / sc).max())
