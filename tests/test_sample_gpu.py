"""Drawing tokens (ds_sample) against its definition in 64 bits, row by row on the CPU. Decisions
are compared exactly; a border or draw within 2^-30 of the mass of a 64-bit evaluation's (the
header's rounding of weights is below 2^-34 of it at these sizes) is left out, and hardly any is."""
import math

import numpy as np
import pytest
import torch

import q4_moe_speculative_gb300 as dsm

pytestmark = pytest.mark.gpu

DEV = "cuda"
CLOSE = 2.0 ** -30


def reference(l, u, T, k, p, mp):
    """(token, its probability, whether any decision is clear) of one row, l as float64."""
    l = np.where(np.isnan(l), -np.inf, l)
    top = l.max()
    if top == -np.inf:
        return -1, 0.0, True
    if not T > 2.0 ** -64:
        return int(np.argmax(l)), 1.0, True
    with np.errstate(invalid="ignore", over="ignore"):
        near = np.where(l == top, 0.0, l - top)
        w = np.exp(near / T)
    order = np.argsort(-l, kind="stable")
    if k > 0:
        order = order[:k]
    clear = True
    # weights of 0 and 1 are exact in both, and so are their sums and (24 bits by 24) the top-p border
    exact = bool(((w == 0) | (w == 1)).all())
    p = 1.0 if math.isnan(p) else p
    if p < 1:
        mass = w[order]
        upto = np.cumsum(mass)
        before = upto - mass
        gap = np.abs(before[1:] - p * upto[-1])
        clear &= exact or len(gap) == 0 or gap.min() > CLOSE * upto[-1]
        order = order[:max(1, int((before < p * upto[-1]).sum()))]
    if mp > 0:
        cut = min(0.0, T * math.log(mp))
        off = near[order]
        clear &= bool((np.abs(off - cut)[off < 0] > 2.0 ** -40 * abs(cut)).all())
        order = order[off >= cut]
    ids = np.sort(order)
    mass = w[ids]
    upto = np.cumsum(mass)
    u = min(max(0.0 if math.isnan(u) else u, 0.0), 1 - 2.0 ** -53)
    clear &= bool(np.abs(upto - u * upto[-1]).min() > CLOSE * upto[-1]) or u == 0.0
    at = min(int((upto <= u * upto[-1]).sum()), len(ids) - 1)
    while mass[at] < 2.0 ** -46:    # no weight in the header's units
        at += 1
    return int(ids[at]), float(mass[at] / upto[-1]), clear


def check(logits, u, T=1.0, k=0, p=1.0, mp=0.0, most_unclear=0.02, **kw):
    got, prob = dsm.sample(logits, u, temperature=T, top_k=k, top_p=p, min_p=mp, **kw)
    got, prob = got.cpu().tolist(), prob.cpu().tolist()
    l, u = logits.cpu().double().numpy(), u.cpu().tolist()
    per = lambda x, b: x[b].item() if isinstance(x, torch.Tensor) else x  # noqa: E731
    f32 = lambda x: float(np.float32(x))  # noqa: E731
    unclear = 0
    for b in range(l.shape[0]):
        tok, pr, clear = reference(l[b], u[b], f32(per(T, b)), per(k, b), f32(per(p, b)),
                                   f32(per(mp, b)))
        if not clear:
            unclear += 1
            continue
        assert got[b] == tok, (b, got[b], tok)
        # the mass off by 2^-33 relative, one rounding to fp32
        assert abs(prob[b] - pr) <= pr * (2.0 ** -24 + 2.0 ** -32) + 1e-45, (b, prob[b], pr)
    assert unclear <= most_unclear * len(got) + 1
    return got


def inputs(B, V, dtype, seed, sigma=2.0):
    g = torch.Generator()
    g.manual_seed(seed)
    z = torch.randn(B, V, generator=g) * sigma
    return z.to(dtype).to(DEV), torch.rand(B, generator=g, dtype=torch.float64).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V", [(1, 1), (5, 2), (7, 33), (40, 1000), (16, 2048), (16, 2049), (9, 4097),
                                 (8, 8200), (6, 32003), (3, 129280), (1, 700_001)])
def test_every_setting_matches_64_bits(B, V, dtype):
    z, u = inputs(B, V, dtype, seed=V)
    check(z, u)
    check(z, u, T=0.7, k=1)
    check(z, u, T=0.7, k=max(1, V // 3))
    check(z, u, T=1.3, p=0.9)
    check(z, u, T=1.0, p=0.3)
    check(z, u, mp=0.05)
    check(z, u, T=0.9, k=50, p=0.95, mp=0.02)
    check(z, u, T=0.0)


def test_settings_per_row():
    B, V = 64, 5000
    z, u = inputs(B, V, torch.float32, seed=1)
    row = torch.arange(B, device=DEV)
    check(z, u, T=(0.3 * (row % 5)).float(), k=(row % 7 * 10).int(), p=(0.4 + 0.1 * (row % 8)).float(),
          mp=(0.03 * (row % 3)).float())
    check(z, u, T=(0.3 * (row % 5)).float(), k=11, p=0.8, mp=(0.03 * (row % 3)).float())


@pytest.mark.parametrize("k,p", [(0, 0.5), (37, 1.0), (37, 0.5), (1, 1.0), (900, 0.999)])
def test_ties_go_to_the_lowest_ids(k, p):
    # few values, many equal: half of them at the border
    g = torch.Generator()
    g.manual_seed(k)
    z = torch.randint(0, 3, (32, 9000), generator=g).float()
    u = torch.rand(32, generator=g, dtype=torch.float64).to(DEV)
    check(z.to(DEV), u, k=k, p=p)
    check((z * -0.0).to(DEV), u, k=k, p=p)                       # all equal, some -0
    check((z.to(torch.bfloat16) * 4 - 20).to(DEV), u, k=k, p=p, T=2.0)


def test_tokens_that_are_masked():
    z, u = inputs(24, 3001, torch.float32, seed=2)
    z[:, ::2] = -float("inf")
    z[:, 1::6] = float("nan")
    z[3, :] = -float("inf")
    z[4, :] = float("nan")
    z[5, 77] = float("inf")
    z[6, 50:60] = float("inf")
    z[7, 3::6] = torch.finfo(torch.float32).min
    for kw in (dict(), dict(k=20), dict(p=0.8), dict(mp=0.1), dict(k=5, p=0.5, mp=0.3), dict(T=0.0)):
        got = check(z, u, **kw)
        assert got[3] == got[4] == -1 and got[5] == 77 and 50 <= got[6] < 60
    low = torch.full((2, 100), torch.finfo(torch.float32).min, device=DEV)
    check(low, u[:2])
    check(low.to(torch.bfloat16), u[:2], k=3)


def test_uniforms_at_the_ends():
    z, _ = inputs(6, 500, torch.float32, seed=3)
    u = torch.tensor([0.0, 1 - 2.0 ** -53, 1.0, 5.0, -1.0, float("nan")], dtype=torch.float64, device=DEV)
    got = check(z, u, T=1.0, most_unclear=1.0)
    w = torch.softmax(z.cpu().double(), -1)
    last = [int((r > 2.0 ** -46 * r.max()).nonzero().max()) for r in w]
    assert got[0] == got[4] == got[5] == 0 and got[1:4] == last[1:4]


def test_settings_at_the_ends():
    z, u = inputs(16, 700, torch.float32, seed=4)
    check(z, u, T=float("inf"))
    check(z, u, T=1e30, k=10)
    check(z, u, T=1e-3)
    check(z, u, T=-1.0)
    check(z, u, T=float("nan"))
    check(z, u, k=700)
    check(z, u, k=2 ** 40)
    check(z, u, k=-3)
    check(z, u, p=0.0)
    check(z, u, p=-2.0)
    check(z, u, p=float("nan"))
    check(z, u, p=5.0)
    check(z, u, mp=1.0)
    check(z, u, mp=3.0)
    check(z, u, mp=1e-30)
    check(z * 1e4, u, p=0.9)
    check(z * 1e-6, u, p=0.9, k=300)


def test_strided_rows_and_other_outputs():
    z, u = inputs(10, 4001, torch.bfloat16, seed=5)
    want = dsm.sample(z[:, :3001].contiguous(), u, top_p=0.8)
    out, prob = (torch.full((10,), -7, dtype=t, device=DEV) for t in (torch.int32, torch.float32))
    got = dsm.sample(z[:, :3001], u, top_p=0.8, out=out, prob=prob)
    assert got[0] is out and got[1] is prob
    assert torch.equal(out, want[0]) and torch.equal(prob, want[1])
    shifted = dsm.sample(z[:, 1:3002], u, top_p=0.8)
    want = dsm.sample(z[:, 1:3002].contiguous(), u, top_p=0.8)
    assert torch.equal(shifted[0], want[0]) and torch.equal(shifted[1], want[1])


@pytest.mark.parametrize("T", [1.0, 0.7, 1.9, 0.013])
def test_weights_are_as_close_as_they_are_said_to_be(T):
    # two tokens: the lighter one, of lower id, is drawn just below its share and not just above. The
    # heavier's weight is exact, the lighter's off by 2^-35 and half a unit (2^-46, against 2^-9 or
    # more), and the draw's place is rounded down to a unit: below 2^-34 of the share together
    g = torch.Generator()
    g.manual_seed(5)
    t32 = float(np.float32(T))
    diff = torch.rand(2000, generator=g).double() * 6.2 * t32
    top = torch.randn(2000, generator=g) * 3
    z = torch.stack([(top.double() - diff).float(), top], 1).to(DEV)
    d = (z[:, 0].double() - z[:, 1].double()).cpu().numpy().astype(np.longdouble)
    w = np.exp(d / np.longdouble(t32))
    share = (w / (1 + w)).astype(np.float64)     # (rounded by 2^-54 of 1, below 2^-43 of it)
    for side, token in ((1 - 2.0 ** -34, 0), (1 + 2.0 ** -34, 1)):
        u = torch.from_numpy(share * side).to(DEV)
        got, _ = dsm.sample(z, u, temperature=T)
        assert bool((got == token).all())


@pytest.mark.parametrize("T,mp,top", [
    (1.634910225868225, 0.6227176189422607, 0.7743950486183167),
    (1.8739752769470215, 0.31074097752571106, 2.190294027328491), (1.0, 0.5, 0.6931472), (2.0, 0.1, 1.0)])
def test_min_p_borders_near_a_logit_of_zero(T, mp, top):
    # max + T log(min_p) is 0 but for a rounding of fp64, so that hundreds of millions of logits around 0
    # have the border's difference (the first two); what is clearly above or below is decided
    row = [top, 1e-3, -1e-3, 1e-12, -1e-12, -5.0, 0.25, -0.25]
    z = torch.tensor([row] * 9, device=DEV)
    u = torch.tensor([0.0, 0.2, 0.4, 0.5, 0.6, 0.7, 0.8, 0.9, 1 - 2.0 ** -53], dtype=torch.float64, device=DEV)
    z[:, 3:5] = -9.0
    check(z, u, T=T, mp=mp)
    z[:, 3:5] = torch.tensor([1e-12, -1e-12])
    got, prob = dsm.sample(z, u, temperature=T, min_p=mp)
    assert set(got.tolist()) <= {0, 1, 3, 4, 6} | ({2, 7} if top == 1.0 else set())


def test_many_rows_of_a_small_vocabulary():
    # one token of weight per row, found whatever the row; then 70,000 rows of three
    B = 70_000
    at = torch.arange(B, device=DEV) % 3
    z = torch.full((B, 3), float("-inf"), device=DEV)
    z[torch.arange(B, device=DEV), at] = 1.0
    u = torch.rand(B, generator=torch.Generator().manual_seed(8), dtype=torch.float64).to(DEV)
    for kw in ({}, dict(top_k=2), dict(top_p=0.5), dict(min_p=0.5)):
        got, prob = dsm.sample(z, u, **kw)
        assert torch.equal(got, at.int()) and bool((prob == 1).all())


@pytest.mark.parametrize("k", [100, 128, 129, 200, 400, 511, 512, 513])
def test_every_way_to_finish_a_top_k(k):
    # kept tokens compared, sorted or counted in bins, with equal logits among them
    g = torch.Generator()
    g.manual_seed(k)
    z = (torch.randn(24, 5000, generator=g) * 8).round().div(8).to(DEV)
    z[:, :300] = torch.randn(24, 300, generator=g).to(DEV) + 4
    u = torch.rand(24, generator=g, dtype=torch.float64).to(DEV)
    check(z, u, k=k)
    check(z, u, k=k, p=0.8, T=1.5)
    check(z, u, k=k, p=0.9, mp=0.05)


def test_frequencies_follow_the_distribution():
    # 200,000 draws of one row: each token's count within 6 standard deviations
    z = torch.randn(200, generator=torch.Generator().manual_seed(6)) * 1.5
    n = 200_000
    u = torch.rand(n, generator=torch.Generator().manual_seed(7), dtype=torch.float64)
    got, _ = dsm.sample(z.expand(n, -1).contiguous().to(DEV), u.to(DEV), temperature=0.8, top_k=40)
    w = torch.softmax(z.double() / 0.8, 0)
    w[torch.argsort(-z)[40:]] = 0
    w /= w.sum()
    count = torch.bincount(got.cpu().long(), minlength=200).double()
    assert bool(((count - n * w).abs() <= 6 * torch.sqrt(n * w * (1 - w)) + 1e-9).all())


def test_no_rows_streams_and_replays():
    e = torch.empty(0, 100, device=DEV)
    assert dsm.sample(e, torch.empty(0, dtype=torch.float64, device=DEV))[0].shape == (0,)
    z, u = inputs(20, 9001, torch.float32, seed=8)
    want = dsm.sample(z, u, top_k=50, top_p=0.9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dsm.sample(z, u, top_k=50, top_p=0.9, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsm.sample(z, u, top_k=50, top_p=0.9, out=want[0], prob=want[1])
    z2, u2 = inputs(20, 9001, torch.float32, seed=9)
    z.copy_(z2)
    u.copy_(u2)
    graph.replay()
    torch.cuda.synchronize()
    got = dsm.sample(z, u, top_k=50, top_p=0.9)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("V", [1025, 2049, 4097, 8193])
def test_clusters_whose_ctas_have_little_to_load(V):
    # the CTAs of a row exchange their largest logits as soon as they can, call behind call
    z, u = inputs(3, V, torch.bfloat16, seed=V)
    want = [check(z, u, **kw) for kw in (dict(), dict(k=40), dict(p=0.9))]
    got = [[dsm.sample(z[i % 3:], u[i % 3:], top_k=k, top_p=p)[0] for k, p in ((0, 1.0), (40, 1.0), (0, 0.9))]
           for i in range(60)]
    for i, each in enumerate(got):
        assert [t.tolist() for t in each] == [w[i % 3:] for w in want]


def test_verify_sample_and_sample_agree_on_a_row():
    # the bonus token of a step of one row is a draw from the whole distribution
    z, u = inputs(30, 3000, torch.float32, seed=10)
    a, _ = dsm.sample(z, u, temperature=0.8)
    b, n = dsm.verify_sample(z[:, None].contiguous(), float(np.float32(0.8)), None, None, None, u[:, None].contiguous())
    assert torch.equal(a, b[:, 0]) and bool((n == 1).all())


@pytest.mark.parametrize("kw", [dict(), dict(top_k=1 << 16), dict(top_p=0.9999999), dict(min_p=1e-12)])
def test_uniforms_beyond_the_end_are_the_last_one(kw):
    # 2^17 - 1 tokens of weight 1 and a last one of 2^-37 or less of it, 2^-54 of the mass: above the last
    # uniform below 1, which leaves 2^-53, and not to be drawn at 1 and beyond either
    z = torch.zeros(4, 1 << 17, device=DEV)
    z[:, -1] = -37 * math.log(2)
    u = torch.tensor([1 - 2.0 ** -53, 1.0, 7.0, float("inf")], dtype=torch.float64, device=DEV)
    got = dsm.sample(z, u, **kw)[0].tolist()
    assert got == [got[0]] * 4 and (got[0] == (1 << 17) - 2 or kw.get("top_p") or kw.get("top_k"))


@pytest.mark.parametrize("T", [3.3e19, 1.7e25, 7.7e28, 1.2e30])
def test_weights_at_high_temperatures(T):
    # as test_weights_are_as_close_as_they_are_said_to_be, with logits of the temperature's size
    g = torch.Generator()
    g.manual_seed(5)
    t32 = float(np.float32(T))
    diff = (torch.rand(2000, generator=g).double() * 6.2 + 1e-3) * t32
    top = torch.randn(2000, generator=g) * 3 * t32
    z = torch.stack([(top.double() - diff).float(), top], 1).to(DEV)
    d = (z[:, 0].double() - z[:, 1].double()).cpu().numpy().astype(np.longdouble)
    w = np.exp(d / np.longdouble(t32))
    share = (w / (1 + w)).astype(np.float64)
    for side, token in ((1 - 2.0 ** -34, 0), (1 + 2.0 ** -34, 1)):
        got, _ = dsm.sample(z, torch.from_numpy(share * side).to(DEV), temperature=T)
        assert bool((got == token).all()), int((got != token).sum())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V", [(2, 311_232), (2, 311_300), (3, 400_003)])
def test_vocabularies_around_what_shared_memory_holds(B, V, dtype):
    # the largest of which a CTA keeps its part, and ones that are read again and again: masked tokens,
    # NaN, infinities, equal logits at the border
    z, u = inputs(B, V, dtype, seed=V)
    for kw in (dict(), dict(k=40), dict(k=5000, p=0.9), dict(T=1.3, p=0.9), dict(mp=0.05), dict(T=0.0)):
        check(z, u, **kw)
    z[:, ::2] = -float("inf")
    z[:, 1::6] = float("nan")
    z[0] = (z[0] * 2).round() / 2
    for kw in (dict(k=700), dict(p=0.7), dict(p=0.9, mp=0.02)):
        check(z, u, **kw)
    z[1, 70::1000] = float("inf")
    assert check(z, u, k=3)[1] % 1000 == 70 and check(z, u, p=0.5)[1] % 1000 == 70
