"""The norms around a block (ds_block_norm) against its formula in 64 bits."""
import pytest
import torch

import paged_ref as ref
import q4_moe_speculative_gb300 as dsm

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-6


def reference(x, y, weight, post, gate, o, xs, ys, eps=EPS):
    """(x, magnitude of its terms, h) in fp64."""
    x = x.double()
    mag = x.abs()
    norm = lambda t, w: t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * (w.double() + o)  # noqa: E731
    if y is not None:
        b = y.double() if post is None else norm(y.double(), post)
        if gate is not None:
            b = b * gate.double()
        x = xs * x + ys * b
        mag = abs(xs) * mag + (ys * b).abs()
    return x, mag, None if weight is None else norm(x, weight)


def check(x, y=None, weight=None, post=None, gate=None, o=0.0, xs=1.0, ys=1.0, got=None, **kw):
    H = x.shape[1]
    if got is None:
        got = dsm.block_norm(x, y, weight=weight, post_weight=post, gate=gate, weight_offset=o,
                             x_scale=xs, y_scale=ys, eps=EPS, **kw)
    want_x, mag, want_h = reference(x, y, weight, post, gate, o, xs, ys)
    x_out, h = got
    # in fp32: the mean's sum of H / threads terms and a tree (at most 32 + 20 roundings, halved by
    # the root), root, quotient, weight, offset, gate and scales: 16 units more; then one rounding
    unit = (26 + 16) * ref.U32
    tol = mag * unit + (ref.HALF_BF16 * want_x.abs() if x.dtype == torch.bfloat16 else 0)
    assert bool(((x_out.double() - want_x).abs() <= tol + 1e-35).all())
    if weight is not None:
        # (h's own norm, and x's error relative to its terms)
        factor = (want_h.abs() / want_x.abs().clamp(min=1e-300))
        spread = torch.sqrt((mag * mag).mean(-1, keepdim=True) / (want_x * want_x).mean(-1, keepdim=True))
        tol = want_h.abs() * (ref.HALF_BF16 + unit * (1 + spread)) + factor * mag * unit
        assert bool(((h.double() - want_h).abs() <= tol + 1e-35).all())
    else:
        assert h is None
    return got


def rows(T, H, dtype=torch.bfloat16, seed=0, sigma=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(T, H, generator=g) * sigma).to(dtype).to(DEV)


def vec(H, seed):
    return rows(1, H, seed=seed)[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (6, 4096), (5, 248), (9, 264), (2, 1032), (7, 5000),
                                 (1, 16384), (700, 320), (400, 1024), (400, 1032), (330, 8192),
                                 (310, 16384), (2, 12296)])
def test_block_norm_matches_64_bits(T, H, dtype):
    x, y = rows(T, H, dtype, 1, 3.0), rows(T, H, seed=2)
    w, p = vec(H, 3), vec(H, 4)
    check(x, y, w, p)
    check(x, y, w, None, vec(H, 5), o=1.0, xs=0.5, ys=-0.25)
    check(x, y, w, p, rows(T, H, seed=6), o=1.0, xs=1.0, ys=0.22)
    check(x, y, None, p, rows(T, H, seed=6))      # the residual stream alone
    got = dsm.block_norm(x, weight=w, eps=EPS)    # the norm alone
    assert got[0] is x
    check(x, weight=w, got=(x if dtype == torch.float32 else x, got[1]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(20001, 8), (30003, 64), (19999, 72), (9001, 128), (9003, 136),
                                 (5001, 256), (2501, 512), (700, 8200), (333, 9000), (309, 12288)])
def test_more_rows_than_fit_at_once(T, H, dtype):
    # rows of part of a warp, a warp or a CTA; each walks over several, the last ones beside none
    x, y = rows(T, H, dtype, 1, 3.0), rows(T, H, seed=2)
    w, p = vec(H, 3), vec(H, 4)
    check(x, y, w, p, rows(T, H, seed=6), o=1.0, xs=0.9, ys=0.22)
    check(x, y, w, None, vec(H, 5))
    want = dsm.block_norm(x, y, weight=w, post_weight=p)
    x1, y1 = x.clone(), y.clone()
    got = dsm.block_norm(x1, y1, weight=w, post_weight=p, x_out=x1, h_out=y1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows(dtype):
    T, H = 37, 520
    wide = rows(T, 3 * H, seed=1)
    x = rows(T, 2 * H, dtype, 2)[:, H:]
    y, gate = wide[:, :H], wide[:, 2 * H:]
    w, p = vec(H, 3), vec(H, 4)
    a = check(x, y, w, p, gate)
    b = dsm.block_norm(x.contiguous(), y.contiguous(), weight=w, post_weight=p,
                       gate=gate.contiguous(), eps=EPS)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    every = rows(2 * T, H, dtype, 5)[::2]
    check(every, y, w, p, gate)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(6, 4096), (500, 640), (400, 6000)])
def test_in_place(T, H, dtype):
    x, y = rows(T, H, dtype, 1), rows(T, H, seed=2)
    w, p = vec(H, 3), vec(H, 4)
    want = dsm.block_norm(x, y, weight=w, post_weight=p)
    x1, y1 = x.clone(), y.clone()
    got = dsm.block_norm(x1, y1, weight=w, post_weight=p, x_out=x1, h_out=y1)
    assert got[0] is x1 and got[1] is y1
    assert torch.equal(x1, want[0]) and torch.equal(y1, want[1])
    if dtype == torch.bfloat16:
        x1, y1 = x.clone(), y.clone()
        dsm.block_norm(x1, y1, weight=w, post_weight=p, x_out=y1, h_out=x1)
        assert torch.equal(y1, want[0]) and torch.equal(x1, want[1])


def test_rows_do_not_depend_on_each_other():
    x, y, w, p = rows(400, 1000, seed=1), rows(400, 1000, seed=2), vec(1000, 3), vec(1000, 4)
    want = dsm.block_norm(x, y, weight=w, post_weight=p)
    x[7], y[9] = float("nan"), float("inf")
    got = dsm.block_norm(x, y, weight=w, post_weight=p)
    keep = torch.tensor([i not in (7, 9) for i in range(400)], device=DEV)
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
        assert bool(a[7].isnan().all()) and bool(a[9].isnan().all())


def test_rows_of_zeros_and_extremes():
    T, H = 4, 256
    x, y = torch.zeros(T, H, device=DEV), torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    w = vec(H, 3)
    a, b = dsm.block_norm(x, y, weight=w, post_weight=w)
    assert not bool(a.any()) and not bool(b.any())
    assert bool(dsm.block_norm(x, weight=w, eps=0.0)[1].isnan().all())
    big = rows(T, H, torch.float32, 5, 2.0 ** 52)
    check(big, rows(T, H, seed=6, sigma=2.0 ** 50), w, w)
    check(big * 2.0 ** -110, rows(T, H, seed=6), w)


def test_no_rows_and_streams():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    a, b = dsm.block_norm(e, e, weight=vec(64, 1))
    assert a.shape == b.shape == (0, 64)
    x, y, w = rows(9, 640, seed=1), rows(9, 640, seed=2), vec(640, 3)
    want = dsm.block_norm(x, y, weight=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dsm.block_norm(x, y, weight=w, stream=s)
    s.synchronize()
    assert all(torch.equal(g, v) for g, v in zip(got, want))


def test_captured_and_replayed():
    x, y, w = rows(6, 4096, torch.float32, 1), rows(6, 4096, seed=2), vec(4096, 3)
    a, b = dsm.block_norm(x, y, weight=w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsm.block_norm(x, y, weight=w, x_out=a, h_out=b)
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want = dsm.block_norm(x, y, weight=w)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 8), (6, 4096), (700, 320), (400, 1032), (310, 9000)])
def test_the_norm_alone_leaves_its_input(T, H, dtype):
    x, w = rows(T, H, dtype, 1, 3.0), vec(H, 3)
    before = x.clone()
    got = dsm.block_norm(x, weight=w, eps=EPS)
    assert got[0] is x and torch.equal(x, before)
    check(x, weight=w, got=got)


@pytest.mark.parametrize("T,H", [(5, 64), (9, 520), (300, 4096), (170, 12296)])
def test_outputs_that_swap_the_inputs_places(T, H):
    # x_out in y's place and h_out in x's, both of which are read in the same pass
    x, y, w, p = rows(T, H, seed=1), rows(T, H, seed=2), vec(H, 3), vec(H, 4)
    want = dsm.block_norm(x, y, weight=w, post_weight=p)
    got = dsm.block_norm(x, y, weight=w, post_weight=p, x_out=y, h_out=x)
    assert got[0] is y and got[1] is x
    assert torch.equal(y, want[0]) and torch.equal(x, want[1])
