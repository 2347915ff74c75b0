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
