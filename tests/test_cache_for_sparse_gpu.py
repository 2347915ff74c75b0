"""The paged cache read by the block selection and the sparse attention: with one key head, bf16
and pages in order, a layer's pages are the [tokens, 128] that both of them take."""
import pytest
import torch

import paged_ref as ref
import q4_moe_speculative_gb300 as dsm

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("page,tokens,Hq", [(16, 640, 16), (64, 2048, 4), (128, 1152, 16)])
def test_sparse_attention_reads_the_cache(page, tokens, Hq):
    # tokens written by the fused pass; all blocks selected give what the paged attention gives,
    # and a part of them the 64-bit result over that part
    D, B4 = 128, 4
    pages = tokens // page
    cache = dsm.PagedCache.zeros(pages, 1, page, D)
    qkv = ref.normal(tokens, Hq + 2, D, seed=page).to(DEV)
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
    q = dsm.qk_norm_rope_write(qkv[:, :Hq], qkv[:, Hq:Hq + 1], qkv[:, Hq + 1:], pos,
                               dsm.rope_frequencies(D), cache, pos)
    k, v = cache.k.view(1, tokens, D), cache.v.view(1, tokens, D)
    last = q[tokens - 1].view(1, 1, Hq, D)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lengths = torch.tensor([tokens], dtype=torch.int32, device=DEV)
    paged = dsm.paged_attention(last, cache, table, lengths)
    blocks = tokens // B4
    every = torch.arange(blocks, dtype=torch.int32, device=DEV).view(1, 1, blocks)
    g = torch.Generator().manual_seed(page)
    some = torch.randperm(blocks, generator=g)[:blocks // 3].sort().values
    part = torch.full((1, 1, blocks), -1, dtype=torch.int32)
    part[0, 0, :len(some)] = some.to(torch.int32)
    part_tokens = (some[:, None] * B4 + torch.arange(B4)).flatten()
    for sel, t, outs in ((every, torch.arange(tokens), [paged]), (part.to(DEV), part_tokens, [])):
        outs = outs + [dsm.sparse_attention(last, k, v, sel, B4)]
        kk, vv = k[0].cpu().double()[t], v[0].cpu().double()[t]
        x = last[0, 0].cpu().double()
        p = torch.softmax(x @ kk.t() * D ** -0.5, -1)
        want = (p @ vv).view(1, 1, Hq, D)
        mag = (p @ vv.abs()).view(1, 1, Hq, D)
        rss = torch.sqrt((p * p) @ (vv * vv)).view(1, 1, Hq, D)
        top = float((x.abs() @ kk.abs().t()).max() * D ** -0.5)
        for out in outs:
            ref.check_attention(out, (want, mag, rss, top), tokens, D)


def test_selection_reads_the_cache():
    # a selection's block keys kept in the cache of a layer of their own
    D, N, R, Hh, K = 128, 320, 3, 4, 64
    cache = dsm.PagedCache.zeros(N // 64, 1, 64, D)
    keys = ref.normal(N, 1, D, seed=3).to(DEV)
    slots = torch.arange(N, dtype=torch.int32, device=DEV)
    dsm.cache_write(cache, keys, keys, slots)
    q = ref.normal(1, R, Hh, D, seed=4).to(DEV)
    head_w = torch.rand(1, R, Hh, device=DEV)
    mask = torch.full((1, R, N // 32), -1, dtype=torch.int32, device=DEV)
    limit = torch.full((1, R), N, dtype=torch.int32, device=DEV)
    want = dsm.select_blocks(keys.view(1, N, D), q, head_w, mask, limit, K)
    got = dsm.select_blocks(cache.k.view(1, N, D), q, head_w, mask, limit, K)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((got[1] == K).all())
