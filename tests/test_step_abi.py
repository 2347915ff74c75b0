"""The C ABI and the binding of the block norm, the attention over shared prefixes and the sampling
reject bad arguments on the host, before anything reaches a GPU (no compute calls here)."""
import pytest
import torch

from test_paged_abi import BAD_CACHES, BAD_POINTERS, BIG, FAKE, cache, lib, paged  # noqa: F401

NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------------- shared prefixes
def prefix(own=None, **kw):
    from q4_moe_speculative_gb300 import _native as N
    d = dict(own=own if own is not None else paged(n_seqs=6), n_prefixes=2, max_prefix_pages=64,
             prefix_table=FAKE, prefix_lengths=FAKE)
    d.update(kw)
    return N.DsPrefixAttnArgs(*[d[f] for f, _ in N.DsPrefixAttnArgs._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(n_prefixes=0), 1), (dict(n_prefixes=-1), 1), (dict(n_prefixes=4), 1),
    (dict(n_prefixes=7), 1), (dict(max_prefix_pages=0), 1), (dict(max_prefix_pages=(1 << 18) + 1), 1),
    (dict(prefix_table=None), 1), (dict(prefix_table=FAKE + 2), 1), (dict(prefix_lengths=None), 1),
    (dict(prefix_lengths=FAKE + 1), 1),
])
def test_prefix_arguments(lib, kw, code):  # noqa: F811
    a = prefix(**kw)
    assert lib.ds_prefix_attention(a, FAKE, FAKE, BIG, None) == code
    pointers = {"prefix_table", "prefix_lengths"} & set(kw)
    assert (lib.ds_prefix_attn_workspace_size(a) > 0) == bool(pointers)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), 1), (dict(n_seqs=4098), 1), (dict(n_rows=0), 1), (dict(n_rows=9), 1),
    (dict(n_heads=30), 1), (dict(max_pages=0), 1), (dict(scale=INF), 1), (dict(scale=3e38), 1),
    (dict(n_heads=4 * 22), 2), (dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(page_table=None), 1),
    (dict(page_table=FAKE + 1), 1), (dict(lengths=None), 1), (dict(lengths=FAKE + 2), 1),
])
def test_prefix_arguments_of_the_sequences(lib, kw, code):  # noqa: F811
    a = prefix(own=paged(**{"n_seqs": 6, **kw}))
    assert lib.ds_prefix_attention(a, FAKE, FAKE, BIG, None) == code


@pytest.mark.parametrize("kw,code", BAD_CACHES + BAD_POINTERS)
def test_prefix_caches(lib, kw, code):  # noqa: F811
    a = prefix(own=paged(n_seqs=6, cache=cache(**kw)))
    assert lib.ds_prefix_attention(a, FAKE, FAKE, BIG, None) == code


def test_prefix_workspace(lib):  # noqa: F811
    a = prefix()
    need = lib.ds_prefix_attn_workspace_size(a)
    assert need > lib.ds_paged_attn_workspace_size(a.own) and need % 256 == 0
    f = lib.ds_prefix_attention
    assert f(a, FAKE, FAKE, need - 1, None) == 3
    assert f(a, FAKE, None, need, None) == 3 and f(a, FAKE, FAKE + 128, need, None) == 3
    assert f(a, None, FAKE, need, None) == 1 and f(a, FAKE + 4, FAKE, need, None) == 1
    assert f(None, FAKE, FAKE, need, None) == 1
    assert lib.ds_prefix_attn_workspace_size(None) == 0
    none = prefix(own=paged(n_seqs=0, q=None, page_table=None, lengths=None), prefix_table=None)
    assert lib.ds_prefix_attn_workspace_size(none) == 0
    assert f(none, None, None, 0, None) == 0


def test_prefix_workspace_of_many_prefixes(lib):  # noqa: F811
    # sums of one row of each of 1024 x 8 heads, not of whole tiles of 128 rows (1 GB)
    a = prefix(own=paged(n_seqs=1024, n_rows=1, n_heads=8, cache=cache(n_heads=8)), n_prefixes=1024)
    assert 0 < lib.ds_prefix_attn_workspace_size(a) < 32 << 20


# ------------------------------------------------------------------------------ block norm
def norm(**kw):
    from q4_moe_speculative_gb300 import _native as N
    d = dict(n_rows=6, hidden=4096, x_format=0, eps=1e-6, weight_offset=0.0, x_scale=1.0, y_scale=1.0,
             x=FAKE, x_stride=4096, y=2 * FAKE, y_stride=4096, post_weight=FAKE, gate=FAKE,
             gate_stride=0, weight=FAKE)
    d.update(kw)
    return N.DsBlockNormArgs(*[d[f] for f, _ in N.DsBlockNormArgs._fields_])


X_OUT, H_OUT = 3 * FAKE, 4 * FAKE


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(n_rows=(1 << 24) + 1), dict(hidden=0), dict(hidden=4), dict(hidden=4100),
    dict(hidden=-8), dict(hidden=16392), dict(x_format=2), dict(x_format=-1), dict(eps=-1.0),
    dict(eps=NAN), dict(eps=INF), dict(weight_offset=INF), dict(x_scale=NAN), dict(y_scale=INF),
    dict(x=None), dict(x=FAKE + 8), dict(x_stride=4088), dict(x_stride=4100), dict(x_stride=-4096),
    dict(x_stride=(1 << 31) + 8), dict(y=FAKE + 2), dict(y_stride=0), dict(y_stride=4097),
    dict(post_weight=FAKE + 4), dict(gate=FAKE + 8), dict(gate_stride=8), dict(gate_stride=-8),
    dict(weight=FAKE + 2),
])
def test_block_norm_arguments(lib, kw):  # noqa: F811
    assert lib.ds_block_norm(norm(**kw), X_OUT, H_OUT, None) == 1


def test_block_norm_outputs(lib):  # noqa: F811
    f = lib.ds_block_norm
    assert f(None, X_OUT, H_OUT, None) == 1
    assert f(norm(), X_OUT, None, None) == 1             # a weight, and nowhere for h
    assert f(norm(), X_OUT + 8, H_OUT, None) == 1 and f(norm(), X_OUT, H_OUT + 2, None) == 1
    assert f(norm(), X_OUT, X_OUT, None) == 1
    assert f(norm(weight=None), None, None, None) == 1   # nothing to write
    assert f(norm(y=None, weight=None), X_OUT, None, None) == 1
    wide = dict(x=FAKE, x_stride=8192, y=2 * FAKE, y_stride=8192)
    assert f(norm(**wide), FAKE, H_OUT, None) == 1       # in place only when contiguous
    assert f(norm(**wide), X_OUT, FAKE, None) == 1
    assert f(norm(**wide), X_OUT, 2 * FAKE, None) == 1
    assert f(norm(**wide), 2 * FAKE, H_OUT, None) == 1
    assert f(norm(x_format=1), 2 * FAKE, H_OUT, None) == 1   # and of the same type
    assert f(norm(x_format=1), X_OUT, FAKE, None) == 1
    assert f(norm(n_rows=0, x=None, y=None), None, None, None) == 0


# -------------------------------------------------------------------------------- sampling
def draw(**kw):
    from q4_moe_speculative_gb300 import _native as N
    d = dict(n_rows=6, n_vocab=1000, logits_format=0, logits=FAKE, logits_stride=1000, u=FAKE,
             temperature=1.0, top_p=1.0, min_p=0.0, top_k=0, temperatures=None, top_ps=None,
             min_ps=None, top_ks=None)
    d.update(kw)
    return N.DsSampleArgs(*[d[f] for f, _ in N.DsSampleArgs._fields_])


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(n_rows=(1 << 20) + 1), dict(n_vocab=0), dict(n_vocab=(1 << 24) + 1),
    dict(logits_format=2), dict(logits=None), dict(logits=FAKE + 1), dict(logits_format=1, logits=FAKE + 2),
    dict(logits_stride=999), dict(logits_stride=(1 << 31) + 1), dict(logits_stride=-1000), dict(u=None),
    dict(u=FAKE + 4), dict(temperatures=FAKE + 2), dict(top_ps=FAKE + 1), dict(min_ps=FAKE + 2),
    dict(top_ks=FAKE + 3),
])
def test_sample_arguments(lib, kw):  # noqa: F811
    assert lib.ds_sample(draw(**kw), FAKE, FAKE, None) == 1


def test_sample_outputs(lib):  # noqa: F811
    f = lib.ds_sample
    assert f(None, FAKE, FAKE, None) == 1 and f(draw(), None, FAKE, None) == 1
    assert f(draw(), FAKE + 2, FAKE, None) == 1 and f(draw(), FAKE, FAKE + 1, None) == 1
    assert f(draw(n_rows=0, logits=None, u=None), None, None, None) == 0


# ------------------------------------------------------------------------------ the binding
def test_the_binding_refuses_host_tensors_and_wrong_shapes(lib):  # noqa: F811
    import q4_moe_speculative_gb300 as dsm
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c = dsm.PagedCache.zeros(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        dsm.prefix_attention(bf(2, 1, 2, 64), c, i32(1, 2), i32(1), i32(2, 2), i32(2))
    with pytest.raises(ValueError):
        dsm.block_norm(bf(3, 64), bf(3, 64), weight=bf(64))
    with pytest.raises(ValueError):
        dsm.sample(torch.zeros(3, 10), torch.zeros(3, dtype=torch.float64))
    for bad in (None, [1.0], 3):
        with pytest.raises(TypeError):
            dsm.block_norm(bad)
        with pytest.raises(TypeError):
            dsm.sample(bad, bad)
        with pytest.raises(TypeError):
            dsm._hidden_rows(bad, "y", torch.bfloat16, (2, 8), torch.device("cpu"))


def test_strides_of_hidden_rows():
    import q4_moe_speculative_gb300 as dsm
    dev, bf = torch.device("cpu"), torch.bfloat16
    t = torch.zeros(6, 64, dtype=bf)
    rows = lambda x: dsm._hidden_rows(x, "y", bf, tuple(x.shape), dev)  # noqa: E731
    assert rows(t) == 64 and rows(t[:, :32]) == 64 and rows(t[::2]) == 128
    assert rows(t[:1]) == 64 and rows(t[:1, :32]) == 32
    with pytest.raises(ValueError):
        rows(t.t())
    with pytest.raises(ValueError):
        dsm._hidden_rows(t, "y", bf, (6, 32), dev)
    with pytest.raises(ValueError):
        dsm._hidden_rows(t.float(), "y", bf, (6, 64), dev)
