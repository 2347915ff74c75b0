"""The C ABI and the binding of the paged-cache operators and the Q4 projection reject bad
arguments on the host, before anything reaches a GPU (no compute calls here)."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from q4_moe_speculative_gb300.build import build_library
    build_library()
    from q4_moe_speculative_gb300 import _native
    return _native.load()


FAKE = 1 << 20  # a 256-aligned address that is never dereferenced: validation fails first
BIG = 1 << 40


def cache(**kw):
    from q4_moe_speculative_gb300 import _native as N
    d = dict(n_pages=100, n_kv_heads=4, page_tokens=64, head_dim=128, format=1, k=FAKE, v=FAKE,
             page_stride=4 * 64 * 128, k_scale=FAKE, v_scale=FAKE, scale_page_stride=4 * 64)
    d.update(kw)
    return N.DsPagedCache(*[d[f] for f, _ in N.DsPagedCache._fields_])


BAD_CACHES = [
    (dict(n_pages=0), 1), (dict(n_pages=1 << 25), 1), (dict(n_kv_heads=0), 1),
    (dict(n_kv_heads=257), 1), (dict(page_tokens=8), 1), (dict(page_tokens=48), 1),
    (dict(page_tokens=256), 1), (dict(head_dim=0), 1), (dict(head_dim=96), 2),
    (dict(head_dim=256), 2), (dict(format=2), 1), (dict(format=-1), 1),
    (dict(page_stride=4 * 64 * 128 - 16), 1), (dict(page_stride=4 * 64 * 128 + 8), 1),
    (dict(page_stride=1 << 40), 1), (dict(scale_page_stride=4 * 64 - 4), 1),
    (dict(scale_page_stride=4 * 64 + 2), 1),
]
BAD_POINTERS = [(dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1),
                (dict(v=FAKE + 2), 1), (dict(k_scale=None), 1), (dict(v_scale=FAKE + 4), 1)]


@pytest.mark.parametrize("kw,code", BAD_CACHES + BAD_POINTERS)
def test_bad_caches(lib, kw, code):
    c = cache(**kw)
    st = 4 * 128 if kw.get("head_dim", 128) == 128 else 4096
    assert lib.ds_cache_write(c, FAKE, st, FAKE, st, FAKE, 5, None) == code
    assert lib.ds_cache_read(c, FAKE, 5, FAKE, FAKE, None) == code
    a = paged(cache=c)
    if (kw, code) in BAD_CACHES:
        assert lib.ds_paged_attn_workspace_size(a) == 0
    assert lib.ds_paged_attention(a, FAKE, FAKE, BIG, None) == code
    n = norm_rope(n_kv_heads=c.n_kv_heads, head_dim=c.head_dim)
    assert lib.ds_qk_norm_rope_write(n, FAKE, st, c, FAKE, FAKE, None) == code


def test_scales_are_ignored_in_bf16(lib):
    c = cache(format=0, k_scale=None, v_scale=None, scale_page_stride=0)
    assert lib.ds_cache_write(c, None, 0, None, 0, None, 0, None) == 0    # nothing to do
    assert lib.ds_cache_read(c, None, 0, None, None, None) == 0


def test_cache_write_and_read_arguments(lib):
    c, st = cache(), 4 * 128
    w = lib.ds_cache_write
    assert w(None, FAKE, st, FAKE, st, FAKE, 5, None) == 1
    for args in ((None, st, FAKE, st, FAKE, 5), (FAKE + 8, st, FAKE, st, FAKE, 5),
                 (FAKE, st - 8, FAKE, st, FAKE, 5), (FAKE, st + 4, FAKE, st, FAKE, 5),
                 (FAKE, st, None, st, FAKE, 5), (FAKE, st, FAKE, 0, FAKE, 5),
                 (FAKE, st, FAKE, -st, FAKE, 5), (FAKE, st, FAKE, st, None, 5),
                 (FAKE, st, FAKE, st, FAKE + 2, 5), (FAKE, st, FAKE, st, FAKE, -1),
                 (FAKE, st, FAKE, st, FAKE, (1 << 24) + 1)):
        assert w(c, *args, None) == 1, args
    r = lib.ds_cache_read
    for args in ((None, 5, FAKE, FAKE), (FAKE, -1, FAKE, FAKE), (FAKE, 5, None, FAKE),
                 (FAKE, 5, FAKE, FAKE + 8), (FAKE + 1, 5, FAKE, FAKE)):
        assert r(c, *args, None) == 1, args


def norm_rope(**kw):
    from q4_moe_speculative_gb300 import _native as N
    d = dict(n_tokens=6, n_heads=16, n_kv_heads=4, head_dim=128, rotary_dim=64, interleaved=0,
             eps=1e-6, q=FAKE, q_stride=None, k=FAKE, k_stride=None, q_weight=FAKE,
             k_weight=FAKE, positions=FAKE, freqs=FAKE)
    d.update(kw)
    for s, h in (("q_stride", "n_heads"), ("k_stride", "n_kv_heads")):
        if d[s] is None:
            d[s] = max(0, d[h] * d["head_dim"])
    return N.DsNormRopeArgs(*[d[f] for f, _ in N.DsNormRopeArgs._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), 1), (dict(n_tokens=(1 << 24) + 1), 1), (dict(n_heads=0), 1),
    (dict(n_heads=257), 1), (dict(n_kv_heads=0), 1), (dict(n_kv_heads=300), 1),
    (dict(head_dim=80), 2), (dict(head_dim=-1), 1), (dict(rotary_dim=-16), 1),
    (dict(rotary_dim=144), 1), (dict(rotary_dim=24), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(q=FAKE + 2), 1), (dict(q_stride=16 * 128 - 8), 1),
    (dict(k_stride=4 * 128 + 4), 1), (dict(q_weight=FAKE + 2), 1), (dict(k_weight=FAKE + 8), 1),
    (dict(positions=None), 1), (dict(freqs=None), 1), (dict(freqs=FAKE + 4), 1),
])
def test_norm_rope_arguments(lib, kw, code):
    a = norm_rope(**kw)
    assert lib.ds_qk_norm_rope(a, FAKE, FAKE, None) == code
    assert lib.ds_qk_norm_rope_write(a, FAKE, 4 * 128, cache(), FAKE, FAKE, None) == code


def test_norm_rope_outputs_and_caches(lib):
    f, w = lib.ds_qk_norm_rope, lib.ds_qk_norm_rope_write
    a = norm_rope()
    assert f(None, FAKE, FAKE, None) == 1
    assert f(a, None, FAKE, None) == 1 and f(a, FAKE, FAKE + 8, None) == 1
    other = FAKE << 1
    strided = norm_rope(q=other, q_stride=24 * 128)    # in place only when contiguous
    assert f(strided, other, FAKE, None) == 1
    assert w(strided, FAKE, 4 * 128, cache(), FAKE, other, None) == 1
    strided = norm_rope(k=other, k_stride=24 * 128)
    assert f(strided, FAKE, other, None) == 1
    assert w(a, FAKE, 4 * 128, cache(n_kv_heads=2, page_stride=1 << 16), FAKE, FAKE, None) == 1
    assert w(a, FAKE, 4 * 128, cache(head_dim=64), FAKE, FAKE, None) == 1
    assert w(a, None, 4 * 128, cache(), FAKE, FAKE, None) == 1
    assert w(a, FAKE, 4 * 128 - 8, cache(), FAKE, FAKE, None) == 1
    assert w(a, FAKE, 4 * 128, cache(), None, FAKE, None) == 1
    assert w(a, FAKE, 4 * 128, cache(), FAKE, None, None) == 1
    none = norm_rope(n_tokens=0, q=None, k=None, positions=None)
    assert f(none, None, None, None) == 0
    assert w(none, None, 0, cache(), None, None, None) == 0


def paged(**kw):
    from q4_moe_speculative_gb300 import _native as N
    d = dict(n_seqs=3, n_rows=6, n_heads=32, max_pages=128, scale=0.1, q=FAKE, cache=cache(),
             page_table=FAKE, lengths=FAKE)
    d.update(kw)
    return N.DsPagedAttnArgs(*[d[f] for f, _ in N.DsPagedAttnArgs._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), 1), (dict(n_seqs=4097), 1), (dict(n_rows=0), 1), (dict(n_rows=9), 1),
    (dict(n_heads=0), 1), (dict(n_heads=30), 1), (dict(n_heads=-4), 1), (dict(max_pages=0), 1),
    (dict(max_pages=(1 << 18) + 1), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(scale=3e38), 1), (dict(n_heads=4 * 22), 2),
    (dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(page_table=None), 1),
    (dict(page_table=FAKE + 1), 1), (dict(lengths=None), 1), (dict(lengths=FAKE + 2), 1),
])
def test_paged_attention_arguments(lib, kw, code):
    a = paged(**kw)
    assert lib.ds_paged_attention(a, FAKE, FAKE, BIG, None) == code
    pointers = {"q", "page_table", "lengths"} & set(kw)
    assert (lib.ds_paged_attn_workspace_size(a) > 0) == bool(pointers)


def test_paged_attention_workspace(lib):
    a = paged()
    need = lib.ds_paged_attn_workspace_size(a)
    assert need > 0 and need % 256 == 0
    f = lib.ds_paged_attention
    assert f(a, FAKE, FAKE, need - 1, None) == 3
    assert f(a, FAKE, None, need, None) == 3 and f(a, FAKE, FAKE + 128, need, None) == 3
    assert f(a, None, FAKE, need, None) == 1 and f(a, FAKE + 4, FAKE, need, None) == 1
    assert f(None, FAKE, FAKE, need, None) == 1
    assert lib.ds_paged_attn_workspace_size(None) == 0
    none = paged(n_seqs=0, q=None, page_table=None, lengths=None)
    assert lib.ds_paged_attn_workspace_size(none) == 0
    assert f(none, None, None, 0, None) == 0


def test_q4_project_arguments(lib):
    from q4_moe_speculative_gb300 import _native as N
    w = N.DsQ4Tiled(FAKE)
    p = lib.ds_q4_project
    assert p(None, 64, 512, FAKE, 6, FAKE, None) == 1
    assert p(N.DsQ4Tiled(None), 64, 512, FAKE, 6, FAKE, None) == 1
    assert p(N.DsQ4Tiled(FAKE + 8), 64, 512, FAKE, 6, FAKE, None) == 1
    for rows, K, R in ((0, 512, 6), (8, 512, 6), (40, 512, 6), ((1 << 24) + 16, 512, 6),
                       (64, 0, 6), (64, 96, 6), (64, 65600, 6), (64, 512, 0), (64, 512, 9)):
        assert p(w, rows, K, FAKE, R, FAKE, None) == 1, (rows, K, R)
    assert p(w, 64, 512, FAKE + 8, 6, FAKE, None) == 1
    assert p(w, 64, 512, FAKE, 6, FAKE + 2, None) == 1
    assert p(w, 64, 512, None, 6, FAKE, None) == 1 and p(w, 64, 512, FAKE, 6, None, None) == 1


# ------------------------------------------------------------------------------ the binding
def test_the_binding_refuses_host_tensors_and_wrong_shapes(lib):
    import q4_moe_speculative_gb300 as dsm
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c = dsm.PagedCache.zeros(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        dsm.cache_read(c, i32(3))
    with pytest.raises(ValueError):
        dsm.cache_write(c, bf(3, 2, 64), bf(3, 2, 64), i32(3))
    with pytest.raises(ValueError):
        dsm.paged_attention(bf(1, 1, 2, 64), c, i32(1, 2), i32(1))
    with pytest.raises(ValueError):
        dsm.qk_norm_rope(bf(3, 2, 64), bf(3, 2, 64), None, None)
    with pytest.raises(ValueError):
        dsm.q4_project(torch.zeros(1, 1, 576, dtype=torch.uint8), bf(1, 64))
    with pytest.raises(ValueError):
        dsm.q4_project(torch.zeros(1, 576, dtype=torch.uint8), bf(1, 64))


def test_the_binding_refuses_what_is_no_tensor():
    import q4_moe_speculative_gb300 as dsm
    dev, bf = torch.device("cpu"), torch.bfloat16
    for bad in (None, [1, 2], 3):
        with pytest.raises(TypeError):
            dsm._need_on(bad, "lengths", torch.int32, (2,), dev)
        with pytest.raises(TypeError):
            dsm._token_rows(bad, "k", (2, 1, 64), dev)
        with pytest.raises(TypeError):
            dsm.q4_project(bad, torch.zeros(1, 64, dtype=bf))


def test_page_strides_of_a_cache():
    from q4_moe_speculative_gb300 import PagedCache
    st = PagedCache._stride
    dev = torch.device("cpu")
    pool = torch.zeros(5, 2, 3, 16, 64, dtype=torch.bfloat16)
    for t in (pool[:, 0], pool[:, 0].transpose(2, 3)):
        with pytest.raises(ValueError):     # a host tensor; and pages that are not contiguous
            st(t, "k", torch.bfloat16, t.shape, dev)
    with pytest.raises(TypeError):
        st(None, "k_scale", torch.float32, (5, 3, 16), dev)


def test_rope_frequencies_on_the_host():
    import math
    from q4_moe_speculative_gb300 import rope_frequencies
    f = rope_frequencies(8, base=100.0, device="cpu")
    want = [round(100.0 ** (-i / 4) / (2 * math.pi) * 2.0 ** 64) for i in range(4)]
    assert all(abs(a - b) <= 2 ** 12 for a, b in zip(f.tolist(), want))
    assert rope_frequencies(0, device="cpu").shape == (0,)
    # half a turn is the same either way round, a whole turn is none
    got = rope_frequencies(inv_freq=[math.pi, -math.pi, 2 * math.pi, 0.0], device="cpu")
    assert got.tolist() == [-(1 << 63), -(1 << 63), 0, 0]
    for bad in (dict(rotary_dim=3), dict(rotary_dim=-2), dict(), dict(inv_freq=[math.inf]),
                dict(rotary_dim=6, inv_freq=[1.0])):
        with pytest.raises(ValueError):
            rope_frequencies(device="cpu", **bad)
