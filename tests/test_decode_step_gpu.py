"""One token of six sequences that share a prompt, from the residual stream to the drawn tokens, by the
operators as a server calls them: block norms, Q4 projections, norms and rotation with the cache's
write, attention over the shared prompt, the MoE layer, and the draw. Each operator's output is held
against 64 bits on the inputs that it got; the whole step is captured and replayed."""
import pytest
import torch

import paged_ref as ref
import synth
import q4_moe_speculative_gb300 as dsm
import test_block_norm_gpu as norms
import test_prefix_attn_gpu as prefix
import test_sample_gpu as draws

pytestmark = pytest.mark.gpu

DEV = "cuda"
H, HQ, KV, D, V, PAGE = synth.TINY_MOE.H, 8, 2, 64, 1008, 16
B, PROMPT = 6, 300


class Model:
    def __init__(self, q8):
        g = torch.Generator()
        g.manual_seed(3)

        def q4(rows, K):
            qs = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
            sc = (torch.rand(rows, K // 32, generator=g) * 0.02 + 0.005).to(torch.float16)
            return dsm.q4_tile(qs.to(DEV), sc.to(DEV))

        def vec(n):
            return (1 + 0.2 * torch.randn(n, generator=g)).to(torch.bfloat16).to(DEV)

        self.qkv, self.o, self.vocab = q4((HQ + 2 * KV) * D, H), q4(H, HQ * D), q4(V, H)
        self.n1, self.n2, self.n3, self.p1, self.p2 = (vec(H) for _ in range(5))
        self.qn, self.kn = vec(D), vec(D)
        self.gate = vec(H)
        self.moe = dsm.MoeLayer.from_dict(synth.moe_layer(synth.TINY_MOE, seed=5, device=DEV), 2)
        self.freqs = dsm.rope_frequencies(D, device=DEV)
        pages = 40
        self.cache = dsm.PagedCache.zeros(pages, KV, PAGE, D, q8=q8, device=DEV)
        slots = torch.arange(pages * PAGE, dtype=torch.int32, device=DEV)
        dsm.cache_write(self.cache, *(torch.randn(pages * PAGE, KV, D, generator=g).to(torch.bfloat16).to(DEV)
                                      for _ in range(2)), slots)
        order = torch.randperm(pages, generator=g).to(torch.int32).to(DEV)
        self.ptable = order[None, :19].contiguous()
        self.plens = torch.tensor([PROMPT], dtype=torch.int32, device=DEV)
        self.table = order[19:19 + 2 * B].view(B, 2).contiguous()
        self.lengths = torch.tensor([1, 5, 16, 17, 9, 30], dtype=torch.int32, device=DEV)

    def step(self, x, u, keep=None):
        """Next tokens of residual rows x [B, H] (fp32); keep: every operator's inputs and outputs."""
        note = (lambda **k: keep.update(k)) if keep is not None else (lambda **k: None)
        at = self.lengths.long() - 1
        slots = (self.table.long()[torch.arange(B, device=DEV), at // PAGE] * PAGE + at % PAGE).int()
        _, h = dsm.block_norm(x, weight=self.n1)
        qkv = dsm.q4_project(self.qkv, h).view(B, HQ + 2 * KV, D)
        q = dsm.qk_norm_rope_write(qkv[:, :HQ], qkv[:, HQ:HQ + KV], qkv[:, HQ + KV:],
                                   (PROMPT + at).int(), self.freqs, self.cache, slots,
                                   q_weight=self.qn, k_weight=self.kn)
        att = dsm.prefix_attention(q[:, None], self.cache, self.ptable, self.plens, self.table,
                                   self.lengths)
        y = dsm.q4_project(self.o, att.view(B, HQ * D))
        x1, h1 = dsm.block_norm(x, y, weight=self.n2, post_weight=self.p1, gate=self.gate)
        z, _, _ = dsm.moe_verify_forward(self.moe, h1)
        x2, h2 = dsm.block_norm(x1, z, weight=self.n3, post_weight=self.p2, y_scale=0.5)
        logits = dsm.q4_project(self.vocab, h2)
        tokens, probs = dsm.sample(logits, u, temperature=0.8, top_k=40, top_p=0.9, min_p=0.02)
        note(x=x, h=h, q=q, att=att, y=y, x1=x1, h1=h1, z=z, x2=x2, h2=h2, logits=logits)
        return tokens, probs, x2


@pytest.mark.parametrize("q8", [False, True])
def test_a_step_of_sequences_that_share_a_prompt(q8):
    m = Model(q8)
    x = norms.rows(B, H, torch.float32, 7, 2.0)
    u = torch.rand(B, generator=torch.Generator().manual_seed(8), dtype=torch.float64).to(DEV)
    k = {}
    tokens, probs, x2 = m.step(x, u, k)
    norms.check(x, weight=m.n1, got=(x, k["h"]))
    prefix.check(k["q"][:, None].contiguous(), m.cache, m.ptable, m.plens, m.table, m.lengths,
                 got=k["att"])
    norms.check(x, k["y"], m.n2, m.p1, m.gate, got=(k["x1"], k["h1"]))
    norms.check(k["x1"], k["z"], m.n3, m.p2, ys=0.5, got=(x2, k["h2"]))
    for tiles, a, out in ((m.o, k["att"].view(B, -1), k["y"]), (m.vocab, k["h2"], k["logits"])):
        want = a.cpu().double() @ ref.q4_weights(tiles).t()
        mag = a.cpu().double().abs() @ ref.q4_weights(tiles).abs().t()
        tol = ref.HALF_BF16 * want.abs() + mag * (a.shape[1] * 2 * ref.U32)
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
    assert draws.check(k["logits"], u, T=0.8, k=40, p=0.9, mp=0.02) == tokens.cpu().tolist()

    # the same step captured: other residual rows, other uniforms, longer contexts
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.step(x, u)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(x, u)
    for seed in (11, 12):
        x.copy_(norms.rows(B, H, torch.float32, seed, 2.0))
        u.copy_(torch.rand(B, generator=torch.Generator().manual_seed(seed), dtype=torch.float64))
        m.lengths.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = m.step(x, u)     # (writes the same keys and values again)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_steps_at_once():
    # two streams, each with its own model and cache
    ms = [Model(False), Model(True)]
    xs = [norms.rows(B, H, torch.float32, 20 + i, 2.0) for i in range(2)]
    u = torch.full((B,), 0.4, dtype=torch.float64, device=DEV)
    want = [m.step(x, u) for m, x in zip(ms, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ms[i].step(xs[i], u))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for step in g:
            assert all(torch.equal(a, b) for a, b in zip(step, w))
