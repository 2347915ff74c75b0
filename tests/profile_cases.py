"""Small workloads that run one kernel family a few times, for single-kernel ncu captures.

    python tests/profile_cases.py moe      # one verify layer (H 4096, 96 + 1 experts, I 1024, R 6)
    python tests/profile_cases.py select   # block select, 43 layers x 6 rows x 16,000 blocks
    python tests/profile_cases.py q8       # paired Q8 projection, 16384 x 4096, R 6
    python tests/profile_cases.py attn     # sparse attention, 43 layers x 6 rows x 512 blocks
    python tests/profile_cases.py accept   # acceptance, 8 steps x 6 rows x 129,280 tokens
    python tests/profile_cases.py paged_few   # paged attention, 8 x 6 rows x 32/8 heads, 16k, Q8
    python tests/profile_cases.py paged_long  # paged attention, 1 x 6 rows x 16/1 heads, 300k, bf16
    python tests/profile_cases.py rows     # norms and rotation of 16,384 tokens x 32 + 8 heads,
                                           # then a Q8 cache's write and read of 32,768 x 8 heads
    python tests/profile_cases.py q4       # Q4 projection, 129,280 x 4096, R 6

Each case holds a few GB on the device at most, with weights / keys larger than L2, and
runs its call `--reps` times (default 4) on synthetic inputs, then checks the workspace
status. Not a test module (no test_ prefix); measurement infrastructure.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

import synth  # noqa: E402
import q4_moe_speculative_gb300 as dsm  # noqa: E402


def run(case: str, reps: int) -> None:
    dev = torch.device("cuda", 0)
    if case == "moe":
        shape = synth.MoeShape(H=4096, E=96, I=1024, k=8)
        layer = dsm.MoeLayer.from_dict(synth.moe_layer(shape, seed=1, device=dev), shape.k)
        x = synth.activations(6, shape.H, seed=2, device=dev)
        ws = torch.empty(dsm.moe_workspace_size(layer, 6), dtype=torch.uint8, device=dev)
        for _ in range(reps):
            dsm.moe_verify_forward(layer, x, workspace=ws)
    elif case == "select":
        sh = synth.SELECT_64K
        d = synth.select_inputs(sh, seed=1, device=dev)
        args = (d["keys"], d["q"], d["head_w"], d["mask"], d["limit"], sh.topk)
        ws = torch.empty(dsm.select_workspace_size(*args), dtype=torch.uint8, device=dev)
        for _ in range(reps):
            dsm.select_blocks(*args, workspace=ws)
    elif case == "q8":
        qs, sc = synth.q8_matrix(16384, 4096, seed=1, device=dev)
        tiles = dsm.q8_tile(qs, sc)
        x = synth.activations(6, 4096, seed=2, device=dev)
        ws = torch.empty(256, dtype=torch.uint8, device=dev)
        for _ in range(reps):
            dsm.q8_project(tiles, x, workspace=ws)
    elif case == "attn":
        T = 75000 * 4
        a = synth.attention_inputs(43, 6, 16, T, seed=1, device=dev)
        rng = np.random.default_rng(2)
        sel = np.sort(np.stack([rng.choice(75000, size=512, replace=False) for _ in range(258)]),
                      axis=1).astype(np.int32).reshape(43, 6, 512)
        st = torch.from_numpy(sel).to(dev)
        ws = None
        for _ in range(reps):
            dsm.sparse_attention(a["q"], a["k"], a["v"], st)
    elif case == "accept":
        d = synth.verify_inputs(8, 6, synth.VOCAB, seed=1)
        t = {k: torch.from_numpy(np.ascontiguousarray(d[k])).to(dev)
             for k in ("logits", "qd", "draft", "u_acc", "u_res")}
        ws = None
        for _ in range(reps):
            dsm.verify_greedy(t["logits"], t["draft"])
            dsm.verify_sample(t["logits"], 1.0, t["qd"], t["draft"], t["u_acc"], t["u_res"])
    elif case in ("paged_few", "paged_long"):
        B, R, Hq, Hkv, n, q8 = (8, 6, 32, 8, 16000, True) if case == "paged_few" else (
            1, 6, 16, 1, 300000, False)
        pages = -(-n // 64)
        cache = dsm.PagedCache.zeros(B * pages, Hkv, 64, 128, q8=q8, device=dev)
        rows = B * pages * 64
        for at in range(0, rows, 1 << 16):   # keys and values by the cache's own write
            slots = torch.arange(at, min(at + (1 << 16), rows), dtype=torch.int32, device=dev)
            dsm.cache_write(cache, *(torch.randn(len(slots), Hkv, 128, device=dev).bfloat16()
                                     for _ in range(2)), slots)
        table = torch.randperm(B * pages, device=dev).to(torch.int32).reshape(B, pages)
        lengths = torch.full((B,), n, dtype=torch.int32, device=dev)
        q = torch.randn(B, R, Hq, 128, device=dev).bfloat16()
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device=dev)
        for _ in range(reps):
            dsm.paged_attention(q, cache, table, lengths, workspace=ws)
    elif case == "rows":
        T = 16384
        q, k = (torch.randn(T, h, 128, device=dev).bfloat16() for h in (32, 8))
        w = torch.ones(128, dtype=torch.bfloat16, device=dev)
        pos = torch.arange(T, dtype=torch.int32, device=dev)
        freqs = dsm.rope_frequencies(128, device=dev)
        cache = dsm.PagedCache.zeros(512, 8, 64, 128, q8=True, device=dev)
        kv = torch.randn(2, 2 * T, 8, 128, device=dev).bfloat16()
        slots = torch.randperm(2 * T, device=dev).to(torch.int32)
        ws = None
        for _ in range(reps):
            dsm.qk_norm_rope(q, k, pos, freqs, q_weight=w, k_weight=w)
            dsm.cache_write(cache, kv[0], kv[1], slots)
            dsm.cache_read(cache, slots)
    elif case == "q4":
        rows, K = 129280, 4096
        tiles = dsm.q4_tile(
            torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=dev),
            (torch.rand(rows, K // 32, device=dev) * 0.01).half())
        x = synth.activations(6, K, seed=2, device=dev)
        ws = None
        for _ in range(reps):
            dsm.q4_project(tiles, x)
    else:
        raise SystemExit(f"unknown case {case}")
    torch.cuda.synchronize()
    if ws is not None:
        assert dsm.workspace_status(ws) == 0
    print(f"{case}: {reps} runs ok")


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("case")
    ap.add_argument("--reps", type=int, default=4)
    args = ap.parse_args()
    run(args.case, args.reps)
