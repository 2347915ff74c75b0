"""Q4 projections (ds_q4_project) against the 64-bit product of the tile-major weights.

Tolerance: a block of 32 exact products is summed in two tensor-core steps (32 additions of
fp32, which may truncate: two units of 2^-24 each), scaled once, and added in a chain of two
blocks for each of a warp's tiles and then of at most 16 warps: n = 32 + 2 ceil(K / 64) + 17
roundings bound it for every split, each of at most sum |W x|. Then half a step of bf16."""
import pytest
import torch

import paged_ref as ref
import synth
import q4_moe_speculative_gb300 as dsm

pytestmark = pytest.mark.gpu


def tiles_of(rows, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qs, sc = synth.q4_matrix((), rows, K, g, "cuda")
    return dsm.q4_tile(qs, sc), qs, sc


def check(y, W, x, K):
    want = x.cpu().double() @ W.t()
    size = x.cpu().double().abs() @ W.abs().t()
    n = 32 + 2 * -(-K // 64) + 17
    err = (y.cpu().double() - want).abs()
    tol = ref.HALF_BF16 * want.abs() + n * 2 * ref.U32 * size
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("rows,K,R", [
    (16, 64, 1), (16, 128, 8), (48, 192, 2), (32, 320, 3), (4096, 64, 5), (2448, 448, 4),
    (16, 8192, 6), (64, 1024, 1), (112, 4096, 3), (4096, 4096, 6), (1040, 4160, 7),
    (2048, 8192, 6), (160, 12352, 8), (16384, 256, 2), (304, 1984, 8), (32, 65536, 8)])
def test_project_matches_64_bits(rows, K, R):
    tiles, qs, sc = tiles_of(rows, K, seed=rows + K + R)
    x = synth.activations(R, K, seed=R, device="cuda")
    y = dsm.q4_project(tiles, x)
    W = ref.q4_weights(tiles)
    if rows * K <= 1 << 22:   # the tiles stand for the planar matrix they were made from
        lo, hi = qs.cpu() & 15, qs.cpu() >> 4
        plain = (torch.stack((lo, hi), -1).view(rows, K).double() - 8) * sc.cpu().double(
        ).repeat_interleave(32, 1)
        assert torch.equal(W, plain)
    check(y, W, x, K)


@pytest.mark.parametrize("rows,K", [(336, 4096), (336, 704), (64, 8192), (2432, 128)])
def test_rows_do_not_depend_on_one_another(rows, K):
    tiles, _, _ = tiles_of(rows, K, seed=3)
    x = synth.activations(8, K, seed=4, device="cuda")
    y = dsm.q4_project(tiles, x)
    assert torch.equal(y, dsm.q4_project(tiles, x))
    for r in range(8):
        assert torch.equal(dsm.q4_project(tiles, x[r:r + 1].contiguous())[0], y[r])
    assert torch.equal(dsm.q4_project(tiles, x[[5, 2, 7]].contiguous()), y[[5, 2, 7]])


def test_infinities_stay_in_their_row():
    tiles, _, _ = tiles_of(64, 256, seed=6)
    x = synth.activations(4, 256, seed=7, device="cuda")
    want = dsm.q4_project(tiles, x)
    x[1, 17] = float("inf")
    x[2, 200] = float("nan")
    y = dsm.q4_project(tiles, x)
    assert torch.equal(y[[0, 3]], want[[0, 3]])
    assert not bool(torch.isfinite(y[1]).any())
    assert bool(torch.isnan(y[2]).all())


def test_given_output_and_stream():
    tiles, _, _ = tiles_of(512, 1024, seed=8)
    x = synth.activations(6, 1024, seed=9, device="cuda")
    want = dsm.q4_project(tiles, x)
    whole = torch.full((8, 512), -3.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = dsm.q4_project(tiles, x, y=whole[:6], stream=side)
    side.synchronize()
    assert got.data_ptr() == whole.data_ptr() and torch.equal(whole[:6], want)
    assert bool((whole[6:] == -3).all())               # rows behind the last stay
    torch.cuda.synchronize()
    got = dsm.q4_project(tiles, x, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
