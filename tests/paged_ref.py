"""Plain implementations in 64 bits of the paged-cache operators and the Q4 projection, for
the tests: written from the formulas of include/dsmoe.h with torch on the CPU."""
import math

import numpy as np
import torch

HALF_BF16 = 2.0 ** -8    # a rounding to bf16 is off by at most this, relative to the value
U32 = 2.0 ** -24         # and one to fp32 by this


def normal(*shape, seed, sigma=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(torch.bfloat16)


def turn_steps(rotary, base=10000.0):
    """(radians per position as fp64, turns per position in units of 2^-64)."""
    f = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1))
    return f, torch.tensor([round(x / (2 * math.pi) * 2.0 ** 64) for x in f.tolist()],
                           dtype=torch.int64)


def norm_rope(x, weight, positions, inv_freq, eps, interleaved):
    """(result, the sum of magnitudes of the two values each result was made from) of
    x [T, heads, D], in fp64."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    mag = x.abs()
    n = 2 * inv_freq.numel()
    if n == 0:
        return x, mag
    a = positions.double()[:, None, None] * inv_freq
    c, s = torch.cos(a), torch.sin(a)
    out, both = x.clone(), mag.clone()
    i = torch.arange(n // 2)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + n // 2)
    u, v = x[..., i], x[..., j]
    out[..., i] = u * c - v * s
    out[..., j] = v * c + u * s
    both[..., i] = both[..., j] = u.abs() + v.abs()
    return out, both


def quantise(x):
    """(codes, fp32 scales) of rows x (bf16 values): exact. 127 x / a with a and x of 8 bits is
    either a half-integer, which fp64 holds, or further than fp64's rounding from one."""
    x = x.double().numpy()
    a = np.abs(x).max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        codes = np.where(a > 0, np.rint(127.0 * x / a), 0.0)
    scale = (a.astype(np.float32) / np.float32(127.0))[..., 0]
    bad = ~np.isfinite(a)
    codes = np.where(bad, 0.0, codes)
    return codes.astype(np.int8), np.where(bad[..., 0], np.float32("nan"), scale)


def flat(t):
    """A cache tensor [pages, heads, page, ...] by slot: [slots, heads, ...]."""
    return t.transpose(1, 2).flatten(0, 1)


def values(cache, side):
    """What the cache stands for, fp64 [slots, heads, D] on the CPU."""
    x = flat(getattr(cache, side)).cpu().double()
    if cache.q8:
        x = x * flat(getattr(cache, side + "_scale")).cpu().double()[..., None]
    return x


def attention(q, cache, table, lengths, scale):
    """(result, sum p |v|, sqrt(sum p^2 v^2), largest sum |q k| scale) in fp64 for
    q [B, R, Hq, D], with bad pages skipped."""
    q = q.cpu().double()
    B, R, H, D = q.shape
    pages, kv, page, _ = cache.k.shape
    k, v = values(cache, "k"), values(cache, "v")
    table, lengths = table.cpu(), lengths.cpu()
    out, mag, rss = (torch.zeros_like(q) for _ in range(3))
    top = 0.0
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page)
        t = torch.arange(n)
        pg = table[b][t // page].long()
        ok = (pg >= 0) & (pg < pages)
        t, slots = t[ok], (pg * page + t % page)[ok]
        for r in range(R):
            sl = slots[t < n - (R - 1 - r)]
            if not len(sl):
                continue
            for h in range(H):
                kk, vv = k[sl, h // (H // kv)], v[sl, h // (H // kv)]
                p = torch.softmax((kk @ q[b, r, h]) * scale, 0)
                out[b, r, h] = p @ vv
                mag[b, r, h] = p @ vv.abs()
                rss[b, r, h] = torch.sqrt((p * p) @ (vv * vv))
                top = max(top, float((kk.abs() @ q[b, r, h].abs()).max() * abs(scale)))
    return out, mag, rss, top


def check_attention(got, ref, n, D):
    """got bf16 against attention()'s result over at most n tokens. Per element, half a step
    of bf16 of the result, and of sum p |v|: two half steps for P (numerator and normaliser),
    twice the score's fp32 error (D products and the scaling, two units each since a tensor
    core may truncate; the exponential's 2^-21), and n sums of fp32. Over all elements: the
    same roundings are independent, so their root mean square is held to half steps of the
    result and of sqrt(sum p^2 v^2), doubled."""
    out, mag, rss, top = ref
    err = (got.cpu().double() - out).abs()
    score = top * (D + 4) * 2 * U32 + 2.0 ** -21
    tol = HALF_BF16 * out.abs() + mag * (2 * HALF_BF16 + 2 * score + n * 2 * U32)
    assert bool((err <= tol + 1e-30).all()), float((err - tol).max())
    rms = lambda x: float(torch.sqrt((x * x).mean()))  # noqa: E731
    allowed = 2 * HALF_BF16 * math.hypot(rms(out), rms(rss)) + rms(mag) * (2 * score + n * 2 * U32)
    assert rms(err) <= allowed + 1e-30, (rms(err), allowed)


def q4_weights(tiles):
    """fp64 [rows, K] of tile-major Q4 (groups of 1), by the header's byte positions."""
    U, Tk, _ = tiles.shape
    t = tiles.cpu().numpy()
    W = np.zeros((U * 16, Tk * 64))
    for row in range(16):
        g, low = row % 8, row // 8
        for k in range(64):
            block, value = k // 32, k % 32
            byte = t[:, :, 16 * (4 * g + value // 8) + 4 * (2 * block + low) + (value % 8) // 2]
            code = ((byte >> (4 * (value % 2))) & 15).astype(np.int64) - 8
            at = 512 + 8 * g + 2 * (2 * block + low)
            sc = np.ascontiguousarray(t[:, :, at:at + 2]).view(np.float16)[..., 0]
            W[row::16, k::64] = code * sc.astype(np.float64)
    return torch.from_numpy(W)
