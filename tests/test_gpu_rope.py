"""Rotary positions and the append to the paged cache against the definition in 64 bits (needs an MI355X).

An output c x1 - s x2 is off by at most: 4 half steps of fp32 in each of c and s (the angle in turns rounded to fp32: half
a step of at most half a turn, 2 pi 2^-26 < 2 half steps; sine and cosine within 2 of their last place; the factor), one for each product and one for the sum, all
relative to mscale (|x1| + |x2|), and half a step of the output's type:
    |y - y64| <= 8 * 2^-24 mscale (|x1| + |x2|) + half step * |y64|   (+ 2^-25 absolute for fp16's smallest values)."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import lut_logits_amd as la
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def check(y, x, positions, freqs, mscale, layout, out, inverse=False):
    want = ref.rotate(x, positions, freqs, mscale, layout, inverse)
    n = len(freqs)
    mag = np.abs(x)
    pair = mag.copy()
    i1, i2 = (np.arange(n), np.arange(n) + n) if layout == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)
    pair[..., i1] = pair[..., i2] = mag[..., i1] + mag[..., i2]
    tol = 8 * 2.0 ** -24 * mscale * pair + 1.01 * ref.HALF_STEP[out] * np.abs(want) + (2.0 ** -25 if out == "f16" else 0) + 1e-37
    err = np.abs(y.astype(np.float64) - want)
    assert (err <= tol).all(), float((err / tol).max())
    assert np.array_equal(y[..., 2 * n:].astype(np.float64), ref.round_to(x[..., 2 * n:], out))


@pytest.mark.parametrize("tokens,heads,size,rot,layout,xt,out,inverse", [
    (1, 1, 2, 2, "half", "f32", "f32", False),
    (1, 8, 256, 256, "half", "f32", "bf16", False),
    (17, 3, 64, 64, "interleaved", "bf16", "bf16", False),
    (33, 5, 80, 32, "half", "f16", "f16", True),
    (33, 5, 80, 32, "interleaved", "f32", "f32", True),
    (50, 2, 66, 66, "half", "f32", "f16", False),          # no whole 8s
    (50, 2, 66, 22, "interleaved", "bf16", "f32", False),
    (16, 1, 512, 512, "half", "f16", "bf16", False),
    (300, 7, 128, 64, "half", "bf16", "bf16", False),
])
def test_rope(tokens, heads, size, rot, layout, xt, out, inverse):
    rng = np.random.default_rng(tokens + size)
    x = ref.round_to(rng.standard_normal((tokens, heads, size)), xt)
    pos = rng.integers(0, 2_000_000, tokens).astype(np.int32)
    pos[0] = 0
    freqs, mscale = la.rope_freqs(rot, scaling="yarn", factor=8.0, device="cpu")
    y = la.rope(dev(x, T[xt]), dev(pos), freqs.cuda(), layout, mscale, inverse, out_dtype=T[out])
    check(host(y.float()), x, pos, freqs.numpy(), mscale, layout, out, inverse)


def test_far_positions_and_negative():
    """Angles at the largest positions are right to the last bits, and negative positions turn back."""
    x = np.ones((4, 1, 64))
    pos = np.array([2 ** 31 - 1, 2 ** 30 + 1, -5, -(2 ** 31)], np.int32)
    freqs, _ = la.rope_freqs(64, device="cpu")
    y = host(la.rope(dev(x, torch.float32), dev(pos), freqs.cuda()))
    # (the product position * frequency itself has 53 bits: 2^31 * 2^-53 radians)
    check(y, x, pos, freqs.numpy(), 1.0, "half", "f32")


def test_in_place_and_strided():
    """Views of a stacked projection, and rotation in x's own memory; the rest of the rows keeps its bits."""
    rng = np.random.default_rng(3)
    stacked = dev(rng.standard_normal((40, 3 * 4 * 64 + 8)), torch.float32)
    before = stacked.clone()
    x = stacked[:, 64:64 + 4 * 64].view(40, 4, 64)
    pos = dev(rng.integers(0, 5000, 40).astype(np.int32))
    freqs, _ = la.rope_freqs(64)
    want = la.rope(x.contiguous(), pos, freqs)
    fresh = la.rope(x, pos, freqs)
    assert torch.equal(fresh, want)
    la.rope(x, pos, freqs, out=x)
    assert torch.equal(x.contiguous(), want)
    assert torch.equal(stacked[:, :64], before[:, :64]) and torch.equal(stacked[:, 64 + 256:], before[:, 64 + 256:])


@pytest.mark.parametrize("size,rot,layout", [(254, 254, "half"), (250, 100, "interleaved"), (66, 22, "half"), (20, 20, "interleaved")])
def test_sizes_of_no_whole_eights(size, rot, layout):
    """Out of place the last items of a head overlap the ones before, in place they do not: the same bits."""
    rng = np.random.default_rng(size)
    x = ref.round_to(rng.standard_normal((70, 5, size)), "bf16")
    pos = rng.integers(0, 5000, 70).astype(np.int32)
    freqs, _ = la.rope_freqs(rot, device="cpu")
    t = dev(x, torch.bfloat16)
    y = la.rope(t, dev(pos), freqs.cuda(), layout)
    check(host(y.float()), x, pos, freqs.numpy(), 1.0, layout, "bf16")
    assert la.rope(t, dev(pos), freqs.cuda(), layout, out=t) is t
    assert torch.equal(t, y)


def test_gradient():
    """inverse=True is the gradient: <rope(x), g> = <x, rope^-1(g)>, against differences of the formula in 64 bits too."""
    rng = np.random.default_rng(4)
    x, g, e = (ref.round_to(rng.standard_normal((9, 2, 48)), "f32") for _ in range(3))
    pos = rng.integers(0, 9000, 9).astype(np.int32)
    freqs, _ = la.rope_freqs(32, device="cpu")
    for layout in ("half", "interleaved"):
        back = host(la.rope(dev(g, torch.float32), dev(pos), freqs.cuda(), layout, 1.25, inverse=True)).astype(np.float64)
        check(back, g, pos, freqs.numpy(), 1.25, layout, "f32", True)
        f = lambda v: (ref.rotate(v, pos, freqs.numpy(), 1.25, layout) * g).sum()  # noqa: E731
        # the map is linear: a central difference is exact up to 64-bit rounding
        slope = (f(x + e) - f(x - e)) / 2
        assert abs(slope - (back * e).sum()) <= 8 * 2.0 ** -24 * 1.25 * 2 * (np.abs(g) @ np.ones(48)).sum() * np.abs(e).max()


APPEND = [
    # new, lens, heads, kv, size, rot, page, layout, in type, cache type, own positions
    ([1], [1], 1, 1, 64, 64, 16, "half", "f32", "bf16", False),
    ([1, 1, 1], [5, 64, 17], 8, 4, 256, 256, 16, "half", "f32", "bf16", True),
    ([40, 0, 1, 33], [40, 9, 100, 65], 6, 2, 128, 64, 32, "interleaved", "bf16", "bf16", False),
    ([16, 16], [16, 48], 4, 4, 80, 40, 16, "half", "f16", "f16", False),
    ([300], [1000], 3, 1, 66, 22, 64, "interleaved", "f32", "f16", True),
    ([130, 7], [130, 261], 2, 2, 64, 64, 128, "half", "bf16", "f16", False),
]


@pytest.mark.parametrize("new,lens,heads,kv,size,rot,page,layout,xt,ct,own_pos", APPEND)
def test_append(new, lens, heads, kv, size, rot, page, layout, xt, ct, own_pos):
    rng = np.random.default_rng(sum(lens) + size)
    b = ref.Batch(rng, new, lens, page)
    q, k, v = (ref.round_to(rng.standard_normal((b.tokens, h, size)), xt) for h in (heads, kv, kv))
    pos = rng.integers(0, 1_000_000, b.tokens).astype(np.int32) if own_pos else b.places()
    freqs, _ = la.rope_freqs(rot, device="cpu")
    cache = la.KVCache(torch.full((b.pages, kv, page, size), 3.0, dtype=T[ct], device="cuda"),
                       torch.full((b.pages, kv, size, page), 3.0, dtype=T[ct], device="cuda"))
    # a stacked projection's views, and rows behind the last sequence
    width = (heads + 2 * kv) * size
    stacked = torch.zeros((b.tokens + 2, width), dtype=T[xt], device="cuda")
    parts = [stacked[:, i:i + n * size].view(-1, n, size) for i, n in ((0, heads), (heads * size, kv), ((heads + kv) * size, kv))]
    for p, a in zip(parts, (q, k, v)):
        p[:b.tokens] = dev(a, T[xt])
    out = torch.full((b.tokens + 2, heads, size), -4.0, dtype=T[ct], device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.cat([dev(pos), torch.zeros(2, dtype=torch.int32, device="cuda")])
    la.rope_append(*parts, cache, dev(b.cu_q), dev(np.array(lens, np.int32)), dev(b.table), freqs.cuda(), layout, 1.0,
                   at if own_pos else None, out, bad)
    assert int(bad) == 0
    check(host(out[:b.tokens].float()), q, pos, freqs.numpy(), 1.0, layout, ct)
    assert bool((out[b.tokens:] == -4).all())
    kp, vp = host(cache.k.float()), host(cache.v.float())
    got_k, got_v = np.zeros((b.tokens, kv, size)), np.zeros((b.tokens, kv, size))
    seen = np.zeros((b.pages, page), bool)
    for s, (m, n) in enumerate(zip(new, lens)):
        for i in range(m):
            j = n - m + i
            p, o = b.table[s, j // page], j % page
            got_k[b.cu_q[s] + i], got_v[b.cu_q[s] + i] = kp[p, :, o], vp[p, :, :, o]
            seen[p, o] = True
    check(got_k, k, pos, freqs.numpy(), 1.0, layout, ct)
    assert np.array_equal(got_v, ref.round_to(v, ct))
    # every other place keeps its bits
    assert (kp.transpose(0, 2, 1, 3)[~seen] == 3).all() and (vp.transpose(0, 3, 1, 2)[~seen] == 3).all()


def test_append_without_pages():
    """Places beyond the table, page ids that are none, and lengths below the number of new tokens: nothing is stored for
    them, they are counted, and the queries are rotated all the same."""
    rng = np.random.default_rng(7)
    heads, kv, size, page = 2, 1, 64, 16
    new, lens = [20, 5, 3], [40, 2, 16]
    cu = np.array([0, 20, 25, 28], np.int32)
    table = np.array([[1, 0], [2, 2], [99, -1]], np.int32)   # sequence 0: places 32.. beyond the table; 2: page 99 of 3
    q, k, v = (ref.round_to(rng.standard_normal((28, h, size)), "f32") for h in (heads, kv, kv))
    freqs, _ = la.rope_freqs(size, device="cpu")
    cache = la.KVCache(torch.zeros((3, kv, page, size), dtype=torch.bfloat16, device="cuda"),
                       torch.zeros((3, kv, size, page), dtype=torch.bfloat16, device="cuda"))
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = la.rope_append(*(dev(a, torch.float32) for a in (q, k, v)), cache, dev(cu), dev(np.array(lens, np.int32)), dev(table),
                         freqs.cuda(), bad_pages=bad)
    places = np.concatenate([np.arange(20, 40), np.arange(-3, 2), np.arange(13, 16)])
    assert int(bad) == 8 + 3 + 3      # places 32..39, -3..-1, and all three of page 99
    check(host(out.float()), q, places, freqs.numpy(), 1.0, "half", "bf16")
    stored = host(cache.v.float()).transpose(0, 3, 1, 2)     # [page][slot][kv][size]
    assert np.array_equal(stored[0, 4:16], ref.round_to(v[0:12], "bf16"))   # places 20..31: second page of sequence 0
    assert np.array_equal(stored[2, 0:2], ref.round_to(v[23:25], "bf16"))
    assert (stored[1] == 0).all() and (stored[0, :4] == 0).all() and (stored[2, 2:] == 0).all()


def test_empty():
    freqs, _ = la.rope_freqs(64)
    assert la.rope(torch.empty((0, 2, 64), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), freqs).shape == (0, 2, 64)
    cache = la.KVCache.empty(1, 1, 16, 64)
    e = torch.empty((0, 1, 64), device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert la.rope_append(e, e, e, cache, z, z[:0], z[:0].view(0, 1), freqs).shape == (0, 1, 64)
