"""The attention operators together, as a decoder layer uses them: 4-bit projections, rotation and append, attention, output
projection; alone, in the decode loop, in graphs and on two streams (needs an MI355X).

Each stage is checked in 64 bits on the inputs that the GPU gave it, with the bounds of that stage's own tests."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import lut_logits_amd as la
import oracle
import test_gpu_composite as composite_test
from gpu_util import dev, host, to_dev
from lut_logits_amd import synth
from lut_logits_amd.composite import AttentionBlock, DecodeLoop
from test_gpu_q4 import bound as q4_bound, upload as q4_upload
from test_gpu_rope import check as rope_check

pytestmark = pytest.mark.gpu


def q4(x, m, y):
    err = np.abs(y - x @ m.dense().T)
    tol = q4_bound(m, x)
    assert (err <= tol).all(), (err / tol).max()


def attn(q, k, v, place, scale, softcap, window, got, size):
    """One token's attention in 64 bits over the rounded keys and values [len][kv][size]; the bound of the kernel of few rows."""
    b = type("B", (), dict(new=[1], lens=[place + 1], cu_q=[0, 1]))()
    want, _, mass = ref.attention(q[None], b, [k], [v], scale, softcap, window)
    dz = scale * (size + 2) * 2.0 ** -24 * float((np.abs(q).max(0) * np.abs(k).max((0, 1))).sum()) + 2.0 ** -20 * softcap
    tol = 1.02 * 2.0 ** -8 * np.abs(want) + (2 * dz + 2.0 ** -19) * mass + 1e-30
    assert (np.abs(got - want[0]) <= tol[0]).all()


@pytest.mark.parametrize("heads,kv,size,window", [(4, 2, 64, 0), (2, 1, 128, 5)])
def test_decode_loop_with_attention(heads, kv, size, window):
    cfg = synth.CONFIGS["tiny"]
    head, _, _ = synth.make_head(cfg)
    rng = np.random.default_rng(21)
    hid, inter, d, K = cfg.D, 160, 2, 64
    layers, blocks, mats = [], [], []
    for i in range(2):
        layers.append(tuple(synth.gen_matrix(rng, r, c, c // d, K, 2, (0.02, 0.005), "f32")
                            for r, c in ((inter, hid), (inter, hid), (hid, inter))))
        qkv = ref.Q4(rng, (heads + 2 * kv) * size, hid, 32, "bf16", i == 1, i == 0)
        out = ref.Q4(rng, hid, heads * size, 64, "f16", False, True)
        mats.append((qkv, out))
        blocks.append(AttentionBlock(q4_upload(qkv), q4_upload(out), heads, kv, size, window if i else 0))
    loop = DecodeLoop(to_dev(head), [tuple(to_dev(m) for m in lay) for lay in layers], softcap=cfg.softcap, max_tokens=24,
                      keep_layers=True, attention=blocks)
    freqs = loop.freqs.cpu().numpy()
    o = oracle.default()
    rms = composite_test._rms
    loop.ids[0] = 7
    tok, tokens = 7, [7]
    for t in range(20):
        loop.step(t)
        row, _ = o.decode_rows(head.codes, head.codebooks, head.cb_is_bf16, np.array([tok], np.int32), False)
        h = row.astype(np.float64) * np.sqrt(head.D)
        for i, (gate, up, down) in enumerate(layers):
            x = host(loop.att_ins[i]).astype(np.float64)
            assert np.allclose(x, rms(h), rtol=0, atol=1e-5 * np.abs(rms(h)).max())
            qkv = host(loop.att_qkv[i]).astype(np.float64)
            q4(x, mats[i][0], qkv)
            q, k, v = np.split(qkv.reshape(1, -1, size), [heads, heads + kv], axis=1)
            rope_check(host(loop.att_q[i].float()), q, [t], freqs, 1.0, "half", "bf16")
            kc = host(loop.caches[i].k.float()).astype(np.float64).transpose(0, 2, 1, 3).reshape(-1, kv, size)[:t + 1]
            vc = host(loop.caches[i].v.float()).astype(np.float64).transpose(0, 3, 1, 2).reshape(-1, kv, size)[:t + 1]
            rope_check(kc[t:].astype(np.float32), k, [t], freqs, 1.0, "half", "bf16")
            assert np.array_equal(vc[t:], ref.round_to(v, "bf16"))
            mid = host(loop.att_mid[i].float()).astype(np.float64)
            attn(host(loop.att_q[i].float()).astype(np.float64)[0], kc, vc, t, size ** -0.5, 50.0, blocks[i].window, mid[0], size)
            y = host(loop.att_outs[i]).astype(np.float64)
            q4(mid.reshape(1, -1), mats[i][1], y)
            h = h + rms(y)
            x = host(loop.ins[i])
            assert np.allclose(x, rms(h), rtol=0, atol=1e-4 * np.abs(rms(h)).max())
            _, _, _, oy = o.mlp(*((m.codes, m.codebooks, False) for m in (gate, up, down)), x)
            composite_test.check_logits(host(loop.outs[i]), oy)
            h = h + rms(host(loop.outs[i]))
        _, logits = o.logits(head.codes, head.codebooks, head.cb_is_bf16, host(loop.last), cfg.softcap)
        tok = int(loop.ids[t + 1].item())
        assert logits[0, tok] >= logits[0].max() - 2e-5 * np.abs(logits).max()
        tokens.append(tok)
    # deterministic, whatever an earlier run left in the cache; the same without the kept buffers
    assert loop.run(7, 20).cpu().tolist() == tokens
    lean = DecodeLoop(loop.head, loop.layers, softcap=cfg.softcap, max_tokens=24, attention=blocks)
    assert lean.run(7, 20).cpu().tolist() == tokens


def test_decode_loop_refusals():
    cfg = synth.CONFIGS["tiny"]
    head, _, _ = synth.make_head(cfg)
    rng = np.random.default_rng(1)
    W = q4_upload(ref.Q4(rng, 256, cfg.D, 32))
    out = q4_upload(ref.Q4(rng, cfg.D, 128, 32))
    with pytest.raises(ValueError):
        AttentionBlock(W, out, 3, 2, 64)
    with pytest.raises(ValueError):
        AttentionBlock(W, out, 4, 2, 64)
    block = AttentionBlock(W, out, 2, 1, 64)
    with pytest.raises(ValueError):
        DecodeLoop(to_dev(head), [], attention=[block])


class Layer:
    """Projections and a cache of one layer, and its attention for a batch of new tokens."""

    def __init__(self, seed, D=96, heads=4, kv=2, size=64, page=16, pages=64):
        rng = np.random.default_rng(seed)
        self.heads, self.kv, self.size = heads, kv, size
        self.wqkv = q4_upload(ref.Q4(rng, (heads + 2 * kv) * size, D, 32, "bf16", True, True))
        self.wo = q4_upload(ref.Q4(rng, D, heads * size, 64, "f32"))
        self.cache = la.KVCache.empty(pages, kv, page, size)
        self.freqs, self.mscale = la.rope_freqs(size, scaling="yarn", factor=4.0)

    def __call__(self, x, cu, lens, table, max_len=0, **kw):
        h, kv, n = self.heads, self.kv, x.shape[0]
        qkv = la.q4_matvec(self.wqkv, x).view(n, h + 2 * kv, self.size)
        where = (self.cache, cu, lens, table)
        q = la.rope_append(qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:], *where, self.freqs, mscale=self.mscale)
        o = la.paged_attn(q, *where, softcap=30.0, max_len=max_len, **kw)
        return la.q4_matvec(self.wo, o.reshape(n, h * self.size))


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def test_prompt_in_chunks_and_tokens():
    """A prompt at once, in chunks, and token by token. Batches sum in another order, so a projection near the middle of two
    bf16 numbers may round the other way: keys, values and queries differ by a step (2^-7 of their size) at most. A score then
    moves by dz <= 2 * 1.01 * 2^-7 scale sum|q||k| (the cap's slope is at most 1), a probability by a factor e^(2 dz), and an
    output by
        ((e^(2 dz) - 1) + 2^-7 + 4 * 2^-8) max|v|
    (the probabilities, a step of the values, and on both sides the roundings of the probabilities and of the output), which the
    output projection adds up with its weights' absolute values."""
    layer = Layer(3)
    x = torch.randn(130, 96, device="cuda")
    table = i32(*range(9)).view(1, 9)
    outs, caches = [], []
    for parts in ([130], [50, 1, 79], [1] * 130):
        layer.cache.k.fill_(float("nan"))
        layer.cache.v.fill_(float("nan"))
        t, y = 0, []
        for n in parts:
            y.append(layer(x[t:t + n].contiguous(), i32(0, n), i32(t + n), table))
            t += n
        outs.append(host(torch.cat(y)).astype(np.float64))
        caches.append((host(layer.cache.k[:9].float()), host(layer.cache.v[:9].float())))
    qkv = la.q4_matvec(layer.wqkv, x).view(130, 8, 64)
    q = host(la.rope(qkv[:, :4], torch.arange(130, dtype=torch.int32, device="cuda"), layer.freqs, mscale=layer.mscale)).astype(np.float64)
    k = np.nan_to_num(caches[0][0]).astype(np.float64)
    dz = 2.02 * 2.0 ** -7 * 64 ** -0.5 * float((np.abs(q).max((0, 1)) * np.abs(k).max((0, 1, 2))).sum())
    vmax = np.nanmax(np.abs(caches[0][1])).astype(np.float64)
    tol = (np.expm1(2 * dz) + 2.0 ** -7 + 4 * 2.0 ** -8) * vmax
    w = np.abs(host(la.q4_matvec(layer.wo, torch.eye(256, device="cuda"))).astype(np.float64))   # |W^T| [256][96]
    for o, (k, v) in zip(outs[1:], caches[1:]):
        for a, b in ((k, caches[0][0]), (v, caches[0][1])):
            assert np.array_equal(np.isnan(a), np.isnan(b))
            assert (np.abs(a - b)[~np.isnan(a)] <= 2.0 ** -7 * np.abs(b)[~np.isnan(b)] + 1e-6).all()
        assert (np.abs(o - outs[0]) <= 1.01 * tol * w.sum(0)).all()


def test_captured_chain_and_shared_workspace():
    """The four calls captured as one graph, replayed on growing sequences, with eager calls between the replays; a second
    graph shares the first one's workspace and runs after it."""
    layer, other = Layer(4), Layer(5)
    x, lens, table = torch.randn(2, 96, device="cuda"), i32(40, 300), torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
    cu = i32(0, 1, 2)
    for a in (layer, other):
        a.cache.k.normal_()
        a.cache.v.normal_()
    ws = la.workspace(la.paged_attn_workspace(layer.cache, 2, 2, 4, 500))
    for a in (layer, other):
        a(x, cu, lens, table, 500, ws=ws)   # warm
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in (layer, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(a(x, cu, lens, table, 500, ws=ws))
        graphs.append(g)
    for i in range(4):
        x.normal_()
        lens += 1
        want = [a(x, cu, lens, table, 500, ws=ws).clone() for a in (layer, other)]
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, want):
            assert torch.equal(o, e), i


def test_two_streams():
    """Two layers at once on two streams, each with its own buffers."""
    layers = [Layer(6), Layer(7)]
    x = torch.randn(60, 96, device="cuda")
    cu, lens, table = i32(0, 60), i32(60), i32(*range(4)).view(1, 4)
    want = [a(x, cu, lens, table) for a in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = layers[i](x, cu, lens, table)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
