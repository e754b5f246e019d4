"""The attention layer's entry points refuse what they cannot run, before anything is launched (no GPU), and the plain forms
that the GPU tests compare with agree with brute force."""
import ctypes
import math

import numpy as np
import pytest
import torch

import layer_ref as ref
import lut_logits_amd as la
from lut_logits_amd import binding as B

P = 0x10000   # an aligned address that no refused call reads


def q4_call(ws=P, ws_bytes=1 << 40, x=P, x2=None, y=P, x_dtype=B.RQ_F32, prologue=B.RQ_PRO_NONE, batch=1, **kw):
    f = dict(rows=64, D=256, group=64, scale_dtype=B.RQ_BF16, codes=P, scales=P, offsets=None, levels=None)
    f.update(kw)
    W = B.rq_q4_matrix(**f)
    return B.lib().rq_q4_matvec(ctypes.byref(W), x, x_dtype, x2, prologue, batch, y, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), B.RQ_ERR_SHAPE), (dict(rows=1 << 31), B.RQ_ERR_SHAPE), (dict(D=0), B.RQ_ERR_SHAPE),
    (dict(D=65537), B.RQ_ERR_SHAPE), (dict(group=16), B.RQ_ERR_SHAPE), (dict(group=0), B.RQ_ERR_SHAPE),
    (dict(group=256), B.RQ_ERR_SHAPE), (dict(scale_dtype=3), B.RQ_ERR_DTYPE), (dict(x_dtype=-1), B.RQ_ERR_DTYPE),
    (dict(prologue=2), B.RQ_ERR_DTYPE), (dict(prologue=1, x_dtype=B.RQ_BF16, x2=P), B.RQ_ERR_DTYPE),
    (dict(prologue=1), B.RQ_ERR_NULL), (dict(prologue=1, x2=P + 2), B.RQ_ERR_ALIGN),
    (dict(batch=-1), B.RQ_ERR_SHAPE), (dict(batch=65536), B.RQ_ERR_SHAPE),
    (dict(codes=None), B.RQ_ERR_NULL), (dict(scales=None), B.RQ_ERR_NULL), (dict(x=None), B.RQ_ERR_NULL), (dict(y=None), B.RQ_ERR_NULL),
    (dict(codes=P + 8), B.RQ_ERR_ALIGN), (dict(scales=P + 4), B.RQ_ERR_ALIGN), (dict(offsets=P + 2), B.RQ_ERR_ALIGN),
    (dict(levels=P + 2), B.RQ_ERR_ALIGN), (dict(x=P + 2), B.RQ_ERR_ALIGN), (dict(y=P + 2), B.RQ_ERR_ALIGN),
    (dict(x=P + 1, x_dtype=B.RQ_BF16), B.RQ_ERR_ALIGN),
    (dict(batch=16, ws=None), B.RQ_ERR_WORKSPACE), (dict(batch=16, ws_bytes=100), B.RQ_ERR_WORKSPACE),
    (dict(batch=16, ws=P + 16), B.RQ_ERR_ALIGN),
    (dict(batch=0), B.RQ_OK), (dict(rows=0), B.RQ_OK),
])
def test_q4_refusals(kw, status):
    assert q4_call(**kw) == status
    if status:
        assert B.lib().rq_last_error()


def test_q4_more_than_a_launch():
    """No split of 2^31 rows x 65536 columns with offsets fits one launch: an error and no launch."""
    assert q4_call(rows=(1 << 31) - 1, D=65536, offsets=P, batch=64, group=32) == B.RQ_ERR_HIP
    W = B.rq_q4_matrix((1 << 31) - 1, 65536, 32, B.RQ_BF16, P, P, P, None)
    assert B.lib().rq_q4_matvec_workspace(ctypes.byref(W), B.RQ_F32, 0, 64) == 0


def test_q4_sizes():
    lib = B.lib()
    assert lib.rq_q4_codes_bytes(17, 129) == 2 * 2 * 1024
    assert lib.rq_q4_scales_bytes(17, 129, 32, B.RQ_F32) == 2 * 2 * 16 * 4 * 4
    assert lib.rq_q4_scales_bytes(17, 129, 128, B.RQ_F16) == 2 * 2 * 16 * 2
    assert lib.rq_q4_codes_bytes(5, 0) == 0 and lib.rq_q4_scales_bytes(5, 64, 48, B.RQ_F32) == 0
    assert lib.rq_q4_codes_bytes((1 << 31) - 1, 65536) == (1 << 27) * 512 * 1024
    W = B.rq_q4_matrix(64, 256, 64, B.RQ_BF16, P, P, None, None)
    assert lib.rq_q4_matvec_workspace(ctypes.byref(W), B.RQ_F32, 0, 1) == 0
    assert lib.rq_q4_matvec_workspace(ctypes.byref(W), B.RQ_F32, 0, 16) >= 16 * 3 * 256 * 2
    assert lib.rq_q4_matvec_workspace(None, B.RQ_F32, 0, 16) == 0
    for bad in (dict(src=None), dict(dst=None), dict(dst=P + 8)):
        a = dict(src=P, dst=P)
        a.update(bad)
        assert lib.rq_pack_q4_codes(a["src"], 4, 64, a["dst"], None) in (B.RQ_ERR_NULL, B.RQ_ERR_ALIGN)
        assert lib.rq_pack_q4_scales(a["src"], 4, 64, 32, B.RQ_F32, a["dst"], None) in (B.RQ_ERR_NULL, B.RQ_ERR_ALIGN)


def rope_call(x=P, x_dtype=B.RQ_F32, tokens=4, heads=2, size=64, xs=128, pos=P, freqs=P, rot=64, layout=0, out=2 * P,
              out_dtype=B.RQ_F32, os_=128):
    return B.lib().rq_rope(x, x_dtype, tokens, heads, size, xs, pos, freqs, rot, layout, 1.0, 0, out, out_dtype, os_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), B.RQ_ERR_SHAPE), (dict(heads=4097), B.RQ_ERR_SHAPE), (dict(size=63), B.RQ_ERR_SHAPE),
    (dict(size=514), B.RQ_ERR_SHAPE), (dict(tokens=-1), B.RQ_ERR_SHAPE), (dict(tokens=1 << 30), B.RQ_ERR_SHAPE),
    (dict(tokens=(1 << 29) + 1, heads=1), B.RQ_ERR_SHAPE), (dict(rot=0), B.RQ_ERR_SHAPE), (dict(rot=66), B.RQ_ERR_SHAPE), (dict(rot=3), B.RQ_ERR_SHAPE), (dict(xs=127), B.RQ_ERR_SHAPE),
    (dict(os_=100), B.RQ_ERR_SHAPE), (dict(layout=2), B.RQ_ERR_DTYPE), (dict(x_dtype=3), B.RQ_ERR_DTYPE), (dict(out_dtype=-1), B.RQ_ERR_DTYPE),
    (dict(x=None), B.RQ_ERR_NULL), (dict(out=None), B.RQ_ERR_NULL), (dict(pos=None), B.RQ_ERR_NULL), (dict(freqs=None), B.RQ_ERR_NULL),
    (dict(x=P + 2), B.RQ_ERR_ALIGN), (dict(out=P + 2), B.RQ_ERR_ALIGN), (dict(freqs=P + 4), B.RQ_ERR_ALIGN), (dict(pos=P + 2), B.RQ_ERR_ALIGN),
    (dict(out=P, os_=192), B.RQ_ERR_SHAPE), (dict(out=P, out_dtype=B.RQ_F16), B.RQ_ERR_SHAPE),
    (dict(tokens=0), B.RQ_OK),
])
def test_rope_refusals(kw, status):
    assert rope_call(**kw) == status


CACHE = dict(pages=8, page_size=16, kv_heads=2, head_dim=64, dtype=B.RQ_BF16, k=P, v=P)
BATCH = dict(seqs=2, tokens=4, max_pages=4, cu_q=P, lens=P, table=P)


def split_kw(kw):
    c, b, rest = dict(CACHE), dict(BATCH), {}
    for k, v in kw.items():
        (c if k in c else b if k in b else rest)[k] = v
    return B.rq_kv_cache(**c), B.rq_seq_batch(**b), rest


SHARED = [
    (dict(pages=0), B.RQ_ERR_SHAPE), (dict(page_size=8), B.RQ_ERR_SHAPE), (dict(page_size=48), B.RQ_ERR_SHAPE),
    (dict(page_size=512), B.RQ_ERR_SHAPE), (dict(kv_heads=0), B.RQ_ERR_SHAPE), (dict(kv_heads=257), B.RQ_ERR_SHAPE),
    (dict(head_dim=0), B.RQ_ERR_SHAPE), (dict(head_dim=65), B.RQ_ERR_SHAPE), (dict(dtype=B.RQ_F32), B.RQ_ERR_DTYPE),
    (dict(k=None), B.RQ_ERR_NULL), (dict(v=P + 8), B.RQ_ERR_ALIGN), (dict(seqs=-1), B.RQ_ERR_SHAPE), (dict(tokens=-1), B.RQ_ERR_SHAPE),
    (dict(tokens=1 << 30), B.RQ_ERR_SHAPE), (dict(max_pages=-1), B.RQ_ERR_SHAPE),
    (dict(seqs=(1 << 22) + 1), B.RQ_ERR_SHAPE), (dict(seqs=1 << 22, max_pages=512), B.RQ_ERR_SHAPE), (dict(cu_q=None), B.RQ_ERR_NULL),
    (dict(lens=None), B.RQ_ERR_NULL), (dict(table=None), B.RQ_ERR_NULL), (dict(lens=P + 2), B.RQ_ERR_ALIGN),
    (dict(heads=3), B.RQ_ERR_SHAPE), (dict(heads=0), B.RQ_ERR_SHAPE), (dict(q_stride=255), B.RQ_ERR_SHAPE), (dict(q=None), B.RQ_ERR_NULL),
    (dict(out=None), B.RQ_ERR_NULL), (dict(out=P), B.RQ_ERR_SHAPE), (dict(bad=P + 1), B.RQ_ERR_ALIGN),
    (dict(seqs=0, cu_q=None, lens=None, table=None), B.RQ_OK), (dict(tokens=0), B.RQ_OK),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(in_dtype=5), B.RQ_ERR_DTYPE), (dict(k_stride=100), B.RQ_ERR_SHAPE), (dict(v_stride=100), B.RQ_ERR_SHAPE),
    (dict(rot=66), B.RQ_ERR_SHAPE), (dict(layout=9), B.RQ_ERR_DTYPE), (dict(freqs=None), B.RQ_ERR_NULL), (dict(kk=None), B.RQ_ERR_NULL),
    (dict(q=P + 2), B.RQ_ERR_ALIGN),
])
def test_append_refusals(kw, status):
    c, b, kw = split_kw(kw)
    a = dict(q=P, kk=P, vv=P, in_dtype=B.RQ_F32, q_stride=256, k_stride=128, v_stride=128, heads=4, pos=None, freqs=P, rot=64,
             layout=0, out=2 * P, bad=None)
    a.update(kw)
    assert B.lib().rq_rope_append(ctypes.byref(b), ctypes.byref(c), a["q"], a["kk"], a["vv"], a["in_dtype"], a["q_stride"], a["k_stride"],
                                  a["v_stride"], a["heads"], a["pos"], a["freqs"], a["rot"], a["layout"], 1.0, a["out"], a["bad"],
                                  None) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(head_dim=96, q_stride=384), B.RQ_ERR_SHAPE), (dict(window=-1), B.RQ_ERR_SHAPE), (dict(scale=0.0), B.RQ_ERR_SHAPE),
    (dict(scale=-0.125), B.RQ_ERR_SHAPE), (dict(scale=math.inf), B.RQ_ERR_SHAPE), (dict(scale=math.nan), B.RQ_ERR_SHAPE), (dict(max_len=-1), B.RQ_ERR_SHAPE),
    (dict(softcap=math.inf), B.RQ_ERR_SHAPE), (dict(softcap=math.nan), B.RQ_ERR_SHAPE), (dict(softcap=1e-39), B.RQ_ERR_SHAPE),
    (dict(q_stride=260), B.RQ_ERR_ALIGN), (dict(q=P + 8), B.RQ_ERR_ALIGN), (dict(out=2 * P + 8), B.RQ_ERR_ALIGN), (dict(lse=P + 2), B.RQ_ERR_ALIGN),
    (dict(tokens=1 << 26), B.RQ_ERR_SHAPE), (dict(seqs=1 << 20, kv_heads=16, heads=16, q_stride=1024, max_pages=1), B.RQ_ERR_SHAPE),
    (dict(ws=None), B.RQ_ERR_WORKSPACE), (dict(ws_bytes=16), B.RQ_ERR_WORKSPACE), (dict(ws=P + 16), B.RQ_ERR_ALIGN),
])
def test_attn_refusals(kw, status):
    c, b, kw = split_kw(kw)
    a = dict(q=P, q_stride=256, heads=4, scale=0.125, softcap=0.0, window=0, max_len=0, out=2 * P, lse=None, bad=None, ws=4 * P, ws_bytes=1 << 40)
    a.update(kw)
    assert B.lib().rq_paged_attn(ctypes.byref(b), ctypes.byref(c), a["q"], a["q_stride"], a["heads"], a["scale"], a["softcap"], a["window"], a["max_len"],
                                 a["out"], a["lse"], a["bad"], a["ws"], a["ws_bytes"], None) == status


def test_attn_workspace():
    c = B.rq_kv_cache(**CACHE)
    w = lambda *a: B.lib().rq_paged_attn_workspace(ctypes.byref(c), *a)  # noqa: E731
    assert w(1, 1, 4, 8192) > 0                      # few workgroups: the keys are split
    assert w(1, 1, 4, 128) == 0                      # a short cache: not
    assert w(1, 1, 4, 0) >= w(1, 1, 4, 8192)         # no bound known
    assert w(8192, 1, 32, 8192) == 0                 # a whole prompt fills the chip
    assert w(0, 0, 4, 100) == 0 and w(1, 1, 3, 100) == 0 and w(-1, 1, 4, 100) == 0


def raises(fn, what):
    with pytest.raises((ValueError, TypeError, RuntimeError)) as e:
        fn()
    assert what in str(e.value), str(e.value)


def test_binding_refusals():
    z = torch.zeros
    i32 = lambda *s: z(s, dtype=torch.int32)  # noqa: E731
    codes, scales = z(2048, dtype=torch.uint8), z(16 * 2 * 2)
    W = la.Q4Matrix(16, 200, 64, codes, scales)
    raises(lambda: la.Q4Matrix(16, 200, 64, codes[1:], scales), "elements")
    raises(lambda: la.Q4Matrix(16, 200, 64, codes, scales[1:]), "elements")
    raises(lambda: la.Q4Matrix(16, 200, 64, codes, scales.double()), "dtype")
    raises(lambda: la.Q4Matrix(16, 200, 64, codes, scales, scales.half()), "dtype")
    raises(lambda: la.Q4Matrix(16, 200, 64, codes, scales, None, z(16)), "dtype")
    raises(lambda: la.Q4Matrix(16, 200, 63, codes, scales), "out of range")
    raises(lambda: la.q4_matvec(codes, z(1, 200)), "Q4Matrix")
    raises(lambda: la.q4_matvec(W, z(1, 199)), "shape")
    raises(lambda: la.q4_matvec(W, z(200)), "shape")
    raises(lambda: la.q4_matvec(W, z(1, 200).double()), "dtype")
    raises(lambda: la.q4_matvec(W, z(200, 2).t()), "contiguous")
    raises(lambda: la.q4_matvec(W, z(2, 200), z(1, 200)), "shape")
    raises(lambda: la.q4_matvec(W, z(1, 200), out=z(1, 15)), "elements")
    raises(lambda: la.q4_matvec(W, z(8, 200), ws=z(16, dtype=torch.uint8)), "elements")
    raises(lambda: la.q4_matvec(W, z(1, 200)), "GPU")
    raises(lambda: la.pack_q4(z(4, 99, dtype=torch.uint8), z(4, 4), 200, 64), "shape")
    raises(lambda: la.pack_q4(z(4, 100, dtype=torch.uint8), z(4, 3), 200, 64), "shape")
    raises(lambda: la.pack_q4(z(4, 100, dtype=torch.uint8), z(4, 4), 200, 64), "GPU")

    f = torch.ones(32, dtype=torch.float64)
    x = z(3, 2, 64)
    raises(lambda: la.rope(x, i32(2), f), "shape")
    raises(lambda: la.rope(x, z(3, dtype=torch.int64), f), "dtype")
    raises(lambda: la.rope(x, i32(3), f.float()), "dtype")
    raises(lambda: la.rope(x.double(), i32(3), f), "dtype")
    raises(lambda: la.rope(z(3, 128), i32(3), f), "shape")
    raises(lambda: la.rope(z(3, 64, 2).transpose(1, 2), i32(3), f), "contiguous")
    raises(lambda: la.rope(z(1, 2, 64).expand(3, 2, 64), i32(3), f), "overlap")
    raises(lambda: la.rope(x, i32(3), f, out=z(3, 2, 63)), "shape")
    raises(lambda: la.rope(x, i32(3), f, out=z(3, 2, 64), out_dtype=torch.float16), "dtype")
    raises(lambda: la.rope(x, i32(3), f), "GPU")

    raises(lambda: la.KVCache(z(4, 1, 16, 64), z(4, 1, 64, 16)), "dtype")
    h = torch.bfloat16
    raises(lambda: la.KVCache(z(4, 1, 16, 64, dtype=h), z(4, 1, 16, 64, dtype=h)), "shape")
    raises(lambda: la.KVCache(z(4, 1, 16, 64, dtype=h), z(4, 1, 64, 16, dtype=torch.float16)), "dtype")
    raises(lambda: la.KVCache(z(4, 1, 64, 16, dtype=h).transpose(2, 3), z(4, 1, 64, 16, dtype=h)), "contiguous")
    cache = la.KVCache(z(4, 1, 16, 64, dtype=h), z(4, 1, 64, 16, dtype=h))
    q, kv, cu, lens, table = z(3, 2, 64, dtype=h), z(3, 1, 64, dtype=h), i32(2), i32(1), i32(1, 2)
    raises(lambda: la.rope_append(q, kv, kv.half(), cache, cu, lens, table, f), "dtype")
    raises(lambda: la.rope_append(q, kv, kv[:2], cache, cu, lens, table, f), "shape")
    raises(lambda: la.rope_append(q, q, kv, cache, cu, lens, table, f), "shape")
    raises(lambda: la.rope_append(q, kv, kv, cache, i32(3), lens, table, f), "shape")
    raises(lambda: la.rope_append(q, kv, kv, cache, cu, lens, table, f, positions=i32(2)), "shape")
    raises(lambda: la.rope_append(q, kv, kv, cache, cu, lens, table, f), "GPU")
    raises(lambda: la.paged_attn(q.half(), cache, cu, lens, table), "dtype")
    raises(lambda: la.paged_attn(z(3, 2, 32, dtype=h), cache, cu, lens, table), "shape")
    raises(lambda: la.paged_attn(q, cache, cu, lens.long(), table), "dtype")
    raises(lambda: la.paged_attn(q, cache, cu, lens, i32(2, 2)), "shape")
    raises(lambda: la.paged_attn(q, cache, cu, lens, table, lse=z(3, 3)), "shape")
    raises(lambda: la.paged_attn(q, cache, cu, lens, table, out=z(3, 2, 64)), "dtype")
    raises(lambda: la.paged_attn(q, cache, cu, lens, table), "GPU")


def test_sizes_kept_are_bounded():
    """A server's batches and lengths change without end: what a handle keeps of them does not grow with them."""
    kept = {}
    for i in range(3 * B._SIZES_KEPT):
        assert B._keep(kept, (i, 1, 4, 2 * i), i) == i and len(kept) <= B._SIZES_KEPT


def test_rope_freqs():
    f, m = la.rope_freqs(8, base=100.0, device="cpu")
    assert m == 1.0 and np.allclose(f.numpy(), [1, 100 ** -0.25, 0.1, 100 ** -0.75], rtol=1e-15)
    lin, _ = la.rope_freqs(8, base=100.0, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(lin.numpy(), f.numpy() / 4, rtol=1e-15)
    ntk, _ = la.rope_freqs(8, base=100.0, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == f[0] and math.isclose(float(ntk[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    yarn, m = la.rope_freqs(128, scaling="yarn", factor=4.0, trained_len=4096, device="cpu")
    plain, _ = la.rope_freqs(128, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(yarn[turns >= 32], plain[turns >= 32]) and torch.allclose(yarn[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15)
    assert bool((yarn <= plain).all()) and bool((yarn >= plain / 4).all()) and math.isclose(m, 1 + 0.1 * math.log(4))
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, scaling="other")):
        with pytest.raises(ValueError):
            la.rope_freqs(device="cpu", **bad)


def test_plain_forms_against_brute_force():
    rng = np.random.default_rng(0)
    m = ref.Q4(rng, 3, 70, 32, "f16", True, True)
    w, packed = m.dense(), m.interchange()
    for r in range(3):
        for k in range(70):
            code = (packed[r, k // 2] >> (4 * (k % 2))) & 15
            assert w[r, k] == m.levels[code] * m.scales[r, k // 32] + m.offsets[r, k // 32]
    x = rng.standard_normal((2, 1, 6))
    y = ref.rotate(x, [0, 3], np.array([0.5, 0.25]), 2.0, "interleaved")
    z = (x[1, 0, 2] + 1j * x[1, 0, 3]) * 2 * np.exp(0.75j)
    assert np.allclose(y[1, 0, 2:4], [z.real, z.imag]) and np.array_equal(y[:, :, 4:], x[:, :, 4:]) and np.allclose(y[0, :, :4], 2 * x[0, :, :4])
    b = ref.Batch(rng, [2], [5], 16)
    q, k, v = rng.standard_normal((2, 2, 4)), [rng.standard_normal((5, 1, 4))], [rng.standard_normal((5, 1, 4))]
    out, lse, _ = ref.attention(q, b, k, v, 0.5, softcap=2.0, window=3)
    for i, place in enumerate((3, 4)):
        for h in range(2):
            e = [math.exp(2 * math.tanh(float(q[i, h] @ k[0][j, 0]) * 0.5 / 2)) for j in range(place - 2, place + 1)]
            assert np.allclose(out[i, h], sum(w * v[0][place - 2 + j, 0] for j, w in enumerate(e)) / sum(e))
            assert math.isclose(lse[i, h], math.log(sum(e)))
