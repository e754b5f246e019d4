"""Products with 4-bit matrices (rq_q4_matvec) against the definition in 64 bits (needs an MI355X).

Two kinds of cases. Exact: integer activations, scales that are powers of two, so that every product and partial sum is
exact in fp32 and the result must be equal; they pin the layout, the tails, the parts and the group sums. Float: a term
passes at most 32 roundings inside its matrix-core step (in whatever order it adds), one for each further step of its
group (4 of at most 3 parts), one for each group's share and its offset's, and 11 when waves and parts are joined:
    |y - y64| <= 2^-24 (32 + 12 + 2 G + 11) * sum_k (|s v| + |o|) |a|
(1.02 of it, since the parts' magnitudes add up to at most 1 + 2^-7 times the activation's)."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import lut_logits_amd as la
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def upload(m):
    st = T[m.scale_dtype]
    return la.pack_q4(dev(m.interchange()), dev(m.scales, st), m.D, m.group,
                      None if m.offsets is None else dev(m.offsets, st), None if m.levels is None else dev(m.levels, torch.bfloat16))


def bound(m, a):
    G = -(-m.D // m.group)
    group = np.arange(m.D) // m.group
    v = np.abs(m.levels[m.codes] if m.levels is not None else m.codes.astype(np.float64) - 8)
    w = v * m.scales[:, group] + (0 if m.offsets is None else np.abs(m.offsets[:, group]))
    return 1.02 * 2.0 ** -24 * (32 + 12 + 2 * G + 11) * (np.abs(a) @ w.T) + 1e-37


CASES = [
    # rows, D, group, B, x type, scale type, offsets, levels
    (1, 1, 32, 1, "f32", "f32", False, False),
    (16, 128, 128, 1, "f32", "bf16", False, True),
    (17, 129, 32, 1, "f32", "f16", True, False),
    (333, 2311, 64, 2, "f32", "bf16", True, True),
    (1000, 515, 128, 3, "bf16", "f32", True, False),
    (257, 4100, 32, 4, "f32", "f32", False, False),
    (257, 4100, 32, 5, "f32", "bf16", True, False),      # activations cut beforehand, columns split over workgroups
    (130, 9216, 64, 16, "f32", "bf16", True, True),
    (130, 700, 64, 16, "bf16", "f16", False, True),
    (95, 1000, 32, 17, "f16", "bf16", True, False),
    (70, 300, 128, 61, "bf16", "f32", True, False),
    (33, 257, 64, 64, "f16", "bf16", False, False),
    (48, 384, 32, 128, "bf16", "bf16", True, True),
    (40, 1111, 64, 130, "f32", "bf16", True, False),     # several batch tiles
    (4700, 640, 64, 1, "bf16", "bf16", False, True),
    (70001, 136, 64, 1, "f32", "bf16", True, False),     # workgroups that walk over the rows
    (70001, 136, 64, 9, "f16", "bf16", False, True),
    (40, 30000, 128, 1, "f32", "bf16", True, False),     # the activations do not fit on chip
]


@pytest.mark.parametrize("rows,D,group,B,xt,st,off,lev", CASES)
def test_exact(rows, D, group, B, xt, st, off, lev):
    rng = np.random.default_rng(rows + D)
    m = ref.Q4(rng, rows, D, group, st, off, lev)
    m.scales = 2.0 ** rng.integers(-2, 3, m.scales.shape).astype(np.float64)
    if off:
        m.offsets = rng.integers(-3, 4, m.offsets.shape) / 4.0
    if lev:
        m.levels = rng.permutation(np.arange(-7, 9)).astype(np.float64)
    # multiples of 1/4 below 2^11 + 1/4: three parts of an fp32 value, two of fp16, one of bf16
    x = {"bf16": rng.integers(-8, 9, (B, D)), "f16": rng.integers(-1023, 1024, (B, D)) if D < 600 else rng.integers(-8, 9, (B, D)),
         "f32": rng.integers(-8, 9, (B, D)) + (rng.integers(0, 2, (B, D)) / 4.0)}[xt].astype(np.float64)
    y = host(la.q4_matvec(upload(m), dev(x, T[xt])))
    want = x @ m.dense().T
    assert np.abs(want).max() < 2 ** 20   # multiples of 1/16 in 24 bits: all sums are exact
    assert y.shape == (B, rows)
    assert np.array_equal(y.astype(np.float64), want)


@pytest.mark.parametrize("rows,D,group,B,xt,st,off,lev", CASES)
def test_float(rows, D, group, B, xt, st, off, lev):
    rng = np.random.default_rng(rows + D + 1)
    m = ref.Q4(rng, rows, D, group, st, off, lev)
    x = ref.round_to(rng.standard_normal((B, D)) * np.exp(rng.standard_normal((B, 1))), xt)
    W = upload(m)
    xd = dev(x, T[xt])
    y = la.q4_matvec(W, xd)
    err = np.abs(host(y).astype(np.float64) - x @ m.dense().T)
    assert (err <= bound(m, x)).all(), (err / bound(m, x)).max()
    assert torch.equal(y, la.q4_matvec(W, xd))


@pytest.mark.parametrize("rows,D,B", [(96, 160, 1), (96, 160, 3), (300, 1300, 16), (64, 9216, 1)])
def test_gelu_prologue(rows, D, B):
    """a = gelu_tanh(x) x2, held as fp32: its own error is at most 8 roundings of |x x2| (tanh within 2 of its last place, the
    sum 1 + tanh, three products and the cubic's two)."""
    rng = np.random.default_rng(D + B)
    m = ref.Q4(rng, rows, D, 32, "f16", True, False)
    x, x2 = (ref.round_to(rng.standard_normal((B, D)) * 1.5, "f32") for _ in range(2))
    a = ref.gelu_tanh(x) * x2
    y = host(la.q4_matvec(upload(m), dev(x, torch.float32), dev(x2, torch.float32), la.RQ_PRO_GELU_TANH_MUL)).astype(np.float64)
    tol = bound(m, a) + 8 * 2.0 ** -24 * (np.abs(x * x2) @ np.abs(m.dense()).T)
    err = np.abs(y - a @ m.dense().T)
    assert (err <= tol).all(), (err / tol).max()


def test_wide_range_of_activations():
    """fp32 activations keep all 24 bits over their whole range: huge, tiny and ordinary values side by side, huge ones
    under zero weights."""
    rng = np.random.default_rng(5)
    m = ref.Q4(rng, 64, 256, 32, "f32", False, False)
    m.codes[:, 0] = 8       # weight 0 under the largest value
    x = np.float32(rng.standard_normal((2, 256))).astype(np.float64)
    x[0, 0], x[1, 0] = 3.4028234e38, -1e30
    x[1, 1:] *= 1e-20
    y = host(la.q4_matvec(upload(m), dev(x, torch.float32))).astype(np.float64)
    finite = x.copy()
    finite[:, 0] = 0
    err = np.abs(y - finite @ m.dense().T)
    assert (err <= bound(m, finite)).all()


def test_infinities_and_nan_stay_in_their_vectors():
    rng = np.random.default_rng(6)
    m = ref.Q4(rng, 40, 130, 32, "bf16", True, False)
    W = upload(m)
    for B in (3, 7):
        x = np.float32(rng.standard_normal((B, 130)))
        clean = host(la.q4_matvec(W, dev(x)))
        x[1, 129], x[2, 5] = np.inf, np.nan
        y = host(la.q4_matvec(W, dev(x)))
        assert np.array_equal(y[[0] + list(range(3, B))], clean[[0] + list(range(3, B))])
        w = m.dense()
        assert np.isnan(y[2]).all()
        assert not np.isfinite(y[1][w[:, 129] != 0]).any()


def test_empty():
    m = ref.Q4(np.random.default_rng(0), 20, 40, 32)
    W = upload(m)
    assert la.q4_matvec(W, torch.empty((0, 40), device="cuda")).shape == (0, 20)
    none = la.pack_q4(torch.empty((0, 20), dtype=torch.uint8, device="cuda"), torch.empty((0, 2), device="cuda"), 40, 32)
    assert la.q4_matvec(none, torch.zeros((3, 40), device="cuda")).shape == (3, 0)


def test_writes_nothing_else():
    """Outputs and workspace inside larger buffers: their surroundings keep their bits."""
    rng = np.random.default_rng(8)
    m = ref.Q4(rng, 77, 300, 64, "bf16", True, True)
    W = upload(m)
    for B in (1, 6):
        x = dev(rng.standard_normal((B, 300)), torch.float32)
        big = torch.full((B * 77 + 64,), 7.0, device="cuda")
        need = la.q4_matvec_workspace(W, B)
        ws = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
        la.q4_matvec(W, x, ws=ws[:max(need, 1)] if need else None, out=big[32:32 + B * 77])
        assert bool((big[:32] == 7).all()) and bool((big[32 + B * 77:] == 7).all())
        assert bool((ws[need:] == 9).all())


def test_graph_replays():
    rng = np.random.default_rng(9)
    m = ref.Q4(rng, 500, 700, 64, "bf16", True, True)
    W = upload(m)
    for B in (1, 9):
        x = dev(rng.standard_normal((B, 700)), torch.float32)
        ws = la.workspace(la.q4_matvec_workspace(W, B))
        y = torch.empty((B, 500), device="cuda")
        la.q4_matvec(W, x, ws=ws, out=y)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            la.q4_matvec(W, x, ws=ws, out=y)
        for i in range(4):
            x.copy_(dev(rng.standard_normal((B, 700)), torch.float32))
            want = la.q4_matvec(W, x)
            y.fill_(-1)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), i


def test_side_stream():
    rng = np.random.default_rng(10)
    m = ref.Q4(rng, 300, 260, 64)
    W = upload(m)
    x = dev(rng.standard_normal((6, 260)), torch.float32)
    want = la.q4_matvec(W, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = la.q4_matvec(W, x)
    s.synchronize()
    assert torch.equal(got, want)
