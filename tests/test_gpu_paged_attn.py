"""Attention over the paged cache (rq_paged_attn) against the definition in 64 bits (needs an MI355X).

Unseen places hold NaN in every case. Tolerance, h being half a step of the 16-bit type:
    |o - o64| <= 1.02 h |o64|                    the output's rounding
               + h mass                          each probability's rounding (kernel of many rows only; mass = sum_j p_j |v_j|)
               + (2 dz + 2^-19) mass             dz: the scores' own error; exponentials within 2^-21, sums in fp32
               + n 2^-25 max|v|  (fp16)          probabilities below fp16's normal range
with dz = scale (size + 2) 2^-24 max sum|q||k|, + 2^-20 cap for the capped tanh."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import lut_logits_amd as la
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    def __init__(self, seed, new, lens, heads, kv, size, page, dtype, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.dtype, self.heads, self.kv, self.size = dtype, heads, kv, size
        self.b = ref.Batch(rng, new, lens, page)
        self.q = ref.round_to(rng.standard_normal((self.b.tokens, heads, size)) * qscale, dtype)
        self.k = [ref.round_to(rng.standard_normal((n, kv, size)), dtype) for n in lens]
        self.v = [ref.round_to(rng.standard_normal((n, kv, size)), dtype) for n in lens]

    def upload(self, fill=np.nan):
        kp, vp = ref.to_pages(self.b, self.k, self.v, self.kv, self.size, fill)
        return la.KVCache(dev(kp, T[self.dtype]), dev(vp, T[self.dtype]))

    def meta(self):
        return dev(self.b.cu_q), dev(np.array(self.b.lens, np.int32)), dev(self.b.table)

    def run(self, **kw):
        return la.paged_attn(dev(self.q, T[self.dtype]), self.upload(), *self.meta(), **kw)

    def tolerance(self, want, mass, softcap=0.0, one_rounding=True):
        h = ref.HALF_STEP[self.dtype]
        top = max([float((np.abs(self.q).max(axis=(0, 1)) * np.abs(k).max(axis=(0, 1))).sum()) for k in self.k if len(k)] + [0.0])
        dz = self.size ** -0.5 * (self.size + 2) * 2.0 ** -24 * top + 2.0 ** -20 * softcap
        sub = max(self.b.lens) * 2.0 ** -25 * max(np.abs(v).max() for v in self.v if len(v)) if self.dtype == "f16" else 0.0
        return 1.02 * h * np.abs(want) + ((h if one_rounding else 0.0) + 2 * dz + 2.0 ** -19) * mass + sub + 1e-30

    def check(self, out, lse=None, softcap=0.0, window=0, one_rounding=True):
        want, want_lse, mass = ref.attention(self.q, self.b, self.k, self.v, self.size ** -0.5, softcap, window)
        got = host(out[:self.b.tokens].float()).astype(np.float64)
        tol = self.tolerance(want, mass, softcap, one_rounding)
        err = np.abs(got - want)
        assert (err <= tol).all(), (float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:5])
        if lse is not None:
            g = host(lse).astype(np.float64)
            none = np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(g), none)
            assert (np.abs(g - want_lse)[~none] <= 2.0 ** -18 * (1 + np.abs(want_lse[~none])) + 2.0 ** -20 * softcap).all()


CASES = [
    # new, lens, heads, kv, size, page, type, softcap, window; few rows a sequence: the kernel of 16 rows
    ([1], [1], 1, 1, 64, 16, "bf16", 0.0, 0),
    ([1], [33], 8, 4, 256, 16, "bf16", 50.0, 0),
    ([1, 1, 1], [5, 700, 128], 4, 1, 128, 32, "f16", 0.0, 0),
    ([1, 1], [1500, 3], 3, 3, 64, 128, "bf16", 0.0, 100),
    ([5, 5, 5], [5, 77, 300], 6, 2, 64, 64, "f16", 30.0, 0),
    ([7], [260], 2, 1, 256, 16, "f16", 0.0, 1),
    ([0, 1, 0, 2], [9, 40, 0, 2], 4, 2, 128, 16, "bf16", 0.0, 0),
    ([1], [2600], 17, 1, 64, 256, "bf16", 0.0, 0),          # 17 heads on one: two tiles of rows
    # many rows: the kernel of 128
    ([40], [40], 4, 2, 64, 16, "bf16", 0.0, 0),
    ([129], [129], 3, 1, 128, 16, "f16", 0.0, 0),
    ([100, 1, 60], [300, 500, 60], 2, 2, 64, 32, "bf16", 30.0, 0),
    ([70], [333], 4, 2, 256, 16, "bf16", 50.0, 64),
    ([200], [1100], 1, 1, 128, 64, "f16", 0.0, 33),
    ([65, 0, 64], [65, 10, 70], 5, 1, 256, 32, "f16", 0.0, 0),
    ([300], [300], 1, 1, 64, 128, "bf16", 0.0, 1),
    ([64, 3], [190, 3], 8, 1, 128, 256, "bf16", 0.0, 100),
]


@pytest.mark.parametrize("new,lens,heads,kv,size,page,dtype,softcap,window", CASES)
def test_against_definition(new, lens, heads, kv, size, page, dtype, softcap, window):
    c = Case(sum(lens) + size, new, lens, heads, kv, size, page, dtype, qscale=3.0 if softcap else 1.0)
    lse = torch.zeros((c.b.tokens, heads), device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    few = c.b.tokens * (heads // kv) <= 32 * len(new)
    out = c.run(softcap=softcap, window=window, lse=lse, bad_pages=bad)
    c.check(out, lse, softcap, window, one_rounding=not few)
    assert int(bad) == 0
    # the bound of the lengths changes how the keys are split, not the result beyond rounding; the same call gives the same bits
    again = c.run(softcap=softcap, window=window, max_len=max(max(lens), 1))
    c.check(again, None, softcap, window, one_rounding=not few)
    assert torch.equal(out, c.run(softcap=softcap, window=window))


@pytest.mark.parametrize("new,size,page,window", [(1, 64, 16, 0), (1, 256, 16, 0), (3, 128, 16, 1500), (70, 64, 16, 0), (70, 128, 32, 0),
                                                  (70, 256, 16, 0), (70, 256, 32, 1200), (70, 128, 16, 1500)])
def test_long_tables(new, size, page, window):
    """More table entries than are looked up at once (64), on both kernels, whatever the page."""
    c = Case(new + size, [new, new], [2100, 2500], 4, 2, size, page, "bf16")
    c.check(c.run(window=window), None, 0.0, window, one_rounding=new > 8)


def test_max_len_exceeded():
    """A bound that is too low changes the split alone."""
    c = Case(1, [1, 40], [900, 1000], 2, 1, 64, 16, "bf16")
    c.check(c.run(max_len=1))


def test_no_visible_key():
    """Empty sequences in the cache, lengths below the number of new tokens, sequences without pages: zeros and -inf."""
    for new in ([3, 2, 4], [40, 33, 50]):
        c = Case(2, new, new, 2, 1, 64, 16, "bf16")
        lens = np.array([0, 1, new[2]], np.int32)
        table = c.b.table.copy()
        table[2] = -1
        lse = torch.full((c.b.tokens, 2), 5.0, device="cuda")
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = la.paged_attn(dev(c.q, torch.bfloat16), c.upload(), dev(c.b.cu_q), dev(lens), dev(table), lse=lse, bad_pages=bad)
        o, z = host(out.float()), host(lse)
        last = new[0] + new[1] - 1            # the only token with a key: sequence 1's last
        rest = np.arange(c.b.tokens) != last
        assert (o[rest] == 0).all() and np.isneginf(z[rest]).all()
        # (the length is one: that key is the cache's first place)
        assert np.array_equal(o[last], np.broadcast_to(c.v[1][0], (2, 64)).astype(np.float32)) and np.isfinite(z[last]).all()
        assert int(bad) == -(-new[2] // 16)


def test_table_shorter_than_length():
    """Places beyond the table are no one's: the result is that of the keys that there are."""
    for n, m in ((100, 1), (100, 50)):
        c = Case(3, [m], [n], 2, 2, 64, 16, "f16")
        out = la.paged_attn(dev(c.q, torch.float16), c.upload(), dev(c.b.cu_q), dev(np.array([n], np.int32)),
                            dev(np.ascontiguousarray(c.b.table[:, :4])))
        got = host(out.float()).astype(np.float64)
        for i in range(m):
            seen = min(n - m + i + 1, 64)
            z = np.einsum("hd,jhd->hj", c.q[i], c.k[0][:seen]) / 8
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            want, mass = np.einsum("hj,jhd->hd", p, c.v[0][:seen]), np.einsum("hj,jhd->hd", p, np.abs(c.v[0][:seen]))
            assert (np.abs(got[i] - want) <= c.tolerance(want, mass)).all()


def test_bad_page_in_the_middle():
    """A page id outside the pool hides its keys from everyone."""
    for new in (1, 60):
        c = Case(4, [new], [200], 2, 1, 128, 32, "bf16")
        table = c.b.table.copy()
        table[0, 2] = c.b.pages       # places 64 .. 95
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = la.paged_attn(dev(c.q, torch.bfloat16), c.upload(), dev(c.b.cu_q), dev(np.array([200], np.int32)), dev(table), bad_pages=bad)
        assert int(bad) == 1
        got = host(out.float()).astype(np.float64)
        keys = np.r_[0:64, 96:200]
        for i in range(new):
            ks = keys[keys <= 200 - new + i]
            z = c.q[i] @ c.k[0][ks, 0].T / np.sqrt(128)
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            want, mass = p @ c.v[0][ks, 0], p @ np.abs(c.v[0][ks, 0])
            assert (np.abs(got[i] - want) <= c.tolerance(want, mass)).all()


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("new,size", [(6, 64), (6, 256), (90, 64), (90, 128), (90, 256)])
def test_later_tokens_do_not_reach_earlier_ones(new, size, value):
    """An infinity or NaN in the keys or values of a token of the chunk reaches the tokens that see it and no others."""
    c = Case(5, [new], [new + 70], 2, 1, size, 16, "bf16")
    place = 70 + new // 2
    clean = host(c.run().float())
    for what in ("v", "k"):
        keep = getattr(c, what)[0].copy()
        getattr(c, what)[0][place, 0, 3] = value
        got = host(c.run().float())
        getattr(c, what)[0][:] = keep
        before, after = np.arange(new) + 70 < place, np.arange(new) + 70 >= place
        # (a chunk that holds such values goes another way through the same sums: to rounding)
        want, _, mass = ref.attention(c.q, c.b, c.k, c.v, size ** -0.5)
        assert (np.abs(got - want) <= c.tolerance(want, mass))[before].all()
        if what == "v":
            assert not np.isfinite(got[after][:, :, 3]).any()
            others = np.delete(np.arange(size), 3)
            assert (np.abs(got - want) <= c.tolerance(want, mass))[after][:, :, others].all()
            if np.isinf(value):
                assert (got[after][:, :, 3] == value).all()
        elif np.isnan(value):
            assert np.isnan(got[after]).all()
    assert np.isfinite(clean).all()


def test_extreme_scores():
    """Scores far apart and far from zero: one key takes all, and nothing overflows."""
    for new in (2, 50):
        c = Case(6, [new], [300], 2, 1, 64, 16, "bf16")
        c.q *= 2.0 ** 12
        c.k[0] *= 2.0 ** 6
        want, _, _ = ref.attention(c.q, c.b, c.k, c.v, 0.125)
        got = host(c.run().float())
        assert np.isfinite(got).all()
        # gaps between the two largest scores dwarf the scores' error in all but a few rows
        z = [np.sort((c.q[i] @ c.k[0][:300 - new + i + 1, 0].T) / 8)[:, -2:] for i in range(new)]
        clear = np.array([(a[:, 1] - a[:, 0]) > 1000 for a in z])
        assert clear.mean() > 0.5
        assert np.array_equal(got[clear], want[clear].astype(np.float32))


def test_strided_queries_and_rows_behind():
    """q as a view of a stacked projection; rows behind the last sequence are left as they are, and so is the memory around
    the workspace."""
    for new in ([1, 1], [50, 20]):
        c = Case(7, new, [300, 222], 4, 2, 64, 16, "f16")
        n = c.b.tokens
        stacked = torch.full((n + 3, 8 * 64), float("nan"), dtype=torch.float16, device="cuda")
        q = stacked[:, 64:64 + 256].view(n + 3, 4, 64)
        q[:n] = dev(c.q, torch.float16)
        out = torch.full((n + 3, 4, 64), 2.5, dtype=torch.float16, device="cuda")
        cache = c.upload()
        need = la.paged_attn_workspace(cache, n + 3, 2, 4)
        assert need > 0
        ws = torch.full((need + 256,), 3, dtype=torch.uint8, device="cuda")
        la.paged_attn(q, cache, *c.meta(), ws=ws, out=out)
        c.check(out)
        assert bool((out[n:] == 2.5).all()) and bool((ws[need:] == 3).all())


@pytest.mark.parametrize("new,lens,lead", [([1, 2], [40, 300], 60), ([70, 130], [70, 900], 400), ([0, 40], [5, 2000], 130)])
def test_rows_before_the_first_sequence(new, lens, lead):
    """cu_q that begins behind row 0: the rows before belong to no sequence and are left as they are."""
    c = Case(6, new, lens, 4, 2, 64, 16, "bf16")
    q = torch.full((lead + c.b.tokens, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    q[lead:] = dev(c.q, torch.bfloat16)
    cu, kept, table = c.meta()
    out, lse = torch.full_like(q, 7.0), torch.full((lead + c.b.tokens, 4), 7.0, device="cuda")
    la.paged_attn(q, c.upload(), cu + lead, kept, table, out=out, lse=lse)
    assert bool((out[:lead] == 7.0).all()) and bool((lse[:lead] == 7.0).all())
    c.check(out[lead:], lse[lead:])


def test_many_sequences():
    """More sequences than one step of the search looks at, some without new tokens."""
    rng = np.random.default_rng(8)
    for most in (3, 40):
        new = [int(x) for x in rng.integers(0, most, 150)]
        lens = [m + int(x) for m, x in zip(new, rng.integers(0, 30, 150))]
        c = Case(9, new, lens, 2, 1, 64, 16, "bf16")
        c.check(c.run())


def test_far_pages():
    """A pool whose pages lie beyond 2^31 elements."""
    page_elems = 256 * 256
    pages = (1 << 31) // page_elems + 40
    k = torch.empty((pages, 1, 256, 256), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((pages, 1, 256, 256), dtype=torch.bfloat16, device="cuda")
    for new in (1, 80):
        c = Case(10, [new], [500], 2, 1, 256, 256, "bf16")
        table = np.array([[pages - 1, pages - 30]], np.int32)
        kp, vp = ref.to_pages(c.b, c.k, c.v, 1, 256, np.nan)
        for i in range(2):
            k[table[0, i]] = dev(kp[c.b.table[0, i]], torch.bfloat16)
            v[table[0, i]] = dev(vp[c.b.table[0, i]], torch.bfloat16)
        out = la.paged_attn(dev(c.q, torch.bfloat16), la.KVCache(k, v), dev(c.b.cu_q), dev(np.array([500], np.int32)), dev(table))
        c.check(out)


def test_graph_replays():
    """Captured once, replayed on other queries and longer sequences: the lengths are read on the device."""
    for new in (1, 40):
        c = Case(11, [new, new], [600, 600], 4, 2, 128, 16, "bf16")
        cache = c.upload(0.0)
        cu, lens, table = c.meta()
        q, out = dev(c.q, torch.bfloat16), torch.empty((2 * new, 4, 128), dtype=torch.bfloat16, device="cuda")
        ws = la.workspace(la.paged_attn_workspace(cache, 2 * new, 2, 4, 600))
        run = lambda: la.paged_attn(q, cache, cu, lens, table, max_len=600, ws=ws, out=out)  # noqa: E731
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        for i, n in enumerate((600, 100, 333, 47)):
            q.copy_(torch.randn_like(q))
            lens.copy_(torch.tensor([n, 600 - n + 40], dtype=torch.int32))
            run()
            want = out.clone()
            out.fill_(-1)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), i


def test_empty():
    cache = la.KVCache.empty(2, 1, 16, 64)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert la.paged_attn(e, cache, z, z[:0], z[:0].view(0, 1)).shape == (0, 2, 64)
    # no sequences: the rows are no one's
    out = torch.full((3, 2, 64), 1.5, dtype=torch.bfloat16, device="cuda")
    la.paged_attn(torch.zeros_like(out), cache, z, z[:0], z[:0].view(0, 1), out=out)
    assert bool((out == 1.5).all())
