"""Plain forms in 64 bits, on the CPU, of the operators around the RQ-coded parts (4-bit products, rotation, paged cache,
attention), written from their definitions, and their inputs."""
import math

import numpy as np

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a step of rounding, relative to the value


def round_to(a, dtype):
    """The values of a rounded to nearest even in dtype, as float64."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64))
    return t.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]).double().numpy()


# ---- 4-bit matrices

class Q4:
    """Codes [rows][D] 0..15, scales and offsets [rows][groups] as float64 values of their type, levels [16] or None."""

    def __init__(self, rng, rows, D, group, scale_dtype="bf16", offsets=False, levels=False):
        G = -(-D // group)
        self.rows, self.D, self.group, self.scale_dtype = rows, D, group, scale_dtype
        self.codes = rng.integers(0, 16, (rows, D)).astype(np.uint8)
        self.scales = round_to(rng.uniform(0.5, 1.5, (rows, G)) * 0.02, scale_dtype)
        self.offsets = round_to(rng.standard_normal((rows, G)) * 0.01, scale_dtype) if offsets else None
        self.levels = round_to(np.sort(rng.standard_normal(16)), "bf16") if levels else None

    def interchange(self):
        """The codes two to a byte, even columns in the low halves."""
        c = np.pad(self.codes, ((0, 0), (0, self.D % 2)))
        return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)

    def dense(self):
        v = self.levels[self.codes] if self.levels is not None else self.codes.astype(np.float64) - 8
        group = np.arange(self.D) // self.group
        w = v * self.scales[:, group]
        return w if self.offsets is None else w + self.offsets[:, group]


def gelu_tanh(x):
    return 0.5 * x * (1 + np.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


# ---- rotation

def rotate(x, positions, freqs, mscale=1.0, layout="half", inverse=False):
    """x [tokens][heads][size] float64."""
    n = len(freqs)
    a = np.asarray(positions, np.float64)[:, None, None] * freqs
    c, s = np.cos(a) * mscale, np.sin(a) * mscale * (-1 if inverse else 1)
    y = x.copy()
    i1, i2 = (np.arange(n), np.arange(n) + n) if layout == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


# ---- sequences and their pages

class Batch:
    """Sequences of `new` tokens out of `lens` kept ones, on pages drawn anywhere from a pool."""

    def __init__(self, rng, new, lens, page_size, spare=3):
        self.new, self.lens, self.page_size = list(new), list(lens), page_size
        need = [-(-max(n, 1) // page_size) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(lens), max(need) + 1), -7, np.int32)   # entries behind a sequence name no page
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.cu_q = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens = int(self.cu_q[-1])

    def places(self):
        return np.concatenate([np.arange(n - m, n) for m, n in zip(self.new, self.lens)] + [np.zeros(0, int)]).astype(np.int32)


def to_pages(batch, k, v, kv_heads, size, fill):
    """The page tensors of per-sequence k, v [len][kv_heads][size]; every place that is no one's holds `fill`."""
    kp = np.full((batch.pages, kv_heads, batch.page_size, size), fill)
    vp = np.full((batch.pages, kv_heads, size, batch.page_size), fill)
    for s in range(len(k)):
        for j in range(len(k[s])):
            p, o = batch.table[s, j // batch.page_size], j % batch.page_size
            kp[p, :, o] = k[s][j]
            vp[p, :, :, o] = v[s][j]
    return kp, vp


def attention(q, batch, k, v, scale, softcap=0.0, window=0):
    """q [tokens][heads][size], k and v per sequence: (out, lse, mass) in 64 bits. mass: sum_j p_j |v_j|, the scale of
    what rounding the probabilities can change. Only seen keys take part: others may hold anything."""
    heads, group = q.shape[1], q.shape[1] // k[0].shape[1]
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    for s, (m, n) in enumerate(zip(batch.new, batch.lens)):
        for i in range(m):
            place = n - m + i
            lo = max(0, place - window + 1) if window else 0
            if place < lo:
                continue
            for h in range(heads):
                ks, vs = k[s][lo:place + 1, h // group], v[s][lo:place + 1, h // group]
                z = ks @ q[batch.cu_q[s] + i, h] * scale
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                top = z.max()
                p = np.exp(z - top)
                t = batch.cu_q[s] + i
                out[t, h], mass[t, h] = p @ vs / p.sum(), p @ np.abs(vs) / p.sum()
                lse[t, h] = top + math.log(p.sum())
    return out, lse, mass
