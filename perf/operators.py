"""The operators that complete a decoder layer around the RQ-coded head and MLP, as measured cases.

- "q4": y[b][r] = sum_k x[b][k] W[r][k] with 4-bit weights W[r][k] = s[r][k/group] * level(code) + o[r][k/group], as the
  attention projections next to an RQ head are kept (level: code - 8, or a table of 16 values); optionally on
  gelu_tanh(x) * x2, as a gated MLP's down projection reads it.
- "rope": rotary positions on a tensor of heads, half or interleaved pairs, part of the head, forwards or (the gradient) backwards.
- "append": one step's q, k and v: q rotated, k rotated and written to a paged cache, v written to it.
- "attn": attention of each sequence's newest tokens over its paged cache: causal, grouped heads, optional softcap and window.

Layouts are the library's serving layouts, which a program holds from load time on:
- 4-bit codes: blocks of 16 rows x 128 columns, 1024 bytes each: [row block][column block][column group of 8 in 32 (4)]
  [row (16)][word (4)][byte (4)]; column 128 cb + 32 word + 8 group + j is the low half of byte j (j < 4) or the high half of byte j - 4.
- scales and offsets: [row block][column block][row (16)][128 / group].
- the paged cache: k [pages][kv heads][page size][head size], v [pages][kv heads][head size][page size].
"""
import math

import numpy as np
import torch

own = False

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = {"f32": F32, "bf16": BF16, "f16": F16}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token through an MLP-sized projection with a 16-level code: the call of which a decode step makes hundreds
        dict(name="q4 one token, projection", kind="q4", rows=9216, cols=2304, group=64, batch=1, x="f32", scales="bf16",
             levels=True, offsets=False, gelu=False),
        # one token through a 256,000-row head kept in 4 bits
        dict(name="q4 one token, head", kind="q4", rows=256000, cols=2304, group=64, batch=1, x="f32", scales="bf16",
             levels=False, offsets=False, gelu=False),
        # sixteen sequences through a gated MLP's down projection, the activation in the call, with offsets
        dict(name="q4 batch of 16, down with gelu", kind="q4", rows=2304, cols=9216, group=32, batch=16, x="f32", scales="f16",
             levels=False, offsets=True, gelu=True),
        # odd sizes everywhere, bf16 activations straight from attention
        dict(name="q4 odd sizes, bf16", kind="q4", rows=5003, cols=2311, group=128, batch=61, x="bf16", scales="f32",
             levels=False, offsets=True, gelu=False),
        # the gradient through the rotation of part of the head, interleaved pairs
        dict(name="rope partial, gradient", kind="rope", tokens=4095, heads=16, size=80, rot=32, layout="interleaved",
             x="f32", out="f32", inverse=True, far=20000),
        # one token of each of 64 sequences: latency
        dict(name="append one token each", kind="append", seqs=64, new=1, ctx=500, heads=8, kv=4, size=256, rot=256,
             page=16, layout="half", x="f32", cache="bf16", far=1000000),
        # a prompt's chunk of three sequences
        dict(name="append prompts", kind="append", seqs=3, new=2700, ctx=2700, heads=32, kv=8, size=128, rot=128,
             page=64, layout="half", x="bf16", cache="bf16", far=0),
        # one sequence, one token, a short context: latency
        dict(name="attn one sequence, one token", kind="attn", seqs=1, new=1, ctx=1000, heads=8, kv=4, size=256, page=16,
             x="bf16", softcap=50.0, window=0),
        # a full decode batch on long contexts: bandwidth
        dict(name="attn decode batch", kind="attn", seqs=64, new=1, ctx=8192, heads=32, kv=8, size=128, page=64, x="bf16",
             softcap=0.0, window=0),
        # checking a few drafted tokens of each sequence
        dict(name="attn drafted tokens", kind="attn", seqs=16, new=5, ctx=3001, heads=24, kv=8, size=64, page=32, x="f16",
             softcap=0.0, window=0),
        # a chunk of a prompt behind a long context
        dict(name="attn chunk on a long context", kind="attn", seqs=1, new=256, ctx=16384, heads=32, kv=8, size=128, page=64,
             x="f16", softcap=0.0, window=0),
        # whole prompts, wide heads, softcap and a sliding window
        dict(name="attn prompts, window", kind="attn", seqs=3, new=4000, ctx=4000, heads=8, kv=4, size=256, page=16, x="bf16",
             softcap=50.0, window=2048),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["q4", "q4", "rope", "append", "attn", "attn", "attn"])
    if kind == "q4":
        batch = _spread(rng, 1, 100)
        cols = _spread(rng, 200, 9300)
        rows = _spread(rng, 500, max(1000, min(100000, int(4e8 / cols / (1 + batch / 8)))))
        gelu = rng.random() < 0.25
        return dict(kind="q4", rows=rows, cols=cols, group=rng.choice([32, 64, 128]), batch=batch,
                    x="f32" if gelu else rng.choice(["f32", "bf16", "f16"]), scales=rng.choice(["bf16", "f16", "f32"]),
                    levels=rng.random() < 0.5, offsets=rng.random() < 0.5, gelu=gelu)
    if kind == "rope":
        size = 2 * rng.randint(16, 128)
        heads = rng.randint(1, 32)
        t = rng.choice(["f32", "bf16", "f16"])
        return dict(kind="rope", tokens=_spread(rng, 1, 4000), heads=heads, size=size, rot=2 * rng.randint(4, size // 2),
                    layout=rng.choice(["half", "interleaved"]), x=t, out=rng.choice([t, "f32"]), inverse=rng.random() < 0.3,
                    far=_spread(rng, 1000, 1000000))
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    size = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if kind == "append":
        seqs = _spread(rng, 1, 64)
        new = _spread(rng, 1, max(2, 6000 // seqs))
        return dict(kind="append", seqs=seqs, new=new, ctx=new + _spread(rng, 1, 500), heads=heads, kv=kv, size=size,
                    rot=rng.choice([size, size // 2]), page=page, layout=rng.choice(["half", "interleaved"]),
                    x=rng.choice(["f32", "bf16"]), cache="bf16", far=_spread(rng, 1000, 1000000))
    if rng.random() < 0.5:   # single or drafted tokens
        seqs, new, ctx = _spread(rng, 1, 64), rng.choice([1, 1, 2, 4, 7]), _spread(rng, 30, 8000)
        ctx = max(new, ctx)
    else:                    # chunks and prompts
        seqs = rng.randint(1, 4)
        new = _spread(rng, 20, 2000)
        ctx = new + (0 if rng.random() < 0.5 else _spread(rng, 10, 4000))
    return dict(kind="attn", seqs=seqs, new=new, ctx=ctx, heads=heads, kv=kv, size=size, page=page, x=rng.choice(["bf16", "f16"]),
                softcap=rng.choice([0.0, 30.0]), window=rng.choice([0, 0, 100, 1024]))


def _lengths(case):
    """(new tokens, length) of every sequence: ragged, fixed by the case. The first has the full length."""
    new, ctx = [], []
    for i in range(case["seqs"]):
        part = 1.0 if i == 0 else 0.35 + 0.65 * ((i * 0.6180339887) % 1.0)
        n = case["new"] if case["new"] <= 8 else max(1, int(case["new"] * part))
        new.append(n)
        ctx.append(max(n, int(case["ctx"] * part)))
    return new, ctx


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, std=1.0, dtype=F32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case)
    if case["kind"] == "q4":
        rb, cb, gb = -(-case["rows"] // 16), -(-case["cols"] // 128), 128 // case["group"]
        st = TYPES[case["scales"]]
        s["codes"] = torch.randint(0, 256, (rb, cb, 4, 16, 4, 4), generator=g, device="cuda", dtype=torch.uint8)
        s["s"] = ((torch.rand(rb, cb, 16, gb, generator=g, device="cuda") + 0.5) * (0.05 if case["levels"] else 0.006)).to(st)
        s["o"] = normal(rb, cb, 16, gb, std=0.01, dtype=st) if case["offsets"] else None
        u = torch.linspace(-1, 1, 16, device="cuda")
        s["levels"] = (u.sign() * u.abs() ** 1.4).to(BF16) if case["levels"] else None
        s["x"] = normal(case["batch"], case["cols"], dtype=TYPES[case["x"]])
        s["x2"] = normal(case["batch"], case["cols"]) if case["gelu"] else None
        if own:
            import lut_logits_amd as la
            s["W"] = la.Q4Matrix(case["rows"], case["cols"], case["group"], s["codes"], s["s"], s["o"], s["levels"])
        return s
    if case["kind"] == "rope":
        s["x"] = normal(case["tokens"], case["heads"], case["size"], dtype=TYPES[case["x"]])
        s["positions"] = torch.from_numpy(rng.integers(0, case["far"], case["tokens"], dtype=np.int32)).cuda()
        s["freqs"], s["mscale"] = _frequencies(case["rot"], 4.0)
        return s
    new, ctx = _lengths(case)
    page, kv, size = case["page"], case["kv"], case["size"]
    need = [-(-n // page) for n in ctx]
    order = rng.permutation(sum(need)).astype(np.int32)   # pages anywhere in the pool
    table = np.zeros((len(ctx), max(need)), np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s["cu_q"], s["lens"] = torch.from_numpy(cu).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["table"] = torch.from_numpy(table).cuda()
    s["max_new"], s["max_len"] = max(new), max(ctx)
    tokens, ct = int(cu[-1]), TYPES[case.get("cache", case["x"])]
    s["k_pages"] = normal(sum(need), kv, page, size, dtype=ct)
    s["v_pages"] = normal(sum(need), kv, size, page, dtype=ct)
    s["q"] = normal(tokens, case["heads"], size, dtype=TYPES[case["x"]])
    if case["kind"] == "append":
        s["k"], s["v"] = normal(tokens, kv, size, dtype=TYPES[case["x"]]), normal(tokens, kv, size, dtype=TYPES[case["x"]])
        s["freqs"], s["mscale"] = _frequencies(case["rot"], 1.0)
        # positions other than the cache's where "far" is set: a long document's tail
        s["positions"] = (torch.from_numpy(rng.integers(0, case["far"], tokens, dtype=np.int32)).cuda() if case["far"] else None)
    if own:
        import lut_logits_amd as la
        s["cache"] = la.KVCache(s["k_pages"], s["v_pages"])
        if case["kind"] == "attn":
            s["ws"] = la.workspace(la.paged_attn_workspace(s["cache"], tokens, len(ctx), case["heads"], max_len=s["max_len"]))
    return s


def _frequencies(rot, stretch):
    """Angles per position in 64 bits, slow ones stretched for long contexts, and the factor on cos and sin."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = 10000.0 ** (-2 * i / rot)
    slow = f * 4096 < 2 * math.pi * 32
    f = np.where(slow, f / stretch, f)
    return torch.from_numpy(f).cuda(), 0.1 * math.log(stretch) + 1.0


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"q4": _q4, "rope": _rope, "append": _append, "attn": _attn}[s["kind"]](s)


def _run_own(s):
    import lut_logits_amd as la

    if s["kind"] == "q4":
        return la.q4_matvec(s["W"], s["x"], s["x2"], la.RQ_PRO_GELU_TANH_MUL if s["gelu"] else la.RQ_PRO_NONE)
    if s["kind"] == "rope":
        return la.rope(s["x"], s["positions"], s["freqs"], layout=s["layout"], mscale=s["mscale"], inverse=s["inverse"],
                       out_dtype=TYPES[s["out"]])
    if s["kind"] == "append":
        q = la.rope_append(s["q"], s["k"], s["v"], s["cache"], s["cu_q"], s["lens"], s["table"], s["freqs"],
                           layout=s["layout"], mscale=s["mscale"], positions=s["positions"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return la.paged_attn(s["q"], s["cache"], s["cu_q"], s["lens"], s["table"], scale=s["size"] ** -0.5, softcap=s["softcap"],
                         window=s["window"], max_len=s["max_len"], ws=s["ws"])


def _q4(s):
    rb, cb = s["codes"].shape[:2]
    rows, cols = s["rows"], s["cols"]
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], 5).permute(0, 3, 1, 4, 2, 5, 6).reshape(rb * 16, cb * 128)
    code = code[:rows, :cols]
    w = s["levels"].float()[code.int()] if s["levels"] is not None else code.float() - 8.0

    def spread(t):
        return t.permute(0, 2, 1, 3).reshape(rb * 16, -1).float().repeat_interleave(s["group"], 1)[:rows, :cols]

    w = w * spread(s["s"])
    if s["o"] is not None:
        w = w + spread(s["o"])
    x = s["x"].float()
    if s["gelu"]:
        x = 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x))) * s["x2"]
    return x @ w.t()


def _rotate(x, positions, freqs, mscale, layout, inverse=False):
    """x [tokens][heads][size] in 32 bits, its first 2 * len(freqs) values of each head rotated; angles in 64 bits."""
    half = freqs.numel()
    a = (positions.double()[:, None] * freqs)[:, None, :]
    c, n = (torch.cos(a) * mscale).float(), (torch.sin(a) * mscale).float()
    n = -n if inverse else n
    if layout == "half":
        x1, x2 = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([x1 * c - x2 * n, x2 * c + x1 * n], -1)
    else:
        x1, x2 = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([x1 * c - x2 * n, x2 * c + x1 * n], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _rope(s):
    return _rotate(s["x"].float(), s["positions"], s["freqs"], s["mscale"], s["layout"], s["inverse"]).to(TYPES[s["out"]])


def _places(s):
    """(sequence, position in it) of every token."""
    t = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu_q"], t, right=True) - 1
    return seq, s["lens"][seq] - s["cu_q"][seq + 1] + t


def _append(s):
    seq, pos = _places(s)
    at = pos if s["positions"] is None else s["positions"]
    ct = s["k_pages"].dtype
    q = _rotate(s["q"].float(), at, s["freqs"], s["mscale"], s["layout"]).to(ct)
    k = _rotate(s["k"].float(), at, s["freqs"], s["mscale"], s["layout"]).to(ct)
    page = s["table"][seq, (pos // s["page"]).long()].long()
    slot = (pos % s["page"]).long()
    s["k_pages"][page, :, slot, :] = k
    s["v_pages"][page, :, :, slot] = s["v"].to(ct)
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attn(s):
    seqs, kv, size, group = len(s["lens"]), s["kv"], s["size"], s["heads"] // s["kv"]
    seq, pos = _places(s)
    row = pos - (s["lens"] - s["cu_q"].diff())[seq]
    k = s["k_pages"][s["table"].long()].permute(0, 2, 1, 3, 4).reshape(seqs, kv, -1, size)
    v = s["v_pages"][s["table"].long()].permute(0, 2, 1, 4, 3).reshape(seqs, kv, -1, size)
    q = torch.zeros(seqs, s["max_new"], s["heads"], size, device="cuda")
    q[seq, row.long()] = s["q"].float()
    q = q.view(seqs, s["max_new"], kv, group, size).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * s["max_new"], size)
    z = torch.matmul(q, k.float().transpose(2, 3).contiguous()) * size ** -0.5
    if s["softcap"]:
        z = s["softcap"] * torch.tanh(z / s["softcap"])
    z = z.view(seqs, kv, group, s["max_new"], -1)
    at = (s["lens"] - s["cu_q"].diff())[:, None] + torch.arange(s["max_new"], device="cuda")
    behind = at[:, :, None] - torch.arange(z.shape[-1], device="cuda")   # how far behind the token a key lies
    seen = (behind >= 0) & (behind < (s["window"] or 1 << 30))
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp_min(-1e30))
    o = torch.matmul(p.view(seqs, kv, -1, z.shape[-1]), v.float().contiguous()).view(seqs, kv, group, s["max_new"], size)
    o = o / p.sum(-1, keepdim=True).clamp_min(1e-37)
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, s["max_new"], s["heads"], size)[seq, row.long()].to(s["q"].dtype)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["kind"] == "q4":
        r, c, b = case["rows"], case["cols"], case["batch"]
        groups = r * -(-c // case["group"]) * (2 if case["offsets"] else 1)
        return {"bytes": r * c / 2 + groups * size[case["scales"]] + b * c * size[case["x"]] * (2 if case["gelu"] else 1) + 4 * b * r,
                "flops": 2.0 * r * c * b}
    if case["kind"] == "rope":
        n = case["tokens"] * case["heads"] * case["size"]
        return {"bytes": n * (size[case["x"]] + size[case["out"]]) + 4 * case["tokens"],
                "flops": 3.0 * case["tokens"] * case["heads"] * case["rot"]}
    new, ctx = _lengths(case)
    h, kv, d, t = case["heads"], case["kv"], case["size"], sum(new)
    if case["kind"] == "append":
        return {"bytes": t * (h + 2 * kv) * d * (size[case["x"]] + size[case["cache"]]) + 4.0 * t,
                "flops": 3.0 * t * (h + kv) * case["rot"]}
    w = case["window"] or 1 << 30
    pairs = sum(min(n - m + i + 1, w) for m, n in zip(new, ctx) for i in range(m))
    keys = sum(min(n, w + m - 1) for m, n in zip(new, ctx))
    return {"bytes": 2 * (2 * t * h * d + 2 * keys * kv * d), "flops": 4.0 * pairs * h * d}


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "q4":
        x = s["x"].double()
        if case["gelu"]:
            x = x * (0.5 + 0.5 * torch.tanh(math.sqrt(2 / math.pi) * x * (1 + 0.044715 * x ** 2))) * s["x2"].double()
        y = torch.empty(case["batch"], case["rows"], dtype=torch.float64, device="cuda")
        k = torch.arange(case["cols"], device="cuda")
        j = k % 8
        for r0 in range(0, case["rows"], 8192):   # rows by rows: every weight found by its own address
            r = torch.arange(r0, min(case["rows"], r0 + 8192), device="cuda")[:, None]
            byte = s["codes"][r // 16, k // 128, k // 8 % 4, r % 16, k // 32 % 4, j % 4]
            code = torch.where(j < 4, byte % 16, byte // 16).long()
            at = (r // 16, k // 128, r % 16, k % 128 // case["group"])
            w = s["s"][at].double() * (s["levels"].double()[code] if case["levels"] else (code - 8).double())
            if case["offsets"]:
                w += s["o"][at].double()
            y[:, r[:, 0]] = (w @ x.t()).t()
        return y
    if case["kind"] == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return _turned(s["x"], s["positions"], s["freqs"], s["mscale"], case["layout"], sign)
    new, ctx = _lengths(case)
    if case["kind"] == "append":
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        places = torch.cat([torch.arange(n - m, n) for m, n in zip(new, ctx)]).cuda()
        at = places if s["positions"] is None else s["positions"]
        q, k = (_turned(s[n], at, s["freqs"], s["mscale"], case["layout"], 1.0) for n in ("q", "k"))
        t = 0
        for i, (m, n) in enumerate(zip(new, ctx)):
            p = torch.arange(n - m, n, device="cuda")
            page, slot = s["table"][i][p // case["page"]].long(), p % case["page"]
            for h in range(case["kv"]):
                k_pages[page, h, slot] = k[t:t + m, h]
                v_pages[page, h, :, slot] = s["v"][t:t + m, h].double()
            t += m
        return {"q": q, "k_pages": k_pages, "v_pages": v_pages}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t = 0
    for i, (m, n) in enumerate(zip(new, ctx)):
        pages = s["table"][i, :-(-n // case["page"])].long()
        query, key = torch.arange(n - m, n, device="cuda")[:, None], torch.arange(n, device="cuda")
        seen = (key <= query) & ((query - key < case["window"]) | (case["window"] == 0))
        for h in range(case["heads"]):
            k = s["k_pages"][pages, h * case["kv"] // case["heads"]].reshape(-1, case["size"])[:n].double()
            v = s["v_pages"][pages, h * case["kv"] // case["heads"]].transpose(1, 2).reshape(-1, case["size"])[:n].double()
            z = s["q"][t:t + m, h].double() @ k.t() / math.sqrt(case["size"])
            if case["softcap"]:
                z = torch.tanh(z / case["softcap"]) * case["softcap"]
            out[t:t + m, h] = torch.softmax(z.masked_fill(~seen, -math.inf), 1) @ v
        t += m
    return out


def _turned(x, positions, freqs, mscale, layout, sign):
    """Each pair as a complex number times mscale * exp(i * sign * position * frequency)."""
    n = freqs.numel()
    x = x.double()
    pairs = (x[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2) if layout == "half" else x[..., :2 * n].unflatten(-1, (n, 2)))
    angle = sign * positions.double()[:, None, None] * freqs
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, mscale), angle))
    turned = turned.transpose(-1, -2).flatten(-2) if layout == "half" else turned.flatten(-2)
    return torch.cat([turned, x[..., 2 * n:]], -1)
