"""Timed cases of the 4-bit K/V cache and of attention with changed scores.

A serving engine that holds its cache in 4 bits rotates the new queries and
keys, writes keys and values into 4-bit pages, and attends over them; models
whose scores are capped by a tanh or biased by distance, batches of packed
documents and prompts with a bidirectional prefix need attention whose scores
and masks are changed on the way.

``op`` of a case:
  append  rotation of q and k, k and v written to their pages in 4 bits, and the
          written rows read back as values
  int4    paged attention over 4-bit pools (decode, chunk, prompt)
  score   paged attention over 2-byte pools with a score cap, a distance bias, a
          document mask or a bidirectional prefix

``run`` computes the operators in plain float32 torch, or with ``own`` set
through the library. ``exact`` is the definition in float64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of 64 requests (32/8 heads): their new tokens.
        dict(name="append-decode", op="append", seqs=64, lens=11, kv_lo=512, kv_hi=8192, q=1,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", rot=128, interleaved=False),
        # Four prompts: every token of theirs, half of each head turned, in f16.
        dict(name="append-prompt", op="append", seqs=4, lens=12, kv_lo=3500, kv_hi=4500, q=0,
             heads=32, kv_heads=8, dim=128, block=32, type="f16", rot=64, interleaved=True),
        # A handful of short requests on a small model: latency.
        dict(name="int4-decode-small", op="int4", seqs=2, lens=21, kv_lo=100, kv_hi=300, q=1,
             heads=8, kv_heads=2, dim=64, block=16, type="f16"),
        # One decode step of 64 requests.
        dict(name="int4-decode", op="int4", seqs=64, lens=22, kv_lo=512, kv_hi=8192, q=1,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16"),
        # A few very long requests, what a 4-bit cache is for.
        dict(name="int4-decode-long", op="int4", seqs=4, lens=23, kv_lo=60000, kv_hi=131072, q=1,
             heads=64, kv_heads=8, dim=128, block=64, type="bf16"),
        # Verification of five drafted tokens for 16 requests.
        dict(name="int4-verify", op="int4", seqs=16, lens=24, kv_lo=1000, kv_hi=16384, q=5,
             heads=32, kv_heads=8, dim=128, block=16, type="f16"),
        # Four prompts attending over what they just wrote.
        dict(name="int4-prompt", op="int4", seqs=4, lens=25, kv_lo=2500, kv_hi=4096, q=0,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16"),
        # Decode of 64 requests of a model that caps its scores.
        dict(name="cap-decode", op="score", seqs=64, lens=31, kv_lo=512, kv_hi=8192, q=1,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", cap=50.0, bias=False,
             docs=False, prefix=False),
        # Its prompts.
        dict(name="cap-prompt", op="score", seqs=4, lens=32, kv_lo=2500, kv_hi=4096, q=0, heads=32,
             kv_heads=8, dim=128, block=16, type="bf16", cap=50.0, bias=False, docs=False,
             prefix=False),
        # A chunk of prompts of a model with a distance bias and a KV head per head.
        dict(name="bias-chunk", op="score", seqs=6, lens=33, kv_lo=1200, kv_hi=3500, q=701,
             heads=16, kv_heads=16, dim=64, block=32, type="f16", cap=0.0, bias=True, docs=False,
             prefix=False),
        # Two rows of packed documents, each attending within its own.
        dict(name="docs-packed", op="score", seqs=2, lens=34, kv_lo=8000, kv_hi=8192, q=0,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", cap=0.0, bias=False, docs=True,
             prefix=False),
        # Prompts whose first part (an image, an instruction) sees itself whole.
        dict(name="prefix-prompt", op="score", seqs=3, lens=35, kv_lo=1500, kv_hi=3500, q=0,
             heads=16, kv_heads=8, dim=256, block=64, type="bf16", cap=30.0, bias=False,
             docs=False, prefix=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "int4", "int4", "int4", "score", "score", "score"))
    case = dict(op=op, lens=rng.randrange(1 << 30), kv_heads=rng.choice((1, 2, 4, 8)),
                dim=rng.choice((64, 128, 128)), block=rng.choice((16, 32, 48, 64, 128)),
                type=rng.choice(("bf16", "f16")))
    case["heads"] = case["kv_heads"] * rng.choice((1, 2, 3, 4, 7, 8))
    kind = rng.choice(("decode", "decode", "chunk", "prompt"))
    if kind == "decode":
        case["seqs"], case["q"] = _log(rng, 1, 64), rng.choice((1, 1, 1, 2, 5))
        case["kv_hi"] = _log(rng, 16, min(65536, 500000 // case["seqs"]))
        case["kv_lo"] = max(1, case["kv_hi"] // rng.randint(1, 16))
    elif kind == "chunk":
        case["seqs"], case["q"] = _log(rng, 1, 6), _log(rng, 9, 600)
        case["kv_hi"] = _log(rng, case["q"], 8192)
        case["kv_lo"] = max(1, case["kv_hi"] // rng.randint(1, 4))
    else:
        case["seqs"], case["q"] = rng.randint(1, 3), 0
        case["kv_hi"] = _log(rng, 16, 3000)
        case["kv_lo"] = max(1, case["kv_hi"] // rng.randint(1, 4))
    if op == "append":
        case["rot"] = case["dim"] // rng.choice((1, 1, 2, 4))
        case["interleaved"] = rng.random() < 0.5
    if op == "score":
        case["dim"] = rng.choice((64, 128, 128, 256))
        case["cap"] = rng.choice((0.0, 20.0, 50.0))
        case["bias"] = rng.random() < 0.4
        case["docs"] = rng.random() < 0.3
        case["prefix"] = rng.random() < 0.3
    return case


def _lengths(case):
    """(kv lengths, query lengths) of the case's sequences."""
    rng = random.Random(case["lens"])
    kv = [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["seqs"])]
    n = case["q"]
    return kv, [k if n == 0 else min(n, k) for k in kv]


def _starts(case, kv):
    """First positions of the documents packed into each sequence."""
    rng, got = random.Random(case["lens"] + 2), []
    for n in kv:
        at = [0]
        while at[-1] + 64 < n:
            at.append(at[-1] + _log(rng, 64, 2000))
        got.append([a for a in at if a < n])
    return got


def _prefixes(case, kv):
    rng = random.Random(case["lens"] + 3)
    return [rng.randint(0, n) for n in kv]


# ------------------------------------------------------------------ inputs
def _pages(case, kv):
    """Pages handed out from a random permutation; one spare page in eight."""
    need = [-(-k // case["block"]) for k in kv]
    total = sum(need) + sum(need) // 8 + 1
    order = list(range(total))
    random.Random(case["lens"] + 1).shuffle(order)
    table, at = [[0] * max(need) for _ in kv], 0
    for s, n in enumerate(need):
        table[s][:n] = order[at:at + n]
        at += n
    return total, torch.tensor(table, dtype=torch.int32, device=DEV)


def _pool4(case, total, gen):
    """(codes uint8 [pages, block, kv heads, dim / 2], scale and minimum f16
    [pages, kv heads, block, 2]) of N(0, 1) values whose heads differ in size."""
    shape = (total, case["block"], case["kv_heads"], case["dim"])
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.linspace(0.5, 2.0, case["kv_heads"], device=DEV)[:, None]
    n, params = _quantized(x)
    return _packed(n), params.transpose(1, 2).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    kv, ql = _lengths(case)
    total, st["table"] = _pages(case, kv)
    block, dim, hk, heads = case["block"], case["dim"], case["kv_heads"], case["heads"]
    tokens, t = sum(ql), TYPES[case["type"]]
    st["kv"], st["ql"], st["max_q"], st["max_k"] = kv, ql, max(ql), max(kv)
    st["lens"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    cu = [0]
    for n in ql:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    st["scale"] = dim ** -0.5
    # q, k and v as a projection leaves them: slices of one packed row.
    qkv = torch.randn((tokens, heads + 2 * hk, dim), generator=gen, device=DEV).to(t)
    st["q"] = qkv[:, :heads]
    if case["op"] == "score":
        # Scores of a few tens, so that a cap bites.
        st["q"] = st["q"] * (4.0 if case["cap"] else 1.0)
        shape = (total, block, hk, dim)
        st["kc"] = torch.randn(shape, generator=gen, device=DEV).to(t)
        st["vc"] = torch.randn(shape, generator=gen, device=DEV).to(t)
        if case["bias"]:
            h = torch.arange(1, heads + 1, device=DEV, dtype=torch.float32)
            st["slopes"] = torch.pow(2.0, -8.0 * h / heads)
        if case["docs"]:
            first = []
            for at, k, n in zip(_starts(case, kv), kv, ql):
                d = torch.tensor(at, device=DEV)
                p = torch.arange(k - n, k, device=DEV)
                first.append(d[torch.searchsorted(d, p, right=True) - 1])
            st["first"] = torch.cat(first).int()
        if case["prefix"]:
            st["prefix"] = torch.tensor(_prefixes(case, kv), dtype=torch.int32, device=DEV)
        return st
    st["kc"], st["kp"] = _pool4(case, total, gen)
    st["vc"], st["vp"] = _pool4(case, total, gen)
    if case["op"] == "append":
        st["k"], st["v"] = qkv[:, heads:heads + hk], qkv[:, heads + hk:]
        pos = torch.cat([torch.arange(k - n, k, device=DEV) for k, n in zip(kv, ql)])
        seq = torch.cat([torch.full((n,), s, device=DEV) for s, n in enumerate(ql)])
        st["pos"] = pos
        st["slots"] = st["table"][seq, pos // block].long() * block + pos % block
        angle = torch.arange(max(kv), device=DEV, dtype=torch.float64)[:, None] * torch.pow(
            10000.0, -torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return st


# ------------------------------------------------------------------ plain form
def _quantized(x):
    """Codes 0 .. 15 (float32) and (scale, minimum) f16 of rows x [..., dim]."""
    x = x.float().clamp(-32752.0, 32752.0)
    lo, hi = x.amin(-1), x.amax(-1)
    params = torch.stack([(hi - lo) * (1.0 / 15.0), lo], -1).half()
    s, m = params[..., 0:1].float(), params[..., 1:2].float()
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    return torch.round((x - m) * inv).clamp(0, 15), params


def _packed(n):
    """Codes as bytes: of each 8 elements the even ones' codes in the low, the
    odd ones' in the high half of a 32-bit word, four bits each in order."""
    n = n.to(torch.uint8).unflatten(-1, (-1, 4, 2)).transpose(-1, -2)    # [.., 8s, parity, 4]
    n = n.flatten(-2).unflatten(-1, (4, 2))
    return (n[..., 0] | (n[..., 1] << 4)).flatten(-2)


def _values(codes, params):
    """float32 values of packed codes [..., dim / 2] and params [..., 2]."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, 2, 4))
    n = n.transpose(-1, -2).flatten(-3)
    return n.float() * params[..., 0:1].float() + params[..., 1:2].float()


def _turned(st, x):
    case = st["case"]
    x = x.float()
    rot, half = case["rot"], case["rot"] // 2
    cs = st["cos_sin"][st["pos"]][:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(st):
    t, block = st["q"].dtype, st["case"]["block"]
    page, row = st["slots"] // block, st["slots"] % block
    kn, kp = _quantized(_turned(st, st["k"]))
    vn, vp = _quantized(st["v"])
    st["kc"][page, row], st["vc"][page, row] = _packed(kn), _packed(vn)
    st["kp"][page, :, row], st["vp"][page, :, row] = kp, vp
    key = _values(st["kc"][page, row], st["kp"][page, :, row])
    value = _values(st["vc"][page, row], st["vp"][page, :, row])
    return dict(q=_turned(st, st["q"]).to(t), key=key.to(t), value=value.to(t))


def _plain_rows(st, pool, params):
    """Every sequence's rows, float32 [sequences, rows, kv heads, dim]."""
    at = st["table"].long()
    if st["case"]["op"] == "score":
        return st[pool][at].flatten(1, 2).float()
    return _values(st[pool][at], st[params][at].transpose(2, 3)).flatten(1, 2)


def _plain_attention(st):
    case, q = st["case"], st["q"]
    cu, lens = st["cu"].long(), st["lens"].long()
    # Queries padded to [sequences, longest, kv heads, group, dim].
    i = torch.arange(st["max_q"], device=DEV)
    ql = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = torch.einsum("sqhgd,skhd->shgqk", q[at].float().unflatten(2, (case["kv_heads"], -1)),
                     _plain_rows(st, "kc", "kp"))
    x *= st["scale"]
    j = torch.arange(x.shape[-1], device=DEV)
    pos = (lens - ql)[:, None] + i                                      # [sequences, longest]
    seen = j <= pos[..., None]
    if case["op"] == "score":
        if case["cap"]:
            x = x.mul_(1.0 / case["cap"]).tanh_().mul_(case["cap"])
        if case["bias"]:
            away = (pos[..., None] - j).abs().float()
            x -= st["slopes"].unflatten(0, (case["kv_heads"], -1))[..., None, None] * \
                away[:, None, None]
        if case["prefix"]:
            seen |= j < st["prefix"].long()[:, None, None]
        if case["docs"]:
            seen &= j >= st["first"].long()[at][..., None]
    seen &= j < lens[:, None, None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.einsum("shgqk,skhd->sqhgd", x, _plain_rows(st, "vc", "vp"))
    o /= total.permute(0, 3, 1, 2, 4)
    lse = (top + torch.log(total))[..., 0].flatten(1, 2)                # [sequences, heads, longest]
    # Back to packed tokens.
    token = torch.arange(q.shape[0], device=DEV)
    s = torch.searchsorted(cu, token, right=True) - 1
    o, lse = o.flatten(2, 3)[s, token - cu[s]], lse[s, :, token - cu[s]].T
    return dict(out=o.to(q.dtype), lse=lse)


# ------------------------------------------------------------------ one pass
def _own(st):
    import paged_kv_varlen_attn_gb300 as pa
    case = st["case"]
    if case["op"] == "append":
        pools = (st["kc"], st["vc"], st["kp"], st["vp"])
        q = pa.rope_and_cache_int4(st["q"], st["k"], st["v"], st["pos"], st["cos_sin"], *pools,
                                   st["slots"], interleaved=case["interleaved"])
        key, value = pa.gather_cache_int4(*pools, st["slots"], st["q"].dtype)
        return dict(q=q, key=key, value=value)
    meta = (st["cu"], st["lens"], st["table"], st["max_q"], st["max_k"], st["scale"])
    if "ws" not in st:   # a workspace that the program keeps
        size = pa.varlen_fwd_int4kv_workspace_size if case["op"] == "int4" else \
            pa.varlen_fwd_workspace_size
        sms = torch.cuda.get_device_properties(DEV).multi_processor_count
        st["ws"] = pa.alloc_workspace(
            size(len(st["kv"]), st["q"].shape[0], st["max_q"], st["max_k"], case["heads"],
                 case["kv_heads"], case["dim"], case["block"], sms), DEV)
    if case["op"] == "int4":
        out, lse = pa.varlen_fwd_int4kv(st["q"], st["kc"], st["vc"], st["kp"], st["vp"], *meta,
                                        True, workspace=st["ws"])
    else:
        out, lse = pa.score_fwd(st["q"], st["kc"], st["vc"], *meta, softcap=case["cap"],
                                alibi_slopes=st.get("slopes"), first_key=st.get("first"),
                                prefix_lens=st.get("prefix"), workspace=st["ws"])
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "append":
        return _plain_append(state)
    return _plain_attention(state)


# ------------------------------------------------------------------ floors
def work(case):
    kv, ql = _lengths(case)
    hk, heads, dim, tokens = case["kv_heads"], case["heads"], case["dim"], sum(ql)
    if case["op"] == "append":
        # q, k, v in, q out; k and v in 4 bits and their scales out, and the
        # rows as values; positions, slots and table rows.
        moved = tokens * (4 * heads * dim + hk * dim * (4 + 1 + 4) + 8 * hk + 16)
        table = 4 * case["rot"] * min(tokens, max(kv))
        return {"bytes": moved + table,
                "flops": tokens * (3 * case["rot"] * (heads + hk) + 8 * hk * dim)}
    pages = 4 * sum(-(-k // case["block"]) for k in kv)
    rest = tokens * heads * (4 * dim + 4) + pages
    if case["op"] == "int4":
        pairs = sum(n * k - n * (n - 1) // 2 for k, n in zip(kv, ql))
        return {"bytes": hk * sum(kv) * (dim + 8) + rest, "flops": 4 * heads * dim * pairs}
    starts = _starts(case, kv) if case["docs"] else [[0]] * len(kv)
    prefix = _prefixes(case, kv) if case["prefix"] else [0] * len(kv)
    pairs = keys = 0
    for k, n, at, pre in zip(kv, ql, starts, prefix):
        ends = at[1:] + [k]
        for a, b in zip(at, ends):   # a document's queries p = max(a, k - n) .. b - 1
            p0 = max(a, k - n)
            if p0 >= b:
                continue
            low = max(p0, min(b, pre))   # queries below it see up to the prefix's end
            pairs += (low - p0) * (pre - a) if low > p0 else 0
            pairs += (b - low) * (low + b + 1) // 2 - (b - low) * a
        first = max((a for a in at if a <= k - n), default=0)
        keys += k - first
    return {"bytes": 4 * hk * dim * keys + rest, "flops": 4 * heads * dim * pairs}


# ------------------------------------------------------------------ definition in 64 bits
def _codes64(st, pool, params, page, row):
    """float64 [rows, kv heads, dim] of the rows at (page, row) of a 4-bit pool."""
    dim = st["case"]["dim"]
    d = torch.arange(dim, device=DEV)
    place = 4 * (d % 2) + d % 8 // 2                 # which four bits of its 32-bit word
    byte = st[pool][page, row][..., d // 8 * 4 + place // 2]
    n = torch.where(place % 2 == 0, byte % 16, byte // 16).double()
    p = st[params][page, :, row].double()
    return n * p[..., :1] + p[..., 1:]


def exact(case, seed):
    st = prepare(case, seed)
    block, hk, dim = case["block"], case["kv_heads"], case["dim"]
    group, t = case["heads"] // hk, st["q"].dtype
    if case["op"] == "append":
        rot = case["rot"]
        cs = st["cos_sin"].double()[st["pos"]][:, None]
        c, s = cs[..., :rot // 2], cs[..., rot // 2:]
        i = torch.arange(rot // 2, device=DEV)
        one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        got = {}
        for name, out in (("q", "q"), ("k", "key"), ("v", "value")):
            x = st[name].double()
            y = x.clone()
            if name != "v":
                y[..., one] = x[..., one] * c - x[..., two] * s
                y[..., two] = x[..., one] * s + x[..., two] * c
            if name != "q":
                low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
                step, low = ((high - low) / 15).half().double(), low.half().double()
                y = torch.clamp(torch.round((y - low) / step), 0, 15) * step + low
            got[out] = y
        return got
    tokens = sum(st["ql"])
    out = torch.zeros((tokens, case["heads"], dim), dtype=torch.float64, device=DEV)
    lse = torch.zeros((case["heads"], tokens), dtype=torch.float64, device=DEV)
    at = 0
    for s, (kv, ql) in enumerate(zip(st["kv"], st["ql"])):
        j = torch.arange(kv, device=DEV)
        page, row = st["table"][s].long()[j // block], j % block
        if case["op"] == "int4":
            key, value = _codes64(st, "kc", "kp", page, row), _codes64(st, "vc", "vp", page, row)
        else:
            key, value = st["kc"][page, row].double(), st["vc"][page, row].double()
        for a in range(0, ql, 2048):
            n = min(2048, ql - a)
            pos = (kv - ql + a + torch.arange(n, device=DEV))[:, None]
            hidden = j > pos
            if st.get("prefix") is not None:
                hidden &= j >= st["prefix"][s]
            if st.get("first") is not None:
                hidden |= j < st["first"][at + a:at + a + n, None]
            for h in range(case["heads"]):
                x = st["q"][at + a:at + a + n, h].double() @ key[:, h // group].T * st["scale"]
                if case.get("cap"):
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case.get("bias"):
                    x = x - st["slopes"][h].double() * (pos - j).abs()
                x[hidden] = -math.inf
                lse[h, at + a:at + a + n] = torch.logsumexp(x, 1)
                out[at + a:at + a + n, h] = torch.softmax(x, 1) @ value[:, h // group]
        at += ql
    return dict(out=out, lse=lse)
