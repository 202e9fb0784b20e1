"""Timed cases of the cache-side operators around paged attention.

One decoder layer that keeps its K/V cache small does, per step: rotate the
new queries and keys (with the per-head norms, if the model has them) and
write K/V into pages; attend with a sliding window and a few first tokens that
stay visible; or, with full attention, add up how much weight every cached key
received and from time to time throw the least used ones out.

``op`` of a case:
  table    rotary cos/sin table of a model's positions, with long-context scaling
  rope     per-head RMS norm + rotation of q and k, k and v written to their pages
  window   paged attention with a sliding window and first tokens (prompt, chunk, decode)
  weights  accumulated attention weight of every cached key
  evict    keep the heaviest keys of each KV head, compact the pages in place

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
        # The table of an 8k-context model, and of a long-context one whose
        # frequencies are interpolated band by band: built once at start-up.
        dict(name="table-8k", op="table", length=8192, rot=128, base=500000.0, scaling="none",
             factor=1.0, orig=8192),
        dict(name="table-128k", op="table", length=131072, rot=128, base=1000000.0,
             scaling="yarn", factor=4.0, orig=32768),
        # One decode step of 64 requests (32/8 heads), with q/k norms.
        dict(name="rope-decode", op="rope", seqs=64, lens=11, kv_lo=512, kv_hi=8192, q=1, heads=32,
             kv_heads=8, dim=128, block=16, type="bf16", fp8=False, rot=128, interleaved=False,
             norm=True),
        # Eight 2048-token prompt chunks; interleaved pairs on half of the head.
        dict(name="rope-chunks", op="rope", seqs=8, lens=12, kv_lo=2048, kv_hi=6144, q=2048,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", fp8=False, rot=64,
             interleaved=True, norm=False),
        # Prompt chunks of a 64/8-head model into an e4m3 cache.
        dict(name="rope-fp8", op="rope", seqs=7, lens=13, kv_lo=600, kv_hi=4096, q=587, heads=64,
             kv_heads=8, dim=128, block=128, type="f16", fp8=True, rot=128, interleaved=False,
             norm=True),
        # Two requests of a small model: what one call costs.
        dict(name="window-small", op="window", seqs=2, lens=21, kv_lo=300, kv_hi=700, q=1, heads=8,
             kv_heads=2, dim=64, block=16, type="f16", fp8=False, window=128, first=4),
        # A decode batch whose layer looks back 1024 keys and at 4 first ones.
        dict(name="window-decode", op="window", seqs=64, lens=22, kv_lo=512, kv_hi=8192, q=1,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", fp8=False, window=1024,
             first=4),
        # Whole prompts through the same layer.
        dict(name="window-prompt", op="window", seqs=4, lens=23, kv_lo=3500, kv_hi=4500, q=0,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", fp8=False, window=1024,
             first=4),
        # Decode step of 64 requests: the new query's weight on every key.
        dict(name="weights-decode", op="weights", seqs=64, lens=31, kv_lo=512, kv_hi=8192, q=1,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", fp8=False),
        # After a prompt: all of its queries' weights.
        dict(name="weights-prompt", op="weights", seqs=2, lens=32, kv_lo=2500, kv_hi=4096, q=0,
             heads=32, kv_heads=8, dim=128, block=16, type="bf16", fp8=False),
        # A decode batch grown a few hundred keys past its budget.
        dict(name="evict-decode", op="evict", seqs=64, lens=41, kv_lo=900, kv_hi=1400, kv_heads=8,
             dim=128, block=16, type="bf16", fp8=False, budget=1024, first=4, recent=256),
        # Long prompts cut down to 2048 keys before decoding starts.
        dict(name="evict-prompt", op="evict", seqs=4, lens=42, kv_lo=12000, kv_hi=16384,
             kv_heads=8, dim=128, block=16, type="bf16", fp8=False, budget=2048, first=4,
             recent=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("table", "rope", "rope", "window", "window", "window", "weights", "weights",
                     "evict", "evict"))
    if op == "table":
        scaling = rng.choice(("none", "linear", "ntk", "yarn", "wavelength"))
        return dict(op=op, length=_log(rng, 1, 131072), rot=2 * rng.randint(8, 64),
                    base=float(rng.choice((10000, 500000, 1000000))), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice((2.0, 4.0, 8.0)),
                    orig=rng.choice((4096, 8192, 32768)))
    case = dict(op=op, lens=rng.randrange(1 << 30), kv_heads=rng.choice((1, 2, 4, 8)),
                dim=rng.choice((64, 128, 128, 256)), block=rng.choice((16, 32, 64, 128)),
                type=rng.choice(("bf16", "f16")), fp8=False)
    if case["dim"] == 128:
        case["fp8"] = rng.random() < 0.35
    if op == "evict":
        case["budget"] = _log(rng, 64, 2048)
        case["first"] = rng.choice((0, 1, 4, 16))
        case["recent"] = rng.randint(0, case["budget"] // 2)
        case["seqs"] = _log(rng, 1, 32)
        top = min(16384, 65536 // case["seqs"])
        case["kv_hi"] = _log(rng, min(case["budget"], top), top)
        case["kv_lo"] = max(1, case["kv_hi"] * rng.randint(5, 10) // 10)
        return case
    case["heads"] = case["kv_heads"] * rng.choice((1, 2, 3, 4, 7, 8))
    kind = rng.choice(("decode", "chunk", "prompt"))
    if kind == "decode":
        case["seqs"], case["q"] = _log(rng, 1, 64), rng.choice((1, 1, 1, 2, 5))
        case["kv_hi"] = _log(rng, 16, 8192)
        case["kv_lo"] = max(1, case["kv_hi"] // rng.randint(1, 16))
    elif kind == "chunk":
        case["seqs"], case["q"] = _log(rng, 1, 6), _log(rng, 9, 600)
        case["kv_hi"] = _log(rng, case["q"], 4096)
        case["kv_lo"] = max(1, case["kv_hi"] // rng.randint(1, 4))
    else:
        case["seqs"], case["q"] = rng.randint(1, 3), 0
        case["kv_hi"] = _log(rng, 16, 2500)
        case["kv_lo"] = max(1, case["kv_hi"] // rng.randint(1, 4))
    if op == "rope":
        case["rot"] = case["dim"] // rng.choice((1, 1, 2, 4))
        case["interleaved"] = rng.random() < 0.5
        case["norm"] = rng.random() < 0.5
    if op == "window":
        case["window"] = _log(rng, 1, 2048)
        case["first"] = rng.choice((0, 1, 4, 16, 100))
    return case


def _lengths(case):
    """(kv lengths, query lengths) of the case's sequences."""
    rng = random.Random(case["lens"])
    kv = [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["seqs"])]
    n = case.get("q", 0)
    return kv, [k if n == 0 else min(n, k) for k in kv]


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


def _pool(case, total, gen):
    """(pool, per-KV-head scale or None) of N(0, 1) values."""
    shape = (total, case["block"], case["kv_heads"], case["dim"])
    x = torch.randn(shape, generator=gen, device=DEV)
    if not case["fp8"]:
        return x.to(TYPES[case["type"]]), None
    scale = torch.linspace(0.02, 0.05, case["kv_heads"], device=DEV)
    codes = (x / scale[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "table":
        # The positions start at 0; the base is the input that may differ.
        st["base"] = case["base"] * (1.0 + (seed % 1009) / 1009.0)
        return st
    kv, ql = _lengths(case)
    total, st["table"] = _pages(case, kv)
    st["kv"], st["ql"] = kv, ql
    st["lens"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    st["kc"], st["ks"] = _pool(case, total, gen)
    block, dim, hk = case["block"], case["dim"], case["kv_heads"]
    if case["op"] == "evict":
        st["vc"], st["vs"] = _pool(case, total, gen)
        # Sums of attention weights: few large, most small, some exactly zero.
        w = torch.rand((total, hk, block), generator=gen, device=DEV)
        st["weights"] = torch.where(w < 0.1, torch.zeros_like(w), w.pow(6) * 3.0)
        return st
    tokens, heads, t = sum(ql), case["heads"], TYPES[case["type"]]
    cu = [0]
    for n in ql:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    st["scale"] = dim ** -0.5
    # q, k and v as a projection leaves them: slices of one packed row.
    qkv = torch.randn((tokens, heads + 2 * hk, dim), generator=gen, device=DEV).to(t)
    st["q"] = qkv[:, :heads]
    if case["op"] == "rope":
        st["k"], st["v"] = qkv[:, heads:heads + hk], qkv[:, heads + hk:]
        st["vc"], st["vs"] = _pool(case, total, gen)
        pos = torch.cat([torch.arange(k - n, k, device=DEV) for k, n in zip(kv, ql)])
        seq = torch.cat([torch.full((n,), s, device=DEV) for s, n in enumerate(ql)])
        st["pos"] = pos
        st["slots"] = st["table"][seq, pos // block].long() * block + pos % block
        angle = torch.arange(max(kv), device=DEV, dtype=torch.float64)[:, None] * torch.pow(
            10000.0, -torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["norm"]:
            st["qw"] = 1.0 + 0.1 * torch.randn(dim, generator=gen, device=DEV)
            st["kw"] = 1.0 + 0.1 * torch.randn(dim, generator=gen, device=DEV)
        return st
    if case["op"] == "window":
        st["vc"], st["vs"] = _pool(case, total, gen)
        if own:
            import paged_kv_varlen_attn_gb300 as pa
            size = pa.varlen_fwd_fp8kv_workspace_size if case["fp8"] else pa.varlen_fwd_workspace_size
            sms = torch.cuda.get_device_properties(DEV).multi_processor_count
            st["ws"] = pa.alloc_workspace(size(len(kv), tokens, max(ql), max(kv), heads, hk, dim,
                                               block, sms), DEV)
        return st
    # weights: the sums so far, and the log-sum-exp that attention returned
    st["weights"] = torch.rand((total, hk, block), generator=gen, device=DEV)
    lse = torch.empty((heads, tokens), device=DEV)
    for s in range(len(kv)):
        key = _rows(st, "kc", "ks", s)
        for a, b, x in _scores(st, s, key, torch.arange(kv[s], device=DEV)):
            lse[:, a:b] = torch.logsumexp(x, -1).flatten(0, 1)
    st["lse"] = lse
    return st


# ------------------------------------------------------------------ plain form
def _rows(st, pool, scale, s, length=None):
    """The first rows of sequence s of a pool, float32 [rows, kv heads, dim]."""
    case, n = st["case"], st["kv"][s] if length is None else length
    rows = st[pool][st["table"][s, :-(-n // case["block"])].long()].flatten(0, 1)[:n]
    if not case["fp8"]:
        return rows.float()
    return rows.view(torch.float8_e4m3fn).float() * st[scale][:, None]


def _scores(st, s, key, at_keys, window=None, first=0):
    """Scaled, masked scores of sequence s against the keys at positions
    at_keys: (first token, last token + 1, [kv heads, group, rows, keys]) per
    chunk of queries."""
    case, kv, ql = st["case"], st["kv"][s], st["ql"][s]
    start = sum(st["ql"][:s])
    step = max(1, (1 << 27) // (case["heads"] * len(at_keys)))
    for a in range(0, ql, step):
        b = min(ql, a + step)
        q = st["q"][start + a:start + b].float().unflatten(1, (case["kv_heads"], -1))
        x = torch.einsum("thgd,khd->hgtk", q, key) * st["scale"]
        at = torch.arange(kv - ql + a, kv - ql + b, device=DEV)[:, None]
        seen = at_keys <= at
        if window is not None:
            seen &= (at_keys > at - window) | (at_keys < first)
        yield start + a, start + b, x.masked_fill_(~seen, -math.inf)


def _plain_table(st):
    case = st["case"]
    rot, base, factor, orig = case["rot"], st["base"], case["factor"], case["orig"]
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    mscale = 1.0
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = torch.pow(base, -2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "wavelength":
        low, high = 1.0, 4.0
        mix = ((orig * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f / factor * (1 - mix) + f * mix
    elif case["scaling"] == "yarn":
        slow, fast = 1.0, 32.0
        lo = max(math.floor(rot * math.log(orig / (fast * 2 * math.pi)) / (2 * math.log(base))), 0)
        hi = min(math.ceil(rot * math.log(orig / (slow * 2 * math.pi)) / (2 * math.log(base))),
                 rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        mscale = 0.1 * math.log(factor) + 1.0
    angle = torch.arange(case["length"], device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([angle.cos() * mscale, angle.sin() * mscale], 1).float()


def _plain_rotate(st, x, weight):
    case = st["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * weight
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


def _plain_store(st, pool, scale, x):
    flat = st[pool].flatten(0, 1)
    if st["case"]["fp8"]:
        x = (x / st[scale][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    flat[st["slots"]] = x.to(flat.dtype)
    return st[pool].view(torch.float8_e4m3fn) if st["case"]["fp8"] else st[pool]


def _plain_rope(st):
    q = _plain_rotate(st, st["q"], st.get("qw")).to(st["q"].dtype)
    key = _plain_store(st, "kc", "ks", _plain_rotate(st, st["k"], st.get("kw")))
    value = _plain_store(st, "vc", "vs", st["v"].float())
    return dict(q=q, key=key, value=value)


def _plain_window(st):
    case, q = st["case"], st["q"]
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    lse = torch.empty((case["heads"], q.shape[0]), device=DEV)
    for s, (kv, ql) in enumerate(zip(st["kv"], st["ql"])):
        # The positions that some query of the sequence sees.
        lo = max(0, kv - ql - case["window"] + 1)
        head = min(case["first"], lo)
        at = torch.cat([torch.arange(head, device=DEV), torch.arange(lo, kv, device=DEV)])
        key, value = _rows(st, "kc", "ks", s), _rows(st, "vc", "vs", s)
        key = torch.cat([key[:head], key[lo:]])
        value = torch.cat([value[:head], value[lo:]])
        for a, b, x in _scores(st, s, key, at, case["window"], case["first"]):
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            total = p.sum(-1, keepdim=True)
            o = torch.einsum("hgtk,khd->thgd", p / total, value)
            out[a:b] = o.flatten(1, 2).to(q.dtype)
            lse[:, a:b] = (top + torch.log(total))[..., 0].flatten(0, 1)
    return dict(out=out, lse=lse)


def _plain_weights(st):
    case, pool = st["case"], st["weights"]
    hk, block = case["kv_heads"], case["block"]
    for s, (kv, ql) in enumerate(zip(st["kv"], st["ql"])):
        key = _rows(st, "kc", "ks", s)
        at = torch.arange(kv, device=DEV)
        got = torch.zeros((hk, kv), device=DEV)
        for a, b, x in _scores(st, s, key, at):
            lse = st["lse"][:, a:b].unflatten(0, (hk, -1))
            got += torch.exp(x - lse[..., None]).sum((1, 2))
        pages, old = _weight_rows(st, s)
        # The call's own keys start from nothing.
        old[:, :kv - ql] += got[:, :kv - ql]
        old[:, kv - ql:kv] = got[:, kv - ql:]
        pool[pages] = old.unflatten(1, (-1, block)).transpose(0, 1)
    return pool


def _weight_rows(st, s):
    """(page ids, float32 [kv heads, rows of those pages]) of sequence s."""
    n = -(-st["kv"][s] // st["case"]["block"])
    pages = st["table"][s, :n].long()
    return pages, st["weights"][pages].transpose(0, 1).flatten(1)


def _plain_evict(st):
    case = st["case"]
    hk, block, budget = case["kv_heads"], case["block"], case["budget"]
    first, recent = case["first"], case["recent"]
    recent = min(recent, budget - first)
    kept = torch.full((len(st["kv"]), hk, budget), -1, dtype=torch.int32, device=DEV)
    lens = torch.clamp(st["lens"], max=budget)
    at = torch.arange(budget, device=DEV)
    for s, kv in enumerate(st["kv"]):
        if kv <= budget:
            kept[s, :, :kv] = at[:kv].int()
            continue
        pages, rows = _weight_rows(st, s)
        middle = rows[:, first:kv - recent].nan_to_num(nan=-math.inf, posinf=math.inf,
                                                       neginf=-math.inf)
        order = torch.sort(middle, dim=1, descending=True, stable=True).indices
        keep = order[:, :budget - first - recent] + first
        keep = torch.cat([at[:first].expand(hk, -1), keep,
                          torch.arange(kv - recent, kv, device=DEV).expand(hk, -1)], 1)
        keep = torch.sort(keep, dim=1).values
        kept[s] = keep.int()
        head = torch.arange(hk, device=DEV)[:, None]
        src = pages[keep // block], keep % block
        dst = pages[at // block], at % block
        for name in ("kc", "vc"):
            st[name][dst[0][None], dst[1][None], head] = st[name][src[0], src[1], head]
        st["weights"][dst[0][None], head, dst[1][None]] = rows.gather(1, keep)
    fp8 = torch.float8_e4m3fn
    return dict(kept=kept, lens=lens, weights=st["weights"],
                key=st["kc"].view(fp8) if case["fp8"] else st["kc"],
                value=st["vc"].view(fp8) if case["fp8"] else st["vc"])


# ------------------------------------------------------------------ one pass
def _own(st):
    import paged_kv_varlen_attn_gb300 as pa
    case = st["case"]
    if case["op"] == "table":
        return pa.rope_table(case["length"], case["rot"], st["base"], scaling=case["scaling"],
                             factor=case["factor"], orig_len=case["orig"], device=DEV)
    fp8 = torch.float8_e4m3fn
    if case["op"] == "rope":
        q = pa.rope_and_cache(st["q"], st["k"], st["v"], st["pos"], st["cos_sin"], st["kc"],
                              st["vc"], st["slots"], interleaved=case["interleaved"],
                              q_norm=st.get("qw"), k_norm=st.get("kw"), eps=1e-6,
                              k_scale=st["ks"], v_scale=st["vs"])
        return dict(q=q, key=st["kc"].view(fp8) if case["fp8"] else st["kc"],
                    value=st["vc"].view(fp8) if case["fp8"] else st["vc"])
    if case["op"] == "evict":
        kept, lens = pa.evict(st["kc"], st["vc"], st["weights"], st["lens"], st["table"],
                              max(st["kv"]), case["budget"], case["first"],
                              min(case["recent"], case["budget"] - case["first"]))
        return dict(kept=kept, lens=lens, weights=st["weights"],
                    key=st["kc"].view(fp8) if case["fp8"] else st["kc"],
                    value=st["vc"].view(fp8) if case["fp8"] else st["vc"])
    meta = (st["cu"], st["lens"], st["table"], max(st["ql"]), max(st["kv"]), st["scale"])
    if case["op"] == "weights":
        return pa.attn_weights(st["q"], st["kc"], st["lse"], st["weights"], *meta, True,
                               k_scale=st["ks"])
    out, lse = pa.window_fwd(st["q"], st["kc"], st["vc"], *meta, case["window"],
                             num_first=case["first"], k_scale=st["ks"], v_scale=st["vs"],
                             workspace=st.get("ws"))
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _own(state)
    return dict(table=_plain_table, rope=_plain_rope, window=_plain_window,
                weights=_plain_weights, evict=_plain_evict)[state["case"]["op"]](state)


# ------------------------------------------------------------------ floors
def _seen(kv, ql, window, first):
    """(query, key) pairs and distinct keys that ql queries at the end of kv
    keys see."""
    pairs = 0
    for p in range(kv - ql, kv):
        pairs += min(p + 1, window + min(first, max(0, p + 1 - window)))
    lo = max(0, kv - ql - window + 1)
    return pairs, kv - lo + min(first, lo)


def work(case):
    op = case["op"]
    if op == "table":
        n = case["length"] * case["rot"]
        return {"bytes": 4 * n, "flops": 4 * n}
    kv, ql = _lengths(case)
    hk, dim, block = case["kv_heads"], case["dim"], case["block"]
    esize = 1 if case["fp8"] else 2
    pages = 4 * sum(-(-k // block) for k in kv)
    if op == "evict":
        rows = sum(case["budget"] - case["first"] for k in kv if k > case["budget"])
        held = sum(k for k in kv if k > case["budget"])
        out = 4 * hk * case["budget"] * len(kv)
        return {"bytes": rows * hk * (4 * dim * esize + 4) + 4 * hk * held + out + pages,
                "flops": hk * held}
    heads, tokens = case["heads"], sum(ql)
    if op == "rope":
        moved = tokens * (4 * heads * dim + hk * dim * (4 + 2 * esize) + 16)
        table = 4 * case["rot"] * min(tokens, max(kv))
        per = 3 * case["rot"] + (3 * dim if case["norm"] else 0)
        return {"bytes": moved + table, "flops": tokens * (heads + hk) * per}
    if op == "window":
        seen = [_seen(k, n, case["window"], case["first"]) for k, n in zip(kv, ql)]
        return {"bytes": 2 * esize * hk * dim * sum(x[1] for x in seen) +
                tokens * heads * (4 * dim + 4),
                "flops": 4 * heads * dim * sum(x[0] for x in seen)}
    pairs = sum(n * k - n * (n - 1) // 2 for k, n in zip(kv, ql))
    old = sum(k - n for k, n in zip(kv, ql))
    return {"bytes": hk * sum(kv) * (dim * esize + 4) + 4 * hk * old +
            tokens * heads * (2 * dim + 4) + pages,
            "flops": 2 * heads * dim * pairs}


# ------------------------------------------------------------------ definition in 64 bits
def _key_rows64(st, name, scale, s):
    """Sequence s of a pool as float64 [kv heads, keys, dim], row by row from
    the page table."""
    case = st["case"]
    j = torch.arange(st["kv"][s], device=DEV)
    x = st[name][st["table"][s].long()[j // case["block"]], j % case["block"]]
    if case["fp8"]:
        x = x.view(torch.float8_e4m3fn).float()
    x = x.double().permute(1, 0, 2)
    return x * st[scale].double()[:, None, None] if case["fp8"] else x


def _codes64(st, name):
    x = st[name]
    return (x.view(torch.float8_e4m3fn).float() if st["case"]["fp8"] else x).double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "table":
        return _exact_table(st)
    if op == "rope":
        return _exact_rope(st)
    if op == "evict":
        return _exact_evict(st)
    hk, group, block = case["kv_heads"], case["heads"] // case["kv_heads"], case["block"]
    tokens = sum(st["ql"])
    out = torch.zeros((tokens, case["heads"], case["dim"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((case["heads"], tokens), dtype=torch.float64, device=DEV)
    sums = st["weights"].double() if op == "weights" else None
    at = 0
    for s, (kv, ql) in enumerate(zip(st["kv"], st["ql"])):
        key = _key_rows64(st, "kc", "ks", s)
        value = _key_rows64(st, "vc", "vs", s) if op == "window" else None
        j = torch.arange(kv, device=DEV)
        page, row = st["table"][s].long()[j // block], j % block
        if op == "weights":   # the call's own keys start from zero
            fresh = j >= kv - ql
            for h in range(hk):
                sums[page, h, row] = torch.where(fresh, 0.0, sums[page, h, row])
        for c in range(0, ql, 1024):
            n = min(1024, ql - c)
            pos = (kv - ql + c + torch.arange(n, device=DEV))[:, None]
            hidden = j > pos
            if op == "window":
                hidden = hidden | ((j <= pos - case["window"]) & (j >= case["first"]))
            for h in range(case["heads"]):
                q = st["q"][at + c:at + c + n, h].double()
                x = (q @ key[h // group].T) * st["scale"]
                x[hidden] = -math.inf
                if op == "weights":
                    x = torch.exp(x - st["lse"][h, at + c:at + c + n, None].double())
                    sums[page, h // group, row] += x.sum(0)
                    continue
                lse[h, at + c:at + c + n] = torch.logsumexp(x, 1)
                out[at + c:at + c + n, h] = torch.softmax(x, 1) @ value[h // group]
        at += ql
    return sums if op == "weights" else dict(out=out, lse=lse)


def _exact_table(st):
    case = st["case"]
    rot, base, factor, orig = case["rot"], st["base"], case["factor"], case["orig"]
    freqs, kind = [], case["scaling"]
    mscale = 0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0

    def pair_of(turns):   # the pair that turns this often within the original length
        return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if kind == "linear":
            f /= factor
        elif kind == "ntk":
            f = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif kind == "wavelength":
            turns = orig * f / (2 * math.pi)
            if turns <= 1.0:
                f /= factor
            elif turns < 4.0:
                share = (turns - 1.0) / 3.0
                f = (1 - share) * f / factor + share * f
        elif kind == "yarn":
            lo = max(math.floor(pair_of(32.0)), 0)
            hi = min(math.ceil(pair_of(1.0)), rot - 1)
            share = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f / factor * share + f * (1 - share)
        freqs.append(f)
    f = torch.tensor(freqs, dtype=torch.float64, device=DEV)
    angle = torch.arange(case["length"], dtype=torch.float64, device=DEV).outer(f)
    return mscale * torch.cat((torch.cos(angle), torch.sin(angle)), -1)


def _exact_rope(st):
    case = st["case"]
    rot, dim = case["rot"], case["dim"]
    cs = st["cos_sin"].double()[st["pos"]]
    i = torch.arange(rot // 2, device=DEV)
    one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + 1e-6) * weight.double()
        y = x.clone()
        c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
        y[..., one] = x[..., one] * c - x[..., two] * s
        y[..., two] = x[..., one] * s + x[..., two] * c
        return y
    key, value = _codes64(st, "kc"), _codes64(st, "vc")
    k, v = turned(st["k"], st.get("kw")), st["v"].double()
    if case["fp8"]:
        k, v = k / st["ks"].double()[:, None], v / st["vs"].double()[:, None]
    page, row = st["slots"] // case["block"], st["slots"] % case["block"]
    key[page, row], value[page, row] = k, v
    return dict(q=turned(st["q"], st.get("qw")), key=key, value=value)


def _exact_evict(st):
    case = st["case"]
    block, budget, first = case["block"], case["budget"], case["first"]
    recent = min(case["recent"], budget - first)
    key, value = _codes64(st, "kc"), _codes64(st, "vc")
    weights = st["weights"].double()
    old = dict(key=key.clone(), value=value.clone(), weights=weights.clone())
    sums, table = st["weights"].cpu(), st["table"].cpu().long()
    kept = torch.full((len(st["kv"]), case["kv_heads"], budget), -1, dtype=torch.int32)
    for s, kv in enumerate(st["kv"]):
        for h in range(case["kv_heads"]):
            if kv <= budget:
                kept[s, h, :kv] = torch.arange(kv, dtype=torch.int32)
                continue
            j = torch.arange(kv)
            w = sums[table[s][j // block], h, j % block].tolist()
            ranked = sorted(range(first, kv - recent), key=lambda k: (-w[k], k))
            keep = sorted(list(range(first)) + ranked[:budget - first - recent] +
                          list(range(kv - recent, kv)))
            kept[s, h] = torch.tensor(keep, dtype=torch.int32)
            src, dst = torch.tensor(keep, device=DEV), torch.arange(budget, device=DEV)
            pages = st["table"][s].long()
            src, dst = (pages[src // block], src % block), (pages[dst // block], dst % block)
            key[dst[0], dst[1], h] = old["key"][src[0], src[1], h]
            value[dst[0], dst[1], h] = old["value"][src[0], src[1], h]
            weights[dst[0], h, dst[1]] = old["weights"][src[0], h, src[1]]
    lens = torch.tensor([min(k, budget) for k in st["kv"]], dtype=torch.int32, device=DEV)
    return dict(kept=kept.to(DEV), lens=lens, weights=weights, key=key, value=value)
