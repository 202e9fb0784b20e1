"""Plain fp64 CPU definitions of the operators around paged attention: the
rotary table, norm + rotation, sliding-window attention with first tokens,
accumulated attention weights, and eviction by them. TEST INFRASTRUCTURE ONLY,
like the rest of this package."""
from __future__ import annotations

import math

import torch

from .paged_attention import gather_kv, kv_head_of

F64 = torch.float64


def rope_rates(rot_dim, base, scaling="none", factor=1.0, orig_len=0.0, low=None, high=None):
    """Radians per position of each pair, as Python floats."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    rates = [base ** (-2 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling == "linear":
        return [f / factor for f in rates]
    if scaling == "wavelength":
        low, high = 1.0 if low is None else low, 4.0 if high is None else high
        out = []
        for f in rates:
            n = orig_len * f / (2 * math.pi)
            keep = min(max((n - low) / (high - low), 0.0), 1.0)
            out.append(keep * f + (1 - keep) * f / factor)
        return out
    if scaling == "yarn":
        low, high = 1.0 if low is None else low, 32.0 if high is None else high

        def pair(n):
            return rot_dim * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(base))
        lo = max(math.floor(pair(high)), 0)
        hi = min(math.ceil(pair(low)), rot_dim - 1)
        out = []
        for i, f in enumerate(rates):
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            out.append(ramp * f / factor + (1 - ramp) * f)
        return out
    return rates


def rope_table(positions, rates, mscale=1.0):
    """[positions, 2 * pairs]: cosines, then sines."""
    angle = torch.as_tensor(positions, dtype=F64)[:, None] * torch.tensor(rates, dtype=F64)
    return mscale * torch.cat([angle.cos(), angle.sin()], 1)


def norm_rotate(x, rows, interleaved, weight=None, eps=0.0):
    """x [tokens, heads, dim] normed (weight given) and rotated by the table
    rows [tokens, rot_dim], in float64, unrounded."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    rot = rows.shape[1]
    y = x.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = rows[:, i].double()[:, None], rows[:, rot // 2 + i].double()[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def window_visible(q_len, kv_len, window, num_first):
    """bool [q_len, kv_len]: which keys each query sees."""
    p = torch.arange(kv_len - q_len, kv_len)[:, None]
    j = torch.arange(kv_len)
    return (j <= p) & ((j > p - window) | (j < num_first))


def _attend(q, k, v, scale, seen, sink=None):
    """One head: q [n, d], k, v [m, d], seen [n, m] -> (out [n, d], lse [n])."""
    x = (q @ k.T) * scale
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    if sink is not None:
        x = torch.cat([x, torch.full((x.shape[0], 1), float(sink), dtype=F64)], 1)
        v = torch.cat([v, v.new_zeros((1, v.shape[1]))])
    lse = torch.logsumexp(x, 1) if x.shape[1] else torch.full((x.shape[0],), -math.inf, dtype=F64)
    p = torch.where(torch.isfinite(lse)[:, None], torch.exp(x - lse[:, None]),
                    torch.zeros_like(x))
    # a key nobody sees contributes nothing, whatever its value holds
    return p @ torch.where((p != 0).any(0)[:, None], v, torch.zeros_like(v)), lse


def window_attention(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table,
                     softmax_scale, window, num_first, sinks=None):
    """(out [T, H, D], lse [H, T]) of causal attention in which query position p
    sees keys j <= p with j > p - window or j < num_first. key_cache and
    value_cache hold the values themselves (dequantized for e4m3 pools)."""
    T, H, D = q.shape
    out = torch.zeros((T, H, D), dtype=F64)
    lse = torch.full((H, T), -math.inf, dtype=F64)
    for s in range(len(seqused_k)):
        a, b, kv = int(cu_seqlens_q[s]), int(cu_seqlens_q[s + 1]), int(seqused_k[s])
        k = gather_kv(key_cache, block_table[s], kv).double()
        v = gather_kv(value_cache, block_table[s], kv).double()
        seen = window_visible(b - a, kv, window, num_first)
        for h in range(H):
            g = kv_head_of(h, H, key_cache.shape[2])
            out[a:b, h], lse[h, a:b] = _attend(q[a:b, h].double(), k[:, g], v[:, g],
                                               softmax_scale, seen,
                                               None if sinks is None else sinks[h])
    return out, lse


def attn_weights(q, key_cache, lse, weights, cu_seqlens_q, seqused_k, block_table,
                 softmax_scale, causal):
    """The updated weights [num_blocks, H_kv, block_size] in float64."""
    T, H, D = q.shape
    bs, hk = key_cache.shape[1], key_cache.shape[2]
    w = weights.double().clone()
    for s in range(len(seqused_k)):
        a, b, kv = int(cu_seqlens_q[s]), int(cu_seqlens_q[s + 1]), int(seqused_k[s])
        n = b - a
        if n == 0 or kv == 0:
            continue
        k = gather_kv(key_cache, block_table[s], kv).double()
        p = torch.arange(kv - n, kv)[:, None]
        seen = torch.arange(kv) <= p if causal else torch.ones((n, kv), dtype=torch.bool)
        got = torch.zeros((hk, kv), dtype=F64)
        for h in range(H):
            g = kv_head_of(h, H, hk)
            row = lse[h, a:b].double()
            x = torch.exp((q[a:b, h].double() @ k[:, g].T) * softmax_scale - row[:, None])
            x = torch.where(seen & torch.isfinite(row)[:, None], x, torch.zeros_like(x))
            got[g] += x.sum(0)
        for j in range(kv):
            page, r = int(block_table[s, j // bs]), j % bs
            w[page, :, r] = (0.0 if j >= kv - n else w[page, :, r]) + got[:, j]
    return w


def evict(key_cache, value_cache, weights, seqused_k, block_table, budget, num_first, num_recent):
    """Updated copies (key_cache, value_cache, weights, kept, lens)."""
    kc, vc, w = key_cache.clone(), value_cache.clone(), weights.clone()
    bs, hk = kc.shape[1], kc.shape[2]
    S = len(seqused_k)
    kept = torch.full((S, hk, budget), -1, dtype=torch.int32)
    lens = torch.zeros(S, dtype=torch.int32)
    for s in range(S):
        kv = int(seqused_k[s])
        lens[s] = min(kv, budget)
        for h in range(hk):
            if kv <= budget:
                kept[s, h, :kv] = torch.arange(kv, dtype=torch.int32)
                continue

            def place(j):
                return int(block_table[s, j // bs]), j % bs

            def heavy(j):
                p, r = place(j)
                x = float(weights[p, h, r])
                return -math.inf if math.isnan(x) else x
            ranked = sorted(range(num_first, kv - num_recent), key=lambda j: (-heavy(j), j))
            keep = sorted(list(range(num_first)) +
                          ranked[:budget - num_first - num_recent] +
                          list(range(kv - num_recent, kv)))
            for d, j in enumerate(keep):
                (pd, rd), (ps, rs) = place(d), place(j)
                kc[pd, rd, h] = key_cache[ps, rs, h]
                vc[pd, rd, h] = value_cache[ps, rs, h]
                w[pd, h, rd] = weights[ps, h, rs]
            kept[s, h] = torch.tensor(keep, dtype=torch.int32)
    return kc, vc, w, kept, lens
