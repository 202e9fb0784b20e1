"""Plain fp64 CPU definitions of the 4-bit cache format and of attention with
changed scores and masks. TEST INFRASTRUCTURE ONLY, like the rest of this
package."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
TOP = 32752.0


def quantize_int4(x):
    """(codes int64 [..., dim], params f16 [..., 2]) of float32 rows x [...,
    dim]: every operation in float32, rounded once, as the format asks."""
    x = x.float()
    nan = x.isnan().any(-1)
    y = x.nan_to_num(nan=0.0, posinf=TOP, neginf=-TOP).clamp(-TOP, TOP)
    low, high = y.min(-1).values, y.max(-1).values
    fifteenth = torch.tensor(1.0 / 15.0, dtype=torch.float32)
    scale, minimum = ((high - low) * fifteenth).half(), low.half()
    inv = torch.where(scale > 0, 1.0 / scale.float(), torch.zeros_like(low))
    codes = ((y - minimum.float()[..., None]) * inv[..., None]).clamp(0, 15).round()
    params = torch.stack([scale, minimum], -1)
    params[nan] = math.nan
    codes[nan] = 0
    return codes.long(), params


def place(d):
    """(byte, low half?) of element d in a row's codes."""
    word, i = divmod(d, 8)
    at = 4 * (i % 2) + i // 2          # which four bits of the word, from the lowest
    return 4 * word + at // 2, at % 2 == 0


def pack_int4(codes):
    """uint8 [..., dim / 2] of codes [..., dim]."""
    out = torch.zeros(codes.shape[:-1] + (codes.shape[-1] // 2,), dtype=torch.int64)
    for d in range(codes.shape[-1]):
        byte, low = place(d)
        out[..., byte] += codes[..., d] << (0 if low else 4)
    return out.to(torch.uint8)


def unpack_int4(packed):
    packed = packed.long()
    out = torch.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), dtype=torch.int64)
    for d in range(out.shape[-1]):
        byte, low = place(d)
        out[..., d] = (packed[..., byte] >> (0 if low else 4)) & 15
    return out


def int4_rows(pool, params, table_row, n, block):
    """float64 values [n, kv heads, dim] of a sequence's first n rows."""
    j = torch.arange(n)
    page, row = table_row.long()[j // block], j % block
    p = params.double()[page, :, row]
    return unpack_int4(pool[page, row]).double() * p[..., :1] + p[..., 1:]


def attend(q, key, value, scale, causal=True, sinks=None, cap=0.0, slopes=None, prefix=0,
           first=None):
    """One sequence: q [ql, H, D], key and value float64 [kv, Hkv, D]. Returns
    (out [ql, H, D], lse [H, ql]) in float64."""
    ql, H, D = q.shape
    kv, hk, _ = key.shape
    out = torch.zeros((ql, H, D), dtype=F64)
    lse = torch.full((H, ql), -math.inf, dtype=F64)
    pos = (kv - ql + torch.arange(ql))[:, None]
    j = torch.arange(kv)[None]
    seen = torch.ones((ql, kv), dtype=torch.bool)
    if causal:
        seen &= (j <= pos) | (j < prefix)
    if first is not None:
        seen &= j >= first.long()[:, None]
    for h in range(H):
        s = q[:, h].double() @ key[:, h // (H // hk)].T * scale
        if cap:
            s = cap * torch.tanh(s / cap)
        if slopes is not None:
            s = s - slopes[h].double() * (pos - j).abs()
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        extra = torch.full((ql, 1), -math.inf if sinks is None else float(sinks[h]), dtype=F64)
        s = torch.cat([s, extra], 1)
        lse[h] = torch.logsumexp(s, 1)
        some = lse[h] > -math.inf
        w = torch.exp(s[:, :-1] - torch.where(some, lse[h], torch.zeros_like(lse[h]))[:, None])
        w = torch.where(seen, w, torch.zeros_like(w))
        # A key that a row does not see adds nothing, whatever it holds.
        v = value[:, h // (H // hk)]
        out[:, h] = torch.where(w[..., None] == 0, torch.zeros((), dtype=F64),
                                w[..., None] * v[None]).sum(1) if v.isnan().any() else w @ v
    return out, lse
