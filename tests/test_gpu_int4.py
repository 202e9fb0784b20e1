"""GPU parity of the 4-bit cache writes, the way back, and attention over 4-bit
pools with their definitions.

Tolerances, from arithmetic:
  * codes and params without a norm: equal (every step is one rounded float32
    operation). With a norm the float32 row is off by a few 2^-24 of its
    largest element, so a code may move by one where the quotient lies that near
    to a border, and the f16 params by one step.
  * scores: with A = scale * sum |q_i| max_i |k_i| over a row, float32 sums of
    at most 256 terms in at most 64 roundings are off by 2^-18 A for sums of
    values. The kernels sum codes and q apart, scale (q.n) + minimum sum q, whose
    parts are up to 3 A (a row's range is at most twice its largest): 3 2^-18 A.
    LSE: that, and 2^-20 (1 + |lse|) for the logarithm and the exponentials.
  * outputs: e = 2 (score error + 2^-20) times the largest |v| of the head from
    the weights; 2^-11 (f16, half a step) of the largest weight x code sum, at
    most the largest row range of V, and of |v| (minimum and range: 3 |v|max);
    half a step of the output type.
"""
import math

import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from oracle import changed_scores as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


# ------------------------------------------------------------------ cache writes
def turned(x, rows, interleaved):
    """x float32 [T, heads, D] rotated by table rows float32 [T, rot], every
    product and sum rounded to float32."""
    rot = rows.shape[1]
    cos, sin = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def new_tokens(seed, T, H, hk, D, bs, dtype, rot=0, packed=True):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((T, H + 2 * hk, D), generator=g) *
           torch.logspace(-2, 2, T)[:, None, None]).to(dtype)
    nb = (T + bs - 1) // bs + 3
    slots = torch.randperm(nb * bs, generator=g)[:T]
    pos = torch.randint(0, 600, (T,), generator=g)
    angle = torch.arange(600, dtype=torch.float64)[:, None] * torch.pow(
        10000.0, -torch.arange(0, max(rot, 2), 2, dtype=torch.float64) / max(rot, 2))
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    d = qkv.to(DEV)
    parts = [d[:, :H], d[:, H:H + hk], d[:, H + hk:]]
    if not packed:
        parts = [p.contiguous() for p in parts]
    return qkv, parts, nb, slots, pos, table


def filled_pools(nb, bs, hk, D, extra=0):
    """Pools of recognisable bytes on the GPU, with `extra` pages' worth between
    pages, and copies on the CPU."""
    codes = [torch.full((nb, (1 + extra) * bs, hk, D // 2), 0xA5 + i, dtype=torch.uint8, device=DEV)
             for i in range(2)]
    params = [torch.full((nb, (1 + extra) * hk, bs, 2), 7.0 + i, dtype=torch.float16, device=DEV)
              for i in range(2)]
    return [c[:, :bs] for c in codes] + [p[:, :hk] for p in params], codes + params


def check_rows(pools, whole, slots, bs, hk, want_codes, want_params, exact=True):
    """The written rows hold the codes and params, the others their bytes."""
    ok = (slots >= 0) & (slots < pools[0].shape[0] * bs)
    at = slots[ok]
    for i in range(2):
        codes, params = pools[i].cpu(), pools[2 + i].cpu()
        got_c, got_p = codes[at // bs, at % bs], params[at // bs, :, at % bs]
        if exact:
            assert torch.equal(got_c, ref.pack_int4(want_codes[i][ok]))
            assert torch.equal(got_p.view(torch.int16), want_params[i][ok].view(torch.int16))
        else:
            moved = (ref.unpack_int4(got_c) - want_codes[i][ok]).abs()
            assert moved.max() <= 1 and moved.float().mean() < 1e-3
            step = (got_p.float() - want_params[i][ok].float()).abs()
            assert (step <= want_params[i][ok].float().abs() * 2.0 ** -10 + 2.0 ** -24).all()
        w = whole[i].cpu()
        flat = torch.ones(w.shape[:2], dtype=torch.bool)
        flat[at // bs, at % bs] = False
        assert (w[flat] == 0xA5 + i).all()
        w = whole[2 + i].cpu()
        left = torch.ones((w.shape[0], w.shape[1], w.shape[2]), dtype=torch.bool)
        for h in range(hk):
            left[at // bs, h, at % bs] = False
        assert (w[left] == 7.0 + i).all()


@pytest.mark.parametrize("T,H,hk,D,bs,dt,rot,inter", [
    (1, 8, 2, 64, 16, "f16", 64, False),
    (37, 4, 1, 128, 16, "bf16", 128, False),
    (300, 8, 8, 128, 48, "f16", 64, True),
    (65, 6, 3, 64, 32, "bf16", 32, True),
    (129, 10, 5, 64, 16, "f16", 16, False),
    (1030, 32, 8, 128, 64, "bf16", 128, False),
])
def test_rope_write_bits(T, H, hk, D, bs, dt, rot, inter):
    dtype = TYPES[dt]
    qkv, (q, k, v), nb, slots, pos, table = new_tokens(T, T, H, hk, D, bs, dtype, rot, T % 2 == 0)
    pools, whole = filled_pools(nb, bs, hk, D, extra=T % 3 == 0)
    out = pa.rope_and_cache_int4(q, k, v, pos.to(DEV), table.to(DEV), *pools, slots.to(DEV),
                                 interleaved=inter)
    kc, kp = ref.quantize_int4(turned(qkv[:, H:H + hk].float(), table[pos], inter))
    vc, vp = ref.quantize_int4(qkv[:, H + hk:].float())
    check_rows(pools, whole, slots, bs, hk, (kc, vc), (kp, vp))
    want = turned(qkv[:, :H].float(), table[pos], inter).to(dtype)
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T,hk,D,bs,dt", [(1, 1, 64, 16, "bf16"), (77, 3, 128, 32, "f16"),
                                          (515, 8, 64, 48, "f16"), (200, 8, 128, 16, "bf16")])
def test_plain_write_and_gather(T, hk, D, bs, dt):
    dtype = TYPES[dt]
    qkv, (_, k, v), nb, slots, _, _ = new_tokens(T + 5, T, 0, hk, D, bs, dtype)
    slots[T // 2] = -1                                # padding
    if T > 3:
        slots[1] = nb * bs + 5                        # past the pool
    pools, whole = filled_pools(nb, bs, hk, D)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.reshape_and_cache_int4(k, v, *pools, slots.to(DEV), dev_status=status)
    assert status.item() == (pa.PA_DEV_BAD_SLOT if T > 3 else 0)
    want = [ref.quantize_int4(qkv[:, i * hk:(i + 1) * hk].float()) for i in range(2)]
    check_rows(pools, whole, slots, bs, hk, [w[0] for w in want], [w[1] for w in want])
    # ... and back: one rounding of code * scale + minimum.
    status.zero_()
    got = pa.gather_cache_int4(*pools, slots.to(DEV), dtype, dev_status=status)
    assert status.item() == (pa.PA_DEV_BAD_SLOT if T > 3 else 0)
    ok = (slots >= 0) & (slots < nb * bs)
    for (codes, params), rows in zip(want, got):
        p = params.float()
        value = (codes.float() * p[..., :1] + p[..., 1:]).to(dtype)
        value[~ok] = 0
        assert torch.equal(rows.cpu().view(torch.int16), value.view(torch.int16))


def test_norm_write():
    T, H, hk, D, bs, rot = 140, 8, 2, 128, 16, 64
    qkv, (q, k, v), nb, slots, pos, table = new_tokens(9, T, H, hk, D, bs, torch.bfloat16, rot)
    g = torch.Generator().manual_seed(2)
    qw, kw = (1 + 0.1 * torch.randn(D, generator=g) for _ in range(2))
    pools, whole = filled_pools(nb, bs, hk, D)
    out = pa.rope_and_cache_int4(q, k, v, pos.to(DEV), table.to(DEV), *pools, slots.to(DEV),
                                 q_norm=qw.to(DEV), k_norm=kw.to(DEV), eps=1e-6)

    def normed(x, w):
        x = x.double()
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    rows = table[pos].double()
    kc, kp = ref.quantize_int4(turned(normed(qkv[:, H:H + hk], kw), rows, False).float())
    vc, vp = ref.quantize_int4(qkv[:, H + hk:].float())
    check_rows(pools, whole, slots, bs, hk, (kc, vc), (kp, vp), exact=False)
    want = turned(normed(qkv[:, :H], qw), rows, False)
    tol = want.abs() * 2.0 ** -8 + want.abs().amax(-1, keepdim=True) * 2.0 ** -19
    assert ((out.cpu().double() - want).abs() <= tol).all()


def test_write_edges():
    # NaN, infinities, constants, values past f16, subnormal ranges.
    hk, D, bs = 1, 128, 16
    x = torch.randn((8, hk, D))
    x[0, 0, 5] = math.nan
    x[1, 0, 6] = math.inf
    x[2, 0, 7] = -math.inf
    x[3] = -2.5
    x[4] *= 1e30
    x[5] *= 1e-7
    x[6] = 0.0
    x[7, 0, :64] = 1e-30
    x = x.bfloat16()
    pools, whole = filled_pools(2, bs, hk, D)
    slots = torch.arange(8) + 3
    pa.reshape_and_cache_int4(x.to(DEV), x.to(DEV), *pools, slots.to(DEV))
    codes, params = ref.quantize_int4(x.float())
    got = pools[2].cpu()[slots // bs, :, slots % bs]
    assert got[0].isnan().all() and torch.equal(got[1:], params[1:])
    packed = pools[0].cpu()[slots // bs, slots % bs]
    assert torch.equal(packed[1:], ref.pack_int4(codes)[1:])
    back = pa.gather_cache_int4(*pools, slots.to(DEV), torch.bfloat16)[0].cpu()
    assert back[0].isnan().all() and not back[1:].isnan().any()


def test_padding_positions():
    T, H, hk, D, bs = 12, 2, 1, 64, 16
    qkv, (q, k, v), nb, slots, pos, table = new_tokens(4, T, H, hk, D, bs, torch.float16, 64)
    pos[3], pos[7] = -1, 600                          # padding, and past the table
    pools, whole = filled_pools(nb, bs, hk, D)
    out = torch.full((T, H, D), 9.0, dtype=torch.float16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.rope_and_cache_int4(q, k, v, pos.to(DEV), table.to(DEV), *pools, slots.to(DEV), out=out,
                           dev_status=status)
    assert status.item() == pa.PA_DEV_BAD_POSITION
    keep = torch.ones(T, dtype=torch.bool)
    keep[3] = keep[7] = False
    assert (out.cpu()[~keep] == 9.0).all()
    kc, kp = ref.quantize_int4(turned(qkv[keep, H:H + hk].float(), table[pos[keep]], False))
    vc, vp = ref.quantize_int4(qkv[keep, H + hk:].float())
    check_rows(pools, whole, slots[keep], bs, hk, (kc, vc), (kp, vp))


# ------------------------------------------------------------------ attention
class Batch:
    """Sequences of (kv, ql) over permuted pages; table entries past a
    sequence's pages are out of range, spare rows hold NaN params."""

    def __init__(self, seqs, H, hk, D, bs, dt, seed=0, spread=1.0, qscale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.H, self.hk, self.D, self.bs, self.dtype = seqs, H, hk, D, bs, TYPES[dt]
        need = [-(-kv // bs) for kv, _ in seqs]
        nb = sum(need) + 3
        order = torch.randperm(nb, generator=g)
        width = max(need + [1]) + 1
        self.table = torch.full((len(seqs), width), 2 ** 30, dtype=torch.int32)
        self.kc, self.vc, self.kp, self.vp = [], [], [], []
        x = torch.randn((2, nb, bs, hk, D), generator=g)
        x *= torch.exp(spread * torch.randn((2, nb, bs, hk, 1), generator=g))
        x += 0.5 * torch.randn((2, 1, 1, hk, D), generator=g)
        pools = [ref.quantize_int4(y) for y in x]
        self.codes = [ref.pack_int4(n) for n, _ in pools]
        self.params = [p.transpose(1, 2).contiguous() for _, p in pools]
        used = torch.zeros((nb, bs), dtype=torch.bool)
        at = 0
        for s, ((kv, _), n) in enumerate(zip(seqs, need)):
            pages = order[at:at + n]
            self.table[s, :n] = pages.int()
            j = torch.arange(kv)
            used[pages[j // bs], j % bs] = True
            at += n
        for p in self.params:
            p.masked_fill_(~used[:, None, :, None], math.nan)
        self.T = sum(q for _, q in seqs)
        self.q = (qscale * torch.randn((self.T, H, D), generator=g)).to(self.dtype)
        self.cu = torch.tensor([0] + [q for _, q in seqs]).cumsum(0).int()
        self.lens = torch.tensor([kv for kv, _ in seqs], dtype=torch.int32)
        self.max_q, self.max_k = max(q for _, q in seqs), max(kv for kv, _ in seqs)
        self.scale = D ** -0.5

    def run(self, causal=True, scale=None, **kw):
        d = [t.to(DEV) for t in (self.q, *self.codes, *self.params, self.cu, self.lens, self.table)]
        return pa.varlen_fwd_int4kv(*d, kw.pop("max_q", self.max_q), kw.pop("max_k", self.max_k),
                                    self.scale if scale is None else scale, causal, **kw)

    def check(self, out, lse, causal=True, scale=None, sinks=None, seqs=None):
        out, lse = out.cpu().double(), lse.cpu().double()
        scale = self.scale if scale is None else scale
        half = torch.finfo(self.dtype).eps / 2
        for s in range(len(self.seqs)) if seqs is None else seqs:
            kv, ql = self.seqs[s]
            if ql == 0:
                continue
            rows = slice(int(self.cu[s]), int(self.cu[s]) + ql)
            key = ref.int4_rows(self.codes[0], self.params[0], self.table[s], kv, self.bs)
            value = ref.int4_rows(self.codes[1], self.params[1], self.table[s], kv, self.bs)
            want, wl = ref.attend(self.q[rows], key, value, scale, causal, sinks)
            q = self.q[rows].double()
            big_k = key.abs().amax((0, 2)) if kv else torch.zeros(self.hk)
            big_v = value.abs().amax((0, 2)) if kv else torch.zeros(self.hk)
            group = self.H // self.hk
            A = abs(scale) * q.abs().sum(-1) * big_k.repeat_interleave(group)      # [ql, H]
            err = A * 3 * 2.0 ** -18
            fin = torch.isfinite(wl)
            assert torch.equal(fin, torch.isfinite(lse[:, rows]))
            lt = err.T + 2.0 ** -20 * (1 + wl.abs())
            assert ((lse[:, rows] - wl).abs() <= lt)[fin].all(), s
            v = big_v.repeat_interleave(group)
            tol = half * want.abs() + (v * (2 * (err + 2.0 ** -20) + 3 * 2.0 ** -11))[..., None]
            off = (out[rows] - want).abs()
            assert (off <= tol + 1e-30).all(), (s, (off - tol).max())


SHORT = [
    # (sequences (kv, ql), H, Hkv, D, block, type)
    ([(1, 1)], 1, 1, 64, 16, "f16"),
    ([(17, 1), (1, 1), (0, 1), (300, 1), (16, 1)], 8, 2, 64, 16, "bf16"),
    ([(100, 1), (700, 1), (64, 0), (65, 1)], 8, 1, 128, 32, "f16"),
    ([(515, 1), (33, 1), (2100, 1)], 32, 8, 128, 16, "bf16"),
    ([(40, 2), (513, 1), (2, 2)], 12, 4, 128, 48, "f16"),              # G = 3
    ([(90, 1), (1000, 1)], 35, 5, 64, 128, "bf16"),                    # G = 7, five KV heads
    ([(200, 5), (3, 5), (1500, 5), (50, 1)], 16, 4, 128, 16, "f16"),   # 20 rows
    ([(200, 4), (3, 4), (700, 3)], 8, 2, 64, 16, "bf16"),              # 16 rows
    ([(600, 1), (31, 1)], 32, 1, 128, 64, "bf16"),                     # G = 32
    ([(400, 2)], 24, 2, 64, 16, "f16"),                                # G = 12: 24 rows
    ([(5000, 1)], 4, 4, 128, 16, "f16"),                               # many ranges of one
    ([(70, 1)] * 100 + [(0, 0)] * 40 + [(900, 1)] * 3, 2, 2, 64, 16, "bf16"),   # many sequences
]


@pytest.mark.parametrize("seqs,H,hk,D,bs,dt", SHORT)
def test_short_queries(seqs, H, hk, D, bs, dt):
    b = Batch(seqs, H, hk, D, bs, dt, seed=len(seqs) + H)
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_short_not_causal_sinks_scales(dt):
    b = Batch([(100, 3), (2, 3), (0, 2), (333, 1)], 8, 2, 128, 16, dt, seed=3)
    sinks = torch.randn(8)
    for scale in (b.scale, -0.2, 0.0):
        for causal in (True, False):
            out, lse = b.run(causal, scale, sinks=sinks.to(DEV))
            b.check(out, lse, causal, scale, sinks)
    out, lse = b.run(False)
    b.check(out, lse, False)


def test_short_large_and_small_numbers():
    # Queries at the ends of bf16, scales of V's rows that differ by 2^20.
    b = Batch([(150, 1), (40, 2)], 4, 2, 128, 16, "bf16", seed=8, spread=3.0)
    b.q[0] *= 1e30
    b.q[1] *= 1e-30
    out, lse = b.run(scale=1e-3)
    b.check(out, lse, scale=1e-3)


def test_bounds_and_workspace_reuse():
    b = Batch([(515, 1), (33, 1), (2100, 1)], 32, 8, 128, 16, "bf16", seed=1)
    ws = pa.alloc_workspace(pa.varlen_fwd_int4kv_workspace_size(
        3, 3, 1, 1 << 30, 32, 8, 128, 16, torch.cuda.get_device_properties(0).multi_processor_count),
        DEV)
    ws.fill_(255)
    out, lse = b.run(workspace=ws, max_k=1 << 30)     # a bound far too large
    out2, lse2 = b.run(workspace=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    b.check(out, lse)


def test_bad_pages_and_lengths():
    b = Batch([(100, 1), (50, 1)], 4, 2, 64, 16, "f16", seed=2)
    b.table[0, 3] = 10 ** 6
    b.table[1, 0] = -5
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = b.run(dev_status=status)
    assert status.item() == pa.PA_DEV_BAD_PAGE
    # Such a page's keys and values read as zeros.
    b.codes = [torch.cat([c, torch.zeros_like(c[:1])]) for c in b.codes]
    b.params = [torch.cat([p, torch.zeros_like(p[:1])]) for p in b.params]
    b.table[0, 3] = b.table[1, 0] = b.codes[0].shape[0] - 1
    b.check(out, lse)
    # Keys above the bound are reported.
    b = Batch([(100, 1), (50, 1)], 4, 2, 64, 16, "f16", seed=2)
    status.zero_()
    b.run(dev_status=status, max_k=60)
    assert status.item() == pa.PA_DEV_BAD_SEQLEN


def test_nan_rows_stay_theirs():
    # A NaN row of V is one sequence's; a later token's is not seen by earlier queries.
    b = Batch([(100, 2), (60, 1)], 4, 2, 128, 16, "f16", seed=5)
    last = b.table[0, 99 // 16]
    b.params[1][last, :, 99 % 16] = math.nan
    out, lse = b.run()
    assert out[1].isnan().all() and not out[0].isnan().any() and not out[2].isnan().any()
    assert not lse.isnan().any()


def test_update_in_the_call():
    # The new tokens written by the call itself: as two calls, bit for bit.
    b = Batch([(100, 1), (37, 2), (16, 1)], 8, 2, 128, 16, "bf16", seed=6)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((b.T, 2, 128), generator=g).bfloat16().to(DEV) for _ in range(2))
    slots = []
    for s, (kv, ql) in enumerate(b.seqs):
        for p in range(kv - ql, kv):
            slots.append(int(b.table[s, p // 16]) * 16 + p % 16)
    slots = torch.tensor(slots, device=DEV)
    pools = [t.to(DEV) for t in (*b.codes, *b.params)]
    meta = [t.to(DEV) for t in (b.cu, b.lens, b.table)]
    one = [t.clone() for t in pools]
    out, lse = pa.varlen_fwd_int4kv(b.q.to(DEV), *one, *meta, b.max_q, b.max_k, b.scale, True,
                                    key=k, value=v, slot_mapping=slots)
    pa.reshape_and_cache_int4(k, v, *pools, slots)
    out2, lse2 = pa.varlen_fwd_int4kv(b.q.to(DEV), *pools, *meta, b.max_q, b.max_k, b.scale, True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for x, y in zip(one, pools):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


LONG = [
    # Prompts, chunks and mixed batches (more than 32 packed rows somewhere).
    ([(33, 33)], 1, 1, 64, 16, "f16"),
    ([(100, 100), (1, 1), (17, 9)], 8, 2, 128, 16, "bf16"),
    ([(300, 300), (129, 40), (0, 20)], 6, 2, 128, 48, "f16"),               # G = 3
    ([(700, 130), (515, 1), (64, 64), (40, 3), (90, 0)], 16, 4, 64, 32, "bf16"),
    ([(260, 260)], 8, 8, 128, 64, "bf16"),                                  # a KV head per head
    ([(400, 7)], 40, 1, 128, 128, "f16"),                                   # G = 40
    ([(3000, 50), (2500, 33)], 8, 2, 128, 16, "bf16"),                      # split over the keys
    ([(128, 128), (256, 129)], 32, 4, 64, 16, "f16"),
]


@pytest.mark.parametrize("seqs,H,hk,D,bs,dt", LONG)
def test_prompts(seqs, H, hk, D, bs, dt):
    b = Batch(seqs, H, hk, D, bs, dt, seed=len(seqs) + D + bs)
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prompts_not_causal_sinks_scales(dt):
    b = Batch([(200, 70), (20, 50)], 8, 2, 128, 16, dt, seed=23)
    sinks = torch.randn(8)
    for scale in (b.scale, -0.2, 0.0):
        for causal in (True, False):
            out, lse = b.run(causal, scale, sinks=sinks.to(DEV))
            b.check(out, lse, causal, scale, sinks)


def test_prompts_large_and_small_numbers():
    b = Batch([(150, 100)], 4, 2, 128, 16, "bf16", seed=28, spread=1.0)
    b.q[:30] *= 1e30
    b.q[30:60] *= 1e-30
    b.q[60] = 0
    out, lse = b.run(scale=1e-3)
    b.check(out, lse, scale=1e-3)


def test_prompt_bad_pages():
    b = Batch([(300, 60)], 4, 2, 128, 16, "f16", seed=29)
    b.table[0, 3] = 10 ** 6
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = b.run(dev_status=status)
    assert status.item() == pa.PA_DEV_BAD_PAGE
    b.codes = [torch.cat([c, torch.zeros_like(c[:1])]) for c in b.codes]
    b.params = [torch.cat([p, torch.zeros_like(p[:1])]) for p in b.params]
    b.table[0, 3] = b.codes[0].shape[0] - 1
    b.check(out, lse)


def test_run_together_and_captured():
    # A prompt and then decode steps as a program runs them, eagerly and captured:
    # rotate and write, attend; the same bits, and the definition's values.
    g = torch.Generator().manual_seed(77)
    H, hk, D, bs, n = 8, 2, 128, 16, 90
    ends = [(0, n), (n, n + 1), (n + 1, n + 2), (n + 2, n + 3)]
    table = torch.randperm(12, generator=g)[None].int()
    rows = pa.rope_table(200, D, device=DEV)
    d_table = table.to(DEV)
    qkv = torch.randn((n + 3, H + 2 * hk, D), generator=g).bfloat16()
    d_qkv = qkv.to(DEV)
    got = []
    for captured in (False, True):
        pools = pa.int4_pools(12, bs, hk, D, DEV)
        for a, b in ends:
            pos = torch.arange(a, b, device=DEV)
            slots = d_table[0, pos // bs].long() * bs + pos % bs
            x = d_qkv[a:b]
            cu = torch.tensor([0, b - a], dtype=torch.int32, device=DEV)
            lens = torch.tensor([b], dtype=torch.int32, device=DEV)
            sms = torch.cuda.get_device_properties(0).multi_processor_count
            ws = pa.alloc_workspace(pa.varlen_fwd_int4kv_workspace_size(
                1, b - a, b - a, b, H, hk, D, bs, sms), DEV)
            q = torch.empty((b - a, H, D), dtype=torch.bfloat16, device=DEV)
            out, lse = torch.empty_like(q), torch.empty((H, b - a), device=DEV)

            def step():
                pa.rope_and_cache_int4(x[:, :H], x[:, H:H + hk], x[:, H + hk:], pos, rows, *pools,
                                       slots, out=q)
                pa.varlen_fwd_int4kv(q, *pools, cu, lens, d_table, b - a, b, D ** -0.5, True,
                                     out=out, lse=lse, workspace=ws)
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
                graph.replay()
                graph.replay()
            else:
                step()
            torch.cuda.synchronize()
            got.append((q.clone(), out.clone(), lse.clone()))
    for one, two in zip(got[:4], got[4:]):
        assert all(torch.equal(x, y) for x, y in zip(one, two))
    cos_sin = rows.cpu()
    kq = ref.quantize_int4(turned(qkv[:, H:H + hk].float(), cos_sin[:n + 3], False))
    vq = ref.quantize_int4(qkv[:, H + hk:].float())
    key, value = (c.double() * p[..., :1].double() + p[..., 1:].double() for c, p in (kq, vq))
    for (a, b), (q, out, lse) in zip(ends, got):
        assert torch.equal(q.cpu(), turned(qkv[a:b, :H].float(), cos_sin[a:b], False).bfloat16())
        want, wl = ref.attend(q.cpu(), key[:b], value[:b], D ** -0.5)
        # Weights 2^-11 and V 2^-11 of values up to 4, scores 3 2^-18 A with A < 40.
        err = 3 * 40 * 2.0 ** -18
        tol = want.abs() * 2.0 ** -8 + 4 * (2 * err + 3 * 2.0 ** -11)
        assert ((out.cpu().double() - want).abs() <= tol).all()
        assert ((lse.cpu().double() - wl).abs() <= err + 1e-5).all()


@pytest.mark.parametrize("seqs,dt", [([(300, 1), (77, 1), (900, 3)], "f16"),
                                     ([(200, 90), (50, 1), (700, 40)], "bf16")])
def test_strided_pools_and_queries_past_32_bits(seqs, dt):
    # Pages of K and V in one tensor, their params in another, pages 2^21 bytes apart over
    # 5 GB; queries that are a slice of a wider row; tokens behind the last sequence.
    H, hk, D, bs = 8, 2, 128, 16
    b = Batch(seqs, H, hk, D, bs, dt, seed=31)
    nb, page = b.codes[0].shape[0], bs * hk * D // 2
    far = 5 * 2 ** 30 // 2 ** 21 - nb                 # the batch's pages are the last ones
    store = torch.empty(((far + nb) * 2 ** 21,), dtype=torch.uint8, device=DEV)
    shape, stride = (far + nb, bs, hk, D // 2), (2 ** 21, hk * D // 2, D // 2, 1)
    codes = [store.as_strided(shape, stride, x * page) for x in (0, 1)]
    params = torch.zeros((far + nb, 2, hk, bs, 2), dtype=torch.float16, device=DEV)
    for x in (0, 1):
        codes[x][far:].copy_(b.codes[x])
        params[far:, x].copy_(b.params[x])
    table = torch.where(b.table < nb, b.table + far, b.table).to(DEV)
    wide = torch.randn((b.T + 5, H + 3, D), device=DEV).to(b.dtype)
    wide[:b.T, 2:2 + H] = b.q.to(DEV)
    out = torch.full((b.T + 5, H, D), 7.0, dtype=b.dtype, device=DEV)
    lse = torch.full((H, b.T + 5), 7.0, device=DEV)
    pa.varlen_fwd_int4kv(wide[:, 2:2 + H], *codes, params[:, 0], params[:, 1], b.cu.to(DEV),
                         b.lens.to(DEV), table, b.max_q, b.max_k, b.scale, True, out=out, lse=lse)
    assert (out[b.T:] == 7.0).all() and (lse[:, b.T:] == 7.0).all()
    b.check(out[:b.T], lse[:, :b.T])
    # The write and the way back at the same far pages; one row asked for twice.
    slots = torch.tensor([(far + nb - 1) * bs + 3, (far + nb - 2) * bs, (far + nb - 1) * bs + 9])
    x = torch.randn((2, 3, hk, D)).to(b.dtype)
    pools = (*codes, params[:, 0], params[:, 1])
    pa.reshape_and_cache_int4(x[0].to(DEV), x[1].to(DEV), *pools, slots.to(DEV))
    again = slots[[0, 1, 2, 0]]
    rows = pa.gather_cache_int4(*pools, again.to(DEV), torch.float16)
    for got, new in zip(rows, x):
        n, p = ref.quantize_int4(new.float())
        want = (n.float() * p[..., :1].float() + p[..., 1:].float()).half()[[0, 1, 2, 0]]
        assert torch.equal(got.cpu(), want)


def test_two_streams_and_two_graphs():
    # Two batches at once on streams of their own; then two graphs that share a
    # workspace, replayed in turn.
    batches = [Batch([(1500, 1), (40, 5), (300, 60)], 8, 2, 128, 16, "f16", seed=41),
               Batch([(700, 1)] * 9 + [(129, 40)], 4, 4, 64, 32, "bf16", seed=42)]
    alone = [b.run() for b in batches]
    args = [[t.to(DEV) for t in (b.q, *b.codes, *b.params, b.cu, b.lens, b.table)] for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in batches]
    got = []
    for _ in range(5):
        for b, d, s in zip(batches, args, streams):
            with torch.cuda.stream(s):
                got.append(pa.varlen_fwd_int4kv(*d, b.max_q, b.max_k, b.scale, True))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[i % 2][0]) and torch.equal(lse, alone[i % 2][1])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = pa.alloc_workspace(max(pa.varlen_fwd_int4kv_workspace_size(
        len(b.seqs), b.T, b.max_q, b.max_k, b.H, b.hk, b.D, b.bs, sms) for b in batches), DEV)
    graphs, outs = [], []
    for b, d in zip(batches, args):
        outs.append((torch.empty_like(d[0]), torch.empty((b.H, b.T), device=DEV)))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pa.varlen_fwd_int4kv(*d, b.max_q, b.max_k, b.scale, True, out=outs[-1][0],
                                 lse=outs[-1][1], workspace=ws)
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, alone):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("hk", [1, 3, 4, 7])
@pytest.mark.parametrize("ql", [1, 20])
def test_lengths_around_every_border(hk, ql):
    # Keys around the pages, the steps of 32 keys, the runs of a block and a key tile.
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]
    b = Batch([(n, min(n, ql)) for n in lens], 2 * hk, hk, 64, 48, "bf16", seed=hk)
    out, lse = b.run()
    b.check(out, lse)
