"""GPU parity of attention with changed scores and masks with its definition.

Tolerances, from arithmetic:
  * scores: float32 sums of at most 256 terms in at most 64 roundings are off by
    2^-18 A, A = scale sum |q_i| max_i |k_i| over a row. A cap has slope at most
    one, and its exponential (2 units of 2^-23), reciprocal (1) and final sum add
    at most 2^-20 cap; a polynomial, 6e-7 of scores up to half the cap or 2e-7 of
    scores up to the cap, less. The bias is rounded twice: 2^-22 of its size.
    LSE: that, and 2^-20 (1 + |lse|) for the logarithm and the exponentials.
  * outputs: 2 (score error + 2^-20) of the largest |v| from the weights, half a
    step of the type for the weights' rounding, of |v|; half a step of the output.
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


class Batch:
    """Sequences of (kv, ql) over permuted pages; spare rows hold NaN, table
    entries past a sequence's pages are out of range."""

    def __init__(self, seqs, H, hk, D, bs, dt, seed=0, qscale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.H, self.hk, self.D, self.bs, self.dtype = seqs, H, hk, D, bs, TYPES[dt]
        need = [-(-kv // bs) for kv, _ in seqs]
        nb = sum(need) + 2
        order = torch.randperm(nb, generator=g)
        self.table = torch.full((len(seqs), max(need + [1])), 2 ** 30, dtype=torch.int32)
        self.kc, self.vc = (torch.randn((nb, bs, hk, D), generator=g).to(self.dtype)
                            for _ in range(2))
        used = torch.zeros((nb, bs), dtype=torch.bool)
        at = 0
        for s, ((kv, _), n) in enumerate(zip(seqs, need)):
            pages = order[at:at + n]
            self.table[s, :n] = pages.int()
            j = torch.arange(kv)
            used[pages[j // bs], j % bs] = True
            at += n
        self.kc[~used] = math.nan
        self.vc[~used] = math.nan
        self.T = sum(q for _, q in seqs)
        self.q = (qscale * torch.randn((self.T, H, D), generator=g)).to(self.dtype)
        self.cu = torch.tensor([0] + [q for _, q in seqs]).cumsum(0).int()
        self.lens = torch.tensor([kv for kv, _ in seqs], dtype=torch.int32)
        self.max_q, self.max_k = max(q for _, q in seqs), max(kv for kv, _ in seqs)
        self.scale = D ** -0.5
        self.g = g

    def slopes(self):
        return torch.pow(2.0, -8.0 * torch.arange(1, self.H + 1) / self.H)

    def documents(self, shortest, longest):
        """First key per token, documents of random lengths."""
        first = []
        for kv, ql in self.seqs:
            at = [0]
            while at[-1] < kv:
                at.append(at[-1] + int(torch.randint(shortest, longest + 1, (1,),
                                                     generator=self.g)))
            d = torch.tensor(at)
            p = torch.arange(kv - ql, kv)
            first.append(d[(torch.searchsorted(d, p, right=True) - 1).clamp(min=0)])
        return torch.cat(first).int()

    def prefixes(self):
        return torch.tensor([int(torch.randint(0, kv + 5, (1,), generator=self.g))
                             for kv, _ in self.seqs], dtype=torch.int32)

    def run(self, scale=None, **kw):
        d = [t.to(DEV) for t in (self.q, self.kc, self.vc, self.cu, self.lens, self.table)]
        kw = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in kw.items()}
        return pa.score_fwd(*d, self.max_q, self.max_k, self.scale if scale is None else scale,
                            **kw)

    def check(self, out, lse, scale=None, softcap=0.0, alibi_slopes=None, prefix_lens=None,
              first_key=None, sinks=None, seqs=None):
        out, lse = out.cpu().double(), lse.cpu().double()
        scale = self.scale if scale is None else scale
        half = torch.finfo(self.dtype).eps / 2
        group = self.H // self.hk
        for s in range(len(self.seqs)) if seqs is None else seqs:
            kv, ql = self.seqs[s]
            if ql == 0:
                continue
            rows = slice(int(self.cu[s]), int(self.cu[s]) + ql)
            j = torch.arange(kv)
            page, row = self.table[s].long()[j // self.bs], j % self.bs
            key, value = self.kc[page, row].double(), self.vc[page, row].double()
            want, wl = ref.attend(
                self.q[rows], key, value, scale, True, sinks, softcap, alibi_slopes,
                0 if prefix_lens is None else min(int(prefix_lens[s]), kv),
                None if first_key is None else first_key[rows])
            q = self.q[rows].double()
            zero = torch.zeros(self.hk, dtype=torch.float64)
            A = abs(scale) * q.abs().sum(-1) * \
                (key.abs().amax((0, 2)) if kv else zero).repeat_interleave(group)
            err = A * 2.0 ** -18 + softcap * 2.0 ** -20
            if alibi_slopes is not None:
                err = err + kv * alibi_slopes.double().abs() * 2.0 ** -22
            v = (value.abs().amax((0, 2)) if kv else zero).repeat_interleave(group)
            fin = torch.isfinite(wl)
            assert torch.equal(fin, torch.isfinite(lse[:, rows]))
            assert ((lse[:, rows] - wl).abs() <= err.T + 2.0 ** -20 * (1 + wl.abs()))[fin].all(), s
            tol = half * want.abs() + (v * (2 * (err + 2.0 ** -20) + half))[..., None]
            off = (out[rows] - want).abs()
            assert (off <= tol + 1e-30).all(), (s, (off - tol).max())


SHAPES = [
    # (sequences (kv, ql), H, Hkv, D, block, type)
    ([(1, 1)], 1, 1, 64, 16, "bf16"),
    ([(100, 1), (700, 1), (64, 0), (65, 1), (0, 1)], 8, 2, 128, 32, "f16"),         # decode
    ([(2000, 1), (3, 1)], 32, 8, 128, 16, "bf16"),
    ([(90, 5), (400, 5), (3, 5)], 12, 4, 64, 48, "f16"),                            # 15 rows
    ([(200, 7), (30, 9)], 8, 2, 128, 16, "bf16"),                                   # 28-36 rows
    ([(300, 300), (129, 129)], 6, 2, 128, 64, "bf16"),                              # prompts, G = 3
    ([(700, 150), (64, 64), (257, 1), (40, 40)], 8, 8, 64, 16, "f16"),              # mixed
    ([(333, 200), (128, 128)], 4, 1, 256, 32, "bf16"),
    ([(500, 1), (70, 2)], 4, 2, 256, 16, "f16"),                                    # decode at 256
]
CHANGES = ["cap", "bias", "docs", "prefix", "cap+bias", "docs+prefix", "cap+bias+docs+prefix"]


def change(b, what):
    kw = {}
    if "cap" in what:
        kw["softcap"] = 12.5
    if "bias" in what:
        kw["alibi_slopes"] = b.slopes()
    if "docs" in what:
        kw["first_key"] = b.documents(1, 150)
    if "prefix" in what:
        kw["prefix_lens"] = b.prefixes()
    return kw


@pytest.mark.parametrize("what", CHANGES)
@pytest.mark.parametrize("seqs,H,hk,D,bs,dt", SHAPES)
def test_shapes(seqs, H, hk, D, bs, dt, what):
    b = Batch(seqs, H, hk, D, bs, dt, seed=len(seqs) * 100 + D, qscale=4.0)
    kw = change(b, what)
    out, lse = b.run(**kw)
    b.check(out, lse, **kw)


def test_nothing_changed_is_plain():
    b = Batch([(300, 300), (40, 1)], 8, 2, 128, 16, "bf16", seed=4)
    out, lse = b.run()
    d = [t.to(DEV) for t in (b.q, b.kc, b.vc, b.cu, b.lens, b.table)]
    out2, lse2 = pa.varlen_fwd(*d, b.max_q, b.max_k, b.scale, True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_split_prompts_and_long_documents():
    # Few rows over many keys: prompts split over their keys, splits that a
    # document's start hides whole.
    b = Batch([(6000, 70), (9000, 40)], 4, 2, 128, 16, "bf16", seed=7, qscale=3.0)
    kw = dict(first_key=b.documents(2500, 4000), softcap=20.0)
    out, lse = b.run(**kw)
    b.check(out, lse, **kw)


def test_rows_that_see_nothing():
    # First keys past a query's own: out 0, lse -inf, or the sink alone.
    for ql in (1, 60):
        b = Batch([(100, ql), (50, ql if ql < 50 else 50)], 8, 2, 128, 16, "f16", seed=9)
        first = torch.zeros(b.T, dtype=torch.int32)
        first[::2] = 2 ** 31 - 1
        out, lse = b.run(first_key=first)
        b.check(out, lse, first_key=first)
        assert not out[::2].any() and (lse[:, ::2] == -math.inf).all()
        sinks = torch.randn(8)
        out, lse = b.run(first_key=first, sinks=sinks)
        b.check(out, lse, first_key=first, sinks=sinks)
        # ... every row.
        first[:] = 100
        out, lse = b.run(first_key=first)
        assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("ql", [1, 100])
def test_sinks_scales_and_ends(ql):
    b = Batch([(150, ql)], 8, 2, 128, 16, "bf16", seed=11, qscale=2.0)
    sinks = torch.randn(8)
    for scale in (0.5, -0.3, 0.0):
        kw = dict(softcap=30.0, alibi_slopes=b.slopes())
        out, lse = b.run(scale, sinks=sinks, **kw)
        b.check(out, lse, scale, sinks=sinks, **kw)
    # Far past the cap, negative slopes, prefix and first keys outside the sequence.
    b.q *= 100
    kw = dict(softcap=5.0, alibi_slopes=-b.slopes() * 0.05,
              first_key=torch.full((b.T,), -7, dtype=torch.int32))
    out, lse = b.run(1.0, prefix_lens=torch.tensor([10 ** 9], dtype=torch.int32), **kw)
    b.check(out, lse, 1.0, prefix_lens=torch.tensor([150]), **kw)


def test_hidden_documents_may_hold_anything():
    # NaN in K and V in front of every query's first key.
    b = Batch([(700, 130)], 4, 2, 128, 16, "bf16", seed=13)
    first = torch.full((130,), 333, dtype=torch.int32)
    j = torch.arange(333)
    page = b.table[0].long()[j // 16]
    out0, lse0 = b.run(first_key=first)
    b.kc[page, j % 16] = math.nan
    b.vc[page, j % 16] = math.nan
    out, lse = b.run(first_key=first)
    assert torch.equal(out, out0) and torch.equal(lse, lse0)
    dec = Batch([(700, 1)], 4, 2, 128, 16, "bf16", seed=14)
    one = torch.tensor([601], dtype=torch.int32)
    out0, lse0 = dec.run(first_key=one)
    j = torch.arange(601)
    dec.kc[dec.table[0].long()[j // 16], j % 16] = math.nan
    dec.vc[dec.table[0].long()[j // 16], j % 16] = math.nan
    out, lse = dec.run(first_key=one)
    assert torch.equal(out, out0) and torch.equal(lse, lse0)


def test_update_in_the_call():
    b = Batch([(100, 1), (37, 20)], 8, 2, 128, 16, "bf16", seed=15)
    k, v = (torch.randn((b.T, 2, 128)).bfloat16() for _ in range(2))
    slots = []
    for s, (kv, ql) in enumerate(b.seqs):
        for p in range(kv - ql, kv):
            slots.append(int(b.table[s, p // 16]) * 16 + p % 16)
    slots = torch.tensor(slots)
    kw = dict(softcap=8.0, prefix_lens=torch.tensor([5, 30], dtype=torch.int32))
    out, lse = b.run(key=k, value=v, slot_mapping=slots, **kw)
    b.kc.view(-1, 2, 128)[slots] = k
    b.vc.view(-1, 2, 128)[slots] = v
    b.check(out, lse, **kw)


def test_capture():
    b = Batch([(100, 1), (300, 90)], 8, 2, 128, 16, "f16", seed=16)
    kw = {k: v.to(DEV) if torch.is_tensor(v) else v
          for k, v in change(b, "cap+bias+docs+prefix").items()}
    d = [t.to(DEV) for t in (b.q, b.kc, b.vc, b.cu, b.lens, b.table)]
    want = pa.score_fwd(*d, b.max_q, b.max_k, b.scale, **kw)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = pa.alloc_workspace(pa.varlen_fwd_workspace_size(
        2, b.T, b.max_q, b.max_k, 8, 2, 128, 16,
        torch.cuda.get_device_properties(0).multi_processor_count), DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.score_fwd(*d, b.max_q, b.max_k, b.scale, out=out, lse=lse, workspace=ws, **kw)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("D,dt", [(64, "f16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("cap", [2.0, 5.0, 12.0, 60.0, 3e6])
def test_caps_of_every_size(D, dt, cap):
    # Scores far past the cap, up to it, up to half of it, a few per cent of it.
    b = Batch([(700, 300), (260, 129)], 6, 2, D, 16, dt, seed=21)
    out, lse = b.run(softcap=cap)
    b.check(out, lse, softcap=cap)
    kw = dict(softcap=cap, alibi_slopes=b.slopes())
    out, lse = b.run(**kw)
    b.check(out, lse, **kw)
    if D < 256:                      # (head size 256 takes positive scales)
        out, lse = b.run(-b.scale, **kw)
        b.check(out, lse, -b.scale, **kw)


def test_hidden_keys_choose_nothing():
    # What the rows past a sequence's end and in front of its documents hold, and the
    # neighbours in the batch, do not change a bit of a capped prompt.
    b = Batch([(300, 140), (200, 64)], 4, 2, 128, 16, "bf16", seed=22)
    first = torch.cat([torch.full((140,), 100), torch.zeros(64)]).int()
    kw = dict(first_key=first, softcap=40.0, alibi_slopes=b.slopes())
    out0, lse0 = b.run(**kw)
    for x in (0.0, 300.0, math.inf):
        b.kc[b.kc.isnan()] = x
        b.vc[b.vc.isnan()] = x
        j = torch.arange(100)
        page = b.table[0].long()[j // 16]
        b.kc[page, j % 16] = x
        b.vc[page, j % 16] = x
        b.q[140:] *= 30
        out, lse = b.run(**kw)
        assert torch.equal(out[:140], out0[:140]) and torch.equal(lse[:, :140], lse0[:, :140])
        used = b.kc == x
        b.kc[used], b.vc[used] = math.nan, math.nan


@pytest.mark.parametrize("ql", [1, 150])
def test_scale_zero_and_negative_without_a_cap(ql):
    b = Batch([(300, ql)], 8, 2, 128, 16, "bf16", seed=23, qscale=2.0)
    first = torch.full((b.T,), 40, dtype=torch.int32)
    for scale in (0.0, -0.2):
        for kw in (dict(first_key=first), dict(alibi_slopes=b.slopes())):
            out, lse = b.run(scale, **kw)
            b.check(out, lse, scale, **kw)


@pytest.mark.parametrize("slope", [8.0, -0.5, 1000.0])
def test_slopes_of_every_size(slope):
    b = Batch([(700, 200), (90, 90)], 4, 4, 64, 16, "f16", seed=24, qscale=3.0)
    kw = dict(alibi_slopes=torch.full((4,), slope))
    out, lse = b.run(**kw)
    b.check(out, lse, **kw)


def test_two_graphs_take_turns_with_one_workspace():
    # Both capture the same workspace; replayed in turn on one stream, each gives what it
    # gave alone.
    b = Batch([(100, 1), (300, 90)], 8, 2, 128, 16, "bf16", seed=25)
    d = [t.to(DEV) for t in (b.q, b.kc, b.vc, b.cu, b.lens, b.table)]
    ws = pa.alloc_workspace(pa.varlen_fwd_workspace_size(
        2, b.T, b.max_q, b.max_k, 8, 2, 128, 16,
        torch.cuda.get_device_properties(0).multi_processor_count), DEV)
    kws = [dict(softcap=9.0), dict(alibi_slopes=b.slopes().to(DEV))]
    graphs, outs, wants = [], [], []
    for kw in kws:
        wants.append(pa.score_fwd(*d, b.max_q, b.max_k, b.scale, **kw))
        outs.append((torch.empty_like(wants[-1][0]), torch.empty_like(wants[-1][1])))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pa.score_fwd(*d, b.max_q, b.max_k, b.scale, out=outs[-1][0], lse=outs[-1][1],
                         workspace=ws, **kw)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    b.check(*outs[0], softcap=9.0)
