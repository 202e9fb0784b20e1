"""GPU parity of sliding-window attention with first tokens against the fp64
definition, on every kernel path: the split-KV kernel (one split and several,
2-byte pools and both FP8 consumers), the tensor-core prefill kernel at every
head size (one split and several), with sinks and with an in-call update.

Tolerance of an output element, from arithmetic: with p_j the softmax weights,
each P entry is rounded to the MMA's operand type (half a step of it, relative
to the entry) and the result to the output type, so the element is off by at
most half a step times (|out| + sum_j p_j |v_j|), the float32 steps adding a
few 2^-24 of the same sums and the scores' own error (1e-4 is far above it).
The definition computes sum_j p_j |v_j| as the attention over |V|. Over
e4m3 pools an f16 query enters Q.K^T as two e4m3 terms of four significant
bits each: the first leaves a remainder of at most 2^-4 of the element's power
of two, the second rounds it by at most 2^-9 of that, so a score is off by at
most ds = 2^-9 scale sum_d |q_d k_d|, a weight by a factor e^(2 ds) at most and
the LSE by ds (bf16 has eight significant bits: exact). (A fixed
1e-2, as for batches whose rows average many keys, does not hold here: a row
that sees two keys has outputs of 4 and more, and 2^-8 * 4 > 1e-2.)"""
import math

import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
import workloads as W
from helpers import LSE_TOL, oracle_pools
from oracle import cache_ops as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


def define(wl, kc, vc, window, first, scale=None, sinks=None):
    """(out, lse, sum_j p_j |v_j|) of the definition."""
    args = (wl.cu_seqlens_q, wl.seqused_k, wl.block_table,
            wl.softmax_scale if scale is None else scale, window, first)
    sinks = None if sinks is None else sinks.double()
    o, l = ref.window_attention(wl.q, kc, vc, *args, sinks=sinks)
    return o, l, ref.window_attention(wl.q, kc, vc.abs(), *args, sinks=sinks)[0]


def check(got, want, ds=0.0):
    (out, lse), (ref_o, ref_l, ref_a) = got, want
    o, l = out.cpu().double(), lse.cpu().double()
    fin = torch.isfinite(ref_l)
    assert torch.equal(fin, torch.isfinite(l))
    half = torch.finfo(out.dtype).eps / 2
    assert ((o - ref_o).abs() <= half * (ref_o.abs() + ref_a) +
            math.expm1(2 * ds) * ref_a + 1e-4).all()
    if fin.any():
        assert (l[fin] - ref_l[fin]).abs().max().item() <= LSE_TOL + ds


def dev(wl):
    return tuple(t.to(DEV) for t in (wl.cu_seqlens_q, wl.seqused_k, wl.block_table))


def hide(wl, kc, vc, window, first, seqs=None):
    """The pools and table as a user that frees what nobody sees may leave
    them: NaN in every unseen row, a stale entry for every unseen page."""
    kc, vc, bt = kc.clone(), vc.clone(), wl.block_table.clone()
    bs = wl.block_size
    seen = torch.zeros(wl.num_blocks * bs, dtype=torch.bool)
    for s, (ql, kv) in enumerate(zip(wl.q_lens, wl.kv_lens)):
        lo = max(0, kv - ql - window + 1)
        for p in range((kv + bs - 1) // bs):
            keys = [j for j in range(p * bs, min(kv, (p + 1) * bs)) if j < first or j >= lo]
            if not keys:
                bt[s, p] = -1 if p % 2 else W.INT32_MAX
            for j in keys:
                seen[int(wl.block_table[s, p]) * bs + j % bs] = True
    kc.view(-1, *kc.shape[2:])[~seen] = float("nan")
    vc.view(-1, *vc.shape[2:])[~seen] = float("nan")
    return kc, vc, bt


CASES = [
    # seed, S, H, hk, D, bs, max_q, max_kv, decode_frac, empty_ok, window, first, dtype
    (701, 5, 8, 2, 64, 16, 1, 200, 1.0, False, 1, 0, torch.bfloat16),     # only its own key
    (702, 6, 32, 8, 128, 16, 1, 3000, 1.0, False, 700, 4, torch.bfloat16),
    (703, 6, 32, 8, 128, 16, 1, 3000, 1.0, False, 64, 0, torch.float16),
    (704, 4, 8, 8, 64, 32, 1, 900, 1.0, False, 130, 300, torch.bfloat16),
    (705, 4, 16, 2, 128, 64, 3, 1500, 0.2, False, 100, 7, torch.bfloat16),  # short queries
    (706, 5, 8, 2, 64, 16, 12, 60, 0.3, True, 5, 2, torch.bfloat16),     # empty rows, D 64
    (707, 3, 16, 2, 128, 32, 300, 700, 0.0, False, 50, 3, torch.bfloat16),
    (708, 2, 32, 8, 128, 128, 200, 4000, 0.0, False, 900, 16, torch.bfloat16),
    (709, 2, 14, 2, 128, 16, 400, 1200, 0.0, False, 257, 129, torch.float16),   # GQA 7
    (710, 2, 8, 2, 64, 16, 500, 1500, 0.0, False, 128, 64, torch.bfloat16),
    (711, 3, 8, 4, 256, 16, 200, 900, 0.3, False, 100, 5, torch.bfloat16),
    (712, 3, 4, 2, 256, 64, 1, 2500, 1.0, False, 1000, 1, torch.float16),
    (713, 3, 12, 4, 128, 16, 80, 500, 0.4, True, 33, 1, torch.bfloat16),
    (714, 1, 200, 1, 128, 16, 3, 300, 0.0, False, 40, 2, torch.bfloat16),   # a wide group
    (715, 2, 32, 8, 128, 16, 700, 700, 0.0, False, 1, 1, torch.bfloat16),
    (716, 2, 8, 1, 128, 16, 260, 6000, 0.0, False, 3000, 4, torch.bfloat16),   # KV splits
]


@pytest.mark.parametrize("seed,S,H,hk,D,bs,mq,mk,dfrac,empty,window,first,dtype", CASES)
def test_window(seed, S, H, hk, D, bs, mq, mk, dfrac, empty, window, first, dtype):
    wl = W.random_case(seed, num_seqs=S, num_heads=H, num_kv_heads=hk, head_size=D,
                       block_size=bs, max_q=mq, max_kv=mk, decode_frac=dfrac, empty_ok=empty,
                       dtype=dtype)
    kc, vc = oracle_pools(wl)
    want = define(wl, kc, vc, window, first)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, window, first)
    out, lse = pa.window_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl), *tail,
                             dev_status=status)
    check((out, lse), want)
    assert int(status) == 0
    # what nobody sees may be anything: the same bits
    hk_, hv_, hbt = hide(wl, kc, vc, window, first)
    o2, l2 = pa.window_fwd(wl.q.to(DEV), hk_.to(DEV), hv_.to(DEV), *dev(wl)[:2], hbt.to(DEV),
                           *tail, dev_status=status)
    assert int(status) == 0
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # looser bounds: the same values (the split of the keys may differ)
    check(pa.window_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl),
                        2 * wl.max_seqlen_q + 40, 3 * wl.max_seqlen_k + 500, *tail[2:]), want)


MANY = [
    # q lengths, kv lengths, H, hk, D, window, first, dtype: more units than SMs
    ([700, 333, 1, 650, 5, 701], [900, 333, 640, 1000, 5, 701], 16, 8, 128, 100, 5, torch.bfloat16),
    ([700, 333, 0, 650, 129], [750, 400, 0, 650, 500], 24, 8, 64, 64, 0, torch.float16),   # G 3
    ([64] * 40, [64 + 13 * i for i in range(40)], 32, 8, 128, 37, 20, torch.bfloat16),     # one tile
    ([2000, 1500], [5000, 4100], 8, 1, 128, 3000, 4, torch.bfloat16),                      # KV splits
    ([2100, 900], [2100, 2300], 7, 1, 64, 1500, 130, torch.float16),                       # G 7, splits
]


@pytest.mark.parametrize("ql,kv,H,hk,D,window,first,dtype", MANY)
def test_window_many_units(ql, kv, H, hk, D, window, first, dtype):
    """Batches of more (item, KV head) units than SMs: items with one and two Q
    tiles, several and no key tiles, whole and split."""
    wl = W._build("many", 3, H, hk, D, 16, ql, kv, torch.Generator().manual_seed(3), dtype=dtype)
    kc, vc = oracle_pools(wl)
    want = define(wl, kc, vc, window, first)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, window, first)
    got = pa.window_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl), *tail, dev_status=status)
    check(got, want)
    assert int(status) == 0
    hk_, hv_, hbt = hide(wl, kc, vc, window, first)
    again = pa.window_fwd(wl.q.to(DEV), hk_.to(DEV), hv_.to(DEV), *dev(wl)[:2], hbt.to(DEV), *tail)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,hk,bs,mq,mk,dfrac,window,first", [
    (32, 8, 16, 1, 2500, 1.0, 600, 4),      # the FP8 decode consumer
    (16, 2, 32, 2, 900, 0.3, 77, 3),        # wider items
    (16, 2, 128, 300, 800, 0.0, 120, 5),    # the prefill kernel
    (8, 1, 16, 260, 3000, 0.0, 1500, 130),
])
def test_window_fp8(H, hk, bs, mq, mk, dfrac, window, first, dtype):
    wl = W.random_case(730 + mq, num_seqs=3, num_heads=H, num_kv_heads=hk, head_size=128,
                       block_size=bs, max_q=mq, max_kv=mk, decode_frac=dfrac, dtype=dtype)
    kc, vc = oracle_pools(wl)
    ks, vs = torch.linspace(0.02, 0.05, hk), torch.linspace(0.03, 0.02, hk)

    def quant(x, s):
        return (x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    qk, qv = quant(kc, ks), quant(vc, vs)
    want = define(wl, qk.float() * ks[:, None], qv.float() * vs[:, None], window, first)
    ds = 0.0
    if dtype == torch.float16:
        aq, ak = wl.q.double().abs(), (qk.float() * ks[:, None]).flatten(0, 1).double().abs()
        ds = 2.0 ** -9 * wl.softmax_scale * max(
            (aq[:, h] @ ak[:, h * hk // H].T).max().item() for h in range(H))
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, window, first)
    kw = dict(k_scale=ks.to(DEV), v_scale=vs.to(DEV))
    out, lse = pa.window_fwd(wl.q.to(DEV), qk.view(torch.uint8).to(DEV),
                             qv.view(torch.uint8).to(DEV), *dev(wl), *tail, **kw)
    check((out, lse), want, ds)
    kn, vn, hbt = hide(wl, kc, vc, window, first)
    kn, vn = quant(kn, ks), quant(vn, vs)      # NaN codes where nobody looks
    o2, l2 = pa.window_fwd(wl.q.to(DEV), kn.view(torch.uint8).to(DEV),
                           vn.view(torch.uint8).to(DEV), *dev(wl)[:2], hbt.to(DEV), *tail, **kw)
    assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("mq,mk,dfrac", [(1, 1500, 1.0), (250, 700, 0.0)])
def test_window_with_sinks_update_and_strided_q(mq, mk, dfrac):
    wl = W.random_case(760 + mq, num_seqs=4, num_heads=16, num_kv_heads=4, head_size=128,
                       block_size=16, max_q=mq, max_kv=mk, decode_frac=dfrac)
    kc, vc = oracle_pools(wl)
    sinks = torch.linspace(-1.0, 3.0, 16)
    window, first = 200, 4
    want = define(wl, kc, vc, window, first, sinks=sinks)
    wide = torch.zeros((wl.total_q, 24, 128), dtype=wl.dtype, device=DEV)
    wide[:, :16] = wl.q.to(DEV)
    dk, dv = wl.pool(0).to(DEV), wl.pool(1).to(DEV)
    out, lse = pa.window_fwd(wide[:, :16], dk, dv, *dev(wl), wl.max_seqlen_q, wl.max_seqlen_k,
                             wl.softmax_scale, window, first, sinks=sinks.to(DEV),
                             key=wl.k_new.to(DEV), value=wl.v_new.to(DEV),
                             slot_mapping=wl.slot_mapping.to(DEV))
    check((out, lse), want)
    assert torch.equal(dk.cpu(), kc) and torch.equal(dv.cpu(), vc)


@pytest.mark.parametrize("D,mq,mk,dfrac", [(128, 1, 900, 1.0), (128, 200, 600, 0.0),
                                           (64, 9, 300, 0.3), (256, 100, 300, 0.2)])
def test_window_that_covers_everything(D, mq, mk, dfrac):
    """A window of at least max_seqlen_k is plain causal attention, bit by
    bit; one key short of it leaves out one key of the longest sequence."""
    wl = W.random_case(770 + D, num_seqs=3, num_heads=8, num_kv_heads=2, head_size=D,
                       block_size=16, max_q=mq, max_kv=mk, decode_frac=dfrac)
    kc, vc = oracle_pools(wl)
    args = (wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl), wl.max_seqlen_q, wl.max_seqlen_k,
            wl.softmax_scale)
    plain = pa.varlen_fwd(*args, True)
    for window, first in ((wl.max_seqlen_k, 0), (2 ** 31 - 1, 2 ** 31 - 1)):
        out, lse = pa.window_fwd(*args, window, first)
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    for window, first in ((wl.max_seqlen_k - 1, 0), (3, 2 ** 31 - 1), (3, wl.max_seqlen_k)):
        check(pa.window_fwd(*args, window, first), define(wl, kc, vc, window, first))


def test_window_nonpositive_scale_and_more_queries_than_keys():
    wl = W.random_case(780, num_seqs=3, num_heads=8, num_kv_heads=2, head_size=64, block_size=16,
                       max_q=90, max_kv=200, decode_frac=0.0)
    kc, vc = oracle_pools(wl)
    for scale in (0.0, -0.2):
        check(pa.window_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl), wl.max_seqlen_q,
                            wl.max_seqlen_k, scale, 30, 2),
              define(wl, kc, vc, 30, 2, scale=scale))
    # fewer keys than queries: the first queries see nothing
    lens = torch.tensor([max(0, q - 5) for q in wl.q_lens], dtype=torch.int32)
    kvs = lens.tolist()
    T = wl.total_q
    ref_o = torch.zeros((T, 8, 64), dtype=torch.float64)
    ref_a = ref_o.clone()
    ref_l = torch.full((8, T), float("-inf"), dtype=torch.float64)
    cu = wl.cu_seqlens_q.tolist()
    sub = [(a + min(5, b - a), b) for a, b in zip(cu, cu[1:])]
    idx = torch.cat([torch.arange(a, b) for a, b in sub])
    cu2 = torch.tensor([0] + torch.tensor(kvs).cumsum(0).tolist(), dtype=torch.int32)
    tail = (cu2, lens, wl.block_table, wl.softmax_scale, 30, 2)
    ref_o[idx], ref_l[:, idx] = ref.window_attention(wl.q[idx], kc, vc, *tail)
    ref_a[idx] = ref.window_attention(wl.q[idx], kc, vc.abs(), *tail)[0]
    got = pa.window_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), dev(wl)[0], lens.to(DEV),
                        dev(wl)[2], wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, 30, 2)
    check(got, (ref_o, ref_l, ref_a))


def test_window_captured_and_repeatable():
    wl = W.random_case(790, num_seqs=8, num_heads=32, num_kv_heads=8, head_size=128,
                       block_size=16, max_q=150, max_kv=2500, decode_frac=0.6)
    kc, vc = oracle_pools(wl)
    d = (wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl))
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, 300, 4)
    ws = pa.alloc_workspace(pa.varlen_fwd_workspace_size(8, wl.total_q, *tail[:2], 32, 8, 128, 16,
                                                         pa._sm_count(DEV)), DEV)
    want = pa.window_fwd(*d, *tail, workspace=ws)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.window_fwd(*d, *tail, out=out, lse=lse, workspace=ws)
    ws.fill_(255)        # the workspace needs no initialisation
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # shorter sequences in the same graph
    d[4].copy_(torch.clamp(d[4] - 7, min=0))
    graph.replay()
    torch.cuda.synchronize()
    again = pa.window_fwd(*d, *tail)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_window_wider_than_32_bits():
    """A window (first tokens) past the C interface's integers is none (all)."""
    wl = W.random_case(77, num_seqs=3, num_heads=8, num_kv_heads=2, head_size=64, block_size=16,
                       max_q=40, max_kv=300)
    kc, vc = (t.to(DEV) for t in oracle_pools(wl))
    args = (wl.q.to(DEV), kc, vc, *dev(wl), wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale)
    plain = pa.varlen_fwd(*args, True)
    for window, first in ((1 << 40, 0), ((1 << 32) + 5, 0), (7, (1 << 32) + 1)):
        got = pa.window_fwd(*args, window, first)
        if window > 7:
            assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
        else:
            check(got, define(wl, kc.cpu(), vc.cpu(), wl.max_seqlen_k, 0))


DECODE = [
    # q lengths, kv lengths, H, hk, D, bs, window, first, dtype: at most 8 packed rows
    ([1], [5000], 8, 1, 128, 16, 4000, 7, torch.bfloat16),          # few sequences: several blocks
    ([1, 1], [17000, 900], 2, 1, 128, 16, 16000, 40, torch.float16),
    ([1], [16700], 1, 1, 64, 64, 16400, 0, torch.bfloat16),         # a window past the kernel's
    ([1], [12500], 2, 1, 128, 16, 12000, 40, torch.float16),        # nearly the longest run of a
    ([1] * 20, [16100 + i for i in range(20)], 1, 1, 64, 32, 16000, 200, torch.bfloat16),   # warp
    ([1] * 40, [1 + 23 * i for i in range(40)], 8, 8, 64, 32, 200, 33, torch.bfloat16),
    ([2, 0, 1, 2, 2], [2, 40, 300, 301, 2], 8, 2, 128, 16, 100, 5, torch.bfloat16),
    ([1, 1, 1], [1, 16, 17], 8, 1, 64, 16, 16, 0, torch.float16),   # one key, a slice, one more
    ([8, 3, 5], [8, 500, 77], 4, 4, 128, 48, 31, 17, torch.float16),   # q rows of one head
    ([1] * 100, [700 + i for i in range(100)], 16, 8, 128, 16, 640, 4, torch.bfloat16),
    ([2] * 90, [600] * 90, 12, 4, 64, 16, 300, 300, torch.bfloat16),   # G 3: 6 rows
    ([1, 1], [3500, 40], 8, 1, 256, 16, 2000, 9, torch.bfloat16),
    ([2] * 30, [300 + 7 * i for i in range(30)], 4, 2, 256, 32, 150, 20, torch.float16),
]


@pytest.mark.parametrize("ql,kv,H,hk,D,bs,window,first,dtype", DECODE)
def test_window_decode(ql, kv, H, hk, D, bs, window, first, dtype):
    """Few packed query rows: every split of the keys over warps and blocks,
    with sinks, and pages that nobody sees."""
    wl = W._build("decode", 5, H, hk, D, bs, ql, kv, torch.Generator().manual_seed(9), dtype=dtype)
    kc, vc = oracle_pools(wl)
    sinks = torch.linspace(-1, 2, H)
    tail = (wl.max_seqlen_q, max(wl.max_seqlen_k, window + 1), wl.softmax_scale, window, first)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for sk in (None, sinks):
        want = define(wl, kc, vc, window, first, sinks=sk)
        skd = None if sk is None else sk.to(DEV)
        got = pa.window_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl), *tail, sinks=skd,
                            dev_status=status)
        check(got, want)
        hk_, hv_, hbt = hide(wl, kc, vc, window, first)
        again = pa.window_fwd(wl.q.to(DEV), hk_.to(DEV), hv_.to(DEV), *dev(wl)[:2], hbt.to(DEV),
                              *tail, sinks=skd, dev_status=status)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ql,kv,H,hk,bs,window,first", [
    ([1], [5000], 8, 1, 16, 4000, 7),
    ([1], [12900], 2, 1, 16, 11000, 9),
    ([1] * 60, [400 + 11 * i for i in range(60)], 16, 8, 16, 500, 4),
    ([2, 1, 0, 2], [2, 33, 50, 900], 8, 2, 48, 65, 40),
])
def test_window_decode_fp8(ql, kv, H, hk, bs, window, first, dtype):
    """e4m3 pools: keys and values are exact in the MMA's types and a query
    keeps its bits, so the tolerance is the 2-byte pools' one."""
    wl = W._build("decode", 8, H, hk, 128, bs, ql, kv, torch.Generator().manual_seed(6),
                  dtype=dtype)
    ks, vs = torch.linspace(0.01, 0.03, hk), torch.linspace(0.02, 0.04, hk)
    codes = [(c.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
             for c, s in zip(oracle_pools(wl), (ks, vs))]
    kd, vd = (c.double() * s.double()[:, None] for c, s in zip(codes, (ks, vs)))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    tail = (wl.max_seqlen_q, max(wl.max_seqlen_k, window + 1), wl.softmax_scale, window, first)
    kw = dict(k_scale=ks.to(DEV), v_scale=vs.to(DEV), dev_status=status)
    raw = [c.view(torch.uint8) for c in codes]
    got = pa.window_fwd(wl.q.to(DEV), *(c.to(DEV) for c in raw), *dev(wl), *tail, **kw)
    check(got, define(wl, kd, vd, window, first))
    nan = hide(wl, *(c.float() for c in codes), window, first)
    raw = [c.to(torch.float8_e4m3fn).view(torch.uint8) for c in nan[:2]]   # NaN bytes
    again = pa.window_fwd(wl.q.to(DEV), *(c.to(DEV) for c in raw), *dev(wl)[:2], nan[2].to(DEV),
                          *tail, **kw)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert int(status) == 0


def test_window_decode_fp8_planned():
    """A window past the unplanned kernel's, over e4m3 pools (bf16 queries are
    exact there too)."""
    wl = W._build("decode", 8, 8, 1, 128, 16, [1], [13000], torch.Generator().manual_seed(6))
    codes = [(c.float() / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn) for c in oracle_pools(wl)]
    kd, vd = (c.double() * torch.tensor([0.02]).double() for c in codes)
    got = pa.window_fwd(wl.q.to(DEV), *(c.view(torch.uint8).to(DEV) for c in codes), *dev(wl), 1,
                        13000, wl.softmax_scale, 12800, 4, k_scale=0.02, v_scale=0.02)
    check(got, define(wl, kd, vd, 12800, 4))


@pytest.mark.parametrize("sink", [False, True])
def test_window_decode_more_queries_than_keys(sink):
    """Queries in front of the first key, and sequences without keys, see
    nothing (a sink apart)."""
    wl = W._build("decode", 7, 8, 2, 64, 16, [2, 2, 1, 2], [60, 60, 60, 60],
                  torch.Generator().manual_seed(4), dtype=torch.float16)
    kc, vc = oracle_pools(wl)
    lens = torch.tensor([1, 0, 0, 60], dtype=torch.int32)
    sinks = torch.linspace(-1, 1, 8) if sink else None
    meta = (wl.cu_seqlens_q, lens, wl.block_table)
    got = pa.window_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *(t.to(DEV) for t in meta), 2, 60,
                        wl.softmax_scale, 20, 3, sinks=None if sinks is None else sinks.to(DEV))
    tail = (*meta, wl.softmax_scale, 20, 3)
    sinks = None if sinks is None else sinks.double()
    o, l = ref.window_attention(wl.q, kc, vc, *tail, sinks=sinks)
    check(got, (o, l, ref.window_attention(wl.q, kc, vc.abs(), *tail, sinks=sinks)[0]))


def test_window_decode_bad_metadata():
    """A page outside the pool reads as zeros and is reported, as are lengths
    past the bounds; a sequence with inconsistent offsets writes nothing."""
    wl = W._build("decode", 6, 8, 2, 128, 16, [1, 1, 1], [400, 300, 200],
                  torch.Generator().manual_seed(4))
    kc, vc = oracle_pools(wl)
    bt = wl.block_table.clone()
    page = int(bt[1, 10])
    bt[1, 10] = wl.num_blocks
    zk, zv = kc.clone(), vc.clone()
    zk[page] = 0
    zv[page] = 0
    args = (wl.q.to(DEV), kc.to(DEV), vc.to(DEV))
    cu, lens, _ = dev(wl)
    tail = (1, wl.max_seqlen_k, wl.softmax_scale, 250, 3)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pa.window_fwd(*args, cu, lens, bt.to(DEV), *tail, dev_status=status)
    assert int(status) == pa.PA_DEV_BAD_PAGE
    check(got, define(wl, zk, zv, 250, 3))
    status.zero_()
    pa.window_fwd(*args, *dev(wl), 1, 350, *tail[2:], dev_status=status)
    assert int(status) == pa.PA_DEV_BAD_SEQLEN
    status.zero_()
    bad = torch.tensor([0, 1, 5, 3], dtype=torch.int32, device=DEV)
    out = torch.full_like(args[0], 7.0)
    pa.window_fwd(*args, bad, lens, dev(wl)[2], *tail, out=out, dev_status=status)
    assert int(status) == pa.PA_DEV_BAD_SEQLEN
    want = define(wl, kc, vc, 250, 3)[0]
    assert (out[0].cpu().double() - want[0]).abs().max() < 0.05
    assert (out[1:] == 7.0).all()


def test_window_decode_captured_scaled_and_on_two_streams():
    """A decode step in a graph, replayed on other lengths, and on two streams
    at once; softmax scales of zero and below."""
    wl = W._build("decode", 11, 16, 4, 128, 16, [1] * 12, [90 + 60 * i for i in range(12)],
                  torch.Generator().manual_seed(2))
    kc, vc = (t.to(DEV) for t in oracle_pools(wl))
    cu, lens, bt = dev(wl)
    q = wl.q.to(DEV)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, 300, 4)
    for scale in (0.0, -0.1):
        check(pa.window_fwd(q, kc, vc, cu, lens, bt, 1, wl.max_seqlen_k, scale, 300, 4),
              define(wl, kc.cpu(), vc.cpu(), 300, 4, scale=scale))
    want = pa.window_fwd(q, kc, vc, cu, lens, bt, *tail)
    ws = pa.alloc_workspace(pa.varlen_fwd_workspace_size(12, 12, 1, wl.max_seqlen_k, 16, 4, 128, 16,
                                                         pa._sm_count(DEV)), DEV)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.window_fwd(q, kc, vc, cu, lens, bt, *tail, out=out, lse=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    short = torch.clamp(lens - 77, min=0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for st, n in zip(streams, (lens, short)):
            with torch.cuda.stream(st):
                got.append(pa.window_fwd(q, kc, vc, cu, n, bt, *tail))
    torch.cuda.synchronize()
    lens.copy_(short)
    graph.replay()
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for x, y in zip(g, (out, lse) if i % 2 else want):
            assert torch.equal(x, y)
