"""GPU parity of the accumulated attention weights and of eviction by them
with their fp64 definitions, and of a run of the operators together.

Tolerance of the weights, from arithmetic: a term exp(x - lse) has the
relative error of its exponent's absolute error. The float32 dot product of D
exact products is off by at most 2 D 2^-24 times scale * |q| |k| (twice the
sequential bound, for the tensor core's order of addition), the products with
scale and log2 e, the LSE's conversion and ex2 by at most 8 * 2^-24 (|x| + |lse|) +
2^-21; the sums add at most n 2^-24 for n terms (all positive).
"""
import math

import pytest
import torch

import oracle
import paged_kv_varlen_attn_gb300 as pa
import workloads as W
from helpers import oracle_pools
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


def rel_bound(wl, kc, lse, extra=1.0):
    D = wl.head_size
    qn = wl.q.double().norm(dim=-1).max().item()
    kn = kc.double().norm(dim=-1).max().item()
    x = abs(wl.softmax_scale) * qn * kn * extra
    fin = lse[torch.isfinite(lse)]
    top = fin.abs().max().item() if fin.numel() else 0.0
    n = max(wl.q_lens) * (wl.num_heads // wl.num_kv_heads) + 2
    return (2 * D * x + 8 * (x + top) + n) * 2.0 ** -24 + 2.0 ** -21


def random_weights(wl, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.rand((wl.num_blocks, wl.num_kv_heads, wl.block_size), generator=g)


WCASES = [
    # seed, S, H, hk, D, bs, max_q, max_kv, causal, decode_frac, empty_ok, dtype
    (901, 1, 1, 1, 64, 16, 1, 1, True, 1.0, False, torch.bfloat16),      # one key
    (902, 6, 32, 8, 128, 16, 1, 900, True, 1.0, False, torch.bfloat16),  # decode
    (903, 5, 8, 8, 64, 32, 1, 300, True, 1.0, False, torch.float16),     # decode, MHA
    (904, 3, 14, 2, 128, 16, 70, 200, True, 0.3, True, torch.bfloat16),  # GQA 7, empty rows
    (905, 2, 16, 2, 128, 128, 300, 700, True, 0.0, False, torch.float16),
    (906, 3, 6, 2, 256, 16, 40, 150, True, 0.3, True, torch.bfloat16),
    (907, 3, 8, 2, 64, 16, 50, 260, False, 0.3, True, torch.bfloat16),   # every key seen
    (908, 1, 200, 1, 128, 16, 3, 90, True, 0.0, False, torch.bfloat16),  # a group of 200 heads
    (909, 2, 12, 4, 128, 64, 260, 1100, True, 0.0, False, torch.bfloat16),
    (910, 2, 8, 1, 256, 32, 130, 400, True, 0.0, False, torch.float16),
    (911, 2, 8, 2, 64, 16, 400, 900, True, 0.0, False, torch.bfloat16),
]


@pytest.mark.parametrize("seed,S,H,hk,D,bs,mq,mk,causal,dfrac,empty,dtype", WCASES)
def test_weights(seed, S, H, hk, D, bs, mq, mk, causal, dfrac, empty, dtype):
    wl = W.random_case(seed, num_seqs=S, num_heads=H, num_kv_heads=hk, head_size=D,
                       block_size=bs, max_q=mq, max_kv=mk, causal=causal, decode_frac=dfrac,
                       empty_ok=empty, dtype=dtype)
    kc, vc = oracle_pools(wl)
    meta = (wl.cu_seqlens_q, wl.seqused_k, wl.block_table)
    _, lse = oracle.varlen_attention(wl.q, kc, vc, *meta, wl.softmax_scale, causal)
    lse = lse.float()
    w0 = random_weights(wl)
    want = ref.attn_weights(wl.q, kc, lse, w0, *meta, wl.softmax_scale, causal)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = w0.to(DEV)
    args = (wl.q.to(DEV), kc.to(DEV), lse.to(DEV))
    margs = tuple(t.to(DEV) for t in meta) + (wl.max_seqlen_q, wl.max_seqlen_k,
                                              wl.softmax_scale, causal)
    got = pa.attn_weights(*args, w, *margs, dev_status=status)
    assert got is w and int(status) == 0
    rel = rel_bound(wl, kc, lse)
    got = got.cpu().double()
    assert ((got - want).abs() <= rel * want.abs()).all()
    untouched = want == w0.double()
    assert torch.equal(got[untouched], w0.double()[untouched])
    # the same bits again, with looser bounds, and with a packed q
    w2 = w0.to(DEV)
    T = wl.total_q
    wide = torch.zeros((T, H + 2, D), dtype=dtype, device=DEV)
    wide[:, :H] = args[0]
    pa.attn_weights(wide[:, :H], *args[1:], w2, *margs[:3], 2 * wl.max_seqlen_q + 50,
                    2 * wl.max_seqlen_k + 77, *margs[5:])
    assert ((w2.cpu().double() - want).abs() <= rel * want.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mq,mk,dfrac", [(1, 700, 1.0), (90, 400, 0.0), (300, 500, 0.2)])
def test_weights_fp8(dtype, mq, mk, dfrac):
    wl = W.random_case(950 + mq, num_seqs=3, num_heads=8, num_kv_heads=2, head_size=128,
                       block_size=32, max_q=mq, max_kv=mk, decode_frac=dfrac, dtype=dtype)
    kc, vc = oracle_pools(wl)
    scale = torch.tensor([0.02, 0.05])
    codes = (kc.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    kd = codes.float() * scale[:, None]
    meta = (wl.cu_seqlens_q, wl.seqused_k, wl.block_table)
    _, lse = oracle.varlen_attention(wl.q, kd, vc, *meta, wl.softmax_scale, True)
    lse = lse.float()
    w0 = random_weights(wl)
    want = ref.attn_weights(wl.q, kd, lse, w0, *meta, wl.softmax_scale, True)
    got = pa.attn_weights(wl.q.to(DEV), codes.view(torch.uint8).to(DEV), lse.to(DEV), w0.to(DEV),
                          *(t.to(DEV) for t in meta), wl.max_seqlen_q, wl.max_seqlen_k,
                          wl.softmax_scale, True, k_scale=scale.to(DEV)).cpu().double()
    assert ((got - want).abs() <= rel_bound(wl, kd, lse) * want.abs()).all()


def test_weights_garbage_past_the_end():
    """NaN keys past a sequence's end and rows that saw nothing change
    nothing; a bad page skips its keys; bad lengths are reported."""
    wl = W.random_case(930, num_seqs=2, num_heads=4, num_kv_heads=2, head_size=64, block_size=16,
                       max_q=50, max_kv=100, decode_frac=0.0)
    kc, vc = oracle_pools(wl)
    meta = (wl.cu_seqlens_q, wl.seqused_k, wl.block_table)
    _, lse = oracle.varlen_attention(wl.q, kc, vc, *meta, wl.softmax_scale, True)
    lse = lse.float()
    lse[1, 3] = float("-inf")
    used = torch.zeros(wl.num_blocks * wl.block_size, dtype=torch.bool)
    for s in range(2):
        j = torch.arange(wl.kv_lens[s])
        used[wl.block_table[s].long()[j // 16] * 16 + j % 16] = True
    kc.view(-1, 2, 64)[~used] = float("nan")
    w0 = random_weights(wl)
    want = ref.attn_weights(wl.q, kc, lse, w0, *meta, wl.softmax_scale, True)
    bt = wl.block_table.clone()
    margs = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, True)
    got = pa.attn_weights(wl.q.to(DEV), kc.to(DEV), lse.to(DEV), w0.to(DEV),
                          *(t.to(DEV) for t in meta), *margs).cpu().double()
    rel = rel_bound(wl, kc[~torch.isnan(kc)].view(-1, 64), lse)
    assert ((got - want).abs() <= rel * want.abs()).all()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bt[0, 0] = wl.num_blocks
    part = pa.attn_weights(wl.q.to(DEV), kc.to(DEV), lse.to(DEV), w0.to(DEV), meta[0].to(DEV),
                           meta[1].to(DEV), bt.to(DEV), *margs, dev_status=status).cpu().double()
    assert int(status) == pa.PA_DEV_BAD_PAGE
    page = int(wl.block_table[0, 0])
    assert torch.equal(part[page], w0.double()[page])
    keep = torch.arange(wl.num_blocks) != page
    assert torch.equal(part[keep], got[keep])
    status.zero_()
    lens = meta[1].clone()
    lens[1] = wl.max_seqlen_k + 10 ** 6
    pa.attn_weights(wl.q.to(DEV), kc.to(DEV), lse.to(DEV), w0.to(DEV), meta[0].to(DEV),
                    lens.to(DEV), meta[2].clamp(0, wl.num_blocks - 1).to(DEV), *margs,
                    dev_status=status)
    assert int(status) & pa.PA_DEV_BAD_SEQLEN


def pools(seed, kv, hk, D, bs, elem, spare=3):
    g = torch.Generator().manual_seed(seed)
    need = [(k + bs - 1) // bs for k in kv]
    nb = sum(need) + spare
    order = torch.randperm(nb, generator=g)
    bt = torch.full((len(kv), max(need + [1])), W.INT32_MAX, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = order[at:at + n].int()
        at += n
    # distinct bit patterns, NaN patterns among them: rows move as bytes
    bits = torch.randint(0, 256, (2, nb, bs, hk, D * elem), generator=g, dtype=torch.uint8)
    w = torch.rand((nb, hk, bs), generator=g)
    return bits[0], bits[1], w, bt, torch.tensor(kv, dtype=torch.int32)


def typed(bits, elem):
    return bits if elem == 1 else bits.view(torch.bfloat16)


ECASES = [
    # kv lengths, hk, D, bs, elem, budget, first, recent
    ([1], 1, 64, 16, 2, 1, 0, 0),
    ([2], 1, 64, 16, 2, 1, 0, 0),
    ([40, 7, 0, 33], 2, 64, 16, 2, 32, 4, 8),
    ([100, 64, 65, 63], 2, 128, 16, 2, 64, 0, 0),
    ([300, 200], 3, 128, 32, 2, 50, 50, 0),            # only first tokens
    ([300, 200], 1, 128, 32, 2, 50, 0, 50),            # only recent ones: a pure shift
    ([300, 2000], 2, 128, 128, 1, 77, 3, 20),          # e4m3
    ([1500, 1100, 900], 2, 256, 16, 2, 1000, 4, 256),  # several chunks of rows
    ([5000], 2, 64, 1024, 2, 4999, 1, 1),              # one key goes
    ([70000], 1, 64, 16, 2, 129, 4, 64),               # candidates beyond shared memory
]


@pytest.mark.parametrize("kv,hk,D,bs,elem,budget,first,recent", ECASES)
def test_evict(kv, hk, D, bs, elem, budget, first, recent):
    kb, vb, w, bt, lens = pools(len(kv) + D, kv, hk, D, bs, elem)
    rk, rv, rw, kept, rlens = ref.evict(kb, vb, w, lens, bt, budget, first, recent)
    dk, dv, dw = typed(kb, elem).to(DEV), typed(vb, elem).to(DEV), w.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, glens = pa.evict(dk, dv, dw, lens.to(DEV), bt.to(DEV), max(kv), budget, first, recent,
                          dev_status=status)
    assert int(status) == 0
    assert torch.equal(got.cpu(), kept) and torch.equal(glens.cpu(), rlens)
    assert torch.equal(dk.cpu().view(torch.uint8), rk)
    assert torch.equal(dv.cpu().view(torch.uint8), rv)
    assert torch.equal(dw.cpu(), rw)


def test_evict_ties_and_odd_weights():
    """Equal weights go to the lowest index; zeros of both signs are equal;
    NaN ranks with -inf; infinities and denormals rank as numbers."""
    kv, hk, bs = [400], 2, 16
    kb, vb, w, bt, lens = pools(77, kv, hk, 64, bs, 2)
    vals = torch.tensor([0.0, -0.0, float("nan"), float("-inf"), float("inf"), 1e-42, -1e-42,
                         1.0, 1.0, -3.0, 3.4e38, 1.0000001])
    g = torch.Generator().manual_seed(6)
    w.copy_(vals[torch.randint(0, len(vals), w.shape, generator=g)])
    for budget, first, recent in ((40, 3, 5), (150, 0, 0), (250, 1, 100), (399, 0, 1), (300, 0, 3)):
        rk, rv, rw, kept, rl = ref.evict(kb, vb, w, lens, bt, budget, first, recent)
        dk, dv, dw = typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV)
        got, _ = pa.evict(dk, dv, dw, lens.to(DEV), bt.to(DEV), 400, budget, first, recent)
        assert torch.equal(got.cpu(), kept)
        assert torch.equal(dw.cpu().view(torch.int32), rw.view(torch.int32))
        assert torch.equal(dk.cpu().view(torch.uint8), rk)


def test_evict_in_place_lengths_strides_and_bad_pages():
    kv, hk, D, bs, budget = [90, 50, 120], 2, 64, 16, 64
    kb, vb, w, bt, lens = pools(5, kv, hk, D, bs, 2)
    rk, rv, rw, kept, rl = ref.evict(kb, vb, w, lens, bt, budget, 2, 10)
    # a combined pool, a weights pool with a padded page stride, new lengths
    # over the old ones, and a looser key bound
    both = torch.stack([typed(kb, 2), typed(vb, 2)], 1).to(DEV)
    wide = torch.zeros((w.shape[0], hk * bs + 16), device=DEV)
    dw = wide[:, :hk * bs].view(-1, hk, bs)
    dw.copy_(w)
    dl = lens.to(DEV)
    out = torch.empty((3, hk, budget), dtype=torch.int32, device=DEV)
    pa.evict(both[:, 0], both[:, 1], dw, dl, bt.to(DEV), 5000, budget, 2, 10, kept=out,
             new_lens=dl)
    assert torch.equal(dl.cpu(), rl) and torch.equal(out.cpu(), kept)
    assert torch.equal(both[:, 0].cpu().contiguous().view(torch.uint8), rk)
    assert torch.equal(both[:, 1].cpu().contiguous().view(torch.uint8), rv)
    assert torch.equal(dw.cpu(), rw) and (wide[:, hk * bs:] == 0).all()
    # a page outside the pool: reported, nothing of it moves, no other
    # sequence is touched
    bad = bt.clone()
    bad[2, 5] = kb.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dk, dv, dw = typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV)
    got, gl = pa.evict(dk, dv, dw, lens.to(DEV), bad.to(DEV), 120, budget, 2, 10,
                       dev_status=status)
    assert int(status) == pa.PA_DEV_BAD_PAGE
    assert torch.equal(got[:2].cpu(), kept[:2]) and torch.equal(gl.cpu(), rl)
    middle = got[2].cpu()
    assert not ((middle >= 80) & (middle < 96)).any()
    status.zero_()
    long = lens.clone()
    long[0], long[1] = 10 ** 7, -4
    pa.evict(dk, dv, dw, long.to(DEV), bt.clamp(0, kb.shape[0] - 1).to(DEV), 120, budget, 2, 10,
             dev_status=status)
    assert int(status) & pa.PA_DEV_BAD_SEQLEN


def test_evict_captured():
    kv, hk, D, bs, budget = [200, 170], 2, 128, 16, 100
    kb, vb, w, bt, lens = pools(9, kv, hk, D, bs, 2)
    dk, dv, dw = typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV)
    kept = torch.empty((2, hk, budget), dtype=torch.int32, device=DEV)
    nl = torch.empty(2, dtype=torch.int32, device=DEV)
    args = (lens.to(DEV), bt.to(DEV), 200, budget, 4, 16, kept, nl)
    pa.evict(dk.clone(), dv.clone(), dw.clone(), *args)      # first call: outside the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.evict(dk, dv, dw, *args)
    g = torch.Generator().manual_seed(31)
    w2 = torch.rand(w.shape, generator=g)
    dw.copy_(w2)
    rk, rv, rw, rkept, rl = ref.evict(kb, vb, w2, lens, bt, budget, 4, 16)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept.cpu(), rkept) and torch.equal(nl.cpu(), rl)
    assert torch.equal(dk.cpu().view(torch.uint8), rk) and torch.equal(dw.cpu(), rw)


def test_prompt_evict_decode():
    """The run of a layer that bounds its cache: norm + rotation + cache write
    of a prompt, attention, its weights, eviction, then a decode step on the
    compacted cache -- against the fp64 definitions on the same tokens."""
    torch.manual_seed(0)
    H, hk, D, bs, dtype = 8, 2, 128, 16, torch.bfloat16
    kv, budget = [230, 90], 128
    T = sum(kv)
    nb = 40
    order = torch.randperm(nb)
    bt = torch.stack([order[:18], order[18:36]]).int()
    cu = torch.tensor([0, kv[0], T], dtype=torch.int32)
    lens = torch.tensor(kv, dtype=torch.int32)
    qkv = torch.randn(T, H + 2 * hk, D).to(dtype)
    pos = torch.cat([torch.arange(k) for k in kv])
    seq = torch.cat([torch.full((k,), s) for s, k in enumerate(kv)])
    slots = bt[seq, pos // bs].long() * bs + pos % bs
    table = pa.rope_table(512, D, 10000.0, device=DEV)
    d = qkv.to(DEV)
    kc, vc = torch.zeros((2, nb, bs, hk, D), dtype=dtype, device=DEV)
    w = torch.zeros((nb, hk, bs), device=DEV)
    cud, ld, btd = cu.to(DEV), lens.to(DEV), bt.to(DEV)
    scale = D ** -0.5
    q = pa.rope_and_cache(d[:, :H], d[:, H:H + hk], d[:, H + hk:], pos.to(DEV), table, kc, vc,
                          slots.to(DEV))
    out, lse = pa.varlen_fwd(q, kc, vc, cud, ld, btd, max(kv), max(kv), scale, True)
    pa.attn_weights(q, kc, lse, w, cud, ld, btd, max(kv), max(kv), scale, True)
    kept, nl = pa.evict(kc, vc, w, ld, btd, max(kv), budget, 4, 32)
    torch.cuda.synchronize()
    # each head of each sequence: the definition on its kept tokens
    rows = ref.rope_table(pos, ref.rope_rates(D, 10000.0))
    k64 = ref.norm_rotate(qkv[:, H:H + hk], rows, False).to(dtype).double()
    v64 = qkv[:, H + hk:].double()
    assert nl.tolist() == [128, 90]
    new = torch.randn(2, H + 2 * hk, D).to(dtype)
    npos = torch.tensor(kv)
    place = torch.tensor([128, 90])
    nslots = bt[torch.arange(2), place // bs].long() * bs + place % bs
    nd = new.to(DEV)
    q1 = pa.rope_and_cache(nd[:, :H], nd[:, H:H + hk], nd[:, H + hk:], npos.to(DEV), table, kc,
                           vc, nslots.to(DEV))
    o1, l1 = pa.varlen_fwd(q1, kc, vc, torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV),
                           nl + 1, btd, 1, budget + 1, scale, True)
    nrows = ref.rope_table(npos, ref.rope_rates(D, 10000.0))
    nk = ref.norm_rotate(new[:, H:H + hk], nrows, False).to(dtype).double()
    nq = ref.norm_rotate(new[:, :H], nrows, False).to(dtype).double()
    for s in range(2):
        for h in range(H):
            g = h // (H // hk)
            idx = kept[s, g, :int(nl[s])].cpu().long() + int(cu[s])
            keys = torch.cat([k64[idx, g], nk[s:s + 1, g]])
            vals = torch.cat([v64[idx, g], new[s:s + 1, H + hk + g].double()])
            x = keys @ nq[s, h] * scale
            ref_l = torch.logsumexp(x, 0)
            ref_o = torch.softmax(x, 0) @ vals
            assert abs(l1[h, s].item() - ref_l.item()) <= 2e-2   # q, k may round apart by a step
            assert (o1[s, h].cpu().double() - ref_o).abs().max().item() <= 2e-2


@pytest.mark.parametrize("kv,bound,first", [(60000, 60000, 5), (5000, 700, 6), (5000, 4999, 3)])
def test_evict_candidates_past_shared_memory(kv, bound, first):
    """More candidates than the selection keeps in shared memory (48k, or what
    the stated bound asks for, which is reported): the same result."""
    kb, vb, w, bt, lens = pools(13, [kv], 1, 64, 64, 2)
    rk, rv, rw, kept, rlens = ref.evict(kb, vb, w, lens, bt, 333, first, 2)
    dk, dv, dw = typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, glens = pa.evict(dk, dv, dw, lens.to(DEV), bt.to(DEV), bound, 333, first, 2,
                          dev_status=status)
    assert int(status) == (pa.PA_DEV_BAD_SEQLEN if kv > bound else 0)
    assert torch.equal(got.cpu(), kept) and torch.equal(glens.cpu(), rlens)
    assert torch.equal(dk.cpu().view(torch.uint8), rk) and torch.equal(dw.cpu(), rw)


@pytest.mark.parametrize("budget,first,recent", [(1500, 5, 7), (12, 5, 7), (8999, 1, 0), (1, 0, 0)])
@pytest.mark.parametrize("seqs", [1, 9, 40])
def test_evict_long_sequences_with_ties(seqs, budget, first, recent):
    """Few distinct weights (kept ties spread over the blocks that share a
    sequence), no candidate kept, all but one, sequences on both sides of the
    budget; with few and many (sequence, head) pairs."""
    kv = [9000, 4800, 6001, 700, 5, 0, 8191, 5003, 9000][:seqs]
    kv += [5000 + 3 * i for i in range(seqs - len(kv))]
    if seqs == 40:
        kv[10:] = [50] * 30
    kb, vb, w, bt, lens = pools(21, kv, 4, 64, 16, 2)
    w = (w * 5).floor()
    rk, rv, rw, kept, rlens = ref.evict(kb, vb, w, lens, bt, budget, first, recent)
    dk, dv, dw = typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV)
    got, glens = pa.evict(dk, dv, dw, lens.to(DEV), bt.to(DEV), max(kv), budget, first, recent)
    assert torch.equal(got.cpu(), kept) and torch.equal(glens.cpu(), rlens)
    assert torch.equal(dk.cpu().view(torch.uint8), rk)
    assert torch.equal(dv.cpu().view(torch.uint8), rv) and torch.equal(dw.cpu(), rw)


def test_evict_long_bad_page():
    """A page outside the pool in a sequence whose candidates several blocks
    share: reported, and the selection is the one with its keys at -inf."""
    kb, vb, w, bt, lens = pools(22, [6000], 2, 64, 16, 2)
    bad = int(bt[0, 200])
    wi = w.clone()
    wi[bad] = float("-inf")
    kept = ref.evict(kb, vb, wi, lens, bt, 1000, 3, 9)[3]
    bt[0, 200] = -5
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, _ = pa.evict(typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV), lens.to(DEV),
                      bt.to(DEV), 6000, 1000, 3, 9, dev_status=status)
    assert int(status) == pa.PA_DEV_BAD_PAGE
    assert torch.equal(got.cpu(), kept)
