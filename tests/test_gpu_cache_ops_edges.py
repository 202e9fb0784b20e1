"""The operators around paged attention at the edges of what a call may be: a
page size that is no power of two, pools whose offsets pass 32 bits, calls in
flight on two streams, captured calls on changed inputs, repeated eviction,
wide block tables. Results are compared with the same operator on an ordinary
layout, bit by bit, or with the fp64 definitions at the tolerances derived in
the operators' own tests."""
import pytest
import torch

import oracle
import paged_kv_varlen_attn_gb300 as pa
import workloads as W
from helpers import oracle_pools
from oracle import cache_ops as ref
from test_gpu_evict import pools, random_weights, rel_bound, typed
from test_gpu_window import check, define

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


def dev(wl):
    return tuple(t.to(DEV) for t in (wl.cu_seqlens_q, wl.seqused_k, wl.block_table))


@pytest.mark.parametrize("bs", [48, 80, 1008])
@pytest.mark.parametrize("mq", [1, 150])
def test_page_sizes_that_are_no_power_of_two(bs, mq):
    wl = W.random_case(41 + bs, num_seqs=3, num_heads=8, num_kv_heads=2, head_size=128,
                       block_size=bs, max_q=mq, max_kv=1300, decode_frac=0.0)
    kc, vc = oracle_pools(wl)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale)
    d = (wl.q.to(DEV), kc.to(DEV), vc.to(DEV))
    check(pa.window_fwd(*d, *dev(wl), *tail, 100, 5), define(wl, kc, vc, 100, 5))
    out, lse = pa.varlen_fwd(*d, *dev(wl), *tail, True)
    w0 = random_weights(wl)
    got = pa.attn_weights(d[0], d[1], lse, w0.to(DEV), *dev(wl), *tail, True).cpu().double()
    want = ref.attn_weights(wl.q, kc, lse.cpu(), w0, wl.cu_seqlens_q, wl.seqused_k,
                            wl.block_table, wl.softmax_scale, True)
    assert ((got - want).abs() <= rel_bound(wl, kc, lse.cpu()) * want.abs()).all()
    kv = [900, 130, 555]
    kb, vb, w, bt, lens = pools(bs, kv, 2, 64, bs, 2)
    rk, rv, rw, kept, rl = ref.evict(kb, vb, w, lens, bt, 100, 3, 20)
    dk, dv, dw = typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV)
    gk, gl = pa.evict(dk, dv, dw, lens.to(DEV), bt.to(DEV), max(kv), 100, 3, 20)
    assert torch.equal(gk.cpu(), kept) and torch.equal(gl.cpu(), rl)
    assert torch.equal(dk.cpu().view(torch.uint8), rk) and torch.equal(dw.cpu(), rw)
    # rotation and cache write into such pages: the bytes of 16-row pages
    T, n = 70, 5
    g = torch.Generator().manual_seed(2)
    x = torch.randn((T, 6, 128), generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.arange(T, device=DEV)
    table = pa.rope_table(T, 128, device=DEV)
    slots = torch.randperm(n * bs, generator=g)[:T].to(DEV)
    res = []
    for rows in (bs, 16):
        k = torch.zeros((n * bs // rows, rows, 2, 128), dtype=torch.bfloat16, device=DEV)
        v = torch.zeros_like(k)
        pa.rope_and_cache(x[:, :2], x[:, 2:4], x[:, 4:], pos, table, k, v, slots)
        res.append((k.flatten(0, 1), v.flatten(0, 1)))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


@pytest.mark.parametrize("mq,mk", [(1, 700), (200, 500)])
def test_offsets_past_32_bits(mq, mk):
    """Pools of more than 2^32 elements (8.6 GB each) with the sequences' pages
    at their far end: the same bits as in a small pool."""
    wl = W.random_case(61 + mq, num_seqs=3, num_heads=8, num_kv_heads=8, head_size=128,
                       block_size=16, max_q=mq, max_kv=mk, decode_frac=0.0)
    kc, vc = (t.to(DEV) for t in oracle_pools(wl))
    far = (1 << 32) // (16 * 8 * 128) + 100
    nb = far + wl.num_blocks
    big_k = torch.empty((nb, 16, 8, 128), dtype=torch.bfloat16, device=DEV)
    big_v = torch.empty_like(big_k)
    big_k[far:], big_v[far:] = kc, vc
    cu, lens, bt = dev(wl)
    bt = bt.clamp(max=wl.num_blocks - 1)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale)
    q = wl.q.to(DEV)
    small = pa.window_fwd(q, kc, vc, cu, lens, bt, *tail, 150, 4)
    large = pa.window_fwd(q, big_k, big_v, cu, lens, bt + far, *tail, 150, 4)
    assert torch.equal(small[0], large[0]) and torch.equal(small[1], large[1])
    _, lse = pa.varlen_fwd(q, kc, vc, cu, lens, bt, *tail, True)
    w = torch.rand((wl.num_blocks, 8, 16), device=DEV)
    wide = torch.zeros((nb, 8, 16), device=DEV)
    wide[far:] = w
    pa.attn_weights(q, kc, lse, w, cu, lens, bt, *tail, True)
    pa.attn_weights(q, big_k, lse, wide, cu, lens, bt + far, *tail, True)
    assert torch.equal(w, wide[far:])
    T = wl.k_new.shape[0]
    table = pa.rope_table(600, 64, device=DEV)
    pos = torch.arange(T, device=DEV) % 600
    slots = wl.slot_mapping.to(DEV)
    new = (wl.k_new.to(DEV), wl.v_new.to(DEV))
    a = pa.rope_and_cache(q, *new, pos, table, kc, vc, slots)
    b = pa.rope_and_cache(q, *new, pos, table, big_k, big_v, slots + far * 16)
    assert torch.equal(a, b) and torch.equal(kc, big_k[far:]) and torch.equal(vc, big_v[far:])
    r1 = pa.evict(kc, vc, w, lens, bt, wl.max_seqlen_k, 64, 2, 10)
    r2 = pa.evict(big_k, big_v, wide, lens, bt + far, wl.max_seqlen_k, 64, 2, 10)
    assert torch.equal(r1[0], r2[0]) and torch.equal(r1[1], r2[1])
    assert torch.equal(kc, big_k[far:]) and torch.equal(vc, big_v[far:])
    assert torch.equal(w, wide[far:])


def test_two_streams_at_once():
    """Calls in flight on two streams, each on its own tensors (no state is
    shared; windowed attention with a workspace of its own each)."""
    wls = [W.random_case(s, num_seqs=6, num_heads=16, num_kv_heads=4, head_size=128,
                         block_size=16, max_q=300, max_kv=900, decode_frac=0.3)
           for s in (81, 82)]
    data = []
    for wl in wls:
        kc, vc = (t.to(DEV) for t in oracle_pools(wl))
        tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale)
        _, lse = pa.varlen_fwd(wl.q.to(DEV), kc, vc, *dev(wl), *tail, True)
        w = torch.rand((wl.num_blocks, 4, 16), device=DEV)
        data.append((wl.q.to(DEV), kc, vc, dev(wl), tail, lse, w))

    def run(d, w, kc, vc):
        q, _, _, meta, tail, lse, _ = d
        out = pa.window_fwd(q, kc, vc, *meta, *tail, 120, 3)
        pa.attn_weights(q, kc, lse, w, *meta, *tail, True)
        kept = pa.evict(kc, vc, w, meta[1], meta[2], tail[1], 200, 4, 50)
        return (*out, w, kc, vc, *kept)
    alone = [run(d, d[6].clone(), d[1].clone(), d[2].clone()) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    copies = [[(d[6].clone(), d[1].clone(), d[2].clone()) for d in data] for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for rep in range(3):
        for d, c, st in zip(data, copies[rep], streams):
            with torch.cuda.stream(st):
                got.append(run(d, *c))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for x, y in zip(g, alone[i % 2]):
            assert torch.equal(x, y)


def test_weights_captured():
    """Both kernels (prompt and decode rows) in a graph, replayed on other
    lengths and queries."""
    wl = W.random_case(91, num_seqs=5, num_heads=16, num_kv_heads=4, head_size=128,
                       block_size=16, max_q=200, max_kv=800, decode_frac=0.4)
    kc, vc = (t.to(DEV) for t in oracle_pools(wl))
    cu, lens, bt = dev(wl)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale)
    q = wl.q.to(DEV)
    _, lse = pa.varlen_fwd(q, kc, vc, cu, lens, bt, *tail, True)
    w0 = torch.rand((wl.num_blocks, 4, 16), device=DEV)
    w = w0.clone()
    pa.attn_weights(q, kc, lse, w, cu, lens, bt, *tail, True)    # first call: no capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.attn_weights(q, kc, lse, w, cu, lens, bt, *tail, True)
    q.mul_(0.5)
    lens.copy_(torch.clamp(lens - 3, min=0))
    w.copy_(w0)
    graph.replay()
    torch.cuda.synchronize()
    again = w0.clone()
    pa.attn_weights(q, kc, lse, again, cu, lens, bt, *tail, True)
    assert torch.equal(w, again)


def test_repeated_eviction_and_growth():
    """Evicting what is already within the budget changes nothing; the cache
    grows again and is cut again."""
    kv, hk, D, bs, budget = [120, 90], 2, 64, 16, 64
    kb, vb, w, bt, lens = pools(13, kv, hk, D, bs, 2)
    dk, dv, dw, dl = typed(kb, 2).to(DEV), typed(vb, 2).to(DEV), w.to(DEV), lens.to(DEV)
    pa.evict(dk, dv, dw, dl, bt.to(DEV), 120, budget, 2, 16, new_lens=dl)
    assert dl.tolist() == [64, 64]
    before = dk.clone(), dv.clone(), dw.clone()
    kept, _ = pa.evict(dk, dv, dw, dl, bt.to(DEV), 120, budget, 2, 16, new_lens=dl)
    assert torch.equal(kept, torch.arange(budget, dtype=torch.int32, device=DEV).expand(2, hk, -1))
    for x, y in zip(before, (dk, dv, dw)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    dl += 20                                        # 20 new tokens per sequence
    k1, v1, w1 = dk.cpu().view(torch.uint8), dv.cpu().view(torch.uint8), dw.cpu()
    want = ref.evict(k1, v1, w1, dl.cpu(), bt, budget, 2, 16)
    kept, nl = pa.evict(dk, dv, dw, dl, bt.to(DEV), 84, budget, 2, 16)
    assert torch.equal(kept.cpu(), want[3]) and nl.tolist() == [64, 64]
    assert torch.equal(dk.cpu().view(torch.uint8), want[0])
    assert torch.equal(dw.cpu(), want[2])


def test_block_table_slices():
    """Columns of a wider table; one whose last row would be read past its
    storage is refused."""
    wl = W.random_case(95, num_seqs=4, num_heads=8, num_kv_heads=2, head_size=64, block_size=16,
                       max_q=30, max_kv=200, decode_frac=0.3)
    kc, vc = (t.to(DEV) for t in oracle_pools(wl))
    cu, lens, bt = dev(wl)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale)
    wide = torch.full((4, bt.shape[1] + 9), 1 << 20, dtype=torch.int32, device=DEV)
    wide[:, :bt.shape[1]] = bt
    q = wl.q.to(DEV)
    a = pa.window_fwd(q, kc, vc, cu, lens, bt, *tail, 20, 2)
    b = pa.window_fwd(q, kc, vc, cu, lens, wide[:, :bt.shape[1]], *tail, 20, 2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide[:, 9:] = bt
    w = torch.zeros((wl.num_blocks, 2, 16), device=DEV)
    with pytest.raises(ValueError):
        pa.window_fwd(q, kc, vc, cu, lens, wide[:, 9:], *tail, 20, 2)
    with pytest.raises(ValueError):
        pa.attn_weights(q, kc, a[1], w, cu, lens, wide[:, 9:], *tail, True)
    with pytest.raises(ValueError):
        pa.evict(kc, vc, w, lens, wide[:, 9:], wl.max_seqlen_k, 32)
    with pytest.raises(ValueError):
        pa.evict(kc, vc, w, lens, bt[:1].expand(4, -1), wl.max_seqlen_k, 32)


def test_oracle_weights_match_the_attention_lse():
    """The weights computed from the library's own LSE sum to the query rows."""
    wl = W.random_case(99, num_seqs=3, num_heads=8, num_kv_heads=2, head_size=128, block_size=16,
                       max_q=120, max_kv=300, decode_frac=0.2)
    kc, vc = oracle_pools(wl)
    ref_o, ref_l = oracle.varlen_attention(wl.q, kc, vc, wl.cu_seqlens_q, wl.seqused_k,
                                           wl.block_table, wl.softmax_scale, True)
    tail = (wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale)
    _, lse = pa.varlen_fwd(wl.q.to(DEV), kc.to(DEV), vc.to(DEV), *dev(wl), *tail, True)
    w = torch.zeros((wl.num_blocks, 2, 16), device=DEV)
    pa.attn_weights(wl.q.to(DEV), kc.to(DEV), lse, w, *dev(wl), *tail, True)
    # each of the T rows of a KV head's 4 query heads has weights of sum 1, to
    # the LSE's own 1e-3
    total = w.double().sum((0, 2)).cpu()
    assert ((total - 4 * wl.total_q).abs() <= 2e-3 * 4 * wl.total_q).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,D,mq", [(8, 128, 1), (8, 128, 300), (14, 64, 400), (4, 256, 260)])
def test_weights_rows_that_saw_nothing_hold_anything(H, D, mq, causal):
    """Queries whose LSE is -inf (padding rows) hold NaN and infinities: the
    same bits as with zeros there."""
    wl = W.random_case(311 + mq, num_seqs=3, num_heads=H, num_kv_heads=2, head_size=D,
                       block_size=16, max_q=mq, max_kv=700, decode_frac=0.0)
    kc, vc = oracle_pools(wl)
    meta = (wl.cu_seqlens_q, wl.seqused_k, wl.block_table)
    _, lse = oracle.varlen_attention(wl.q, kc, vc, *meta, wl.softmax_scale, causal)
    lse = lse.float()
    blind = torch.rand(lse.shape, generator=torch.Generator().manual_seed(5)) < 0.05
    blind[1, 0] = True
    lse[blind] = float("-inf")
    w0 = random_weights(wl)
    got = []
    for fill in (0.0, float("nan"), float("inf")):
        q = wl.q.clone()
        q[blind.T] = fill
        got.append(pa.attn_weights(q.to(DEV), kc.to(DEV), lse.to(DEV), w0.to(DEV), *dev(wl),
                                   wl.max_seqlen_q, wl.max_seqlen_k, wl.softmax_scale, causal))
    want = ref.attn_weights(torch.where(blind.T[..., None], torch.zeros_like(wl.q), wl.q), kc, lse,
                            w0, *meta, wl.softmax_scale, causal)
    rel = rel_bound(wl, kc, lse)
    assert ((got[0].cpu().double() - want).abs() <= rel * want.abs()).all()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
