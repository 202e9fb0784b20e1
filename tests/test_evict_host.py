"""Accumulated attention weights and eviction, checks that need no GPU: the
fp64 definitions on small hand-made inputs, and the refusals of
pa_attn_weights and pa_evict (made on the host before any CUDA call)."""
import ctypes

import pytest
import torch

import oracle
import paged_kv_varlen_attn_gb300 as pa
import workloads as W
from oracle import cache_ops as ref
from paged_kv_varlen_attn_gb300 import _build

FAKE = 0x10000   # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


@pytest.mark.parametrize("causal", [True, False])
def test_weights_sum_to_the_rows(causal):
    """Every query row's weights sum to 1, so what a call adds to the keys of
    a KV head is its query tokens times the heads of the group."""
    wl = W.random_case(31, num_seqs=4, num_heads=6, num_kv_heads=2, head_size=64, block_size=16,
                       max_q=20, max_kv=50, decode_frac=0.3)
    kc, vc = wl.pool(0), wl.pool(1)
    meta = (wl.cu_seqlens_q, wl.seqused_k, wl.block_table)
    _, lse = oracle.varlen_attention(wl.q, kc, vc, *meta, wl.softmax_scale, causal)
    w0 = torch.full((wl.num_blocks, 2, 16), 5.0)
    w = ref.attn_weights(wl.q, kc, lse, w0, *meta, wl.softmax_scale, causal)
    for s in range(4):
        q, k = wl.q_lens[s], wl.kv_lens[s]
        j = torch.arange(k)
        rows = w[wl.block_table[s].long()[j // 16], :, j % 16]          # [k, hk]
        old = 5.0 * (k - q)
        assert torch.allclose(rows.sum(0), torch.full((2,), old + 3 * q, dtype=torch.float64))


def test_evict_by_hand():
    bs, w = 16, torch.zeros(2, 1, 16)
    weights = [9, 1, 5, 5, 0, 7, 5, 2, 0, 3]     # keys 0 .. 9 on page 1
    w[1, 0, :10] = torch.tensor(weights, dtype=torch.float32)
    kc = torch.arange(2 * bs * 64).view(2, bs, 1, 64).int()
    vc = -kc
    bt = torch.tensor([[1]])
    nk, nv, nw, kept, lens = ref.evict(kc, vc, w, torch.tensor([10]), bt, 6, 2, 1)
    # first 0, 1; last 9; of 2 .. 8 the heaviest three: 7 (key 5), then the
    # fives of lowest index (keys 2 and 3)
    assert kept[0, 0].tolist() == [0, 1, 2, 3, 5, 9] and lens.tolist() == [6]
    assert torch.equal(nk[1, :6], kc[1, [0, 1, 2, 3, 5, 9]])
    assert torch.equal(nv[1, :6], vc[1, [0, 1, 2, 3, 5, 9]])
    assert nw[1, 0, :6].tolist() == [9, 1, 5, 5, 7, 3]
    assert torch.equal(nk[1, 6:], kc[1, 6:]) and torch.equal(nk[0], kc[0])


def call_weights(lib, **kw):
    a = dict(q=FAKE, qs=32 * 128, kc=FAKE, cbs=16 * 8 * 128, lse=FAKE, cu=FAKE, lens=FAKE, bt=FAKE,
             bts=4, S=2, T=2, mq=1, mk=64, H=32, hk=8, D=128, bs=16, nb=10, scale=0.088, causal=1,
             w=FAKE, ws=128, fp8=None, dtype=0)
    a.update(kw)
    return lib.pa_attn_weights(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), pa.PA_ERR_INVALID_ARG),
    (dict(H=30), pa.PA_ERR_INVALID_ARG),
    (dict(D=96), pa.PA_ERR_UNSUPPORTED),
    (dict(dtype=3), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=8), pa.PA_ERR_BLOCK_SIZE),
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(kc=None), pa.PA_ERR_INVALID_ARG),
    (dict(lse=None), pa.PA_ERR_INVALID_ARG),
    (dict(lse=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(w=None), pa.PA_ERR_INVALID_ARG),
    (dict(w=FAKE + 4), pa.PA_ERR_INVALID_ARG),
    (dict(ws=124), pa.PA_ERR_INVALID_ARG),
    (dict(ws=130), pa.PA_ERR_INVALID_ARG),
    (dict(cu=None), pa.PA_ERR_INVALID_ARG),
    (dict(qs=100), pa.PA_ERR_INVALID_ARG),
    (dict(cbs=16 * 8 * 128 + 4), pa.PA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), pa.PA_ERR_INVALID_ARG),
    (dict(causal=3), pa.PA_ERR_INVALID_ARG),
    (dict(fp8=(None, FAKE)), pa.PA_ERR_INVALID_ARG),
    (dict(fp8=(FAKE + 2, FAKE)), pa.PA_ERR_INVALID_ARG),
    (dict(fp8=(FAKE, None), D=64, qs=32 * 64, cbs=16 * 8 * 64), pa.PA_ERR_UNSUPPORTED),
    (dict(S=1 << 30, mk=1 << 20), pa.PA_ERR_INVALID_ARG),      # more blocks than a launch has
    (dict(mk=(1 << 30) + 1), pa.PA_ERR_INVALID_ARG),
    (dict(T=1 << 29), pa.PA_ERR_INVALID_ARG),                  # packed rows
    (dict(S=0, T=0), pa.PA_OK),
    (dict(T=0, q=None, lse=None), pa.PA_OK),                   # no queries: nothing to add
])
def test_weights_refusals(lib, kw, code):
    if kw.get("fp8"):
        kw = dict(kw, fp8=ctypes.byref(pa.KvFp8(*kw["fp8"])))
    assert call_weights(lib, **kw) == code


def call_evict(lib, **kw):
    a = dict(kc=FAKE, vc=FAKE, cbs=16 * 8 * 128, w=FAKE, ws=128, lens=FAKE, bt=FAKE, bts=4, S=2,
             mk=64, hk=8, D=128, bs=16, nb=10, elem=2, budget=32, first=4, recent=8, kept=FAKE,
             nl=FAKE)
    a.update(kw)
    return lib.pa_evict(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), pa.PA_ERR_INVALID_ARG),
    (dict(budget=0), pa.PA_ERR_INVALID_ARG),
    (dict(budget=(1 << 30) + 1), pa.PA_ERR_INVALID_ARG),
    (dict(first=-1), pa.PA_ERR_INVALID_ARG),
    (dict(recent=-1), pa.PA_ERR_INVALID_ARG),
    (dict(first=20, recent=13), pa.PA_ERR_INVALID_ARG),
    (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), pa.PA_ERR_INVALID_ARG),
    (dict(elem=4), pa.PA_ERR_UNSUPPORTED),
    (dict(elem=1, D=64), pa.PA_ERR_UNSUPPORTED),
    (dict(D=32), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=24), pa.PA_ERR_BLOCK_SIZE),
    (dict(kc=None), pa.PA_ERR_INVALID_ARG),
    (dict(vc=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(cbs=16 * 8 * 128 - 8), pa.PA_ERR_INVALID_ARG),
    (dict(elem=1, cbs=16 * 8 * 128 + 8), pa.PA_ERR_INVALID_ARG),
    (dict(w=None), pa.PA_ERR_INVALID_ARG),
    (dict(ws=127), pa.PA_ERR_INVALID_ARG),
    (dict(lens=None), pa.PA_ERR_INVALID_ARG),
    (dict(kept=None), pa.PA_ERR_INVALID_ARG),
    (dict(nl=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(S=0, kc=None, kept=None), pa.PA_OK),
])
def test_evict_refusals(lib, kw, code):
    assert call_evict(lib, **kw) == code


def test_binding_refuses_wrong_shapes():
    c = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    w, n = torch.zeros(4, 8, 16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):                       # not CUDA tensors
        pa.evict(c, c, w, n, torch.zeros((2, 4), dtype=torch.int32), 64, 32)
    for bad in (w[:, :4], w.double(), w.transpose(1, 2)):
        with pytest.raises(ValueError):
            pa._weights_stride(bad, 4, 16, 8)
