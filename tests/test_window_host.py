"""Sliding-window attention with first tokens, checks that need no GPU: the
fp64 definition against brute force and plain causal attention, and the
refusals of pa_window_fwd (made on the host before any CUDA call)."""
import ctypes
import math

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


def test_visible_keys_by_hand():
    seen = ref.window_visible(3, 8, 2, 1)        # queries at positions 5, 6, 7
    assert [[j for j in range(8) if row[j]] for row in seen.tolist()] == [
        [0, 4, 5], [0, 5, 6], [0, 6, 7]]
    assert ref.window_visible(4, 2, 5, 9).sum(1).tolist() == [0, 0, 1, 2]   # positions -2 .. 1


def test_definition_against_brute_force():
    wl = W.random_case(41, num_seqs=3, num_heads=4, num_kv_heads=2, head_size=64, block_size=16,
                       max_q=12, max_kv=40, decode_frac=0.3)
    kc, vc = wl.pool(0), wl.pool(1)
    meta = (wl.cu_seqlens_q, wl.seqused_k, wl.block_table)
    out, lse = ref.window_attention(wl.q, kc, vc, *meta, 0.2, 5, 2)
    at = 0
    for s in range(3):
        for i in range(wl.q_lens[s]):
            p = wl.kv_lens[s] - wl.q_lens[s] + i
            for h in range(4):
                e, o = 0.0, torch.zeros(64, dtype=torch.float64)
                for j in range(p + 1):
                    if j > p - 5 or j < 2:
                        pg, r = int(wl.block_table[s, j // 16]), j % 16
                        w = math.exp(0.2 * float(wl.q[at, h].double() @ kc[pg, r, h // 2].double()))
                        e += w
                        o += w * vc[pg, r, h // 2].double()
                assert abs(lse[h, at].item() - math.log(e)) < 1e-9
                assert (out[at, h] - o / e).abs().max().item() < 1e-9
            at += 1
    full = ref.window_attention(wl.q, kc, vc, *meta, 0.2, 1000, 0)
    want = oracle.varlen_attention(wl.q, kc, vc, *meta, 0.2, True)
    assert torch.allclose(full[0], want[0]) and torch.allclose(full[1], want[1])


def call(lib, **kw):
    a = dict(upd=None, q=FAKE, qs=32 * 128, kc=FAKE, vc=FAKE, cbs=16 * 8 * 128, cu=FAKE, lens=FAKE,
             bt=FAKE, bts=4, S=2, T=2, mq=1, mk=64, H=32, hk=8, D=128, bs=16, nb=10, scale=0.088,
             window=16, first=4, opts=None, out=FAKE, lse=None, ws=FAKE, wsb=1 << 20, dtype=0)
    a.update(kw)
    return lib.pa_window_fwd(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(window=0), pa.PA_ERR_INVALID_ARG),
    (dict(window=-5), pa.PA_ERR_INVALID_ARG),
    (dict(first=-1), pa.PA_ERR_INVALID_ARG),
    (dict(D=96), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=24), pa.PA_ERR_BLOCK_SIZE),
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), pa.PA_ERR_INVALID_ARG),
    (dict(opts="sink"), pa.PA_ERR_INVALID_ARG),                # misaligned sinks
    (dict(D=64, qs=32 * 64, cbs=16 * 8 * 64, opts="fp8"), pa.PA_ERR_UNSUPPORTED),
    (dict(upd=-1), pa.PA_ERR_INVALID_ARG),
    (dict(D=256, qs=32 * 256, cbs=16 * 8 * 256, scale=-0.1), pa.PA_ERR_UNSUPPORTED),
    (dict(S=0, T=0), pa.PA_OK),
])
def test_window_refusals(lib, kw, code):
    kw = dict(kw)
    if "upd" in kw:
        kw["upd"] = ctypes.byref(pa.KvUpdate(FAKE, FAKE, 1024, 1024, FAKE, kw["upd"]))
    desc = pa.KvFp8(FAKE, FAKE)
    if kw.get("opts") == "sink":
        kw["opts"] = ctypes.byref(pa.AttnOpts(FAKE + 2, None))
    elif kw.get("opts") == "fp8":
        kw["opts"] = ctypes.byref(pa.AttnOpts(None, ctypes.pointer(desc)))
    assert call(lib, **kw) == code


def test_window_reaches_the_workspace_check(lib):
    """The largest window and first count pass the argument checks; with no
    workspace the call stops at PA_ERR_WORKSPACE (PA_ERR_CUDA without a GPU)."""
    big = 2 ** 31 - 1
    for kw in (dict(window=big, first=big), dict(window=1, first=0), dict(window=63, first=big)):
        assert call(lib, ws=None, wsb=0, **kw) in (pa.PA_ERR_WORKSPACE, pa.PA_ERR_CUDA)


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.window_fwd(q, c, c, i, i[:2], torch.zeros((2, 4), dtype=torch.int32), 1, 8, 0.1, 4)
