"""Argument checks of the operators around attention that need no GPU: the
limits of a launch, integers past 32 bits, outputs beside their inputs."""
import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from paged_kv_varlen_attn_gb300 import _build
from test_evict_host import call_weights
from test_rope_host import call_rope


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


@pytest.mark.parametrize("S,mk,hk,ok", [
    (1 << 10, 128 * ((1 << 18) - 1), 8, True),      # 2^31 - 8192 blocks
    (1 << 10, 128 * ((1 << 18) - 1) + 1, 8, False),   # 2^31
    ((1 << 30) - 1, 128, 2, True),                  # 2^31 - 2
    ((1 << 30) - 1, 0, 2, True),
    (1 << 30, 1, 2, False),
    (1 << 30, 1 << 30, 2048, False),                # 2^64: a product that wraps to nothing
])
def test_weights_largest_grid(lib, S, mk, hk, ok):
    """One block per 128 keys of a sequence and KV head: a call is refused only
    past what a launch holds (no queries: an accepted call launches nothing)."""
    got = call_weights(lib, S=S, mk=mk, H=hk, hk=hk, D=64, qs=hk * 64, cbs=16 * hk * 64,
                       ws=16 * hk, T=0, mq=0)
    assert got == (pa.PA_OK if ok else pa.PA_ERR_INVALID_ARG)


BIG = [(1 << 32) + 5, -(1 << 32) + 5, 1 << 31, -(1 << 31) - 1]


@pytest.mark.parametrize("v", BIG)
def test_integers_past_32_bits_are_refused(lib, v):
    """ctypes passes the low 32 bits of an integer; the binding refuses what
    does not fit, before it looks at any tensor."""
    c = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    q, w = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 8, 16)
    n, bt = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32)
    cu, lse = torch.zeros(3, dtype=torch.int32), torch.zeros(8, 2)
    calls = [lambda: pa.evict(c, c, w, n, bt, v, 32),
             lambda: pa.evict(c, c, w, n, bt, 64, v),
             lambda: pa.evict(c, c, w, n, bt, 64, 32, v),
             lambda: pa.evict(c, c, w, n, bt, 64, 32, 0, v),
             lambda: pa.attn_weights(q, c, lse, w, cu, n, bt, v, 64, 0.1, True),
             lambda: pa.attn_weights(q, c, lse, w, cu, n, bt, 1, v, 0.1, True),
             lambda: pa.window_fwd(q, c, c, cu, n, bt, v, 64, 0.1, 16),
             lambda: pa.window_fwd(q, c, c, cu, n, bt, 1, v, 0.1, 16),
             lambda: pa.rope_table(v, 2, device="meta"),
             lambda: pa.rope_table(2, v, device="meta")]
    if v < 0:      # a window (first tokens) past the integers is all; below them, nothing
        calls += [lambda: pa.window_fwd(q, c, c, cu, n, bt, 1, 64, 0.1, v),
                  lambda: pa.window_fwd(q, c, c, cu, n, bt, 1, 64, 0.1, 16, v)]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_rope_table_longer_than_32_bits_is_refused(lib):
    q = torch.empty((1, 2, 128), dtype=torch.bfloat16, device="meta")
    c = torch.empty((1, 16, 2, 128), dtype=torch.bfloat16, device="meta")
    i = torch.empty(1, dtype=torch.int64, device="meta")
    table = torch.empty(((1 << 32) + 8, 64), device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        pa.rope_and_cache(q, q, q, i, table, c, c, i)


ROW = 32 * 128
FAR = 1 << 24    # 16-byte aligned, never dereferenced: validation fails first


@pytest.mark.parametrize("n,os,off", [
    (4, 4 * ROW, 3 * ROW + 8),        # the next row of q begins inside
    (4, 4 * ROW, ROW - 8),
    (4, 4 * ROW, -ROW + 8),
    (4, 4 * ROW, 4 * ROW),            # other rows of q
    (4, 4 * ROW, -8 * ROW),
    (4, 2 * ROW, 3 * ROW),            # strides apart: any common range
    (1, 2 * ROW, ROW - 8),
])
def test_rope_output_that_overlaps_its_input(lib, n, os, off):
    """q_out lies off elements from q, whose rows are four rows apart."""
    assert call_rope(lib, n=n, q=FAR, qs=4 * ROW, out=FAR + 2 * off, os=os) == \
        pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("given", [("key",), ("value",), ("slot_mapping",), ("key", "value"),
                                   ("value", "slot_mapping"), ("key", "slot_mapping")])
def test_window_update_is_whole_or_none(lib, given):
    """New tokens without one of key, value and slots: refused, not left out."""
    m = dict(device="meta")
    q = torch.empty((2, 8, 128), dtype=torch.bfloat16, **m)
    c = torch.empty((4, 16, 8, 128), dtype=torch.bfloat16, **m)
    n, bt = torch.empty(2, dtype=torch.int32, **m), torch.empty((2, 4), dtype=torch.int32, **m)
    cu = torch.empty(3, dtype=torch.int32, **m)
    new = dict(key=q, value=q, slot_mapping=torch.empty(2, dtype=torch.int64, **m))
    with pytest.raises(ValueError, match="go together"):
        pa.window_fwd(q, c, c, cu, n, bt, 1, 64, 0.1, 16, **{k: new[k] for k in given})
