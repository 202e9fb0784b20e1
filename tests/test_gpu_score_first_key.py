"""Attention with first keys at the ends of int32: negative ones count as 0."""
import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from test_gpu_score import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


SHAPES = [
    ([(700, 1), (90, 1), (3000, 1)], 8, 2, 128, "bf16"),        # decode
    ([(500, 5), (64, 3)], 8, 4, 64, "f16"),                     # short queries
    ([(700, 300), (260, 129)], 6, 2, 128, "f16"),               # prompts
    ([(300, 200), (150, 150)], 4, 4, 64, "bf16"),
    ([(300, 140), (700, 1)], 4, 2, 256, "bf16"),
]


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("seqs,H,hk,D,dt", SHAPES)
def test_first_keys_at_the_ends_of_the_range(seqs, H, hk, D, dt, cap):
    # Negative: as 0, bit for bit. Past every key: nothing is seen.
    b = Batch(seqs, H, hk, D, 16, dt, seed=33)
    zero = torch.zeros(b.T, dtype=torch.int32)
    want, want_lse = b.run(softcap=cap, first_key=zero)
    for low in (-2 ** 31, -2 ** 31 + 100, -2 ** 30, -1):
        out, lse = b.run(softcap=cap, first_key=zero + low)
        assert torch.equal(out, want) and torch.equal(lse, want_lse), low
    mixed = zero.clone()
    mixed[::3] = -2 ** 31
    out, lse = b.run(softcap=cap, first_key=mixed)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse = b.run(softcap=cap, first_key=zero + (2 ** 31 - 1))
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("seqs,H,hk,D,dt", SHAPES)
def test_window_beside_a_cap_and_a_bias(seqs, H, hk, D, dt):
    # A window of w tokens as first keys, position - w + 1.
    b = Batch(seqs, H, hk, D, 16, dt, seed=34)
    pos = torch.cat([torch.arange(kv - ql, kv) for kv, ql in seqs])
    for w in (1, 50, 129):
        kw = dict(softcap=20.0, alibi_slopes=b.slopes(), first_key=(pos - w + 1).int())
        out, lse = b.run(**kw)
        b.check(out, lse, **kw)
