"""Attention with caps far above the scores.

Tolerances: as in test_gpu_score.py, but for the cap, whose rounding does not grow with
it: a capped score is off by at most 2^-20 of itself (a polynomial, or a quotient
where the score is at least 0.46 of the cap) and 2^-20 of the cap up to 128.
"""
import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from oracle import changed_scores as ref
from test_gpu_score import Batch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


def check(b, out, lse, cap, slopes=None, first_key=None, scale=None):
    out, lse = out.cpu().double(), lse.cpu().double()
    scale = b.scale if scale is None else scale
    half = torch.finfo(b.dtype).eps / 2
    for s, (kv, ql) in enumerate(b.seqs):
        rows = slice(int(b.cu[s]), int(b.cu[s]) + ql)
        j = torch.arange(kv)
        page, row = b.table[s].long()[j // b.bs], j % b.bs
        key, value = b.kc[page, row].double(), b.vc[page, row].double()
        want, wl = ref.attend(b.q[rows], key, value, scale, True, None, cap, slopes, 0,
                              None if first_key is None else first_key[rows])
        G = b.H // b.hk
        A = abs(scale) * b.q[rows].double().abs().sum(-1) * \
            key.abs().amax((0, 2)).repeat_interleave(G)
        err = A * 2.0 ** -18 + A.clamp(max=cap) * 2.0 ** -20 + min(cap, 128.0) * 2.0 ** -20
        if slopes is not None:
            err = err + kv * slopes.double().abs() * 2.0 ** -22
        lse_off = (lse[:, rows] - wl).abs() - err.T - 2.0 ** -20 * (1 + wl.abs())
        assert lse_off.max() <= 0, (s, lse_off.max())
        v = value.abs().amax((0, 2)).repeat_interleave(G)
        tol = half * want.abs() + (v * (2 * (err + 2.0 ** -20) + half))[..., None]
        off = (out[rows] - want).abs() - tol
        assert off.max() <= 0, (s, off.max())


SHAPES = [
    ([(700, 1), (90, 1), (3000, 1)], 8, 2, 128, "bf16"),        # decode
    ([(500, 5), (64, 3)], 8, 4, 64, "f16"),                     # short queries
    ([(700, 300), (260, 129)], 6, 2, 128, "f16"),               # prompts
    ([(300, 200), (150, 150)], 4, 4, 64, "bf16"),
    ([(300, 140), (700, 1)], 4, 2, 256, "bf16"),
]


@pytest.mark.parametrize("cap", [100.0, 150.0, 1e3, 1e5, 3e6, 1e30])
@pytest.mark.parametrize("seqs,H,hk,D,dt", SHAPES)
def test_large_caps(seqs, H, hk, D, dt, cap):
    b = Batch(seqs, H, hk, D, 16, dt, seed=31)
    out, lse = b.run(softcap=cap)
    check(b, out, lse, cap)
    kw = dict(softcap=cap, alibi_slopes=b.slopes())
    out, lse = b.run(**kw)
    check(b, out, lse, cap, b.slopes())


@pytest.mark.parametrize("seqs,H,hk,D,dt", SHAPES[:4])
def test_scores_up_to_a_large_cap(seqs, H, hk, D, dt):
    # Some rows' scores reach the cap, others stay far below it.
    b = Batch(seqs, H, hk, D, 16, dt, seed=32)
    b.q[::2] *= 300
    for cap, scale in ((400.0, b.scale), (1000.0, -b.scale)):
        out, lse = b.run(scale, softcap=cap)
        check(b, out, lse, cap, scale=scale)
