"""The definition of changed scores and masks against closed forms, and the
refusals of pa_score_fwd (host only: nothing is launched)."""
import ctypes as C
import math

import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from oracle import changed_scores as ref

INVALID, UNSUPPORTED, WORKSPACE = 1, 3, 4


@pytest.fixture(scope="module")
def lib():
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    return pa.load_library()


def seen_by(ql, kv, **kw):
    """Which keys each query sees: values are unit vectors, keys are zero."""
    out, lse = ref.attend(torch.zeros((ql, 1, 64)), torch.zeros((kv, 1, 64), dtype=torch.float64),
                          torch.eye(kv, 64, dtype=torch.float64)[:, None], 1.0, **kw)
    return [[j for j in range(kv) if out[i, 0, j] > 0] for i in range(ql)], lse


def test_masks():
    assert seen_by(3, 5)[0] == [[0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 3, 4]]
    assert seen_by(3, 5, prefix=4)[0] == [[0, 1, 2, 3], [0, 1, 2, 3], [0, 1, 2, 3, 4]]
    first = torch.tensor([1, 3, 3])
    assert seen_by(3, 5, first=first)[0] == [[1, 2], [3], [3, 4]]
    got, lse = seen_by(3, 5, first=torch.tensor([3, 9, 0]), prefix=5)
    assert got == [[3, 4], [], [0, 1, 2, 3, 4]]
    assert lse[0, 1] == -math.inf and abs(lse[0, 2] - math.log(5)) < 1e-12


def test_scores():
    # One key: the LSE is its score.
    q, k = torch.full((1, 1, 64), 0.5), torch.full((1, 1, 64), 2.0, dtype=torch.float64)
    one = lambda **kw: float(ref.attend(q, k, k, 0.25, **kw)[1])
    assert one() == 16.0
    assert abs(one(cap=10.0) - 10 * math.tanh(1.6)) < 1e-12
    # The second query's bias on keys 0, 1 is 2 s and s; on its own, none.
    q, k = torch.zeros((1, 2, 64)), torch.zeros((3, 1, 64), dtype=torch.float64)
    _, lse = ref.attend(q, k, k, 1.0, slopes=torch.tensor([0.0, 0.5]))
    assert abs(float(lse[0]) - math.log(3)) < 1e-12
    assert abs(float(lse[1]) - math.log(math.exp(-1.0) + math.exp(-0.5) + 1)) < 1e-12


HK, D, BS = 2, 128, 16


@pytest.fixture(scope="module")
def mem():
    keep = [torch.empty(1 << 16, dtype=torch.uint8) for _ in range(9)]
    return [(t.data_ptr() + 15) // 16 * 16 for t in keep], keep


def call(lib, p, cap=0.0, slopes=None, prefix=None, first=None, fp8=False, **kw):
    a = dict(q=p[0], kc=p[1], vc=p[2], out=p[3], H=4, d=D, bs=BS, scale=0.1, dtype=0, T=1, mq=1,
             ws=0, size=0)
    a.update(kw)
    score = pa.Score(cap, slopes, prefix, first)
    opts = pa.AttnOpts(None, C.pointer(pa.KvFp8(p[4], p[5]))) if fp8 else None
    return lib.pa_score_fwd(None, a["q"], a["H"] * a["d"], a["kc"], a["vc"], BS * HK * a["d"], p[6],
                            p[7], p[8], 4, 1, a["T"], a["mq"], 64, a["H"], HK, a["d"], a["bs"], 4,
                            a["scale"], C.byref(score), C.byref(opts) if opts else None, a["out"],
                            None, a["ws"], a["size"], a["dtype"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(cap=-1.0), INVALID), (dict(cap=math.nan), INVALID), (dict(cap=math.inf), INVALID),
    (dict(cap=3e38), INVALID), (dict(cap=1e-38, scale=1e10), INVALID),
    (dict(slopes=2), INVALID), (dict(prefix=6), INVALID), (dict(first=1), INVALID),
    (dict(cap=1.0, fp8=True), UNSUPPORTED), (dict(fp8=True), UNSUPPORTED),
    (dict(cap=1.0, scale=math.nan), INVALID), (dict(cap=1.0, H=3), INVALID),
    (dict(cap=1.0, d=80), UNSUPPORTED), (dict(cap=1.0, d=256, scale=-1.0), UNSUPPORTED),
    (dict(cap=1.0, bs=8), 2), (dict(cap=1.0, dtype=5), UNSUPPORTED), (dict(cap=1.0, q=0), INVALID),
    (dict(cap=1.0, T=0), 0)])
def test_refusals(lib, mem, kw, want):
    assert call(lib, mem[0], **kw) == want


def test_binding_refuses(lib):
    with pytest.raises(ValueError):
        pa.score_fwd(*([torch.zeros(1)] * 6), 1, 1, 1.0, softcap=2.0)
