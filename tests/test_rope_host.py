"""Rotary positions, checks that need no GPU: the fp64 definition against
closed forms, and the refusals of pa_rope_table and pa_rope_and_cache (made on
the host before any CUDA call)."""
import cmath
import ctypes
import math

import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from oracle import cache_ops as ref
from paged_kv_varlen_attn_gb300 import _build

FAKE = 0x10000   # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def test_definition_is_a_complex_rotation():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 2, 8), generator=g, dtype=torch.float64)
    pos, rates = [0, 5, 77], ref.rope_rates(6, 100.0)
    rows = ref.rope_table(pos, rates)
    for inter in (False, True):
        y = ref.norm_rotate(x, rows, inter)
        assert torch.equal(y[..., 6:], x[..., 6:])
        for t, p in enumerate(pos):
            for i, f in enumerate(rates):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 3)
                for h in range(2):
                    z = complex(x[t, h, a], x[t, h, b]) * cmath.exp(1j * p * f)
                    assert abs(complex(y[t, h, a], y[t, h, b]) - z) < 1e-12


def test_norm_definition():
    x = torch.tensor([[[3.0, 4.0, 0.0, 0.0]]])
    rows = ref.rope_table([0], [1.0])
    y = ref.norm_rotate(x, rows, False, torch.tensor([1.0, 2.0, 1.0, 1.0]), eps=0.0)
    r = 1 / math.sqrt(25 / 4)
    assert torch.allclose(y.flatten(), torch.tensor([3 * r, 8 * r, 0, 0], dtype=torch.float64))


def test_scaled_rates():
    """Limits of each scaling: the fastest pair of a band-wise scaling keeps
    its rate, the slowest is divided by the factor; the NTK base moves the
    slowest pair by exactly the factor and leaves the fastest."""
    plain = ref.rope_rates(128, 10000.0)
    for kind in ("wavelength", "yarn"):
        f = ref.rope_rates(128, 10000.0, kind, 4.0, 4096)
        assert f[0] == plain[0] and abs(f[-1] * 4 / plain[-1] - 1) < 1e-12
        assert all(p / 4 * (1 - 1e-12) <= x <= p * (1 + 1e-12) for x, p in zip(f, plain))
    f = ref.rope_rates(128, 10000.0, "ntk", 4.0)
    assert f[0] == 1.0 and abs(f[-1] * 4 / plain[-1] - 1) < 1e-12
    assert ref.rope_rates(128, 10000.0, "linear", 4.0)[3] == plain[3] / 4


def scaling(**kw):
    a = dict(kind=4, factor=4.0, orig_len=4096.0, low=1.0, high=32.0, mscale=1.0)
    a.update(kw)
    return ctypes.byref(pa.RopeScaling(*a.values()))


def test_table_refusals(lib):
    def call(out=FAKE, n=8, rot=64, base=1e4, s=None):
        return lib.pa_rope_table(out, n, rot, base, s, None)
    bad = pa.PA_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(n=(1 << 30) + 1), dict(rot=0), dict(rot=7), dict(rot=258), dict(base=0.0),
               dict(base=-2.0), dict(base=float("nan")), dict(base=float("inf")),
               dict(out=None), dict(out=FAKE + 4),
               dict(s=scaling(kind=5)), dict(s=scaling(kind=-1)), dict(s=scaling(factor=0.0)),
               dict(s=scaling(factor=float("inf"))), dict(s=scaling(kind=1, factor=-1.0)),
               dict(s=scaling(orig_len=0.0)), dict(s=scaling(low=0.0)),
               dict(s=scaling(high=1.0)), dict(s=scaling(high=float("nan"))),
               dict(s=scaling(mscale=float("nan"))), dict(base=1.0, s=scaling()),
               dict(rot=2, s=scaling(kind=2)), dict(base=1e300, s=scaling(kind=2, factor=1e30))):
        assert call(**kw) == bad, kw
    assert call(n=0, out=None) == pa.PA_OK        # no positions: nothing to do
    with pytest.raises(ValueError):
        pa.rope_table(4, 64, scaling="other", device="cpu")
    with pytest.raises(ValueError):
        pa.rope_table(4, 64, device="cpu")


def rope(**kw):
    a = dict(cos_sin=FAKE, table_len=100, rot_dim=128, interleaved=0, q_norm=None, k_norm=None,
             norm_eps=1e-6)
    a.update(kw)
    return pa.Rope(*a.values())


def call_rope(lib, r=None, **kw):
    a = dict(pos=FAKE, q=FAKE, qs=32 * 128, out=FAKE + (1 << 24), os=32 * 128, key=FAKE,
             value=FAKE, ks=1024, vs=1024, slots=FAKE, n=4, kc=FAKE, vc=FAKE, cbs=16 * 1024, H=32,
             hk=8, D=128, bs=16, nb=10, fp8=None, dtype=0, rope=True, update=True)
    a.update(kw)
    u = pa.KvUpdate(a["key"], a["value"], a["ks"], a["vs"], a["slots"], a["n"])
    return lib.pa_rope_and_cache(
        ctypes.byref(r or rope()) if a["rope"] else None, a["pos"], a["q"], a["qs"], a["out"],
        a["os"], ctypes.byref(u) if a["update"] else None, a["kc"], a["vc"], a["cbs"], a["H"],
        a["hk"], a["D"], a["bs"], a["nb"], a["fp8"], a["dtype"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rope=False), pa.PA_ERR_INVALID_ARG),
    (dict(update=False), pa.PA_ERR_INVALID_ARG),
    (dict(n=-1), pa.PA_ERR_INVALID_ARG),
    (dict(H=0), pa.PA_ERR_INVALID_ARG),
    (dict(H=1 << 22, qs=1 << 30, os=1 << 30), pa.PA_ERR_INVALID_ARG),   # row offsets past 32 bits
    (dict(hk=0), pa.PA_ERR_INVALID_ARG),
    (dict(D=96), pa.PA_ERR_UNSUPPORTED),
    (dict(dtype=2), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=24), pa.PA_ERR_BLOCK_SIZE),
    (dict(pos=None), pa.PA_ERR_INVALID_ARG),
    (dict(pos=FAKE + 4), pa.PA_ERR_INVALID_ARG),
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(out=None), pa.PA_ERR_INVALID_ARG),
    (dict(qs=32 * 128 - 8), pa.PA_ERR_INVALID_ARG),
    (dict(os=32 * 128 + 4), pa.PA_ERR_INVALID_ARG),
    (dict(out=FAKE, os=32 * 128 + 8), pa.PA_ERR_INVALID_ARG),          # overlaps q
    (dict(out=FAKE + 16), pa.PA_ERR_INVALID_ARG),
    (dict(out=FAKE + 2 * 4 * 32 * 128 - 16), pa.PA_ERR_INVALID_ARG),
    (dict(key=None), pa.PA_ERR_INVALID_ARG),
    (dict(slots=FAKE + 4), pa.PA_ERR_INVALID_ARG),
    (dict(cbs=16 * 1024 - 8), pa.PA_ERR_INVALID_ARG),
    (dict(D=64, qs=32 * 64, os=32 * 64, fp8="scales"), pa.PA_ERR_UNSUPPORTED),
    (dict(fp8="none"), pa.PA_ERR_INVALID_ARG),
    (dict(n=0, q=None, pos=None), pa.PA_OK),                           # no tokens
])
def test_rope_refusals(lib, kw, code):
    if kw.get("fp8") is not None:
        desc = pa.KvFp8(FAKE, FAKE) if kw["fp8"] == "scales" else pa.KvFp8(None, FAKE)
        kw = dict(kw, fp8=ctypes.byref(desc))
    r = rope(rot_dim=64) if kw.get("D") == 64 else None
    assert call_rope(lib, r, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(table_len=-1),
    dict(interleaved=2), dict(cos_sin=None), dict(cos_sin=FAKE + 4), dict(q_norm=FAKE + 4),
    dict(k_norm=FAKE + 8), dict(norm_eps=-1e-6), dict(norm_eps=float("nan"))])
def test_rope_descriptor_refusals(lib, kw):
    assert call_rope(lib, rope(**kw)) == pa.PA_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        pa.rope_and_cache(q, q, q, i, torch.zeros(4, 128), c, c, i)
