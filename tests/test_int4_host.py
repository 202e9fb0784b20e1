"""The 4-bit format's definition against closed forms, and the refusals of the
entry points over 4-bit pools (host only: nothing is launched)."""
import ctypes as C

import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from oracle import changed_scores as ref

INVALID, BLOCK, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    return pa.load_library()


def test_codes_of_a_ramp():
    # 0, 1, .., 15 repeated: scale 1, minimum 0, the codes are the values.
    x = torch.arange(128).remainder(16).float()
    codes, params = ref.quantize_int4(x[None])
    assert torch.equal(codes[0], x.long())
    assert params[0].tolist() == [1.0, 0.0]


def test_ties_to_even_and_ends():
    # Minimum -2 and scale 0.25 are exact: -2 + 0.25 (n + 0.5) lies between two
    # codes and goes to the even one.
    x = torch.full((64,), -2.0)
    x[1] = 1.75
    x[2:17] = -2.0 + 0.25 * (torch.arange(15) + 0.5)
    codes, params = ref.quantize_int4(x[None])
    assert params[0].tolist() == [0.25, -2.0]
    assert codes[0, :17].tolist() == [0, 15] + [0, 2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14, 14]


def test_constant_rows_infinities_and_nan():
    x = torch.full((4, 64), 3.5)
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    x[3] = 0.0
    codes, params = ref.quantize_int4(x)
    assert params[0].tolist() == [0.0, 3.5] and not codes[0].any()
    assert params[1, 1] == 3.5 and codes[1, 7] == 15 and not codes[1, :7].any()
    assert params[2].isnan().all() and not codes[2].any()
    assert params[3].tolist() == [0.0, 0.0]


def test_half_a_step():
    # A value is off by at most half a scale, the rounding of the minimum, and
    # what the scale's rounding leaves over the fifteenth code.
    g = torch.Generator().manual_seed(5)
    x = torch.randn((500, 128), generator=g) * torch.logspace(-3, 3, 500)[:, None]
    codes, params = ref.quantize_int4(x)
    got = codes * params[:, :1].double() + params[:, 1:].double()
    step = params[:, :1].double()
    slack = 15 * step * 2.0 ** -11 + params[:, 1:].double().abs() * 2.0 ** -11 + 2.0 ** -24
    assert ((got - x.double()).abs() <= step / 2 + slack).all()


def test_places_of_the_codes():
    # Word w: elements 8w, 8w + 2, .. in its low half, 8w + 1, .. in its high.
    codes = torch.arange(64).remainder(16)
    packed = ref.pack_int4(codes)
    words = packed.view(torch.int32)
    for w in range(8):
        for i in range(8):
            shift = 4 * (i // 2) + 16 * (i % 2)
            assert (int(words[w]) >> shift) & 15 == int(codes[8 * w + i])
    assert torch.equal(ref.unpack_int4(packed), codes)


# ------------------------------------------------------------------ refusals
HK, D, BS, NB = 2, 128, 16, 4


def buf(n=1 << 16):
    t = torch.empty(n + 64, dtype=torch.uint8)
    p = t.data_ptr()
    return t, (p + 15) // 16 * 16


@pytest.fixture(scope="module")
def mem():
    keep = [buf() for _ in range(10)]
    return [p for _, p in keep], keep


def write(lib, p, **kw):
    a = dict(key=p[0], value=p[1], ks=HK * D, vs=HK * D, kc=p[2], vc=p[3], page=BS * HK * D // 2,
             kp=p[4], vp=p[5], pp=HK * BS, slots=p[6], n=0, hk=HK, d=D, bs=BS, nb=NB, dtype=0)
    a.update(kw)
    desc = None if a["kp"] is False else C.byref(pa.KvInt4(a["kp"], a["vp"], a["pp"]))
    return lib.pa_reshape_and_cache_int4(a["key"], a["value"], a["ks"], a["vs"], a["kc"], a["vc"],
                                         a["page"], desc, a["slots"], a["n"], a["hk"], a["d"],
                                         a["bs"], a["nb"], a["dtype"], None, None)


WRITES = [
    (dict(kp=False), INVALID), (dict(n=-1), INVALID), (dict(d=256), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(bs=24), BLOCK),
    (dict(bs=2048), BLOCK), (dict(n=1, key=0), INVALID), (dict(n=1, slots=0), INVALID),
    (dict(n=1, kp=0), INVALID), (dict(n=1, vp=0), INVALID), (dict(n=1, page=BS * HK * D // 2 - 16),
                                                             INVALID),
    (dict(n=1, page=BS * HK * D // 2 + 8), INVALID), (dict(n=1, pp=HK * BS - 1), INVALID),
    (dict(n=1, ks=HK * D - 8), INVALID), (dict(n=1, vs=HK * D + 4), INVALID),
]


@pytest.mark.parametrize("kw,want", WRITES)
def test_write_refusals(lib, mem, kw, want):
    assert write(lib, mem[0], **kw) == want


def test_write_misaligned(lib, mem):
    p = mem[0]
    for name in ("key", "value", "kc", "vc"):
        at = dict(key=p[0], value=p[1], kc=p[2], vc=p[3])[name]
        assert write(lib, p, n=1, **{name: at + 8}) == INVALID
    assert write(lib, p, n=1, kp=p[4] + 4) == INVALID
    assert write(lib, p, n=1, pp=HK * BS + 2) == INVALID
    assert write(lib, p, n=1, slots=p[6] + 4) == INVALID
    assert write(lib, p) == 0                     # nothing to write


def gather(lib, p, **kw):
    a = dict(kc=p[2], vc=p[3], page=BS * HK * D // 2, kp=p[4], vp=p[5], pp=HK * BS, slots=p[6], n=1,
             hk=HK, d=D, bs=BS, nb=NB, key=p[7], value=p[8], dtype=0)
    a.update(kw)
    return lib.pa_gather_cache_int4(a["kc"], a["vc"], a["page"],
                                    C.byref(pa.KvInt4(a["kp"], a["vp"], a["pp"])), a["slots"],
                                    a["n"], a["hk"], a["d"], a["bs"], a["nb"], a["key"], a["value"],
                                    a["dtype"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(hk=0), INVALID), (dict(d=256), UNSUPPORTED),
    (dict(dtype=7), UNSUPPORTED), (dict(bs=8), BLOCK), (dict(kc=0), INVALID),
    (dict(slots=0), INVALID), (dict(key=0), INVALID), (dict(value=0), INVALID),
    (dict(pp=1), INVALID), (dict(page=16), INVALID), (dict(hk=1 << 22), INVALID), (dict(n=0), 0)])
def test_gather_refusals(lib, mem, kw, want):
    assert gather(lib, mem[0], **kw) == want


def rope(lib, p, rot=64, interleaved=0, null_rope=False, desc=True, **kw):
    a = dict(heads=2, n=0, page=BS * HK * D // 2, qs=2 * D, d=D, pos=p[9], table=p[8])
    a.update(kw)
    r = pa.Rope(a["table"], 8, rot, interleaved, None, None, 1e-6)
    u = pa.KvUpdate(p[0], p[1], HK * D, HK * D, p[6], a["n"])
    kv = C.byref(pa.KvInt4(p[4], p[5], HK * BS)) if desc else None
    return lib.pa_rope_and_cache_int4(None if null_rope else C.byref(r), a["pos"], p[7], a["qs"],
                                      p[7], a["qs"], C.byref(u), p[2], p[3], a["page"], kv,
                                      a["heads"], HK, a["d"], BS, NB, 0, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(null_rope=True), INVALID), (dict(desc=False), INVALID), (dict(rot=8), INVALID),
    (dict(rot=24), INVALID), (dict(rot=144), INVALID), (dict(interleaved=2), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(heads=0), INVALID), (dict(n=1, pos=0), INVALID),
    (dict(n=1, table=0), INVALID), (dict(n=1, qs=D), INVALID), (dict(n=1, page=16), INVALID),
    (dict(), 0)])
def test_rope_refusals(lib, mem, kw, want):
    assert rope(lib, mem[0], **kw) == want


def attend(lib, p, desc=True, **kw):
    a = dict(update=None, q=p[0], qs=4 * D, kc=p[2], vc=p[3], page=BS * HK * D // 2, cu=p[6],
             lens=p[7], bt=p[8], row=4, seqs=1, T=1, mq=1, mk=64, H=4, hk=HK, d=D, bs=BS, nb=NB,
             scale=0.1, causal=1, sinks=None, out=p[9], lse=None, ws=0, size=0, dtype=0, kp=p[4],
             pp=HK * BS)
    a.update(kw)
    kv = C.byref(pa.KvInt4(a["kp"], p[5], a["pp"])) if desc else None
    return lib.pa_varlen_fwd_int4kv(
        a["update"], a["q"], a["qs"], a["kc"], a["vc"], a["page"], a["cu"], a["lens"], a["bt"],
        a["row"], a["seqs"], a["T"], a["mq"], a["mk"], a["H"], a["hk"], a["d"], a["bs"], a["nb"],
        a["scale"], a["causal"], kv, a["sinks"], a["out"], a["lse"], a["ws"], a["size"],
        a["dtype"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(desc=False), INVALID), (dict(H=3), INVALID), (dict(d=256), UNSUPPORTED),
    (dict(H=2 * 129), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(bs=20), BLOCK),
    (dict(page=BS * HK * D // 2 - 16), INVALID), (dict(kp=0), INVALID), (dict(pp=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(causal=2), INVALID), (dict(mk=(1 << 30) + 1),
                                                                     INVALID),
    (dict(q=0), INVALID), (dict(cu=0), INVALID), (dict(mq=-1), INVALID), (dict(T=0), 0),
    (dict(seqs=0, T=0), 0)])
def test_attention_refusals(lib, mem, kw, want):
    assert attend(lib, mem[0], **kw) == want


def test_workspace_sizes(lib):
    size = pa.varlen_fwd_int4kv_workspace_size
    assert size(4, 4, 1, 4096, 32, 8, 256, 16, 152) == 0
    assert size(4, 4, 1, 4096, 8 * 129, 8, 128, 16, 152) == 0
    decode, verify, prompt = (size(4, 4 * q, q, 4096, 32, 8, 128, 16, 152) for q in (1, 5, 900))
    assert 0 < decode <= verify <= prompt
    # The key bound of a decode batch does not matter.
    assert size(4, 4, 1, 1 << 30, 32, 8, 128, 16, 152) == decode


def test_binding_refuses(lib):
    with pytest.raises(ValueError):
        pa.varlen_fwd_int4kv(*([torch.zeros(1)] * 8), 1, 1, 1.0, True)
    with pytest.raises(ValueError):
        pa.reshape_and_cache_int4(*([torch.zeros(1)] * 7))
