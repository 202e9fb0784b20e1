"""GPU parity of the rotary table and of the norm + rotation + cache write
with their fp64 definitions.

Tolerances, from arithmetic:
  * table: the phase is exact to 1e-9 radian (a 64-bit fraction of a turn per
    position), the float32 remainder, sinpi / cospi and the product with
    mscale are each off by at most 2 units of 2^-24: 6 * 2^-24 * mscale.
  * rotated values: one rounding to the output type (half a step) of a float32
    value that is off by a few 2^-24 of the head's largest element (norm: sum
    of D squares, rsqrt, two products; rotation: two products, one add): at
    most 16 * 2^-24 of it.
"""
import math

import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
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


TABLES = [
    (1, 2, 10000.0, dict()),
    (300, 16, 10000.0, dict()),
    (1000, 30, 500.0, dict()),                        # a width that is no power of two
    (777, 256, 10000.0, dict(scaling="linear", factor=4.0)),
    (5000, 128, 500000.0, dict(scaling="ntk", factor=8.0)),
    (5000, 128, 500000.0, dict(scaling="wavelength", factor=8.0, orig_len=8192)),
    (5000, 64, 500000.0, dict(scaling="wavelength", factor=3.0, orig_len=2048, low=2, high=9)),
    (5000, 128, 1000000.0, dict(scaling="yarn", factor=4.0, orig_len=32768)),
    (5000, 64, 10000.0, dict(scaling="yarn", factor=16.0, orig_len=64, mscale=1.0)),
    (400, 64, 10000.0, dict(scaling="yarn", factor=2.0, orig_len=4096, low=3, high=3.5)),
    (1100000, 32, 10000.0, dict()),                   # positions past a million
]


@pytest.mark.parametrize("n,rot,base,kw", TABLES)
def test_table(n, rot, base, kw):
    got = pa.rope_table(n, rot, base, device=DEV, **kw).cpu().double()
    pos = list(range(n)) if n <= 5000 else list(range(0, n, 997)) + [n - 2, n - 1]
    mscale = kw.get("mscale")
    if mscale is None:
        mscale = 0.1 * math.log(kw["factor"]) + 1 if kw.get("scaling") == "yarn" else 1.0
    okw = {k: v for k, v in kw.items() if k != "mscale"}
    want = ref.rope_table(pos, ref.rope_rates(rot, base, **okw), mscale)
    tol = mscale * (6 * 2.0 ** -24 + 2e-9)
    assert (got[pos] - want).abs().max().item() <= tol


def batch(seed, T, H, hk, D, bs, dtype, rot, packed, table_len=600):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((T, H + 2 * hk, D), generator=g).to(dtype)
    nb = (T + bs - 1) // bs + 3
    slots = torch.randperm(nb * bs, generator=g)[:T]
    pos = torch.randint(0, table_len, (T,), generator=g)
    table = ref.rope_table(range(table_len), ref.rope_rates(rot, 10000.0)).float()
    d = qkv.to(DEV)
    parts = [d[:, :H], d[:, H:H + hk], d[:, H + hk:]]
    if not packed:
        parts = [p.contiguous() for p in parts]
    return qkv, parts, nb, slots, pos, table


def head_tol(y, dtype, inflate):
    """Half a step of the output type plus float32 slack of the head's scale."""
    eps = torch.finfo(dtype).eps
    tiny = torch.finfo(dtype).smallest_normal * eps / 2   # half a subnormal step
    big = y.abs().amax(-1, keepdim=True).clamp(min=1e-30) * inflate
    return y.abs() * (eps / 2) * (1 + eps) + 16 * 2.0 ** -24 * big + tiny


CASES = [
    # T, H, hk, D, bs, dtype, rot, interleaved, norm, packed
    (1, 1, 1, 64, 16, torch.bfloat16, 64, False, False, True),
    (1, 8, 2, 128, 16, torch.float16, 128, False, True, True),
    (7, 5, 5, 64, 16, torch.bfloat16, 32, True, True, True),       # odd head count: half items
    (37, 3, 1, 64, 32, torch.float16, 16, False, True, False),
    (64, 32, 8, 128, 16, torch.bfloat16, 128, False, True, True),
    (129, 28, 4, 128, 64, torch.bfloat16, 64, True, False, True),
    (50, 6, 2, 128, 16, torch.bfloat16, 96, False, True, True),    # rot no power of two
    (33, 6, 3, 256, 16, torch.float16, 256, False, True, True),
    (20, 2, 1, 256, 1024, torch.bfloat16, 48, True, False, True),
    (700, 16, 2, 128, 128, torch.bfloat16, 128, True, True, True),
    (6000, 8, 1, 64, 16, torch.bfloat16, 64, False, False, True),  # a warp takes whole tokens
]


@pytest.mark.parametrize("T,H,hk,D,bs,dtype,rot,inter,norm,packed", CASES)
def test_rope_and_cache(T, H, hk, D, bs, dtype, rot, inter, norm, packed):
    qkv, (q, k, v), nb, slots, pos, table = batch(T + D, T, H, hk, D, bs, dtype, rot, packed)
    g = torch.Generator().manual_seed(1)
    qw, kw = [1 + 0.2 * torch.randn(D, generator=g) for _ in range(2)] if norm else (None, None)
    kc = torch.full((nb, bs, hk, D), 7.0, dtype=dtype)
    vc = torch.full((nb, bs, hk, D), -7.0, dtype=dtype)
    dk, dv = kc.to(DEV), vc.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pa.rope_and_cache(q, k, v, pos.to(DEV), table.to(DEV), dk, dv, slots.to(DEV), inter,
                            None if qw is None else qw.to(DEV),
                            None if kw is None else kw.to(DEV), 1e-5, dev_status=status)
    rows = table[pos]
    want = ref.norm_rotate(qkv[:, :H], rows, inter, qw, 1e-5)
    inflate = 2.0 if not norm else 4.0      # rotation and weights may enlarge an element
    assert ((out.cpu().double() - want).abs() <= head_tol(want, dtype, inflate)).all()
    # the pool: rotated keys and copied values in their slots, nothing else
    want_k = ref.norm_rotate(qkv[:, H:H + hk], rows, inter, kw, 1e-5)
    got_k = dk.cpu().flatten(0, 1)[slots].double()
    assert ((got_k - want_k).abs() <= head_tol(want_k, dtype, inflate)).all()
    vc.view(-1, hk, D)[slots] = qkv[:, H + hk:]
    assert torch.equal(dv.cpu(), vc)
    rest = torch.ones(nb * bs, dtype=torch.bool)
    rest[slots] = False
    assert (dk.cpu().flatten(0, 1)[rest] == 7.0).all()
    assert int(status) == 0
    # in place on q: the same bits
    pa.rope_and_cache(q, k, v, pos.to(DEV), table.to(DEV), dk, dv, slots.to(DEV), inter,
                      None if qw is None else qw.to(DEV), None if kw is None else kw.to(DEV),
                      1e-5, out=q)
    assert torch.equal(q, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter,rot,norm", [(False, 128, True), (True, 64, False)])
def test_rope_fp8(dtype, inter, rot, norm):
    T, H, hk, D, bs = 90, 8, 4, 128, 32
    qkv, (q, k, v), nb, slots, pos, table = batch(5, T, H, hk, D, bs, dtype, rot, True)
    ks, vs = torch.tensor([0.01, 0.03, 0.5, 3.0]), torch.tensor([0.02, 0.3, 1.0, 0.004])
    kw = torch.linspace(0.5, 2, D) if norm else None
    dk = torch.zeros((nb, bs, hk, D), dtype=torch.uint8, device=DEV)
    dv, rv, rk = dk.clone(), dk.clone(), dk.clone()
    pa.rope_and_cache(q, k, v, pos.to(DEV), table.to(DEV), dk, dv, slots.to(DEV), inter, None,
                      None if kw is None else kw.to(DEV), 1e-6, k_scale=ks.to(DEV),
                      v_scale=vs.to(DEV))
    # values: the bytes of the plain quantizing scatter
    pa.reshape_and_cache_fp8(k, v, rk, rv, slots.to(DEV), ks, vs)
    assert torch.equal(dv, rv)
    got = dk.view(torch.float8_e4m3fn).float().cpu().flatten(0, 1)[slots].double()
    want = ref.norm_rotate(qkv[:, H:H + hk], table[pos], inter, kw, 1e-6) / ks.double()[:, None]
    want = want.clamp(-448, 448)
    # half an e4m3 step (2^-4 relative, 2^-10 below the smallest normal) plus
    # the float32 slack in front of it
    slack = 64 * 2.0 ** -24 * want.abs().amax(-1, keepdim=True)
    tol = torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10) + slack
    assert ((got - want).abs() <= tol).all()


def test_rope_padding_and_bad_metadata():
    """Padding (negative position or slot) and metadata outside the table or
    the pool: those tokens are skipped, the others as without them."""
    T, H, hk, D, bs, dtype = 12, 4, 2, 64, 16, torch.bfloat16
    qkv, (q, k, v), nb, slots, pos, table = batch(3, T, H, hk, D, bs, dtype, 64, True, 50)
    dk = torch.full((nb, bs, hk, D), 3.0, dtype=dtype, device=DEV)
    dv = dk.clone()
    good = pa.rope_and_cache(q, k, v, pos.to(DEV), table.to(DEV), dk.clone(), dv.clone(),
                             slots.to(DEV))
    p2, s2 = pos.clone(), slots.clone()
    p2[1], p2[4], s2[7], s2[9] = -1, 50, -5, nb * bs
    out = torch.full((T, H, D), 9.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.rope_and_cache(q, k, v, p2.to(DEV), table.to(DEV), dk, dv, s2.to(DEV), out=out,
                      dev_status=status)
    assert int(status) == pa.PA_DEV_BAD_POSITION | pa.PA_DEV_BAD_SLOT
    skipped = torch.zeros(T, dtype=torch.bool)
    skipped[[1, 4]] = True
    assert (out[skipped.to(DEV)] == 9.0).all()
    assert torch.equal(out[~skipped.to(DEV)], good[~skipped.to(DEV)])
    uncached = skipped.clone()
    uncached[[7, 9]] = True
    flat = dk.cpu().flatten(0, 1)
    assert (flat[slots[uncached]] == 3.0).all()
    assert (flat[slots[~uncached]] != 3.0).any(-1).all()
    # padding alone sets no bit, and a call without tokens is nothing
    p2, s2 = pos.clone(), slots.clone()
    p2[3], s2[5] = -7, -1
    status.zero_()
    pa.rope_and_cache(q, k, v, p2.to(DEV), table.to(DEV), dk, dv, s2.to(DEV), dev_status=status)
    assert int(status) == 0
    e = torch.empty(0, dtype=torch.int64, device=DEV)
    pa.rope_and_cache(q[:0], k[:0], v[:0], e, table.to(DEV), dk, dv, e)


def test_rope_values_that_do_not_turn():
    """Infinities and NaN stay with their own pair; elements past rot_dim are
    copied bit by bit."""
    T, H, hk, D, bs = 2, 2, 1, 64, 16
    for inter in (False, True):
        qkv, (q, k, v), nb, slots, pos, table = batch(8, T, H, hk, D, bs, torch.float16, 32, True)
        q[0, 0, 3] = float("inf")
        q[0, 1, 40] = float("nan")
        q[1, 0, 63] = float("-inf")
        kc = torch.zeros((nb, bs, hk, D), dtype=torch.float16, device=DEV)
        out = pa.rope_and_cache(q, k, v, pos.to(DEV), table.to(DEV), kc, kc.clone(),
                                slots.to(DEV), inter)
        assert torch.equal(out[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16))
        touched = {2, 3} if inter else {3, 19}
        for i in range(32):
            assert bool(torch.isfinite(out[0, 0, i])) == (i not in touched)
        assert torch.isfinite(out[1, 0, :32]).all() and torch.isfinite(out[0, 1, :32]).all()


def test_rope_combined_pool_graph_and_stream():
    """A combined [num_blocks, 2, ...] pool (page stride of two pages), a
    captured call replayed on new inputs, and a call on a side stream."""
    T, H, hk, D, bs, dtype = 40, 8, 2, 128, 16, torch.bfloat16
    qkv, (q, k, v), nb, slots, pos, table = batch(4, T, H, hk, D, bs, dtype, 128, True)
    pos, slots, table = pos.to(DEV), slots.to(DEV), table.to(DEV)
    both = torch.zeros((nb, 2, bs, hk, D), dtype=dtype, device=DEV)
    kc, vc = torch.zeros((2, nb, bs, hk, D), dtype=dtype, device=DEV)
    want = pa.rope_and_cache(q, k, v, pos, table, kc, vc, slots)
    got = pa.rope_and_cache(q, k, v, pos, table, both[:, 0], both[:, 1], slots)
    assert torch.equal(got, want)
    assert torch.equal(both[:, 0], kc) and torch.equal(both[:, 1], vc)
    # graph
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.rope_and_cache(q, k, v, pos, table, kc, vc, slots, out=out)
        side.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pa.rope_and_cache(q, k, v, pos, table, kc, vc, slots, out=out)
    torch.cuda.current_stream().wait_stream(side)
    pos.add_(1)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    k2, v2 = kc.clone(), vc.clone()
    assert torch.equal(pa.rope_and_cache(q, k, v, pos, table, kc, vc, slots), out)
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
