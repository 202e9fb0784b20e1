"""4-bit pools whose rows hold what the cache writes do not write."""
import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
from test_gpu_int4_ranges import Pools

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


@pytest.mark.parametrize("share", [0.5, 1.0])
@pytest.mark.parametrize("kv,ql,H,hk,D,dt", [
    ([300, 1, 70, 2000], 1, 8, 2, 128, "bf16"), ([300, 40, 70], 3, 8, 4, 64, "f16"),
    ([400, 33], 2, 24, 2, 128, "f16"), ([300, 129], 100, 4, 2, 128, "bf16"),
    ([200, 64], 64, 8, 8, 64, "f16"),
])
def test_negative_scales(kv, ql, H, hk, D, dt, share):
    # A value is code x scale + minimum, whatever the scale's sign.
    b = Pools(kv, [min(ql, n) for n in kv], H, hk, D, 16, dt, 41)
    g = torch.Generator(device=DEV).manual_seed(2)
    for p in b.params:
        flip = torch.rand(p.shape[:3], device=DEV, generator=g) < share
        p[..., 0] = torch.where(flip, -p[..., 0], p[..., 0])
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("D,dt,G", [(128, "bf16", 2), (64, "f16", 2), (128, "f16", 8)])
def test_infinite_scale_of_a_hidden_key(D, dt, G):
    # The last token's scale of V is infinite: the tokens in front of it do not see it.
    b = Pools([90, 40, 1000], [3, 3, 3], 2 * G, 2, D, 16, dt, 42)
    rows = [(b.table[s, (n - 1) // 16].item(), (n - 1) % 16) for s, n in enumerate(b.kv)]
    for page, row in rows:
        b.params[1][page, :, row] = 0.0
    want, want_lse = b.run()
    for page, row in rows:
        b.params[1][page, :, row, 0] = float("inf")
    out, lse = b.run()
    blind = [i for i in range(9) if i % 3 != 2]
    assert torch.equal(out[blind], want[blind]) and torch.equal(lse[:, blind], want_lse[:, blind])
