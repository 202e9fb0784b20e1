"""4-bit decode where a block has three KV heads and a warp without one, over ranges of
many slices: the ring of copies goes round several times.

Tolerances as in test_gpu_int4.py.
"""
import pytest
import torch

from test_gpu_int4_ranges import Pools

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()


LENGTHS = {
    "equal": [8200] * 24,                                   # 10, 20 and 30 slices a range
    "unequal": [1, 20000, 33, 0, 70000, 5, 5, 90000, 64, 12345],
    "tiny": [n % 41 for n in range(3000)],
}


@pytest.mark.parametrize("kind", sorted(LENGTHS))
@pytest.mark.parametrize("hk,D,dt,G,tokens", [
    (3, 128, "bf16", 8, 1), (3, 128, "f16", 1, 2), (6, 128, "f16", 4, 1), (9, 128, "bf16", 2, 1),
    (15, 128, "bf16", 1, 1), (3, 64, "f16", 4, 1), (9, 64, "bf16", 8, 1), (3, 128, "bf16", 8, 2),
    (6, 128, "f16", 8, 4),
])
def test_three_heads_a_block(kind, hk, D, dt, G, tokens):
    kv = LENGTHS[kind]
    b = Pools(kv, [tokens] * len(kv), G * hk, hk, D, 16, dt, hk + G)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = b.run(dev_status=status)
    assert status.item() == 0
    b.check(out, lse)
    for _ in range(3):
        again, lse2 = b.run()
        assert torch.equal(out, again) and torch.equal(lse, lse2)
