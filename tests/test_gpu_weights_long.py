"""Accumulated weights of a sequence so long that (keys x heads of the group)
passes 32 bits, on the tensor-core kernel."""
import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


@pytest.mark.parametrize("blind", [False, True])
def test_keys_times_group_past_32_bits(blind):
    """64 query heads on one KV head of 64, 34,000,000 keys (4.4 GB): key j of
    the last, partial query tile (and, with blind, of the first, one of whose
    rows saw nothing) is 64 (past - j) > 2^31 packed rows away for the first
    445,000 keys. Every page holds the same 1,024 rows, so a key in front of
    the queries gets the sum of its row.

    Tolerance: a term's exponent is off by the float32 dot product of D
    products, at most 2 D 2^-24 scale |q| |k| (twice the sequential bound), and
    by 8 * 2^-24 (|x| + |lse|) + 2^-21 of the products, the LSE's conversion
    and ex2; n positive terms add n 2^-24."""
    H, D, bs, kv, qn, dtype = 64, 64, 1024, 34_000_000, 3, torch.bfloat16
    past, nb = kv - qn, (kv + bs - 1) // bs
    assert past * H > 2 ** 31 and (nb - 1) * bs < past
    g = torch.Generator().manual_seed(17)
    q = torch.randn((qn, H, D), generator=g).to(dtype)
    page = torch.randn((bs, 1, D), generator=g).to(dtype)
    lse = 2 + torch.rand((H, qn), generator=g)
    if blind:
        lse[5, 0] = float("-inf")
    scale = D ** -0.5
    kc = page.to(DEV).expand(nb, bs, 1, D).contiguous()
    w = torch.zeros((nb, 1, bs), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.attn_weights(q.to(DEV), kc, lse.to(DEV), w,
                    torch.tensor([0, qn], dtype=torch.int32, device=DEV),
                    torch.tensor([kv], dtype=torch.int32, device=DEV),
                    torch.arange(nb, dtype=torch.int32, device=DEV)[None], qn, kv, scale, True,
                    dev_status=status)
    assert int(status) == 0
    x = torch.einsum("ihd,rd->hir", q.double(), page[:, 0].double()) * scale
    p = torch.exp(x - lse.double()[..., None])           # [H, query, row of a page]
    p[torch.isinf(lse)] = 0.0
    qk = scale * (q.double().norm(dim=-1).max() * page.double().norm(dim=-1).max()).item()
    rel = (2 * D * qk + 8 * (qk + 3) + qn * H) * 2.0 ** -24 + 2.0 ** -21
    want = p.sum((0, 1))
    got = w[:nb - 1, 0].double()                         # pages in front of the queries
    assert ((got - want.to(DEV)).abs() <= rel * want.to(DEV)).all()
    tail = w[nb - 1, 0].cpu().double()
    for r in range(bs):
        j = (nb - 1) * bs + r
        seen = p[:, max(0, j - past):, r].sum() if j < kv else 0.0
        assert abs(tail[r] - seen) <= rel * seen
