"""Pools of no pages (num_blocks = 0): every page is outside the pool and reads as
zeros, whatever lies at the pool's address."""
import math

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


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("kv,ql,D", [([16, 0, 40], 1, 128), ([48, 20, 33], 20, 128),
                                     ([40, 40], 40, 64), ([40, 16], 1, 256)])
def test_pool_of_no_pages(scored, kv, ql, D):
    S, H, hk, bs = len(kv), 8, 2, 16
    T = S * ql
    q = torch.randn((T, H, D), device=DEV).bfloat16()
    pool = torch.randn((4, bs, hk, D), device=DEV).bfloat16()
    cu = torch.arange(0, T + 1, ql, dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv, dtype=torch.int32, device=DEV)
    table = torch.zeros((S, 3), dtype=torch.int32, device=DEV)
    out = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((H, T), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = pa.alloc_workspace(pa.varlen_fwd_workspace_size(S, T, ql, 48, H, hk, D, bs, sms), DEV)
    front = (q.data_ptr(), H * D, pool.data_ptr(), pool.data_ptr(), bs * hk * D, cu.data_ptr(),
             lens.data_ptr(), table.data_ptr(), 3, S, T, ql, 48, H, hk, D, bs, 0, D ** -0.5)
    back = (out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), pa.PA_BF16,
            status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    lib = pa.load_library()
    if scored:
        score = pa.Score(30.0, None, None, None)
        code = lib.pa_score_fwd(None, *front, score, None, *back)
    else:
        code = lib.pa_varlen_fwd(*front, 1, *back)
    torch.cuda.synchronize()
    assert code == pa.PA_OK and status.item() == pa.PA_DEV_BAD_PAGE
    assert (out == 0).all()
    for s, n in enumerate(kv):
        for i in range(ql):
            seen = max(n - ql + i + 1, 0)
            want = math.log(seen) if seen else -math.inf
            got = lse[:, s * ql + i]
            assert (got == want).all() or ((got - want).abs() <= 2.0 ** -20 * (1 + want)).all()
