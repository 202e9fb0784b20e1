"""Windowed decode over e4m3 pools with bf16 queries near either end of the
type's range: the kernel brings each query row into f16's range by a power of
two, so a row is as exact there as anywhere. Tolerances as derived in
test_gpu_window (a bf16 query is exact in the product)."""
import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa
import workloads as W
from helpers import oracle_pools
from test_gpu_window import check, define, dev

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


@pytest.mark.parametrize("exps,kexp", [
    ([118] * 4, -118),                  # row maxima of 2^119 and more
    ([125] * 4, -125),                  # up to the type's largest values
    ([-120] * 4, 118),
    ([-132] * 4, 126),                  # rows of subnormal numbers alone
    ([124, 0, -60, -126], -124),        # beside each other: most rows' scores are near zero
])
def test_rows_at_the_ends_of_the_range(exps, kexp):
    H, hk, window, first = 8, 2, 500, 4
    wl = W._build("range", 12, H, hk, 128, 16, [1, 1, 1], [700, 90, 1200],
                  torch.Generator().manual_seed(12))
    codes = [(c.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)
             for c, s in zip(oracle_pools(wl), (1.0, 0.03))]
    codes[0].view(torch.uint8).view(-1, 128)[::7] = 0          # keys of zeros
    q = wl.q.clamp(-3.9, 3.9).double()
    for h in range(H):
        q[:, h] *= 2.0 ** exps[h % 4]
    wl.q = q.to(torch.bfloat16)
    assert torch.isfinite(wl.q).all() and (wl.q != 0).any(-1).all()
    ks = torch.full((hk,), 2.0 ** kexp)
    kd, vd = codes[0].double() * 2.0 ** kexp, codes[1].double() * torch.tensor(0.03).double()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pa.window_fwd(wl.q.to(DEV), *(c.view(torch.uint8).to(DEV) for c in codes), *dev(wl), 1,
                        wl.max_seqlen_k, wl.softmax_scale, window, first, k_scale=ks.to(DEV),
                        v_scale=torch.full((hk,), 0.03, device=DEV), dev_status=status)
    assert int(status) == 0
    check(got, define(wl, kd, vd, window, first))
