"""4-bit pools whose rows hold what the cache writes do not write, and pools of no pages."""
import ctypes

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


def test_pool_of_no_pages():
    # num_blocks = 0: every page is outside the pool and reads as zeros, whatever lies at
    # the pool's address.
    b = Pools([16, 0, 40], [1, 1, 1], 4, 2, 128, 16, "bf16", 43)
    lib = pa.load_library()
    out = torch.full((3, 4, 128), 9.0, dtype=b.dtype, device=DEV)
    lse = torch.zeros((4, 3), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.zeros((3, 3), dtype=torch.int32, device=DEV)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = pa.alloc_workspace(pa.varlen_fwd_int4kv_workspace_size(3, 3, 1, 40, 4, 2, 128, 16, sms),
                            DEV)
    desc = pa.KvInt4(b.params[0].data_ptr(), b.params[1].data_ptr(), 2 * 16)
    code = lib.pa_varlen_fwd_int4kv(
        None, b.q.data_ptr(), 4 * 128, b.codes[0].data_ptr(), b.codes[1].data_ptr(), 16 * 2 * 64,
        b.cu.data_ptr(), b.lens.data_ptr(), table.data_ptr(), 3, 3, 3, 1, 40, 4, 2, 128, 16, 0,
        b.scale, 1, ctypes.byref(desc), None, out.data_ptr(), lse.data_ptr(), ws.data_ptr(),
        ws.numel(), pa.PA_BF16, status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == pa.PA_OK and status.item() == pa.PA_DEV_BAD_PAGE
    assert (out == 0).all()
    want = torch.tensor([16.0, 0.0, 40.0]).log().expand(4, 3)
    assert torch.equal(lse.cpu()[:, 1], want[:, 1])
    assert ((lse.cpu() - want).abs()[:, ::2] <= 2.0 ** -20 * 5).all()
