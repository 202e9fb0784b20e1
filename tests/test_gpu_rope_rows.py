"""Rotated queries written between the rows of the queries they come from."""
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


@pytest.mark.parametrize("T", [1, 2, 33])
def test_output_rows_by_turns_with_the_input(T):
    """One buffer [T, 4, H, D]: q in one of its columns, q_out in another (ahead
    of it or behind), the other two left as they were; the same bits as into a
    buffer of its own."""
    H, hk, D, bs, dtype = 6, 2, 128, 16, torch.bfloat16
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, 4, H, D), generator=g).to(dtype).to(DEV)
    kv = torch.randn((T, 2, hk, D), generator=g).to(dtype).to(DEV)
    pos = torch.arange(T, device=DEV) * 3
    table = pa.rope_table(128, D, device=DEV)
    kc, vc = torch.zeros((2, 3, bs, hk, D), dtype=dtype, device=DEV)
    tail = (kv[:, 0], kv[:, 1], pos, table, kc, vc, torch.arange(T, device=DEV))
    for a, b in ((0, 1), (3, 0), (1, 2), (2, 0)):
        buf = x.clone()
        want = pa.rope_and_cache(buf[:, a], *tail)
        pa.rope_and_cache(buf[:, a], *tail, out=buf[:, b])
        assert torch.equal(buf[:, b], want)
        rest = [i for i in range(4) if i != b]
        assert torch.equal(buf[:, rest], x[:, rest])
