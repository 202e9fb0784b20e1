"""4-bit decode whose lengths change on the stream, shortly before the call reads them."""
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


def test_lengths_written_just_before():
    # Lengths change on the stream between calls that share a workspace, nothing waits.
    b = Pools([4000] * 40, [1] * 40, 8, 2, 128, 16, "bf16", 44)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = pa.alloc_workspace(pa.varlen_fwd_int4kv_workspace_size(40, 40, 1, 4000, 8, 2, 128, 16,
                                                                sms), DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    steps = torch.randint(0, 4001, (30, 40), device=DEV, generator=g, dtype=torch.int32)
    wants = []
    for n in steps:
        b.lens.copy_(n)
        torch.cuda.synchronize()
        wants.append(b.run(workspace=ws))
        torch.cuda.synchronize()
    got = []
    for n in steps:
        b.lens.copy_(n)
        got.append(b.run(workspace=ws))
    for x, y in zip(got, wants):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
