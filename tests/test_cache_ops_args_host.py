"""Argument checks of the operators around attention that need no GPU: the
limits of a launch, integers past 32 bits, outputs beside their inputs."""
import pytest

import paged_kv_varlen_attn_gb300 as pa
from paged_kv_varlen_attn_gb300 import _build
from test_evict_host import call_weights


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


@pytest.mark.parametrize("S,mk,hk,ok", [
    (1 << 10, 128 * ((1 << 18) - 1), 8, True),      # 2^31 - 8192 blocks
    (1 << 10, 128 * ((1 << 18) - 1) + 1, 8, False),   # 2^31
    ((1 << 30) - 1, 128, 2, True),                  # 2^31 - 2
    ((1 << 30) - 1, 0, 2, True),
    (1 << 30, 1, 2, False),
    (1 << 30, 1 << 30, 2048, False),                # 2^64: a product that wraps to nothing
])
def test_weights_largest_grid(lib, S, mk, hk, ok):
    """One block per 128 keys of a sequence and KV head: a call is refused only
    past what a launch holds (no queries: an accepted call launches nothing)."""
    got = call_weights(lib, S=S, mk=mk, H=hk, hk=hk, D=64, qs=hk * 64, cbs=16 * hk * 64,
                       ws=16 * hk, T=0, mq=0)
    assert got == (pa.PA_OK if ok else pa.PA_ERR_INVALID_ARG)
