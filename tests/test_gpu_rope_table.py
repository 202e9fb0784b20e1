"""The rotary table to the bound of the polynomials that it is computed with.

With u = 2^-24 (a float32 rounding is off by at most u of the value, and by u/2
of the power of two above a value below 1) and x in [-1, 1] the remainder in
eighths of a turn, sin(pi/4 x) = x S(x^2) and cos(pi/4 x) = C(x^2):
  * x is a rounded integer: u |x d/dx| of either function, at most 0.56 u; x^2
    is rounded once: 0.08 u of the sine, 0.28 u of the cosine;
  * the sine's last step and its product with x are rounded below 1, 0.5 u each,
    the steps before them add 0.07 u, the float32 coefficients 0.42 u (2.5e-8):
    2.2 u in all;
  * the cosine's last step is rounded below 1, 0.5 u, the one before it below
    1/2, 0.25 u, the others add 0.03 u, the coefficients 0.13 u (7.3e-9): 1.8 u;
  * mscale, unless 1, is rounded to float32 and multiplied once: 2 u more;
  * the phase is off by 1e-9 radian at most and its remainder, cut to 32 bits,
    by 4e-10."""
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


@pytest.mark.parametrize("n,rot,base,mscale", [
    (1, 2, 10000.0, 1.0), (3001, 128, 500000.0, 1.0), (4097, 256, 10000.0, 1.2079441541679836),
    (1000003, 16, 100.0, 1.0), (20011, 34, 1.0, 0.3),
])
def test_table_to_its_own_bound(n, rot, base, mscale):
    got = pa.rope_table(n, rot, base, mscale=mscale, device=DEV).cpu().double()
    pos = list(range(n)) if n <= 20011 else list(range(0, n, 499)) + [n - 1]
    want = ref.rope_table(pos, ref.rope_rates(rot, base), mscale)
    tol = mscale * ((2.2 if mscale == 1.0 else 4.2) * 2.0 ** -24 + 1.4e-9)
    assert (got[pos] - want).abs().max().item() <= tol
