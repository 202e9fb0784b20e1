"""4-bit decode of batches whose ranges of slices hold several sequences, for every
arrangement of KV heads and key runs in a block.

The pools are random codes with random scales and minima; the definition is
evaluated in float64 on the device, all sequences of a batch. Tolerances as in
test_gpu_int4.py.
"""
import pytest
import torch

import paged_kv_varlen_attn_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_varlen_attn_gb300 import _build
    _build.build()
    pa.load_library()


class Pools:
    """Sequences of the lengths kv, ql tokens each (0: none), over permuted pages; rows
    of a page past its sequence have NaN scales."""

    def __init__(self, kv, ql, H, hk, D, bs, dt, seed):
        g = torch.Generator().manual_seed(seed)
        d = torch.Generator(device=DEV).manual_seed(seed)
        self.kv, self.H, self.hk, self.D, self.bs = kv, H, hk, D, bs
        need = [-(-n // bs) for n in kv]
        nb = sum(need) + 3
        order = torch.randperm(nb, generator=g).int()
        self.table = torch.full((len(kv), max(need) + 1), 2 ** 30, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.table = self.table.to(DEV)
        self.codes = [torch.randint(0, 256, (nb, bs, hk, D // 2), dtype=torch.uint8, device=DEV,
                                    generator=d) for _ in range(2)]
        self.params = []
        for _ in range(2):
            scale = 0.3 * torch.exp(0.5 * torch.randn((nb, hk, bs), device=DEV, generator=d))
            low = -7.5 * scale + 0.3 * torch.randn((nb, hk, bs), device=DEV, generator=d)
            self.params.append(torch.stack([scale, low], -1).half())
        used = torch.zeros((nb, bs), dtype=torch.bool, device=DEV)
        for s, n in enumerate(kv):
            j = torch.arange(n, device=DEV)
            used[self.table[s].long()[j // bs], j % bs] = True
        for p in self.params:
            p.masked_fill_(~used[:, None, :, None], float("nan"))
        self.q_lens = list(ql)
        self.T = sum(ql)
        self.dtype = TYPES[dt]
        self.q = torch.randn((self.T, H, D), device=DEV, generator=d).to(self.dtype)
        self.cu = torch.tensor([0] + self.q_lens).cumsum(0).int().to(DEV)
        self.lens = torch.tensor(kv, dtype=torch.int32, device=DEV)
        self.scale = D ** -0.5

    def run(self, **kw):
        return pa.varlen_fwd_int4kv(self.q, *self.codes, *self.params, self.cu, self.lens,
                                    self.table, max(self.q_lens), max(self.kv), self.scale, True,
                                    **kw)

    def rows(self, x, s):
        """float64 [kv heads, keys, D] of sequence s, of K (x = 0) or V."""
        n = self.kv[s]
        j = torch.arange(n, device=DEV)
        page, row = self.table[s].long()[j // self.bs], j % self.bs
        words = self.codes[x][page, row].contiguous().view(torch.int32)
        shifts = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=DEV)
        codes = ((words.long()[..., None] >> shifts) & 15).flatten(-2).double()
        p = self.params[x].double()[page, :, row]
        return (codes * p[..., :1] + p[..., 1:]).transpose(0, 1)

    def check(self, out, lse):
        half = torch.finfo(self.dtype).eps / 2
        G, hk = self.H // self.hk, self.hk
        first = 0
        wrong = []
        for s, (n, ql) in enumerate(zip(self.kv, self.q_lens)):
            rows = slice(first, first + ql)
            first += ql
            if ql == 0:
                continue
            got = out[rows].double().view(ql, hk, G, self.D).permute(1, 2, 0, 3)
            got_lse = lse[:, rows].double().view(hk, G, ql)
            if n == 0:
                if (got != 0).any() or (got_lse != -float("inf")).any():
                    wrong.append(s)
                continue
            q = self.q[rows].double().view(ql, hk, G, self.D).permute(1, 2, 0, 3)
            key, value = self.rows(0, s), self.rows(1, s)
            score = torch.einsum("hgqd,hkd->hgqk", q, key) * self.scale
            pos = n - ql + torch.arange(ql, device=DEV)
            seen = torch.arange(n, device=DEV) <= pos[:, None]
            score.masked_fill_(~seen, -float("inf"))
            want_lse = torch.logsumexp(score, -1)
            blind = want_lse == -float("inf")
            weight = torch.exp(score - want_lse.masked_fill(blind, 0.0)[..., None])
            want = torch.einsum("hgqk,hkd->hgqd", weight, value)
            big_k, big_v = key.abs().amax((1, 2)), value.abs().amax((1, 2))
            err = self.scale * q.abs().sum(-1) * big_k[:, None, None] * 3 * 2.0 ** -18
            lse_ok = (got_lse - want_lse).abs() <= err + 2.0 ** -20 * (1 + want_lse.abs())
            lse_ok |= blind & (got_lse == want_lse)
            tol = half * want.abs() + (big_v[:, None, None] *
                                       (2 * (err + 2.0 ** -20) + 3 * 2.0 ** -11))[..., None]
            if not (lse_ok.all() and ((got - want).abs() <= tol).all()):
                wrong.append(s)
        assert not wrong, f"{len(wrong)} of {len(self.kv)}: {wrong[:20]}"


def lengths(kind):
    g = torch.Generator().manual_seed(7)
    if kind == "long-then-short":
        return [8192] * 32 + [20] * 8
    if kind == "mixed":
        return torch.randint(16, 4097, (200,), generator=g).tolist()
    if kind == "empty-between":
        return [30000, 0] * 16
    if kind == "one-long":
        return [33, 5, 64, 200000, 1, 90, 31]
    return [int(n) for n in torch.randint(0, 65, (2000,), generator=g)]     # "tiny"


KINDS = ["long-then-short", "mixed", "empty-between", "one-long", "tiny"]


# One, two and four runs of keys in a block, in one and several groups of heads; 8 rows
# and up to 32.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hk,D,dt,G,tokens", [
    (1, 128, "bf16", 8, 1), (1, 64, "f16", 2, 3), (2, 128, "f16", 4, 1), (2, 64, "bf16", 8, 3),
    (2, 128, "bf16", 8, 3), (5, 128, "bf16", 2, 1), (5, 64, "f16", 10, 3), (7, 64, "bf16", 1, 1),
    (7, 128, "f16", 5, 3), (10, 128, "f16", 4, 1), (10, 64, "bf16", 3, 3), (4, 128, "bf16", 2, 1),
])
def test_ranges_of_several_sequences(kind, hk, D, dt, G, tokens):
    kv = lengths(kind)
    b = Pools(kv, [tokens] * len(kv), G * hk, hk, D, 16 if hk % 2 else 64, dt, hk + D)
    out, lse = b.run()
    b.check(out, lse)
    again, lse2 = b.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_padded_batch_in_a_graph():
    # Captured once for 48 sequences; replayed as sequences end and their places are empty.
    b = Pools([9000] * 48, [1] * 48, 16, 2, 128, 16, "bf16", 3)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = pa.alloc_workspace(pa.varlen_fwd_int4kv_workspace_size(48, 48, 1, 9000, 16, 2, 128, 16,
                                                                sms), DEV)
    out, lse = b.run(workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(workspace=ws, out=out, lse=lse)
    for step in range(3):
        b.kv = [0 if s % 3 < step else 9000 - 100 * s for s in range(48)]
        b.lens.copy_(torch.tensor(b.kv, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        b.check(out, lse)
