"""Selections whose candidates exceed shared memory in the variants for long
sequences: clusters of blocks (few sequence and head pairs) and single blocks
(many). Kept rows and moves are compared with a stable sort of the weights."""
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


@pytest.mark.parametrize("kv,hk,levels", [
    ([260_001], 1, 0),                    # past 48k candidates per block of four
    ([260_001, 200_007, 90], 2, 7),       # the same with ties over the blocks
    ([53_000], 160, 0),                   # past 48k in one block
    ([53_000, 4_500], 80, 5),
])
def test_candidates_past_shared_memory(kv, hk, levels):
    D, bs, budget, first, recent = 64, 64, 1500, 5, 33
    g = torch.Generator().manual_seed(len(kv) + hk)
    need = [(k + bs - 1) // bs for k in kv]
    nb = sum(need)
    order = torch.randperm(nb, generator=g)
    bt = torch.full((len(kv), max(need)), 1 << 30, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = order[at:at + n].int()
        at += n
    w = torch.randn((nb, hk, bs), generator=g)
    if levels:
        w = (w * levels).round()
    lens = torch.tensor(kv, dtype=torch.int32)
    gd = torch.Generator(device=DEV).manual_seed(1)
    kc = torch.randint(-2 ** 15, 2 ** 15, (nb, bs, hk, D), generator=gd, dtype=torch.int16,
                       device=DEV).view(torch.bfloat16)
    vc = kc.view(torch.int16).flip(0).contiguous().view(torch.bfloat16)
    k0, v0, w0 = kc.clone(), vc.clone(), w.to(DEV)
    wd = w0.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept, nl = pa.evict(kc, vc, wd, lens.to(DEV), bt.to(DEV), max(kv), budget, first, recent,
                        dev_status=status)
    assert int(status) == 0 and nl.tolist() == [min(k, budget) for k in kv]
    k1, v1, w1 = k0.clone(), v0.clone(), w0.clone()
    for s, k in enumerate(kv):
        if k <= budget:
            assert (kept[s, :, :k].cpu() == torch.arange(k)).all() and (kept[s, :, k:] == -1).all()
            continue
        pages = bt[s].long()[:need[s]]
        seq = w[pages].permute(1, 0, 2).reshape(hk, -1)[:, :k]             # [head, key]
        rank = seq[:, first:k - recent].sort(dim=1, descending=True, stable=True)[1]
        some = rank[:, :budget - first - recent].sort(dim=1)[0] + first
        ends = [torch.arange(a, b).expand(hk, -1) for a, b in ((0, first), (k - recent, k))]
        want = torch.cat([ends[0], some, ends[1]], 1)
        assert torch.equal(kept[s].cpu().long(), want)
        src, dst = want.to(DEV), torch.arange(budget, device=DEV).expand(hk, -1)
        head = torch.arange(hk, device=DEV)[:, None]
        pd = pages.to(DEV)
        sp, sr, dp, dr = pd[src // bs], src % bs, pd[dst // bs], dst % bs
        k1[dp, dr, head], v1[dp, dr, head] = k0[sp, sr, head], v0[sp, sr, head]
        w1[dp, head, dr] = w0[sp, head, sr]
    assert torch.equal(kc.view(torch.int16), k1.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), v1.view(torch.int16))
    assert torch.equal(wd, w1)
