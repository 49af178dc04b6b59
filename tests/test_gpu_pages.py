"""Pages of any number of entries through the calls that take them: csa2_append_kv and csa2_decode_step (the others
refuse a page_size that is no power of two)."""
import pytest
import torch

from tests.helpers import K

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def two_caches(B, ratio, page, entries):
    """The same room as pages in a shuffled order and as one row a sequence, and the slot in each of entry n of b."""
    k = K()
    n = -(-entries // page)
    perm = torch.randperm(B * n + 2, generator=torch.Generator().manual_seed(page))[:B * n].view(B, n)
    paged = k.GlobalKVCache(B, ratio, num_slots=(B * n + 2) * page, page_table=perm.to(torch.int32).to(DEV), page_size=page)
    flat = k.GlobalKVCache(B, ratio, seq_stride=entries)
    for p in paged.planes + flat.planes:
        p.fill_(0xA5)
    e = torch.arange(entries)
    at = perm[:, e // page] * page + e % page
    return paged, flat, at.to(DEV)


@pytest.mark.parametrize("page", [1, 3, 48, 64, 100])
@pytest.mark.parametrize("ratio", [1, 2])
def test_append(page, ratio):
    k = K()
    B, T = 3, 130
    paged, flat, at = two_caches(B, ratio, page, T)
    stages = [torch.zeros((B, ratio, 640), device=DEV) if ratio > 1 else None for _ in range(2)]
    kv, ix = make((T, B, 512), 1), make((T, B, 128), 2)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for t in range(T):
        pos = torch.full((B,), t, dtype=torch.int32, device=DEV)
        for c, s in zip((paged, flat), stages):
            k.csa2_append_kv(kv[t], ix[t], pos, c, stage=s, err=err)
    assert k.csa2_check(err) == 0 and torch.equal(paged.num_entries, flat.num_entries)
    for p, f in zip(paged.planes, flat.planes):
        assert torch.equal(p[at.flatten()], f)
        rest = torch.ones(len(p), dtype=torch.bool, device=DEV)
        rest[at.flatten()] = False
        assert (p[rest] == 0xA5).all()


@pytest.mark.parametrize("page", [48, 128])
def test_decode_step(page):
    """Full, Reuse and dense layers over one cache that grows from nothing: the selections and outputs of a paged cache and
    of one without pages are the same bits."""
    k = K()
    B, T, L, kk = 2, 150, 3, 16
    plan = [(k.MODE["full"], -1, 0), (k.MODE["reuse"], 0, 0), (k.MODE["dense"], -1, 0)]
    paged, flat, _ = two_caches(B, 1, page, T)
    kv, ix = make((T, 1, B, 512), 3), make((T, 1, B, 128), 4)
    got = []
    for c in (paged, flat):
        pos = torch.zeros(B, dtype=torch.int32, device=DEV)
        new_kv, new_ix = torch.empty_like(kv[0]), torch.empty_like(ix[0])
        codes, scale = torch.zeros((L, B, 128, 512), dtype=torch.uint8, device=DEV), torch.zeros((L, B, 128), device=DEV)
        idx = torch.full((L, B, kk), -1, dtype=torch.int32, device=DEV)
        o, lse = torch.zeros((L, B, 64, 512), device=DEV), torch.zeros((L, B, 64), device=DEV)
        step = k.DecodeStep(plan, [c], [T], pos, 512 ** -0.5, kk, 0, make((L, B, 64, 512), 5), make((L, B, 512), 6), codes, scale,
                            idx, o, lse, q_ix=make((L, B, 64, 128), 7), w=make((L, B, 64), 8), new_kv=new_kv, new_ix=new_ix)
        ws = torch.empty(max(step.workspace_size(), 1), dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        rows = []
        for t in range(T):
            pos.fill_(t)
            new_kv.copy_(kv[t])
            new_ix.copy_(ix[t])
            step.run(ws, err=err)
            if t % 29 == 0 or t == T - 1:
                rows += [idx[:2].clone(), o.clone(), lse.clone()]
        assert k.csa2_check(err) == 0
        got.append(rows)
    assert all(torch.equal(a, b) for a, b in zip(*got))
