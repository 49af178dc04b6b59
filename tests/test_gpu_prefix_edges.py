"""csa2_prefix_attn where its warps hand tiles to one another."""
import numpy as np
import pytest
import torch

from tests.helpers import ATOL_MAX, K, to_np
from tests.test_gpu_prefix import DEV, TAU, Batch, check, everything, make

pytestmark = pytest.mark.gpu


def test_tiles_change_hands_under_memory_traffic():
    """Tiles that the loader copies and tiles that the producers dequantise alternate within a block (short tails and a
    window behind 1 to 9 shared tiles, several rows a block) while other streams keep the memory system busy, so that each
    writer falls behind the other: no wait runs out, and every call gives the bits of an undisturbed one."""
    k = K()
    batches = [Batch(140, [11 * (b % 5) for b in range(70)], 1, 16, 128, 6, seed=41),
               Batch(1300, [7 * (b % 9) for b in range(45)], 2, 64, 128, 3, seed=42),
               Batch(400, [200 * (b % 2) for b in range(60)], 1, 16, 100, 4, seed=43)]
    for t in batches:
        assert t.B * t.Q * (t.S // 128) >= 400  # dequantised ahead
        o, lse = t.run()
        check(o, lse, tuple(to_np(x) for x in everything(t)), f"prefix {t.S}")
        ws = torch.empty(k.csa2_prefix_workspace_size(t.B, t.Q, t.most), dtype=torch.uint8, device=DEV)
        big = torch.empty(1 << 28, dtype=torch.float32, device=DEV)
        scattered = torch.randint(0, big.numel(), (1 << 22,), device=DEV)
        traffic = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        outs = []
        for _ in range(20):
            with torch.cuda.stream(traffic[0]):
                big[:1 << 27].copy_(big[1 << 27:])
            with torch.cuda.stream(traffic[1]):
                big[scattered]
            outs.append(t.run(ws=ws))
        torch.cuda.synchronize()
        assert k.csa2_check(t.err) == 0
        for o2, lse2 in outs:
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def rising(t, heads):
    """The given heads' logits rise along the keys by 8 bits a tile (the lag is 5), up to 4 tau |q|: a reference moves in
    all but a few of the tiles."""
    up = torch.nn.functional.normalize(torch.randn(512, generator=torch.Generator().manual_seed(5)), dim=0).to(DEV)
    n = t.S
    rise = torch.arange(n, device=DEV)[:, None] / n * 4.0
    t.prefix = t._pack(0, 0, make((n, 512), 6) * 0.05 + up * rise)
    top = 8 * 0.6931 * n / 128  # in natural units
    t.q[:, :, heads] = (up * (top / 4.0 / TAU)).to(torch.bfloat16)
    return top


@pytest.mark.parametrize("S,tails,window,Q", [(2000, [3, 200], 128, 1), (3000, [0, 9, 300, 1, 70], 100, 5)])
def test_references_move_in_every_tile(S, tails, window, Q):
    """Weights written twice in tile after tile, in one head and in all, beside heads whose references stay; the same bits
    every time.  A logit is a sum of 32 products of the tensor core, each sum off by 2^-23 of its size at most: 2^-18 of the
    largest logit, which a weight and lse are off by too, and an output by twice that times the largest value."""
    for heads in (slice(5, 6), slice(0, 64)):
        t = Batch(S, tails, 1, 16, window, Q, seed=44)
        off = rising(t, heads) * 2.0 ** -18
        wo, wl = (to_np(x) for x in everything(t))
        runs = [t.run() for _ in range(10)]
        assert K().csa2_check(t.err) == 0
        o, lse = (to_np(x).astype(np.float64) for x in runs[0])
        size = max(np.abs(t.prefix).max(), 4.0)
        assert np.abs(lse - wl).max() <= 1e-4 + off
        assert np.abs(o - wo).max() <= ATOL_MAX * size / 4 + 2 * off * size
        for o, lse in runs[1:]:
            assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])


@pytest.mark.parametrize("S,B,Q", [(50, 3, 1), (300, 3, 1), (2500, 3, 1), (12800, 4, 1), (140, 70, 6)])
def test_heads_that_are_not_finite_are_nan(S, B, Q):
    """A NaN or an infinity in a query head makes its output and its lse NaN, whether its row lies in one block or in
    several (an lse of -inf would say that it sees no key)."""
    t = Batch(S, [3] * B, 1, 16, 128, Q, seed=45)
    t.q[0, 0, 7, 100], t.q[1, 0, 0, 0], t.q[2, 0, 63, 511] = float("inf"), float("nan"), -float("inf")
    t.q[1, 0, 20] = float("nan")
    o, lse = t.run()
    assert K().csa2_check(t.err) == 0
    bad = torch.zeros((B, Q, 64), dtype=torch.bool, device=DEV)
    bad[0, 0, 7] = bad[1, 0, 0] = bad[1, 0, 20] = bad[2, 0, 63] = True
    assert torch.isnan(lse[bad]).all() and torch.isnan(o[bad]).all()
    assert torch.isfinite(lse[~bad]).all() and torch.isfinite(o[~bad]).all()


@pytest.mark.parametrize("S,B", [(30, 3), (150, 3), (12800, 4)])
def test_a_window_scale_that_is_nan_is_seen(S, B):
    """A window token whose scale is NaN makes every head of the queries that see it NaN, as csa2_sparse_attn does; the
    other sequences, and one whose ring holds it outside the window, are as before (of 33 entries position -18's slot is
    outside it for both)."""
    k = K()
    t = Batch(S, [3] * B, 1, 16, 100, 1, seed=46)
    wo, wl = (to_np(x) for x in everything(t))
    ring = t.ring
    t.scale[1, (int(t.q_pos[1, 0]) - 50) % ring] = float("nan")
    t.scale[2, (int(t.q_pos[2, 0]) - 100) % ring] = float("nan")  # one position too old
    o, lse = t.run()
    assert k.csa2_check(t.err) == 0
    inside = int(t.q_pos[1, 0]) >= 50
    assert inside == (S > 30)
    if inside:
        assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    for b in (0, 2) if inside else (0, 1, 2):
        check(o[b], lse[b], (wo[b], wl[b]), f"b={b}")
    od, _ = k.csa2_sparse_attn("reuse", t.q, t.q_pos, t.cache, TAU, t.most, idx_in=torch.zeros((B, 1, 1), dtype=torch.int32, device=DEV),
                                k=1, swa_codes=t.codes, swa_scale=t.scale, window=100)
    assert torch.isnan(od[1]).all() == inside and torch.isfinite(od[0]).all()


@pytest.mark.parametrize("S,tails,Q", [(140, [11 * (b % 5) for b in range(70)], 6), (300, [3000] + [1] * 39, 1)])
def test_workspace_of_the_prefix_alone(S, tails, Q):
    """A workspace of the prefix's own size, between guards that stay as they are."""
    k = K()
    t = Batch(S, tails, 1, 16, 128, Q, seed=47)
    n, guard = k.csa2_prefix_workspace_bytes(t.B, Q, t.most, S), 4096
    assert n <= k.csa2_prefix_workspace_size(t.B, Q, t.most)
    room = torch.full((n + 2 * guard,), 0xFF, dtype=torch.uint8, device=DEV)
    o, lse = t.run(ws=room[guard:guard + n])
    assert k.csa2_check(t.err) == 0 and (room[:guard] == 0xFF).all() and (room[guard + n:] == 0xFF).all()
    check(o, lse, tuple(to_np(x) for x in everything(t)), f"prefix {S}")
    with pytest.raises(RuntimeError, match="workspace"):
        t.run(ws=room[guard:guard + n - 1])


@pytest.mark.parametrize("B,Q", [(31, 1), (32, 1), (33, 1), (11, 3), (8, 4), (147, 1), (148, 1), (149, 1), (1, 33)])
@pytest.mark.parametrize("S,spread", [(0, 40), (600, 1), (300, 900), (2600, 2)])
def test_row_counts_where_the_plan_changes(B, Q, S, spread):
    """Rows that one warp plans and rows that the block does (32, 33), as many rows as blocks, one more; equal rows and
    rows of unequal length, one of them seeing nothing."""
    t = Batch(S, [(spread * ((7 * b) % 11)) // 10 for b in range(B)], 1, 16, 100 if S % 600 else 0, Q, seed=48)
    if B > 2:
        t.q_pos[B // 2] = -1
    o, lse = t.run()
    assert K().csa2_check(t.err) == 0
    check(o, lse, tuple(to_np(x) for x in everything(t)), f"{B} x {Q} rows over {S}")
