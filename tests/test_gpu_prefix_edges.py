"""csa2_prefix_attn where its warps hand tiles to one another."""
import pytest
import torch

from tests.helpers import K, to_np
from tests.test_gpu_prefix import DEV, Batch, check, everything

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
