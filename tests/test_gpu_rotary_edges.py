"""csa2_rotate and the rotating cache writes at sizes where their kernels take other paths: wide heads, blocks of several
trips, runs of several entries."""
import numpy as np
import pytest
import torch

from tests.helpers import K, to_np
from tests.test_gpu_rotary import DEV, check_rotated, make, table

pytestmark = pytest.mark.gpu
BOTH = (torch.float32, torch.bfloat16)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("tokens,heads,dim,rot,first", [
    (1, 1, 4096, 64, 4032), (8, 3, 2304, 64, 0), (8, 1, 4096, 4096, 0), (1, 2, 8192, 8192, 0), (2, 1, 6152, 4112, 8),
    (3, 2, 2057, 6, 3)])
def test_rotate_wide_heads(tokens, heads, dim, rot, first, layout):
    k = K()
    rotary = k.Rotary(table(rot)[0].to(DEV), first, layout, 1.25)
    pos = torch.randint(0, 1 << 20, (tokens,), device=DEV, dtype=torch.int32)
    for xd in BOTH:
        x = make((tokens, heads, dim), 3, xd)
        for od in BOTH:
            check_rotated(k.csa2_rotate(x, pos, rotary, out_dtype=od), x, pos, rotary)
        y = x.clone()
        assert k.csa2_rotate(y, pos, rotary, inverse=True, out=y) is y
        check_rotated(y, x, pos, rotary, inverse=True)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotate_blocks_of_several_trips(layout):
    """Enough tokens that a block takes all heads of its token, more than it has in flight at once: the bits of the same
    tokens in calls of a few, which the oracle checks."""
    k = K()
    T, H, D = 2500, 64, 512
    rotary = k.Rotary(table(64)[0].to(DEV), 448, layout, 1.25)
    pos = torch.randint(0, 1 << 20, (T,), device=DEV, dtype=torch.int32)
    pos[7] = -1
    some = torch.tensor([0, 1, 6, 8, 1000, 2367, 2368, 2499], device=DEV)
    for xd in BOTH:
        x = make((T, H, D), 5, xd)
        for od in BOTH:
            out = torch.full((T, H, D), 7.0, device=DEV, dtype=od)
            k.csa2_rotate(x, pos, rotary, out=out)
            assert (out[7] == 7).all()
            few = k.csa2_rotate(x[some], pos[some].contiguous(), rotary, out_dtype=od)
            check_rotated(few, x[some], pos[some], rotary)
            assert torch.equal(out[some], few)
            for at in range(0, T, 625):  # every token, 625 at a time (blocks of fewer heads)
                part = slice(at, at + 625)
                small = torch.full((625, H, D), 7.0, device=DEV, dtype=od)
                k.csa2_rotate(x[part], pos[part], rotary, out=small)
                assert torch.equal(small, out[part])
        y = x.clone()
        k.csa2_rotate(y, pos, rotary, out=y)
        keep = pos >= 0
        assert torch.equal(y[keep], k.csa2_rotate(x, pos, rotary)[keep]) and torch.equal(y[7], x[7])
