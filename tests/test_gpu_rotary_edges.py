"""csa2_rotate and the rotating cache writes at sizes where their kernels take other paths: wide heads, blocks of several
trips, runs of several entries."""
import numpy as np
import pytest
import torch

from oracle import rotary as R
from tests.helpers import K, to_np
from tests.test_gpu_rotary import DEV, check_rotated, make, planes_of, rot_args, table

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


# ------------------------------------------------------------------ runs of several entries
def one_table(scale=1.125):
    """Rotations of the main and the indexer values by one table, as the runs need it."""
    step = table(64, scaling="yarn", factor=16.0, original_len=65536)[0].to(DEV)
    return K().Rotary(step, 448, "interleaved", scale), K().Rotary(step, 32, "half", scale)


def warps_at_once(dtype):
    return torch.cuda.get_device_properties(0).multi_processor_count * (24 if dtype == torch.bfloat16 else 20)


def room(B, ratio, entries, page, gap=None):
    """A cache of `entries` entries a sequence in shuffled pages, filled with 0xA5; page `gap` (b, p) is left out."""
    k = K()
    n = -(-entries // page)
    perm = torch.randperm(B * n, generator=torch.Generator().manual_seed(3)).view(B, n).to(torch.int32).to(DEV)
    if gap:
        perm[gap] = -1
    c = k.GlobalKVCache(B, ratio, num_slots=B * n * page, page_table=perm, page_size=page)
    for p in c.planes:
        p.fill_(0xA5)
    return c


@pytest.mark.parametrize("dtype,ratio,B,times,more,weights,main_only", [
    (torch.bfloat16, 1, 3, 1, 3, False, False), (torch.bfloat16, 2, 2, 3, 5, True, False), (torch.bfloat16, 1, 5, 17, 11, False, False),
    (torch.bfloat16, 1, 3, 64, 4, False, False), (torch.float32, 1, 2, 1, 5, True, False), (torch.float32, 2, 3, 4, 6, False, False),
    (torch.float32, 1, 4, 21, 9, False, False), (torch.bfloat16, 2, 2, 9, 7, False, True)])
def test_pack_in_runs(dtype, ratio, B, times, more, weights, main_only):
    """More entries than the device has warps at once, so that a warp takes a run of them: across the ends of sequences with
    unequal first entries, around a page outside the cache.  Every byte is that of the same tokens in chunks of a few
    hundred, where a warp takes one entry; and some of the oracle's."""
    k = K()
    fit = warps_at_once(dtype)
    n = -(-(times * fit + more) // B)
    assert n * B > times * fit
    T = n * ratio + (ratio > 1)  # (a token that completes no entry)
    kv, ix = make((B, T, 512), 41, dtype), make((B, T, 128), 42, dtype)
    w = torch.rand((B, T), device=DEV) if weights else None
    first = [(0, 1003, 17, 5)[b] if b < 4 else 31 for b in range(B)]
    page = 64
    rk, ri = one_table()
    if main_only:
        ri = None
    hats = lambda: (torch.full((B, n, 512), 9.0, dtype=torch.bfloat16, device=DEV), torch.full((B, n, 128), 9.0, dtype=torch.bfloat16, device=DEV))  # noqa: E731
    a, b_ = (room(B, ratio, max(first) + n, page, (1, (first[1] + n // 2) // page)) for _ in range(2))
    (kh, ih), (kh2, ih2), err = hats(), hats(), torch.zeros(2, dtype=torch.int32, device=DEV)
    fe = torch.tensor(first, dtype=torch.int32, device=DEV)
    k.csa2_pack_kv_rotary(kv, ix, fe, a, rk, ri, pool_w=w, kv_hat=kh, ix_hat=ih, err=err[:1])
    assert k.csa2_check(err[:1]) == 5
    gone = [j for j in range(n) if (first[1] + j) // page == (first[1] + n // 2) // page]
    assert (kh[1, gone] == 9).all() and (ih[1, gone] == 9).all() and len(gone) == page
    chunk = 331
    for b in range(B):
        view = b_.seq_view(b)
        for j in range(0, n, chunk):
            m = min(chunk, n - j)
            s = slice(j * ratio, (j + m) * ratio)
            hk, hi = kh2[b, j:j + m][None], ih2[b, j:j + m][None]
            k.csa2_pack_kv_rotary(kv[b:b + 1, s].contiguous(), ix[b:b + 1, s].contiguous(), fe[b:b + 1] + j, view, rk, ri,
                                  pool_w=None if w is None else w[b:b + 1, s].contiguous(), kv_hat=hk, ix_hat=hi, err=err[1:])
    assert torch.equal(kh, kh2) and torch.equal(ih, ih2)
    for x, y in zip(a.planes, b_.planes):
        assert torch.equal(x, y)
    rng = np.random.default_rng(5)
    for b in range(B):
        for j in [0, n - 37] + list(rng.integers(0, n - 37, 2)):
            j = int(j)
            if b == 1 and set(range(j, j + 37)) & set(gone):
                continue
            s = slice(j * ratio, (j + 37) * ratio)
            want = R.pack_entries(to_np(kv[b, s]), to_np(ix[b, s]), first[b] + j, ratio, rot_args(rk), rot_args(ri), None if w is None else to_np(w[b, s]))
            for x, y in zip(planes_of(a, b, first[b] + j + np.arange(37))[0], want):
                np.testing.assert_array_equal(x, y.reshape(x.shape))


@pytest.mark.parametrize("dtype,ratio", [(torch.bfloat16, 1), (torch.bfloat16, 2), (torch.float32, 1)])
def test_append_is_the_pack_in_runs(dtype, ratio):
    """The same tokens appended one at a time and packed at once in runs of several entries: the same bytes."""
    k = K()
    B, n, first = 8, 1100, 5
    assert B * n > 2 * warps_at_once(dtype)
    kv, ix = make((B, n * ratio, 512), 51, dtype), make((B, n * ratio, 128), 52, dtype)
    rk, ri = one_table()
    a, b = room(B, ratio, first + n, 16), room(B, ratio, first + n, 16)
    fe = torch.full((B,), first, dtype=torch.int32, device=DEV)
    k.csa2_pack_kv_rotary(kv, ix, fe, a, rk, ri)
    stage = torch.zeros((B, ratio, 640), device=DEV) if ratio > 1 else None
    for t in range(n * ratio):
        k.csa2_append_kv_rotary(kv[:, t].contiguous(), ix[:, t].contiguous(), fe * ratio + t, b, rk, ri, stage=stage)
    assert (b.num_entries == first + n).all()
    for x, y in zip(a.planes, b.planes):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ the gradient
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("xd,od", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_gradient_through_autograd(layout, xd, od):
    """x from a wider tensor, in a scaled rotation; rows of padding tokens have no gradient."""
    k = K()
    T, H, D = 9, 3, 48
    rotary = k.Rotary(table(16)[0].to(DEV), 8, layout, 1.5)
    pos = torch.randint(0, 1 << 20, (T,), device=DEV, dtype=torch.int32)
    pos[4] = -1
    keep = pos >= 0
    for inverse in (False, True):
        wide = make((T, H * D + 8), 61, xd).requires_grad_()
        y = k.csa2_rotate(wide[:, 8:].view(T, H, D), pos, rotary, inverse=inverse, out_dtype=od)
        assert y.requires_grad and y.dtype == od
        check_rotated(y.detach()[keep], wide.detach()[:, 8:].view(T, H, D)[keep], pos[keep], rotary, inverse)
        dy = make((T, H, D), 62, od)
        y.backward(dy)
        got = wide.grad[:, 8:].view(T, H, D)
        assert wide.grad.dtype == xd and (wide.grad[:, :8] == 0).all() and (got[4] == 0).all()
        check_rotated(got[keep], dy[keep], pos[keep], rotary, not inverse)
    x = make((T, H, D), 63, xd).requires_grad_()
    k.csa2_rotate(x, pos, rotary, out_dtype=od)[keep].sum().backward()  # a gradient without memory of its own
    check_rotated(x.grad[keep], torch.ones((T, H, D), dtype=od, device=DEV)[keep], pos[keep], rotary, True)
    # a difference quotient of the (linear) operator is its derivative up to rounding
    if xd == od == torch.float32:
        dy = make((T, H, D), 64)
        x.grad = None
        k.csa2_rotate(x, pos, rotary).backward(dy)
        for h, d in ((0, 8), (1, 15), (2, 23), (0, 3)):
            e = torch.zeros_like(x)
            e[:, h, d] = 0.5
            with torch.no_grad():
                df = k.csa2_rotate(x + e, pos, rotary).double() - k.csa2_rotate(x - e, pos, rotary).double()
            np.testing.assert_allclose(to_np((df * dy.double())[keep].sum((-1, -2))), to_np(x.grad[keep][:, h, d]), atol=H * D * 2.0 ** -20 * 16)


def test_where_no_gradient_is_asked_for():
    """Without grad mode, into a given tensor and with a table or positions changed since: no graph, or an error."""
    k = K()
    rotary = k.Rotary(table(16)[0].to(DEV), 0, "half", 1.0)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    x = make((4, 2, 16), 65).requires_grad_()
    with torch.no_grad():
        assert not k.csa2_rotate(x, pos, rotary).requires_grad
    assert not k.csa2_rotate(x, pos, rotary, out=torch.zeros((4, 2, 16), device=DEV)).requires_grad
    for changed in (pos, rotary.step):
        y = k.csa2_rotate(x, pos, rotary)
        changed.add_(1)
        with pytest.raises(RuntimeError, match="modified"):
            y.sum().backward()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_a_scaled_rotation_is_taken_back_by_the_reciprocal_scale(layout):
    """The inverse keeps the scale, which makes it the gradient: after a rotation scaled by g it gives g^2 times the turned
    dims.  The rotation by the same table and 1 / g takes it back: twice the tolerance of a rotation, and the rounding of
    1 / g (below a third of it)."""
    k = K()
    g = 0.1 * np.log(16) + 1
    a = k.Rotary(table(64)[0].to(DEV), 448, layout, g)
    back = k.Rotary(a.step, 448, layout, 1 / a.scale)
    x, pos = make((50, 64, 512), 66), torch.randint(0, 1 << 20, (50,), device=DEV, dtype=torch.int32)
    y = k.csa2_rotate(x, pos, a)
    i, j = R.pair_dims(32, 448, layout)
    size = (x[..., i].abs() + x[..., j].abs()).repeat(1, 1, 2)
    at = np.concatenate((i, j))
    once = k.csa2_rotate(y, pos, back, inverse=True)
    assert ((once - x)[..., at].abs() <= size * 2.0 ** -19).all() and torch.equal(once[..., :448], x[..., :448])
    twice = k.csa2_rotate(y, pos, a, inverse=True)
    assert ((twice / g ** 2 - x)[..., at].abs() <= size * 2.0 ** -19).all()
    assert ((twice - x)[..., at].abs() > 0.5 * x[..., at].abs() - size * 2.0 ** -19).all()  # g^2 = 1.63
