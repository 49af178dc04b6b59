"""Rotary operators on the GPU against the float64 oracle: rotation of heads, and the cache writes that turn entries.

Tolerances of csa2_rotate: the turn rounded to fp32 is off by 2^-25 of a turn at most (2^-22.3 rad), sincospi by two
units in the last place (2^-23), the two products and their sum by 3 * 2^-24 of |a| + |b|: below 2^-21 of it; bf16
results by half a step more, 2^-8 of the value.  The cache writes turn in float64 and round once: bytes must be equal.
"""
import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import rotary as R
from tests.helpers import K, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def table(rot, **kw):
    step, scale = K().csa2_rotary_table(rot, **kw)
    return step, scale


def np_step(rotary):
    return to_np(rotary.step).astype(np.uint64)


def make(shape, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def check_rotated(got, x, pos, rotary, inverse=False):
    x64 = to_np(x).astype(np.float64)
    p = np.broadcast_to(to_np(pos)[..., None], x.shape[:-1])
    want = R.turn(x64, p, np_step(rotary), rotary.first, rotary.layout, np.float32(rotary.scale).astype(np.float64), inverse)
    n = rotary.step.numel()
    i, j = R.pair_dims(n, rotary.first, rotary.layout)
    tol = np.zeros_like(want)
    size = (np.abs(x64[..., i]) + np.abs(x64[..., j])) * abs(rotary.scale) * 2.0 ** -21
    tol[..., i], tol[..., j] = size, size
    if got.dtype == torch.bfloat16:
        tol += (np.abs(want) + tol) * 2.0 ** -8 + 1e-38
    d = np.abs(to_np(got).astype(np.float64) - want)
    assert (d <= tol).all(), f"off by up to {(d / np.maximum(tol, 1e-300)).max():.3g} times the tolerance"
    if got.dtype == x.dtype:  # dims that are not turned are copied bit for bit
        rest = np.setdiff1d(np.arange(x.shape[-1]), np.concatenate([i, j]))
        assert torch.equal(got[..., rest], x[..., rest])


SHAPES = [  # tokens, heads, dim, rot, first
    (1, 1, 2, 2, 0), (1, 64, 512, 64, 448), (5, 64, 512, 64, 448), (7, 3, 128, 128, 0), (33, 64, 128, 64, 64),
    (300, 1, 512, 512, 0), (9, 5, 48, 16, 8), (4, 2, 51, 6, 3), (3, 2, 30, 14, 16), (2, 7, 72, 34, 2), (1030, 2, 64, 32, 0)]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("tokens,heads,dim,rot,first", SHAPES)
def test_rotate_shapes(tokens, heads, dim, rot, first, layout):
    k = K()
    rotary = k.Rotary(table(rot)[0].to(DEV), first, layout, 1.25)
    pos = torch.randint(0, 1 << 20, (tokens,), device=DEV, dtype=torch.int32)
    for xd in (torch.float32, torch.bfloat16):
        x = make((tokens, heads, dim), 3, xd)
        for od in (torch.float32, torch.bfloat16):
            for inverse in (False, True):
                check_rotated(k.csa2_rotate(x, pos, rotary, inverse=inverse, out_dtype=od), x, pos, rotary, inverse)
        y = x.clone()
        assert k.csa2_rotate(y, pos, rotary, out=y) is y  # in place
        assert torch.equal(y, k.csa2_rotate(x, pos, rotary))


def test_rotate_far_positions_and_scalings():
    k = K()
    pos = torch.tensor([0, 1, 65535, 1 << 20, (1 << 24) + 1, (1 << 31) - 1], device=DEV, dtype=torch.int32)
    x = make((6, 4, 128), 5)
    for kw in (dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
               dict(scaling="yarn", factor=16.0, original_len=65536)):
        rotary = k.Rotary.table(64, first=64, layout="half", device=DEV, **kw)
        check_rotated(k.csa2_rotate(x, pos, rotary), x, pos, rotary)
    assert torch.equal(k.csa2_rotate(x, pos, k.Rotary.table(64, device=DEV))[0], x[0])  # position 0: no turn


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotate_strides_and_padding_rows(layout):
    """Heads inside a wider row, heads outermost, an expanded input, odd offsets; rows of padding tokens (negative
    positions) and everything between the heads of out stay as they were."""
    k = K()
    rotary = k.Rotary.table(32, first=16, layout=layout, device=DEV)
    T, H, D = 11, 6, 64
    pos = torch.arange(100, 100 + T, device=DEV, dtype=torch.int32)
    pos[[0, 4, 10]] = -1
    keep = pos >= 0
    for pad, off in ((0, 0), (8, 0), (13, 5), (8, 8)):
        rows = make((T, H * D + pad), 7, torch.bfloat16)
        x = rows[:, off:off + H * D].view(T, H, D) if off + H * D <= H * D + pad else rows[:, :H * D].view(T, H, D)
        for od in (torch.float32, torch.bfloat16):
            wide = torch.full((H, T, D + 3), 7.0, device=DEV, dtype=od)
            out = wide[:, :, 1:1 + D].transpose(0, 1)  # heads outermost, odd row starts
            k.csa2_rotate(x, pos, rotary, out=out)
            check_rotated(out[keep], x[keep], pos[keep], rotary)
            assert (out[~keep] == 7).all() and (wide[..., 0] == 7).all() and (wide[..., 1 + D:] == 7).all()
    x = make((1, 1, D), 8).expand(T, H, D)
    check_rotated(k.csa2_rotate(x, pos, rotary)[keep], x[keep], pos[keep], rotary)
    with pytest.raises(RuntimeError, match="SHAPE"):
        k.csa2_rotate(x, pos, rotary, out=torch.zeros(1, 1, D, device=DEV).expand(T, H, D))
    xb = make((3, 5, H, D), 9)
    pb = torch.arange(15, device=DEV, dtype=torch.int32).view(3, 5)
    check_rotated(k.csa2_rotate(xb, pb, rotary), xb, pb, rotary)
    with pytest.raises(ValueError):
        k.csa2_rotate(xb.transpose(0, 1), pb.t(), rotary)


def test_rotate_gradient():
    """The inverse with the same scale is the gradient: against the formula's transpose, and against differences (the
    operator is linear, so a difference quotient is the derivative up to rounding)."""
    k = K()
    for layout in ("interleaved", "half"):
        rotary = k.Rotary(table(16)[0].to(DEV), 4, layout, 1.5)
        pos = torch.tensor([3, 70000], device=DEV, dtype=torch.int32)
        x, dy = make((2, 3, 24), 1), make((2, 3, 24), 2)
        dx = k.csa2_rotate(dy, pos, rotary, inverse=True)
        lhs = (dy.double() * k.csa2_rotate(x, pos, rotary).double()).sum()
        assert abs(float(lhs - (dx.double() * x.double()).sum())) <= 2 * 144 * 2.0 ** -20 * 16
        for d in range(24):
            e = torch.zeros_like(x)
            e[..., d] = 0.5
            df = (k.csa2_rotate(x + e, pos, rotary).double() - k.csa2_rotate(x - e, pos, rotary).double())
            np.testing.assert_allclose(to_np((df * dy.double()).sum(-1)), to_np(dx[..., d]), atol=24 * 2.0 ** -20 * 16)


def test_rotate_nothing_and_not_finite():
    k = K()
    rotary = k.Rotary.table(16, device=DEV)
    for shape in ((0, 3, 16), (3, 0, 16)):
        assert k.csa2_rotate(torch.zeros(shape, device=DEV), torch.zeros(shape[0], dtype=torch.int32, device=DEV), rotary).shape == shape
    x = make((1, 2, 32), 1)
    x[0, 0, 3], x[0, 1, 20] = float("inf"), float("nan")
    y = k.csa2_rotate(x, torch.tensor([5], dtype=torch.int32, device=DEV), rotary)
    bad = ~torch.isfinite(y)
    assert bad[0, 0, 2:4].all() and bad[0, 1, 20] and bad.sum() == 3  # its own pair and no other value


# ------------------------------------------------------------------ cache writes
def planes_of(cache, b, n):
    """The four planes' rows of entries n of sequence b."""
    if cache.page_table is None:
        at = b * cache.seq_stride + n
    else:
        at = to_np(cache.page_table)[b][n // cache.page_size].astype(np.int64) * cache.page_size + n % cache.page_size
    return [to_np(p)[at] for p in cache.planes], at


def new_cache(B, ratio, entries, page=0):
    k = K()
    if not page:
        c = k.GlobalKVCache(B, ratio, seq_stride=entries)
    else:
        n = -(-entries // page)
        perm = torch.randperm(B * n + 3, generator=torch.Generator().manual_seed(1))[:B * n]
        c = k.GlobalKVCache(B, ratio, num_slots=(B * n + 3) * page, page_table=perm.view(B, n).to(torch.int32).to(DEV),
                            page_size=page)
    for p in c.planes:
        p.fill_(0xA5)
    return c


def rot_args(r):
    return None if r is None else (np_step(r), r.first, r.layout, np.float64(np.float32(r.scale)))


def rotations(kind):
    k = K()
    if kind == "tail64":
        step, scale = table(64, scaling="yarn", factor=16.0, original_len=65536)
        step = step.to(DEV)
        return k.Rotary(step, 448, "interleaved", scale), k.Rotary(step, 64, "interleaved", scale)
    if kind == "half":
        return k.Rotary.table(64, 448, "half", DEV), k.Rotary.table(64, 64, "half", DEV)
    if kind == "unequal":  # another number of dims, an odd first, another scale
        return k.Rotary.table(512, 0, "half", DEV), k.Rotary(table(30)[0].to(DEV), 5, "interleaved", -0.75)
    if kind == "shared_unequal":  # one table, two layouts
        step = table(128)[0].to(DEV)
        return k.Rotary(step, 3, "half", 1.0), k.Rotary(step, 0, "interleaved", 2.0)
    return (k.Rotary.table(64, 448, "interleaved", DEV), None) if kind == "main" else (None, k.Rotary.table(128, 0, "half", DEV))


PACKS = [  # ratio, page, B, T, first entry, dtype, rotations, pooling
    (1, 0, 1, 1, 0, torch.bfloat16, "tail64", "mean"), (1, 16, 3, 37, 5, torch.float32, "half", "mean"),
    (2, 0, 2, 75, 3, torch.bfloat16, "unequal", "mean"), (2, 64, 2, 130, 60, torch.float32, "tail64", "weights"),
    (3, 16, 2, 50, 0, torch.bfloat16, "shared_unequal", "mean"), (4, 0, 1, 41, 1000, torch.float32, "main", "gates"),
    (2, 0, 1, 64, 0, torch.bfloat16, "index", "gates"), (128, 0, 1, 300, 7, torch.bfloat16, "tail64", "mean"),
    (8, 0, 1, 7, 0, torch.bfloat16, "tail64", "mean")]


@pytest.mark.parametrize("ratio,page,B,T,first,dtype,kind,pooling", PACKS)
def test_pack_bytes(ratio, page, B, T, first, dtype, kind, pooling):
    k = K()
    n = T // ratio
    cache = new_cache(B, ratio, first + n + 2, page)
    rk, ri = rotations(kind)
    kv, ix = make((B, T, 512), 11, dtype), make((B, T, 128), 12, dtype)
    kv[0, 0, 32:48], kv[0, 0, 448:480] = 0, 0  # blocks of zeros
    fe = torch.full((B,), first, dtype=torch.int32, device=DEV)
    w = torch.rand((B, T), device=DEV) if pooling == "weights" else None
    g = (make((B, T, 512), 13), make((B, T, 128), 14)) if pooling == "gates" else None
    kh, ih = make((B, n, 512), 1, torch.bfloat16), make((B, n, 128), 1, torch.bfloat16)
    err = err_word()
    k.csa2_pack_kv_rotary(kv, ix, fe, cache, rk, ri, pool_w=w, gate_kv=g and g[0], gate_ix=g and g[1], kv_hat=kh, ix_hat=ih, err=err)
    assert k.csa2_check(err) == 0
    touched = np.zeros(cache.num_slots, bool)
    for b in range(B):
        want = R.pack_entries(to_np(kv[b]), to_np(ix[b]), first, ratio, rot_args(rk), rot_args(ri), None if w is None else to_np(w[b]),
                              g and (to_np(g[0][b]), to_np(g[1][b])))
        got, at = planes_of(cache, b, first + np.arange(n))
        touched[at] = True
        for name, x, y in zip(("kv codes", "kv scales", "ix codes", "ix scales"), got, want):
            np.testing.assert_array_equal(x, y.reshape(x.shape), err_msg=f"{name} b={b}")
        if n:
            np.testing.assert_array_equal(to_np(kh[b]).astype(np.float64), F.unpack_main(want[0], want[1]))
            np.testing.assert_array_equal(to_np(ih[b]).astype(np.float64), F.unpack_indexer(want[2], want[3]))
    for p in cache.planes:
        assert (to_np(p)[~touched] == 0xA5).all()  # nothing else is written


def scale_border_latents():
    """fp32 latents whose blocks' largest values are 6 times a border between two scales, or a neighbour of that, from
    subnormal ones to 2^125, and whose other values are at or next to borders between two codes of such a scale."""
    rng = np.random.default_rng(7)
    f = np.float32

    def neighbours(v):
        v = np.asarray(v, f)
        return np.concatenate([np.nextafter(v, f(0)), v, np.nextafter(v, f(np.inf))])

    with np.errstate(over="ignore"):
        step = np.unique(np.concatenate([np.arange(0, 16) * 2.0 ** -9, *(np.arange(8, 16) * 2.0 ** e for e in range(-9, 6))]))
    step = step[step <= 448]
    main = neighbours(6 * np.concatenate([step, (step[1:] + step[:-1]) / 2]))
    main = main[main > 0]
    index = neighbours(np.ldexp(f(6), np.arange(-150, 123)))
    index = index[index > 0]
    entries = max(-(-len(main) // 32), -(-len(index) // 4))
    kv, ix = np.zeros((entries, 512), f), np.zeros((entries, 128), f)
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], f)
    for x, tops, width in ((kv, main, 16), (ix, index, 32)):
        for n, top in enumerate(tops):
            e, at = divmod(n, x.shape[1] // width)
            scale = F.e4m3_decode(F.e4m3_encode(f(top) / f(6))) if width == 16 else np.ldexp(1.0, int(F.e8m0_ceil_exponent(np.array([f(top) / f(6)], f))[0]))
            v = neighbours((np.float64(scale) * border[rng.integers(0, 7, 16)]).astype(f))
            v = np.minimum(rng.permutation(v)[:width] * rng.choice([-1, 1], width), top).astype(f)
            v = np.where(np.abs(v) > top, top, v)
            v[rng.integers(0, width)] = top * rng.choice([-1, 1])
            x[e, width * at:width * (at + 1)] = v
    return kv, ix


def test_pack_at_the_borders_of_scales_and_codes():
    k = K()
    kv, ix = scale_border_latents()
    E = kv.shape[0]
    (mc, ms), (xc, xs) = F.pack_main(kv), F.pack_indexer(ix)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, b = torch.from_numpy(kv)[None].to(DEV), torch.from_numpy(ix)[None].to(DEV)
    turned = k.Rotary(torch.zeros(64, dtype=torch.int64, device=DEV))  # angles of 0: the values stay
    two = k.Rotary(torch.zeros(32, dtype=torch.int64, device=DEV))
    for kind in ("plain", "runs", "single", "append"):
        cache, err = new_cache(E if kind == "append" else 1, 1, 1 if kind == "append" else E), err_word()
        if kind == "plain":
            k.csa2_pack_kv(a, b, zero, cache, err=err)
        elif kind == "append":
            k.csa2_append_kv_rotary(a[0], b[0], torch.zeros(E, dtype=torch.int32, device=DEV), cache, turned, two, err=err)
        else:
            k.csa2_pack_kv_rotary(a, b, zero, cache, two if kind == "runs" else turned, two, err=err)
        assert k.csa2_check(err) == 0
        for plane, want in zip(cache.planes, (mc, ms, xc, xs)):
            assert (to_np(plane).reshape(E, -1) == np.asarray(want).reshape(E, -1)).all(), kind


def test_pack_without_rotations_is_the_plain_pack():
    k = K()
    kv, ix = make((2, 40, 512), 1, torch.bfloat16), make((2, 40, 128), 2, torch.bfloat16)
    fe = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    a, b = new_cache(2, 2, 30), new_cache(2, 2, 30)
    k.csa2_pack_kv(kv, ix, fe, a)
    k.csa2_pack_kv_rotary(kv, ix, fe, b, None, None)
    assert all(torch.equal(x, y) for x, y in zip(a.planes, b.planes))


def test_pack_reports_entries_outside_the_cache():
    k = K()
    rk, ri = rotations("tail64")
    kv, ix = make((1, 8, 512), 1), make((1, 8, 128), 2)
    cache, err = new_cache(1, 1, 5), err_word()
    kh = torch.full((1, 8, 512), 9.0, dtype=torch.bfloat16, device=DEV)
    k.csa2_pack_kv_rotary(kv, ix, torch.zeros(1, dtype=torch.int32, device=DEV), cache, rk, ri, kv_hat=kh, err=err)
    assert k.csa2_check(err) == 5
    assert (kh[0, 5:] == 9).all() and (kh[0, :5] != 9).any()
    want = R.pack_entries(to_np(kv[0, :5]), to_np(ix[0, :5]), 0, 1, rot_args(rk), rot_args(ri))
    for x, y in zip(planes_of(cache, 0, np.arange(5))[0], want):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("ratio,page,dtype", [(1, 16, torch.bfloat16), (2, 0, torch.float32), (3, 16, torch.bfloat16)])
def test_append_is_the_bulk_pack(ratio, page, dtype):
    """Tokens appended one at a time (sequences at different phases, one of them padding) give the bytes of the chunk
    packed at once; hats of completed entries are the codes' values, the other rows stay."""
    k = K()
    B, T = 4, 25
    rk, ri = rotations("tail64")
    kv, ix = make((B, T, 512), 21, dtype), make((B, T, 128), 22, dtype)
    cache = new_cache(B, ratio, 40, page)
    stage = torch.zeros((B, ratio, 640), device=DEV) if ratio > 1 else None
    first = torch.tensor([0, 4 * ratio, 7 * ratio, 0], device=DEV, dtype=torch.int32)
    err = err_word()
    for t in range(T):
        pos = first + t
        pos[3] = -1
        kh = torch.full((B, 512), 9.0, dtype=torch.bfloat16, device=DEV)
        ih = torch.full((B, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        k.csa2_append_kv_rotary(kv[:, t].contiguous(), ix[:, t].contiguous(), pos, cache, rk, ri, stage=stage, kv_hat=kh, ix_hat=ih, err=err)
        done = (to_np(pos) >= 0) & (to_np(pos) % ratio == ratio - 1)
        for b in range(B):
            if not done[b]:
                assert (kh[b] == 9).all() and (ih[b] == 9).all()
            else:
                rows, _ = planes_of(cache, b, np.array([int(pos[b]) // ratio]))
                np.testing.assert_array_equal(to_np(kh[b])[None], F.unpack_main(rows[0], rows[1]))
                np.testing.assert_array_equal(to_np(ih[b])[None], F.unpack_indexer(rows[2], rows[3]))
    assert k.csa2_check(err) == 0
    for b in range(3):
        e0, n = int(first[b]) // ratio, T // ratio
        assert int(cache.num_entries[b]) == e0 + n
        want = R.pack_entries(to_np(kv[b]), to_np(ix[b]), e0, ratio, rot_args(rk), rot_args(ri))
        for x, y in zip(planes_of(cache, b, e0 + np.arange(n))[0], want):
            np.testing.assert_array_equal(x, y)
    assert int(cache.num_entries[3]) == 0


@pytest.mark.parametrize("B,T,ring,dtype,rot,first,layout", [
    (1, 1, 128, torch.bfloat16, 64, 448, "interleaved"), (3, 200, 130, torch.float32, 64, 448, "half"),
    (2, 50, 256, torch.bfloat16, 512, 0, "half"), (2, 129, 128, torch.bfloat16, 6, 17, "interleaved")])
def test_window_bytes(B, T, ring, dtype, rot, first, layout):
    k = K()
    rotary = k.Rotary.table(rot, first, layout, DEV)
    x = make((B, T, 512), 31, dtype)
    x[0, 0] = 0
    start = torch.tensor([5, 1000000, 70001][:B], device=DEV, dtype=torch.int32)
    pos = start[:, None] + torch.arange(T, device=DEV, dtype=torch.int32)
    pos[B - 1, :T // 3] = -1  # leading padding of a ragged batch
    codes = torch.full((B, ring, 512), 0xA5, dtype=torch.uint8, device=DEV)
    scale = torch.full((B, ring), 3.0, device=DEV)
    k.csa2_pack_swa_rotary(x, pos, codes, scale, rotary, err=err_word())
    want_c, want_s = np.full((B, ring, 512), 0xA5, np.uint8), np.full((B, ring), 3.0, np.float32)
    for b in range(B):
        p = to_np(pos[b])
        c, s = F.pack_swa(R.turn_entries(to_np(x[b]), p, rot_args(rotary)))
        for t in range(max(0, T - ring), T):
            if p[t] >= 0:
                want_c[b, p[t] % ring], want_s[b, p[t] % ring] = c[t], s[t]
    np.testing.assert_array_equal(to_np(scale), want_s)
    np.testing.assert_array_equal(to_np(codes), want_c)


def test_captured_and_on_another_stream():
    """A decode step's rotation and append, captured on a side stream and replayed on new inputs and positions."""
    k = K()
    rk, ri = rotations("tail64")
    B = 5
    q, kv, ix = make((B, 64, 512), 1, torch.bfloat16), make((B, 512), 2, torch.bfloat16), make((B, 128), 3, torch.bfloat16)
    pos = torch.arange(B, device=DEV, dtype=torch.int32)
    cache, out = new_cache(B, 1, 64), torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            k.csa2_rotate(q, pos, rk, out=out)
            k.csa2_append_kv_rotary(kv, ix, pos, cache, rk, ri)
    for step in range(3):
        q.copy_(make(q.shape, 10 + step, q.dtype))
        kv.copy_(make(kv.shape, 20 + step, kv.dtype))
        pos += 7
        graph.replay()
        torch.cuda.synchronize()
        check_rotated(out, q, pos, rk)
        for b in range(B):
            e = int(pos[b])
            want = R.pack_entries(to_np(kv[b])[None], to_np(ix[b])[None], e, 1, rot_args(rk), rot_args(ri))
            for x, y in zip(planes_of(cache, b, np.array([e]))[0], want):
                np.testing.assert_array_equal(x, y)


def test_offsets_behind_four_gigabytes():
    """Tokens 2^31 values apart; entries, appended tokens and their groups in pages behind 2^32 bytes of the planes."""
    k = K()
    rk, ri = rotations("tail64")
    far = (1 << 31) + 64
    pos = torch.tensor([77, 900001], device=DEV, dtype=torch.int32)
    x = torch.empty(far + 3 * 512, dtype=torch.bfloat16, device=DEV).as_strided((2, 3, 512), (far, 512, 1))
    x.copy_(make((2, 3, 512), 1, torch.bfloat16))
    got = k.csa2_rotate(x, pos, rk)
    check_rotated(got, x.contiguous(), pos, rk)
    x.zero_()
    assert k.csa2_rotate(got, pos, rk, out=x) is x
    assert torch.equal(x.contiguous(), k.csa2_rotate(got, pos, rk))
    del x
    page, n = 256, (1 << 24) // 256 + 3
    cache = k.GlobalKVCache(2, 1, num_slots=(n + 4) * page, page_size=page,
                            page_table=torch.tensor([[n, n + 2], [n + 3, n + 1]], dtype=torch.int32, device=DEV))
    kv, ix = make((2, 300, 512), 2, torch.bfloat16), make((2, 300, 128), 3, torch.bfloat16)
    k.csa2_pack_kv_rotary(kv, ix, torch.zeros(2, dtype=torch.int32, device=DEV), cache, rk, ri, err=(err := err_word()))
    last = make((2, 512), 4, torch.bfloat16), make((2, 128), 5, torch.bfloat16)
    k.csa2_append_kv_rotary(*last, torch.full((2,), 300, dtype=torch.int32, device=DEV), cache, rk, ri, err=err)
    assert k.csa2_check(err) == 0 and cache.num_entries.tolist() == [301, 301]
    for b in range(2):
        rows = torch.cat((kv[b], last[0][b:b + 1])), torch.cat((ix[b], last[1][b:b + 1]))
        want = R.pack_entries(to_np(rows[0]), to_np(rows[1]), 0, 1, rot_args(rk), rot_args(ri))
        for got, w in zip(planes_of(cache, b, np.arange(301))[0], want):
            np.testing.assert_array_equal(got, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_results_on_a_stream_of_their_own(dtype):
    """A new output for a stream that is not the current one."""
    k = K()
    rk, _ = rotations("tail64")
    x, pos = make((500, 64, 512), 6, dtype), torch.arange(500, device=DEV, dtype=torch.int32)
    want = k.csa2_rotate(x, pos, rk)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = k.csa2_rotate(x, pos, rk, stream=side)
    torch.full_like(x, 3.0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
