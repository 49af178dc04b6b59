"""Rotary tables and the refusals of the rotary and shared-prefix entry points (no GPU: no call here reaches a
kernel), and pins of the rotary oracle."""
import ctypes
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from oracle import rotary as R

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.fixture(scope="module")
def pkg():
    from compressed_sparse_attention_score_b200 import build
    build.build()
    import compressed_sparse_attention_score_b200 as k
    return k


def frequencies(rot, base, scaling="none", factor=1, original=0, fast=32, slow=1):
    """The frequencies from their definition, in 60 digits."""
    b, s = Decimal(base), Decimal(factor)
    if scaling == "ntk":
        b = b * (s.ln() * rot / (rot - 2)).exp()
    f = [(-Decimal(2 * i) / rot * b.ln()).exp() for i in range(rot // 2)]
    if scaling == "linear":
        f = [v / s for v in f]
    if scaling == "yarn":
        def pair_of(turns):
            return Decimal(rot) * (Decimal(original) / (2 * PI * Decimal(turns))).ln() / (2 * Decimal(base).ln())
        lo = max(int(pair_of(fast).to_integral_value(rounding="ROUND_FLOOR")), 0)
        hi = min(int(pair_of(slow).to_integral_value(rounding="ROUND_CEILING")), rot - 1)
        ramp = [min(Decimal(1), max(Decimal(0), (Decimal(i) - lo) / (hi - lo))) for i in range(rot // 2)]
        f = [v / s * r + v * (1 - r) for v, r in zip(f, ramp)]
    return f


@pytest.mark.parametrize("rot,kw", [
    (64, {}), (2, {}), (128, {"base": 500000.0}), (64, {"scaling": "linear", "factor": 8.0}),
    (64, {"scaling": "ntk", "factor": 4.0}), (64, {"scaling": "yarn", "factor": 16.0, "original_len": 65536}),
    (96, {"scaling": "yarn", "factor": 40.0, "original_len": 4096, "base": 10000.0}),
    (64, {"scaling": "yarn", "factor": 1.0, "original_len": 4096})])
def test_table_against_the_formulas(pkg, rot, kw):
    step, scale = pkg.csa2_rotary_table(rot, **kw)
    want = frequencies(rot, kw.get("base", 10000.0), kw.get("scaling", "none"), kw.get("factor", 1.0),
                       kw.get("original_len", 0))
    # the extended-precision exponential is off by a few units of 2^-64 times its argument (below 14): 2^-58 relative
    for got, f in zip(step.numpy().astype(np.uint64).tolist(), want):
        exact = f / (2 * PI) * 2 ** 64
        assert abs(Decimal(int(got)) - exact) <= exact / 2 ** 58 + 1
    factor = kw.get("factor", 1.0)
    assert scale == pytest.approx(0.1 * np.log(factor) + 1 if kw.get("scaling") == "yarn" else 1.0, rel=1e-7)


@pytest.mark.parametrize("original_len,all_the_way", [(65536, False), (4096, True)])
def test_table_keeps_fast_pairs_and_slows_the_others(pkg, original_len, all_the_way):
    """The slowest pair turns 65536 / (2 pi 10^(4 * 31 / 32)) = 1.4 times over 65536 positions, more than beta_slow:
    only over 4096 positions is it divided by the whole factor."""
    plain, _ = pkg.csa2_rotary_table(64)
    yarn, _ = pkg.csa2_rotary_table(64, scaling="yarn", factor=16.0, original_len=original_len)
    ratio = plain.double() / yarn.double()
    assert ratio[0] == 1.0 and (abs(float(ratio[-1]) - 16.0) < 1e-9) == all_the_way and 1.0 < ratio[-1] < 16.0 + 1e-9
    assert bool((ratio[1:] >= ratio[:-1] - 1e-12).all())


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=-2), dict(base=1.0),
                                dict(base=float("nan")), dict(base=float("inf")), dict(factor=0.5),
                                dict(rot_dim=2, scaling="ntk", factor=2.0), dict(scaling="yarn", factor=2.0),
                                dict(scaling="yarn", factor=2.0, original_len=100, beta_fast=1.0, beta_slow=1.0),
                                dict(scaling="yarn", factor=2.0, original_len=100, beta_slow=0.0)])
def test_table_refusals(pkg, kw):
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        pkg.csa2_rotary_table(**{"rot_dim": 64, **kw})


def test_table_refuses_null_and_bad_scaling(pkg):
    lib = pkg.raw()
    buf = (ctypes.c_uint64 * 32)()
    assert lib.csa2_rotary_table(64, 1e4, 0, 1.0, 0, 0.0, 0.0, None, None) == 1
    assert lib.csa2_rotary_table(64, 1e4, 4, 1.0, 0, 0.0, 0.0, ctypes.addressof(buf), None) == 1
    assert lib.csa2_rotary_table(64, 1e4, 0, 1.0, 0, 0.0, 0.0, ctypes.addressof(buf), None) == 0


# ------------------------------------------------------------------ refusals through the C ABI
@pytest.fixture()
def memory():
    buf = ctypes.create_string_buffer(4096)
    memory.keep = buf
    return (ctypes.addressof(buf) + 255) & ~255


def rotary(pkg, addr, rot_dim=64, first=0, layout=0, scale=1.0):
    r = pkg.csa2_rotary()
    r.step, r.rot_dim, r.first, r.layout, r.scale = addr, rot_dim, first, layout, scale
    return r


BAD_ROTARY = [(dict(step=None), 1), (dict(step=4), 1), (dict(rot_dim=0), 1), (dict(rot_dim=63), 1), (dict(rot_dim=-64), 1),
              (dict(layout=2), 1), (dict(layout=-1), 1), (dict(first=-1), 2), (dict(first=449), 2),
              (dict(rot_dim=514), 2), (dict(first=2147483647), 2), (dict(scale=float("nan")), 1),
              (dict(scale=float("inf")), 1)]


@pytest.mark.parametrize("bad,status", BAD_ROTARY)
def test_bad_rotations_are_refused(pkg, memory, bad, status):
    r = rotary(pkg, memory)
    for name, v in bad.items():
        setattr(r, name, memory + v if name == "step" and v else v)
    lib, a, br = pkg.raw(), memory, ctypes.byref(r)
    assert lib.csa2_rotate(a, 1, 32768, 512, a + 512, 1, 32768, 512, 1, 1, 512, a, br, 0, None) == status
    assert lib.csa2_pack_swa_rotary(a, 1, 1, 1, a, br, a, a, 128, None, None) == status
    c = cache(pkg, a)
    assert lib.csa2_pack_kv_rotary(a, a, 1, None, None, None, 1, 1, a, br, None, ctypes.byref(c), None, None, None, None) == status
    assert lib.csa2_append_kv_rotary(a, a, 1, 1, a, None, br, None, ctypes.byref(c), None, None, None, None) == status


def cache(pkg, a, **kw):
    c = pkg.csa2_cache()
    c.kv_codes = c.kv_scales = c.ix_codes = c.ix_scales = c.num_entries = a
    c.batch, c.ratio, c.num_slots, c.seq_stride = 1, 1, 4, 4
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def test_rotate_refusals(pkg, memory):
    lib, a, r = pkg.raw(), memory, rotary(pkg, memory)

    def call(x=a, xd=1, xt=128, xh=64, o=a + 1024, od=1, ot=128, oh=64, tokens=2, heads=2, dim=64, pos=a, rot=r):
        return lib.csa2_rotate(x, xd, xt, xh, o, od, ot, oh, tokens, heads, dim, pos, rot and ctypes.byref(rot), 0, None)
    for kw, status in [(dict(tokens=-1), 1), (dict(heads=-1), 1), (dict(dim=0), 1), (dict(x=None), 1), (dict(o=None), 1),
                       (dict(pos=None), 1), (dict(rot=None), 1), (dict(xd=2), 1), (dict(od=-1), 1), (dict(x=a + 1), 1),
                       (dict(o=a + 1026, od=0), 1), (dict(xt=-128), 1), (dict(ot=64), 2), (dict(oh=32), 2),
                       (dict(ot=0), 2), (dict(o=a, od=0, ot=128), 1), (dict(o=a, ot=256), 1), (dict(dim=32), 2)]:
        assert call(**kw) == status, kw
    assert call(tokens=0, x=None) == 0 and call(heads=0, x=None) == 0  # no work


def test_pack_append_window_refusals(pkg, memory):
    lib, a, r = pkg.raw(), memory, rotary(pkg, memory)
    br, wide = ctypes.byref(r), ctypes.byref(rotary(pkg, memory, rot_dim=128, first=2))

    def pack(kv=a, ix=a, dt=1, w=None, gk=None, gi=None, B=1, T=1, fe=a, rk=br, ri=br, c=cache(pkg, a), kh=None, ih=None):
        return lib.csa2_pack_kv_rotary(kv, ix, dt, w, gk, gi, B, T, fe, rk, ri, c and ctypes.byref(c), kh, ih, None, None)
    for kw, status in [(dict(B=-1), 1), (dict(T=-1), 1), (dict(c=None), 1), (dict(kv=None), 1), (dict(ix=None), 1),
                       (dict(fe=None), 1), (dict(dt=2), 1), (dict(gk=a), 1), (dict(gi=a), 1), (dict(w=a, gk=a, gi=a), 1),
                       (dict(kv=a + 8), 1), (dict(ix=a + 4), 1), (dict(ix=a + 8, dt=0), 1), (dict(gk=a + 4, gi=a), 1),
                       (dict(ri=wide), 2), (dict(kh=a + 8), 1), (dict(ih=a + 4), 1), (dict(B=2), 2),
                       (dict(c=cache(pkg, a, ratio=0)), 1)]:
        assert pack(**kw) == status, kw
    assert pack(B=0, kv=None) == 0 and pack(T=0, kv=None) == 0

    def append(kv=a, ix=a, dt=1, B=1, pos=a, stage=None, rk=br, ri=br, c=cache(pkg, a), kh=None, ih=None):
        return lib.csa2_append_kv_rotary(kv, ix, dt, B, pos, stage, rk, ri, c and ctypes.byref(c), kh, ih, None, None)
    for kw, status in [(dict(B=-1), 1), (dict(c=None), 1), (dict(kv=None), 1), (dict(pos=None), 1), (dict(dt=7), 1),
                       (dict(c=cache(pkg, a, ratio=2)), 1), (dict(c=cache(pkg, a, ratio=2), stage=a + 4), 1),
                       (dict(kv=a + 2), 1), (dict(ri=wide), 2), (dict(kh=a + 8), 1), (dict(B=2), 2)]:
        assert append(**kw) == status, kw
    assert append(B=0, kv=None) == 0

    def window(x=a, dt=1, B=1, T=1, pos=a, rot=br, codes=a, scale=a, R_=128):
        return lib.csa2_pack_swa_rotary(x, dt, B, T, pos, rot, codes, scale, R_, None, None)
    for kw, status in [(dict(B=-1), 1), (dict(T=-1), 1), (dict(R_=0), 1), (dict(x=None), 1), (dict(pos=None), 1),
                       (dict(rot=None), 1), (dict(codes=None), 1), (dict(scale=None), 1), (dict(dt=3), 1),
                       (dict(x=a + 8), 1), (dict(codes=a + 8), 1)]:
        assert window(**kw) == status, kw
    assert window(T=0, x=None) == 0


def test_prefix_refusals(pkg, memory):
    lib, a = pkg.raw(), memory
    size = lib.csa2_prefix_workspace_size(1, 1, 64)
    assert size > 0 and lib.csa2_prefix_workspace_size(0, 1, 64) == 0 and lib.csa2_prefix_workspace_size(1, -1, 64) == 0

    def call(q=a, B=1, Q=1, pos=a, S=4, most=64, c=cache(pkg, a), codes=None, scale=None, ring=0, window=128, o=a, od=1,
             lse=a, ws=a, n=size):
        return lib.csa2_prefix_attn(q, B, Q, pos, 1.0, S, most, c and ctypes.byref(c), codes, scale, ring, window, o, od,
                                    lse, ws, n, None, None)
    for kw, status in [(dict(B=-1), 1), (dict(Q=-1), 1), (dict(S=-1), 1), (dict(most=-1), 1), (dict(c=None), 1),
                       (dict(q=None), 1), (dict(pos=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(od=2), 1),
                       (dict(q=a + 8), 1), (dict(o=a + 8), 1), (dict(codes=a, ring=128), 1),
                       (dict(codes=a, scale=a, ring=127), 1), (dict(codes=a, scale=a, ring=256, window=129), 1),
                       (dict(codes=a, scale=a, ring=128, window=0), 1), (dict(codes=a + 8, scale=a, ring=128), 1),
                       (dict(ws=None), 1), (dict(ws=a + 8), 1), (dict(n=size - 1), 1), (dict(B=2), 2),
                       (dict(c=cache(pkg, a, seq_stride=0)), 1)]:
        assert call(**kw) == status, kw
    assert call(B=0, q=None) == 0 and call(Q=0, q=None) == 0


def test_binding_refuses_cpu_tensors_and_bad_shapes(pkg):
    step = torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkg.Rotary(step)                       # a host table
    with pytest.raises(ValueError):
        pkg.Rotary(step.int())
    x, pos = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    holder = type("Table", (), {"step": step})()
    for args in [(x, pos, holder), (x, pos.long(), holder), (x, pos[:1], holder), (x[0, 0], pos, holder)]:
        with pytest.raises(ValueError):
            pkg.csa2_rotate(*args)
    q = torch.zeros(1, 1, 64, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        host = type("Cache", (), {"kv_codes": torch.zeros(4, 256, dtype=torch.uint8)})()
        pkg.csa2_prefix_attn(q, torch.zeros(1, 1, dtype=torch.int32), host, 1.0, 16, 4, ws=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        pkg.csa2_prefix_attn(q.float(), torch.zeros(1, 1, dtype=torch.int32), None, 1.0, 16, 4)


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_oracle_turns_by_position_differences(pkg, layout):
    step = pkg.csa2_rotary_table(16)[0].numpy().astype(np.uint64)
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 32))
    turn = lambda x, p: R.turn(x, np.asarray(p), step, 8, layout)  # noqa: E731
    a = turn(q, 1000003) @ turn(k, 1000000)
    assert a == pytest.approx(turn(q, 3) @ turn(k, 0), abs=1e-12)
    assert abs(a - turn(q, 4) @ turn(k, 0)) > 1e-3
    back = R.turn(turn(q, 12345), np.asarray(12345), step, 8, layout, inverse=True)
    np.testing.assert_allclose(back, q, atol=1e-14)
    np.testing.assert_array_equal(turn(q, 77)[:8], q[:8])
    np.testing.assert_array_equal(turn(q, 77)[24:], q[24:])


def test_oracle_against_complex_numbers(pkg):
    step = pkg.csa2_rotary_table(8)[0].numpy().astype(np.uint64)
    x = np.random.default_rng(2).standard_normal((5, 8))
    pos = np.array([0, 1, 7, 1000, 70000])
    z = (x[:, 0::2] + 1j * x[:, 1::2]) * np.exp(1j * pos[:, None] * 10000.0 ** (-np.arange(4) / 4))
    got = R.turn(x, pos, step, 0, "interleaved")
    np.testing.assert_allclose(got[:, 0::2] + 1j * got[:, 1::2], z, atol=1e-10)  # pos x frequency in fp64: 2^-53 70000
