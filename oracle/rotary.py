"""Oracle of the rotary operators: plain numpy in float64.

The angle of pair i at position p is p * step[i] 2^64ths of a turn, modulo one turn; uint64
arithmetic wraps there by itself.
"""
import numpy as np

from . import csa2 as C
from . import formats as F


def angles(pos, step):
    """cos, sin [.., n] of positions pos [..] for steps [n] (uint64)."""
    p = np.asarray(pos, np.int64).astype(np.uint64)[..., None]
    with np.errstate(over="ignore"):
        turn = (p * np.asarray(step, np.uint64)).astype(np.int64).astype(np.float64) * 2.0 ** -64
    return np.cos(2 * np.pi * turn), np.sin(2 * np.pi * turn)


def pair_dims(n, first, layout):
    """Dims of the first and second element of the n pairs."""
    i = np.arange(n)
    return (first + 2 * i, first + 2 * i + 1) if layout == "interleaved" else (first + i, first + n + i)


def turn(x, pos, step, first, layout, scale=1.0, inverse=False):
    """x [.., d] float64 turned at positions pos [..]."""
    y = np.array(x, np.float64)
    c, s = angles(pos, step)
    s = -s if inverse else s
    i, j = pair_dims(len(step), first, layout)
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i] = (a * c - b * s) * scale
    y[..., j] = (a * s + b * c) * scale
    return y


def turn_entries(x, pos, rot):
    """fp32 values turned in float64 and rounded once to fp32; rot = (step, first, layout, scale) or None."""
    x = np.asarray(x, np.float32)
    return x if rot is None else turn(x, pos, *rot).astype(np.float32)


def pack_entries(lat_kv, lat_ix, first_entry, ratio, rot_kv, rot_ix, pool_w=None, gates=None):
    """Tokens [T, 512], [T, 128] of one sequence -> the four planes' rows of its new entries."""
    if gates is None:
        kv, ix = C.compress(lat_kv, ratio, pool_w), C.compress(lat_ix, ratio, pool_w)
    else:
        kv, ix = C.compress_gated(lat_kv, gates[0], ratio), C.compress_gated(lat_ix, gates[1], ratio)
    pos = (first_entry + np.arange(len(kv))) * ratio
    return F.pack_main(turn_entries(kv, pos, rot_kv)) + F.pack_indexer(turn_entries(ix, pos, rot_ix))


def prefix_attention(keys_prefix, keys_own, q, pos, ratio, tau, swa=None, window=128):
    """One query token: heads q [64, 512] at position pos over the prefix's entries, then its own, as far as it
    sees them, joined with its window (codes [R, 512], scale [R])."""
    keys = np.concatenate([keys_prefix, keys_own])[:max(0, (pos + 1) // ratio) if pos >= 0 else 0]
    o, lse = C.attend(q, keys, tau)
    if swa is not None:
        o, lse = C.merge(o, lse, *C.swa_attention(q, pos, swa[0], swa[1], window, tau))
    return o, lse
