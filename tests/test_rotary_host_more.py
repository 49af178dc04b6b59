"""Host side of the rotary and shared-prefix entry points: choices that are made before a launch (no GPU: the calls that
would launch run in a process that sees no device)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def without_a_device(code, timeout=60):
    """Runs code in a process that sees no CUDA device, so that nothing it launches can run."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    return subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=timeout)


@pytest.fixture(scope="module")
def pkg():
    from compressed_sparse_attention_score_b200 import build
    build.build()
    import compressed_sparse_attention_score_b200 as k
    return k


ROTATE = """
import ctypes
lib = ctypes.CDLL("compressed_sparse_attention_score_b200/libcsa2.so")
class Rotary(ctypes.Structure):
    _fields_ = [("step", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("first", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("scale", ctypes.c_float)]
P, L, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
lib.csa2_rotate.argtypes = [P, I, L, L, P, I, L, L, I, I, I, P, ctypes.POINTER(Rotary), I, P]
a = 1 << 20  # never read: there is no device
for tokens, heads, dim, rot in %r:
    for layout in (0, 1):
        for out in (a, a + (1 << 30)):
            r = Rotary(a, rot, 0, layout, 1.0)
            s = lib.csa2_rotate(a, 1, heads * dim, dim, out, 1, heads * dim, dim, tokens, heads, dim, a, ctypes.byref(r), 0, None)
            assert s == 4, s  # the launch fails, CSA2_ERR_CUDA
print("done")
"""


def test_rotate_of_wide_heads_reaches_its_launch(pkg):
    """Heads of more than 256 units of eight values, with too few tokens to fill a GPU: the choice of heads per block
    ends."""
    sizes = [(1, 1, 4096, 64), (1, 8, 2304, 64), (8, 64, 4096, 64), (100, 1, 2112, 64), (1, 1, 8192, 8192), (3, 5, 4096, 4096),
             (1, 3, 2057, 6), (1, 1, 1 << 20, 2), (2000, 64, 512, 64)]
    r = without_a_device(ROTATE % (sizes,))
    assert r.stdout.strip() == "done", r.stdout + r.stderr


def test_workspace_goes_by_the_prefix(pkg):
    """A prefix of none or of a few entries does not ask for room for every entry that a sequence may have, more entries
    never ask for less, and the size without a prefix is enough for all of them."""
    size, fit = pkg.csa2_prefix_workspace_size, pkg.csa2_prefix_workspace_bytes
    assert fit(8, 1, 1 << 20, 0) == fit(8, 1, 1 << 20, 1000) < 64 << 20 < 1 << 30 < size(8, 1, 1 << 20)
    assert fit(8, 1, 1 << 20, 1 << 19) - fit(8, 1, 1 << 20, 0) == pytest.approx(512 << 20, rel=1e-3)
    for B, Q, most in ((1, 1, 64), (4, 1, 12800), (70, 6, 200), (32, 1, 8229), (3, 2, 1 << 20)):
        sizes = [fit(B, Q, most, p) for p in (0, 1, 127, 128, 4000, most // 2, most, 2 * most, 2 ** 31 - 1)]
        assert sizes[:4] == sorted(sizes[:4]) and max(sizes) == sizes[-1] == sizes[-3] == size(B, Q, most) and min(sizes) > 0
    assert fit(0, 1, 64, 4) == fit(1, -1, 64, 4) == fit(1, 1, -1, 4) == fit(1, 1, 64, -1) == 0


@pytest.mark.parametrize("astray", ["kv_codes", "kv_scales", "ix_codes", "ix_scales", "num_entries", "page_table"])
def test_every_tensor_of_a_cache_is_on_the_calls_device(pkg, astray):
    from compressed_sparse_attention_score_b200 import _lib

    class On:
        def __init__(self, device):
            self.get_device = lambda: device

    class Cache:
        kv_codes = kv_scales = ix_codes = ix_scales = num_entries = page_table = On(0)
        desc = staticmethod(_lib.csa2_cache)

    c = Cache()
    _lib._cache_on(c, 0)
    setattr(c, astray, On(1))
    with pytest.raises(ValueError, match="device"):
        _lib._cache_on(c, 0)
