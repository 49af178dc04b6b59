"""csa2_prefix_attn against the float64 oracle, and a decode step that uses the rotary operators with it.

Tolerances: keys are exact in fp16 and so is the prescaled query; the weights are rounded to fp16 (2^-11 relative,
2^-29 of the row's largest absolute), so an output is off by at most 2^-11 of the largest |value| (about 4 here):
ATOL_MAX, and much less on average; bf16 outputs by half a step, 2^-8 of the value, more.  lse is fp32 throughout.
"""
import numpy as np
import pytest
import torch

from oracle import csa2 as OC
from oracle import formats as F
from oracle import rotary as R
from tests.helpers import ATOL_MAX, ATOL_MEAN, K, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
TAU = 512 ** -0.5


def make(shape, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


class Batch:
    """B sequences on a shared prefix of S entries, with tails of their own, packed through the library."""

    def __init__(self, S, tails, ratio=4, page=16, window=128, Q=1, seed=0, std=1.0, slack=0):
        k = K()
        self.B, self.Q, self.S, self.ratio, self.tails = len(tails), Q, S, ratio, tails
        self.most = S + max(tails) + slack
        B = self.B
        whole = S // page if page else 0
        if page:
            n = max(-(-self.most // page), 1)
            t = torch.zeros((B, n), dtype=torch.long)
            t[:, :whole] = torch.arange(whole)
            t[:, whole:] = whole + torch.arange(B * (n - whole)).view(B, n - whole)
            used = whole + B * (n - whole)
            perm = torch.randperm(used, generator=torch.Generator().manual_seed(seed))
            self.table = perm[t].to(torch.int32).to(DEV)
            self.cache = k.GlobalKVCache(B, ratio, num_slots=used * page, page_table=self.table, page_size=page)
        else:
            self.cache = k.GlobalKVCache(B, ratio, seq_stride=max(self.most, 1))
        self.values = [None] * B
        view = self.cache
        pre = make((1, S, 512), seed + 1) * std
        self.prefix = self._pack(0, 0, pre[0]) if S else np.zeros((0, 512))
        for b, n in enumerate(tails):
            own = make((1, n, 512), seed + 10 + b) * std
            self.values[b] = self._pack(b, S, own[0]) if n else np.zeros((0, 512))
            view.num_entries[b] = S + n
        last = [(S + n) * ratio + (b % ratio) - 1 for b, n in enumerate(tails)]
        self.q_pos = torch.tensor([[p - (Q - 1) + i for i in range(Q)] for p in last], dtype=torch.int32, device=DEV)
        self.q = make((B, Q, 64, 512), seed + 3, torch.bfloat16)
        self.codes = self.scale = None
        self.window = window
        if window:
            self.ring = window + Q + 3
            x = make((B, self.ring, 512), seed + 4, torch.bfloat16) * std
            slots = self.q_pos[:, -1:] - self.ring + 1 + torch.arange(self.ring, device=DEV)
            self.codes = torch.zeros((B, self.ring, 512), dtype=torch.uint8, device=DEV)
            self.scale = torch.zeros((B, self.ring), device=DEV)
            k.csa2_pack_swa(x, slots.to(torch.int32), self.codes, self.scale)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def _pack(self, b, first, rows):
        """Entries of exactly these rows (ratio 1 view), and their values."""
        k, c = K(), self.cache
        view = k.GlobalKVCache(c.batch, 1, num_slots=c.num_slots, page_table=c.page_table, page_size=c.page_size,
                               planes=c.planes, num_entries=c.num_entries) if c.page_table is not None else \
            k.GlobalKVCache(c.batch, 1, seq_stride=c.seq_stride, planes=c.planes, num_entries=c.num_entries)
        view = view.seq_view(b)
        k.csa2_pack_kv(rows[None].contiguous(), torch.zeros((1, len(rows), 128), device=DEV),
                       torch.tensor([first], dtype=torch.int32, device=DEV), view)
        codes, scales = F.pack_main(to_np(rows))
        return F.unpack_main(codes, scales)

    def run(self, **kw):
        k = K()
        args = dict(swa_codes=self.codes, swa_scale=self.scale, window=self.window or 128, err=self.err)
        o, lse = k.csa2_prefix_attn(self.q, self.q_pos, self.cache, TAU, self.most, self.S, **{**args, **kw})
        return o, lse

    def want(self, b, i):
        swa = (to_np(self.codes[b]), to_np(self.scale[b])) if self.window else None
        return R.prefix_attention(self.prefix, self.values[b], to_np(self.q[b, i]).astype(np.float64),
                                  int(self.q_pos[b, i]), self.ratio, TAU, swa, self.window)


def check(o, lse, want, what):
    wo, wl = want
    go, gl = to_np(o).astype(np.float64), to_np(lse).astype(np.float64)
    np.testing.assert_array_equal(np.isneginf(gl), np.isneginf(wl), err_msg=what)
    big = max(1.0, np.abs(wo).max() / 4)
    d = np.abs(go - wo)
    half = np.abs(wo) * 2.0 ** -8 if o.dtype == torch.bfloat16 else 0.0
    assert (d <= ATOL_MAX * big + half).all(), f"{what}: o off by {d.max():.3g}"
    assert np.maximum(d - half, 0).mean() <= ATOL_MEAN * big, f"{what}: o off by {d.mean():.3g} on average"
    fin = np.isfinite(wl)
    assert (np.abs(gl[fin] - wl[fin]) <= 1e-4).all(), f"{what}: lse off by {np.abs(gl[fin] - wl[fin]).max():.3g}"


CASES = [  # S, tails, ratio, page, window, Q
    (0, [0], 1, 0, 0, 1),                       # nothing at all: o = 0, lse = -inf
    (0, [0, 3], 1, 0, 128, 1),                  # windows, one of them empty of entries
    (1, [0, 0, 1], 1, 16, 0, 1),                # one key
    (127, [1, 0], 4, 16, 1, 1), (128, [0, 5], 4, 16, 0, 1), (129, [3, 130], 4, 16, 100, 1),
    (96, [17, 2], 4, 64, 128, 1), (300, [40, 0, 77], 2, 256, 128, 3), (257, [9], 128, 16, 128, 1),
    (40, [3, 20], 1, 0, 128, 6), (1000, [1, 300, 44, 0, 513], 4, 64, 128, 2), (2500, [7] * 9, 4, 256, 128, 1),
    (6, [2], 1, 16, 5, 12),                     # more queries than tokens: the first ones stand before the sequence
]


@pytest.mark.parametrize("S,tails,ratio,page,window,Q", CASES)
def test_against_the_oracle(S, tails, ratio, page, window, Q):
    t = Batch(S, tails, ratio, page, window, Q)
    for od in (torch.float32, torch.bfloat16):
        o, lse = t.run(o_dtype=od)
        assert K().csa2_check(t.err) == 0
        for b in range(t.B):
            for i in range(Q):
                check(o[b, i], lse[b, i], t.want(b, i), f"{od} b={b} i={i}")


def test_long_prefix_over_many_blocks():
    t = Batch(20011, [5, 0, 260], 4, 256, 128, 1, seed=5)
    o, lse = t.run()
    assert K().csa2_check(t.err) == 0
    for b in range(t.B):
        check(o[b, 0], lse[b, 0], t.want(b, 0), f"b={b}")


def test_many_rows():
    """More query rows than the GPU has blocks; every one against the oracle's neighbours, some against the oracle."""
    t = Batch(140, [11 * (b % 5) for b in range(70)], 1, 16, 128, 4, seed=6)
    o, lse = t.run(o_dtype=torch.bfloat16)
    assert K().csa2_check(t.err) == 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    for b in range(0, 70, 9):
        for i in range(4):
            check(o[b, i], lse[b, i], t.want(b, i), f"b={b} i={i}")


def test_is_dense_attention_where_the_tables_share():
    """With prefix pages in every sequence's table, csa2_sparse_attn's dense mode computes the same."""
    k = K()
    t = Batch(512, [30, 0, 200], 4, 64, 128, 1, seed=7)  # the prefix ends with a page: the tables agree below it
    o, lse = t.run()
    od, ld = k.csa2_sparse_attn("dense", t.q, t.q_pos, t.cache, TAU, t.most, swa_codes=t.codes, swa_scale=t.scale, err=t.err)
    assert k.csa2_check(t.err) == 0
    assert float((o - od).abs().max()) <= 2 * ATOL_MAX and float((lse - ld).abs().max()) <= 1e-4
    o0, l0 = k.csa2_prefix_attn(t.q, t.q_pos, t.cache, TAU, t.most, 0, swa_codes=t.codes, swa_scale=t.scale)  # no sharing
    assert float((o0 - od).abs().max()) <= 2 * ATOL_MAX and float((l0 - ld).abs().max()) <= 1e-4


def test_entries_that_are_not_visible_do_not_count():
    """Slots behind a sequence's last entry, and prefix slots of the other sequences, hold bytes that would decode to
    NaN (an E4M3 scale of 0x7F): nothing of them reaches an output."""
    t = Batch(200, [9, 0, 40], 4, 0, 128, 2, seed=8, slack=100)
    live = np.zeros(t.cache.num_slots, bool)
    for b, n in enumerate(t.tails):
        at = b * t.cache.seq_stride
        live[at + (0 if b == 0 else t.S):at + t.S + n] = True
    dead = torch.from_numpy(~live).to(DEV)
    t.cache.kv_scales[dead] = 0x7F
    t.cache.kv_codes[dead] = 0xFF
    o, lse = t.run()
    assert K().csa2_check(t.err) == 0
    for b in range(3):
        for i in range(2):
            check(o[b, i], lse[b, i], t.want(b, i), f"b={b} i={i}")


def test_steep_and_large():
    """Logits far apart (one key takes nearly all the weight, wherever it stands), and values of a thousand."""
    for where in (0, 700, 1290, 1310):
        t = Batch(1300, [20, 3], 1, 256, 128, 1, seed=9)
        key = t.prefix[where] if where < t.S else t.values[0][where - t.S]
        t.q[0, 0, 5] = torch.from_numpy(key * 20).to(DEV).to(torch.bfloat16)
        o, lse = t.run()
        for b in range(2):
            check(o[b, 0], lse[b, 0], t.want(b, 0), f"where={where} b={b}")
    t = Batch(200, [20, 3], 1, 256, 128, 1, seed=9, std=400.0)
    t.q = (t.q / 400).contiguous()
    o, lse = t.run()
    for b in range(2):
        check(o[b, 0], lse[b, 0], t.want(b, 0), f"large b={b}")


def test_negative_positions_and_short_counts():
    """A padded query (negative position) attends nothing; a sequence whose num_entries is below the prefix sees only
    that many of its entries."""
    t = Batch(90, [10, 10, 10], 2, 16, 128, 1, seed=10)
    t.q_pos[1, 0] = -1
    t.cache.num_entries[2] = 33
    o, lse = t.run()
    assert K().csa2_check(t.err) == 0
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    check(o[0, 0], lse[0, 0], t.want(0, 0), "b=0")
    t.prefix, t.values[2] = t.prefix[:33], t.values[2][:0]
    check(o[2, 0], lse[2, 0], t.want(2, 0), "b=2")


def test_device_errors():
    k = K()
    t = Batch(100, [30, 30], 4, 16, 128, 1, seed=11)
    o, lse = t.run(o=None)
    k.csa2_prefix_attn(t.q, t.q_pos, t.cache, TAU, 120, 100, swa_codes=t.codes, swa_scale=t.scale, err=t.err)
    assert k.csa2_check(t.err) == 2  # sees 130 entries, max_entries says 120
    t = Batch(100, [30, 30], 4, 16, 128, 1, seed=11)
    t.cache.page_table[1, 7] = -1    # a page of sequence 1's own entries
    o, lse = t.run()
    assert k.csa2_check(t.err) == 5
    check(o[0, 0], lse[0, 0], t.want(0, 0), "the other sequence")
    gone = np.arange(100, 130)
    t.values[1] = t.values[1][~((gone >= 112) & (gone < 128))]
    t.ratio = 1
    check(o[1, 0], lse[1, 0], t.want(1, 0), "its other entries")
    t = Batch(100, [30, 30], 4, 16, 128, 1, seed=11)
    t.cache.page_table[0, 0] = 1 << 20  # a page of the prefix outside the cache
    t.run()
    assert k.csa2_check(t.err) == 5


def test_again_captured_and_on_another_stream():
    """Two different calls in one workspace after another, the same call twice (equal bits), a captured graph replayed
    with other inputs, on a side stream."""
    k = K()
    a, b = Batch(700, [5, 90], 4, 16, 128, 1, seed=12), Batch(90, [7, 9, 4], 4, 16, 0, 2, seed=13)
    n = max(k.csa2_prefix_workspace_size(t.B, t.Q, t.most) for t in (a, b))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    oa, la = a.run(ws=ws)
    ob, lb = b.run(ws=ws)
    oa2, la2 = a.run(ws=ws)
    assert torch.equal(oa, oa2) and torch.equal(la, la2)
    for t, o, lse in ((a, oa, la), (b, ob, lb)):
        for i in range(t.B):
            check(o[i, 0], lse[i, 0], t.want(i, 0), f"b={i}")
    o, lse = torch.zeros_like(oa), torch.zeros_like(la)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            a.run(ws=ws, o=o, lse=lse)
    for step in range(2):
        a.q.copy_(make(a.q.shape, 40 + step, torch.bfloat16))
        if step:
            a.cache.num_entries[1] = 700 + 12
            a.values[1] = a.values[1][:12]
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            check(o[i, 0], lse[i, 0], a.want(i, 0), f"replay {step} b={i}")


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_decode_steps_with_rotation(layout):
    """The operators together, as a decode loop uses them: the shared prefix packed with rotation once, then for every
    token each sequence's query heads turned, its latent appended (two tokens an entry) and its window token written
    with rotation, the attention over prefix, own entries and window, and the outputs turned back."""
    k = K()
    B, r, S, steps = 3, 2, 64, 7
    rot = k.Rotary.table(64, 448, layout, DEV, scaling="yarn", factor=4.0, original_len=64)
    rix = k.Rotary(rot.step, 64, layout, rot.scale)
    arg = (to_np(rot.step).astype(np.uint64), 448, layout, np.float64(np.float32(rot.scale)))
    cache = k.GlobalKVCache(B, r, seq_stride=S + 16)
    prompt, pix = make((1, S * r, 512), 1, torch.bfloat16), make((1, S * r, 128), 2, torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    view = cache.seq_view(0)
    k.csa2_pack_kv_rotary(prompt, pix, torch.zeros(1, dtype=torch.int32, device=DEV), view, rot, rix, err=err)
    cache.num_entries.fill_(S)
    pre = F.unpack_main(*R.pack_entries(to_np(prompt[0]), to_np(pix[0]), 0, r, arg, None)[:2])
    ring = 128
    codes, scale = torch.zeros((B, ring, 512), dtype=torch.uint8, device=DEV), torch.zeros((B, ring), device=DEV)
    stage = torch.zeros((B, r, 640), device=DEV)
    seen = make((B, ring, 512), 3, torch.bfloat16)  # the prompt's last tokens in each window
    before = S * r - ring + torch.arange(ring, device=DEV, dtype=torch.int32)
    k.csa2_pack_swa_rotary(seen, before.repeat(B, 1).contiguous(), codes, scale, rot, err=err)
    lat, lix = make((B, steps, 512), 4, torch.bfloat16), make((B, steps, 128), 5, torch.bfloat16)
    for t in range(steps):
        p = S * r + t
        pos = torch.full((B,), p, dtype=torch.int32, device=DEV)
        q, x = make((B, 64, 512), 50 + t, torch.bfloat16), make((B, 1, 512), 70 + t, torch.bfloat16)
        seen = torch.cat((seen, x), 1)
        qr = k.csa2_rotate(q, pos, rot)
        k.csa2_append_kv_rotary(lat[:, t].contiguous(), lix[:, t].contiguous(), pos, cache, rot, rix, stage=stage, err=err)
        k.csa2_pack_swa_rotary(x, pos[:, None], codes, scale, rot, err=err)
        o, lse = k.csa2_prefix_attn(qr[:, None], pos[:, None], cache, TAU, S + 16, S, swa_codes=codes, swa_scale=scale,
                                    err=err)
        back = k.csa2_rotate(o[:, 0], pos, rot, inverse=True, out_dtype=torch.bfloat16)
        assert k.csa2_check(err) == 0
        n = (t + 1) // r
        for b in range(B):
            own = F.unpack_main(*R.pack_entries(to_np(lat[b, :n * r]), to_np(lix[b, :n * r]), S, r, arg, None)[:2]) if n else np.zeros((0, 512))
            heads = R.turn(to_np(q[b]).astype(np.float64), np.full(64, p), *arg)
            heads = torch.from_numpy(heads).to(torch.bfloat16).double().numpy()  # what the attention is given
            wc, wsc = F.pack_swa(R.turn_entries(to_np(seen[b, -128:]), p - 127 + np.arange(128), arg))
            near = F.unpack_swa(wc, wsc)
            wo, wl = OC.attend(heads, np.concatenate([pre, own, near]), TAU)
            # a query value next to a border between two bf16 numbers may fall to either side: 2^-8 of a few of 512
            # terms of a logit, 1e-2 at most
            assert np.abs(to_np(lse[b, 0]) - wl).max() <= 1e-2
            assert np.abs(to_np(o[b, 0]) - wo).max() <= 1e-2
            turned = R.turn(to_np(o[b, 0]).astype(np.float64), np.full(64, p), *arg, inverse=True)
            np.testing.assert_allclose(to_np(back[b]), turned, rtol=2.0 ** -8, atol=1e-5)


# ------------------------------------------------------------------ the prefix dequantised ahead (many rows or a long prefix)
def everything(t, values=None):
    """Plain float64 attention of every query of the batch on the GPU: o [B][Q][64][512], lse."""
    o = torch.zeros((t.B, t.Q, 64, 512), dtype=torch.float64, device=DEV)
    lse = torch.full((t.B, t.Q, 64), -float("inf"), dtype=torch.float64, device=DEV)
    pre = torch.from_numpy(t.prefix).to(DEV)
    for b in range(t.B):
        own = torch.from_numpy(t.values[b]).to(DEV)
        count = int(t.cache.num_entries[b])
        for i in range(t.Q):
            p = int(t.q_pos[b, i])
            if p < 0:
                continue
            keys = torch.cat((pre, own))[:min(count, (p + 1) // t.ratio)]
            if t.gone is not None:
                keys = keys[~t.gone[b, :len(keys)]]
            if t.window:
                at = torch.arange(max(0, p - t.window + 1), p + 1, device=DEV) % t.ring
                codes = t.codes[b, at].view(torch.float8_e4m3fn).double()
                keys = torch.cat((keys, codes * t.scale[b, at].double()[:, None]))
            if len(keys):
                x = t.q[b, i].double() @ keys.T * TAU
                lse[b, i] = torch.logsumexp(x, -1)
                o[b, i] = torch.softmax(x, -1) @ keys
    return o, lse


Batch.gone = None
AHEAD = [  # S, tails, ratio, page, window, Q: at least 4 rows and 400 row-tiles of the prefix
    (10500, [5, 0, 260, 128, 33], 4, 256, 128, 1), (12800, [0, 1, 127, 300], 1, 16, 0, 1),
    (140, [11 * (b % 5) for b in range(70)], 1, 16, 128, 6), (1300, [7 * (b % 9) for b in range(45)], 2, 64, 0, 1),
    (400, [b % 4 for b in range(40)], 1, 0, 100, 4), (129, [200 * (b % 2) for b in range(410)], 4, 64, 0, 1)]


@pytest.mark.parametrize("S,tails,ratio,page,window,Q", AHEAD)
def test_prefix_dequantised_ahead(S, tails, ratio, page, window, Q):
    t = Batch(S, tails, ratio, page, window, Q, seed=21)
    assert t.B * Q >= 4 and t.B * Q * (S // 128) >= 400
    t.cache.num_entries[1] = min(int(t.cache.num_entries[1]), S // 2)  # one row sees half of the prefix
    if t.B > 4:
        t.q_pos[4] = -1                                                 # and one nothing
    ws = torch.full((K().csa2_prefix_workspace_size(t.B, Q, t.most),), 0xFF, dtype=torch.uint8, device=DEV)
    wo, wl = everything(t)
    for od in (torch.float32, torch.bfloat16):
        o, lse = t.run(o_dtype=od, ws=ws)
        assert K().csa2_check(t.err) == 0
        check(o, lse, (to_np(wo), to_np(wl)), f"{od}")
    o2, lse2 = t.run(o_dtype=torch.bfloat16, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_pages_outside_the_cache_in_a_prefix_dequantised_ahead():
    """Pages of the prefix that lie outside the cache: reported, their entries left out of every row, whether before,
    between or behind the good ones."""
    for pages in ((0,), (100, 101, 333), (656,)):
        t = Batch(10500, [5, 0, 260, 128, 33], 4, 16, 128, 1, seed=22)
        t.gone = torch.zeros((5, 10500 + 300), dtype=torch.bool, device=DEV)
        for n, page in enumerate(pages):
            t.cache.page_table[0, page] = (-1, 1 << 20, -7)[n]
            t.gone[:, 16 * page:min(16 * page + 16, 10500)] = True
            t.gone[0, 16 * page:16 * page + 16] = True  # (the prefix's last page holds sequence 0's first own entries)
        o, lse = t.run()
        assert K().csa2_check(t.err) == 5
        check(o, lse, tuple(to_np(x) for x in everything(t)), f"pages {pages}")


def test_short_bound_with_a_prefix_dequantised_ahead():
    """max_entries below the prefix: reported, and only that many entries count."""
    k = K()
    t = Batch(12900, [0, 1, 127, 300], 1, 16, 128, 1, seed=23)
    o, lse = k.csa2_prefix_attn(t.q, t.q_pos, t.cache, TAU, 12801, 12900, swa_codes=t.codes, swa_scale=t.scale, err=t.err)
    assert k.csa2_check(t.err) == 2
    t.cache.num_entries.clamp_(max=12801)
    check(o, lse, tuple(to_np(x) for x in everything(t)), "bounded")


@pytest.mark.parametrize("S,B", [(300, 3), (12800, 4)])
def test_heads_that_are_not_finite_stay_alone(S, B):
    """Infinities and NaN in some query heads: every other head is as without them."""
    t = Batch(S, [3] * B, 1, 16, 128, 1, seed=24)
    wo, wl = everything(t)
    t.q[0, 0, 7, 100], t.q[1, 0, 0, 0], t.q[2, 0, 63, 511] = float("inf"), float("nan"), -float("inf")
    o, lse = t.run()
    assert K().csa2_check(t.err) == 0
    keep = torch.ones((B, 1, 64), dtype=torch.bool, device=DEV)
    keep[0, 0, 7] = keep[1, 0, 0] = keep[2, 0, 63] = False
    check(o[keep], lse[keep], (to_np(wo[keep]), to_np(wl[keep])), "the other heads")


def test_two_calls_at_once_and_a_captured_one():
    """Two streams with a workspace each, over one cache; then the long call captured and replayed on other queries."""
    t = Batch(12800, [0, 1, 127, 300], 1, 16, 128, 1, seed=25)
    u = Batch(12800, [0, 1, 127, 300], 1, 16, 128, 1, seed=25)
    u.q.copy_(make(u.q.shape, 77, torch.bfloat16))
    want = [tuple(to_np(x) for x in everything(x)) for x in (t, u)]
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s, got in zip((t, u), streams, outs):
            with torch.cuda.stream(s):
                got.append(x.run())
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        for o, lse in got:
            check(o, lse, w, "two streams")
    ws = torch.empty(K().csa2_prefix_workspace_size(t.B, 1, t.most), dtype=torch.uint8, device=DEV)
    o, lse = torch.zeros_like(outs[0][0][0]), torch.zeros_like(outs[0][0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run(ws=ws, o=o, lse=lse)
        t.run(ws=ws, o=o, lse=lse)  # (one after the other in one workspace)
    t.q.copy_(u.q)
    for _ in range(2):
        ws.fill_(0xFF)
        graph.replay()
    torch.cuda.synchronize()
    check(o, lse, tuple(to_np(x) for x in everything(t)), "replayed")


def test_very_large_and_very_small_logits():
    """Softmax scales that spread the logits over millions, and that leave them all but equal; keys of one repeated value
    (every weight the same, whatever the reference)."""
    k = K()
    for S, B in ((700, 2), (12800, 4)):
        t = Batch(S, [3] * B, 1, 16, 0, 1, seed=26)
        for tau in (1e-6, 3.0, 1e5):
            o, lse = k.csa2_prefix_attn(t.q, t.q_pos, t.cache, tau, t.most, t.S, err=t.err)
            x = torch.einsum("bqhd,nd->bqhn", t.q.double(), torch.from_numpy(t.prefix).to(DEV))
            own = torch.stack([torch.einsum("qhd,nd->qhn", t.q[b].double(), torch.from_numpy(t.values[b]).to(DEV)) for b in range(B)])
            x = torch.cat((x, own), -1) * float(np.float32(tau))
            wl = torch.logsumexp(x, -1)
            assert torch.isfinite(o).all() and torch.isfinite(lse).all()
            # logits are fp32: off by a few 2^-24 of their size
            size = x.abs().amax(-1)
            assert bool(((lse.double() - wl).abs() <= 1e-4 + size * 2.0 ** -21).all())
            if tau <= 3.0:
                vals = [torch.cat((torch.from_numpy(t.prefix).to(DEV), torch.from_numpy(t.values[b]).to(DEV))) for b in range(B)]
                wo = torch.stack([torch.softmax(x[b], -1) @ vals[b] for b in range(B)])
                check(o, lse, (to_np(wo), to_np(lse.double())), f"tau {tau}")


def test_memory_of_its_own_on_another_stream():
    """Outputs and a workspace that the call makes itself, for a stream that is not the current one: what the current
    stream allocates and fills right after it does not get into them."""
    t = Batch(2000, [5, 0, 33], 4, 16, 128, 1, seed=31)
    want = t.run()
    side = torch.cuda.Stream()
    n = K().csa2_prefix_workspace_size(t.B, t.Q, t.most)
    for _ in range(5):
        torch.cuda.synchronize()
        o, lse = t.run(stream=side)
        for _ in range(3):
            torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_the_last_position_and_single_entry_pages():
    """Position 2^31 - 1 sees every entry, and a window that is in the ring by position; pages of one entry."""
    t = Batch(150, [4, 70], 1, 1, 0, 1, seed=32)
    o, lse = t.run()
    for b in range(2):
        check(o[b, 0], lse[b, 0], t.want(b, 0), f"b={b}")
    t.q_pos.fill_(2 ** 31 - 1)
    o2, lse2 = t.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and K().csa2_check(t.err) == 0


def test_entries_behind_four_gigabytes():
    """A prefix and own entries in a cache whose planes pass 2^32 bytes, in pages at its end."""
    t = Batch(300, [40, 7], 4, 256, 0, 1, seed=33)
    want = t.run()
    page = t.cache.page_size
    far = (1 << 24) // page + 5  # 2^24 entries of 256 code bytes
    used = t.cache.num_slots // page
    big = K().GlobalKVCache(t.B, 4, num_slots=(far + used) * page, page_table=t.table + far, page_size=page,
                            num_entries=t.cache.num_entries)
    for new, old in zip(big.planes, t.cache.planes):
        new[far * page:] = old
    o, lse = K().csa2_prefix_attn(t.q, t.q_pos, big, TAU, t.most, t.S, err=t.err)
    assert K().csa2_check(t.err) == 0 and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    t.cache = big
    o, lse = K().csa2_prefix_attn(t.q[:, :1].repeat(1, 250, 1, 1).contiguous(), t.q_pos.repeat(1, 250).contiguous(), big, TAU,
                                  t.most, t.S, err=t.err)  # (dequantised ahead)
    for b in range(2):
        check(o[b, 249], lse[b, 249], t.want(b, 0), f"ahead b={b}")
