"""Cases of the rotary operators, the rotating cache writes and the shared-prefix attention.

Every case runs in two forms.  With `own` false, `run` computes the operator in its plain form
(elementary torch operations, fp32 or fp64); with `own` true it makes the library's calls:

  rotate   csa2_rotate: rotary positions on query heads, indexer queries or attention outputs
  pack     csa2_pack_kv_rotary: a chunk of tokens pooled, rotated and written into the FP4 cache
  append   csa2_append_kv_rotary: one token per sequence into the (paged) FP4 cache
  window   csa2_pack_swa_rotary: sliding-window tokens rotated and written into the FP8 ring
  prefix   csa2_prefix_attn: attention of a batch whose sequences share their first entries

An angle is a number of turns modulo one: position times a 64-bit step (2^64 steps to a turn).
"""
import math

import torch

own = False

DEV = "cuda"
D, DI, H = 512, 128, 64
NAMED = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the query heads of one decode step of eight sequences near 2^20 tokens, the last 64 of 512 dims
        {"name": "rotate_decode", "op": "rotate", "tokens": 8, "heads": 64, "dim": 512, "rot": 64, "first": 448,
         "layout": "interleaved", "inverse": False, "x": "bf16", "out": "bf16", "pos": 1048000, "pad": 0, "factor": 16.0},
        # the query heads of a prefill chunk: 8192 tokens after a prefix of 262144
        {"name": "rotate_prefill", "op": "rotate", "tokens": 8192, "heads": 64, "dim": 512, "rot": 64, "first": 448,
         "layout": "interleaved", "inverse": False, "x": "bf16", "out": "bf16", "pos": 262144, "pad": 0, "factor": 4.0},
        # attention outputs turned back before the output projection (fp32 to bf16), an odd number of rows;
        # as a gradient of `rotate` this is the backward direction
        {"name": "rotate_back", "op": "rotate", "tokens": 1021, "heads": 64, "dim": 512, "rot": 64, "first": 448,
         "layout": "half", "inverse": True, "x": "f32", "out": "bf16", "pos": 70000, "pad": 0, "factor": 1.0},
        # one token of 64 ragged sequences appended to a paged cache that pools two tokens per entry
        {"name": "append_64", "op": "append", "B": 64, "ratio": 2, "page": 256, "rot": 64, "layout": "interleaved",
         "x": "bf16", "last": 16384, "factor": 4.0},
        # a prefill chunk written at two tokens per entry
        {"name": "pack_chunk", "op": "pack", "B": 1, "T": 8192, "ratio": 2, "page": 0, "rot": 64,
         "layout": "interleaved", "x": "bf16", "first_entry": 131072, "factor": 4.0},
        # the prompts of a batch written into pages, one entry per token
        {"name": "pack_batch", "op": "pack", "B": 8, "T": 16411, "ratio": 1, "page": 256, "rot": 64,
         "layout": "half", "x": "bf16", "first_entry": 77, "factor": 16.0},
        # the window tokens of a prefill chunk of eight sequences
        {"name": "window_chunk", "op": "window", "B": 8, "T": 1151, "R": 1280, "rot": 64, "layout": "interleaved",
         "x": "bf16", "pos": 4096, "factor": 1.0},
        # two short sequences on a short shared prompt: latency
        {"name": "prefix_short", "op": "prefix", "B": 2, "Q": 1, "prefix": 96, "most_own": 17, "ratio": 4, "page": 64,
         "window": 128, "out": "bf16"},
        # 32 sessions on one system prompt of 2^20 tokens, 128 tokens per entry, and their window
        {"name": "prefix_sessions", "op": "prefix", "B": 32, "Q": 1, "prefix": 8192, "most_own": 37, "ratio": 128,
         "page": 256, "window": 128, "out": "bf16"},
        # a batch with unequal tails on a prefix that ends inside a page, no window
        {"name": "prefix_ragged", "op": "prefix", "B": 13, "Q": 1, "prefix": 2999, "most_own": 700, "ratio": 4,
         "page": 256, "window": 0, "out": "bf16"},
        # several query tokens of each sequence at once (drafted tokens checked, a short chunk)
        {"name": "prefix_drafts", "op": "prefix", "B": 16, "Q": 6, "prefix": 4096, "most_own": 96, "ratio": 1,
         "page": 256, "window": 128, "out": "bf16"},
        # the longest: 16 sequences on 65536 shared entries
        {"name": "prefix_long", "op": "prefix", "B": 16, "Q": 1, "prefix": 65536, "most_own": 512, "ratio": 4,
         "page": 256, "window": 128, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "pack", "append", "window", "prefix", "prefix"])
    layout = rng.choice(["interleaved", "half"])
    factor = rng.choice([1.0, 4.0, 16.0])
    x = rng.choice(["bf16", "f32"])
    if op == "rotate":
        dim = rng.choice([128, 512])
        rot = rng.choice([16, 32, 64, 96, 128])
        return {"op": op, "tokens": _log(rng, 1, 3000), "heads": rng.choice([1, 3, 8, 64]), "dim": dim, "rot": rot,
                "first": rng.choice([0, dim - rot]), "layout": layout, "inverse": rng.random() < 0.5, "x": x,
                "out": rng.choice(["bf16", "f32"]), "pos": _log(rng, 1, 1 << 20), "pad": rng.choice([0, 8, 640]),
                "factor": factor}
    if op == "append":
        return {"op": op, "B": _log(rng, 1, 128), "ratio": rng.choice([1, 2, 4]), "page": rng.choice([0, 16, 64, 256]),
                "rot": rng.choice([32, 64, 128]), "layout": layout, "x": x, "last": _log(rng, 8, 16384), "factor": factor}
    if op == "pack":
        B = _log(rng, 1, 16)
        return {"op": op, "B": B, "T": _log(rng, 4, 65536 // B), "ratio": rng.choice([1, 2, 4]),
                "page": rng.choice([0, 16, 64, 256]), "rot": rng.choice([32, 64, 128]), "layout": layout, "x": x,
                "first_entry": rng.choice([0, rng.randint(1, 3000)]), "factor": factor}
    if op == "window":
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "T": _log(rng, 1, 16384 // B), "R": rng.choice([128, 200, 1280]),
                "rot": rng.choice([32, 64, 128, 512]), "layout": layout, "x": x, "pos": _log(rng, 1, 1 << 20),
                "factor": factor}
    B, Q = _log(rng, 1, 48), rng.choice([1, 1, 1, 2, 5])
    return {"op": op, "B": B, "Q": Q, "prefix": rng.choice([0, 1]) if rng.random() < 0.1 else _log(rng, 16, min(32768, 1048576 // (B * Q))),
            "most_own": _log(rng, 1, 600), "ratio": rng.choice([1, 2, 4, 128]), "page": rng.choice([0, 16, 64, 256]),
            "window": rng.choice([0, 1, 100, 128]), "out": "bf16"}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000 + k)
    return g


def _normal(shape, seed, k, dtype):
    return torch.randn(shape, generator=_gen(seed, k), device=DEV, dtype=torch.float32).to(dtype)


def _ints(lo, hi, shape, seed, k):
    """Whole numbers lo .. hi (both ends among them)."""
    return torch.randint(lo, hi + 1, shape, generator=_gen(seed, k), device=DEV)


def _steps(rot, factor, base=10000.0, original=65536, fast=32.0, slow=1.0):
    """2^64ths of a turn per position for each pair: base^(-2i/rot), and for factor > 1 the YaRN blend
    (pairs that turn often keep their frequency, slow ones are divided by the factor)."""
    got = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if factor > 1.0:
            def dim_of(turns):
                return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(math.floor(dim_of(fast)), 0), min(math.ceil(dim_of(slow)), rot - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / factor * ramp + f * (1.0 - ramp)
        n = int(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64)
        got.append(n - (1 << 64) if n >= (1 << 63) else n)
    return torch.tensor(got, dtype=torch.int64, device=DEV)


def _gain(factor):
    return 1.0 if factor <= 1.0 else 0.1 * math.log(factor) + 1.0


def _slots(B, entries, page, seed):
    """(page table or None, slots in all): room for `entries` entries of each of B sequences."""
    if page == 0:
        return None, B * entries
    n = -(-entries // page)
    perm = torch.randperm(B * n, generator=_gen(seed, 90), device=DEV)
    return perm.view(B, n).to(torch.int32), B * n * page


def _planes(slots):
    return [torch.zeros((slots, w), dtype=torch.uint8, device=DEV) for w in (256, 32, 64, 4)]


def prepare(case, seed):
    op = case["op"]
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if op == "prefix":
        return _prepare_prefix(s, case, seed)
    s["step"], s["gain"] = _steps(case["rot"], case["factor"]), _gain(case["factor"])
    if op == "rotate":
        T, NH, dim = case["tokens"], case["heads"], case["dim"]
        rows = _normal((T, NH * dim + case["pad"]), seed, 1, NAMED[case["x"]])
        s["x"] = rows[:, :NH * dim].view(T, NH, dim)  # heads inside a wider row where pad > 0
        s["pos"] = (case["pos"] + torch.arange(T, device=DEV) + _ints(0, 64, (1,), seed, 2)).to(torch.int32)
        s["out"] = torch.empty((T, NH, dim), dtype=NAMED[case["out"]], device=DEV)
        return s
    B, dt = case["B"], NAMED[case["x"]]
    if op == "window":
        s["x"] = _normal((B, case["T"], D), seed, 1, dt)
        s["pos"] = (case["pos"] + _ints(0, 500, (B, 1), seed, 2) + torch.arange(case["T"], device=DEV)).to(torch.int32)
        s["codes"] = torch.zeros((B, case["R"], D), dtype=torch.uint8, device=DEV)
        s["scale"] = torch.zeros((B, case["R"]), dtype=torch.float32, device=DEV)
        return s
    r = case["ratio"]
    if op == "append":
        s["pos"] = _ints(0, case["last"] - 1, (B,), seed, 2).to(torch.int32)
        s["pos"][::2] = s["pos"][::2] // r * r + r - 1  # about half and more complete an entry
        s["per"] = case["last"] // r + 1
        s["lat_kv"], s["lat_ix"] = _normal((B, D), seed, 3, dt), _normal((B, DI), seed, 4, dt)
        s["stage"] = _normal((B, r, D + DI), seed, 5, dt).to(torch.float32) if r > 1 else None
        s["num_entries"] = (s["pos"] // r).to(torch.int32)
        s["kv_hat"], s["ix_hat"] = (torch.zeros((B, w), dtype=torch.bfloat16, device=DEV) for w in (D, DI))
    else:
        T = case["T"]
        s["lat_kv"], s["lat_ix"] = _normal((B, T, D), seed, 3, dt), _normal((B, T, DI), seed, 4, dt)
        s["first_entry"] = torch.full((B,), case["first_entry"], dtype=torch.int32, device=DEV)
        s["per"] = case["first_entry"] + T // r
        s["num_entries"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["kv_hat"], s["ix_hat"] = (torch.zeros((B, T // r, w), dtype=torch.bfloat16, device=DEV) for w in (D, DI))
    s["table"], slots = _slots(B, max(s["per"], 1), case["page"], seed)
    s["planes"] = _planes(slots)
    return s


def _prepare_prefix(s, case, seed):
    B, Q, S, r, W = case["B"], case["Q"], case["prefix"], case["ratio"], case["window"]
    tail = _ints(0, case["most_own"], (B,), seed, 2)
    entries = S + tail  # per sequence, its shared entries among them
    most = S + case["most_own"]
    if case["page"]:
        n, whole = -(-most // case["page"]), S // case["page"]
        table = torch.empty((B, n), dtype=torch.long, device=DEV)
        table[:, :whole] = torch.arange(whole, device=DEV)  # whole pages of the prefix: the same for all
        table[:, whole:] = whole + torch.arange(B * (n - whole), device=DEV).view(B, n - whole)  # its end: sequence 0's
        used = whole + B * (n - whole)
        s["table"] = torch.randperm(used, generator=_gen(seed, 90), device=DEV)[table].to(torch.int32)
        slots = used * case["page"]
    else:
        s["table"], slots = None, B * most
    s["per"], s["most"] = most, most
    # entries as the packer writes them: normal latents, quantised
    kv, sc = [], []
    for at in range(0, slots, 1 << 15):
        x = _normal((min(1 << 15, slots - at), D), seed, 100 + (at >> 15), torch.float32)
        c, e = _encode_main(x)
        kv.append(c), sc.append(e)
    s["planes"] = [torch.cat(kv), torch.cat(sc), torch.zeros((slots, 64), dtype=torch.uint8, device=DEV),
                   torch.zeros((slots, 4), dtype=torch.uint8, device=DEV)]
    s["num_entries"] = entries.to(torch.int32)
    last = entries * r + _ints(0, r - 1, (B,), seed, 3) - 1  # the last query sees every entry
    s["q_pos"] = (last[:, None] - (Q - 1) + torch.arange(Q, device=DEV)).to(torch.int32)  # below 0: sees nothing
    s["q"] = _normal((B, Q, H, D), seed, 4, torch.bfloat16)
    s["tau"] = 1.0 / math.sqrt(D)
    if W:
        s["R"] = W + Q
        x = _normal((B, s["R"], D), seed, 5, torch.float32)
        s["scale"] = x.abs().amax(-1) / 448.0
        s["codes"] = (x / s["scale"][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s["o"] = torch.empty((B, Q, H, D), dtype=NAMED[case["out"]], device=DEV)
    s["lse"] = torch.empty((B, Q, H), dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------------------------ the library's calls
def _rotary(s, first):
    import compressed_sparse_attention_score_b200 as k
    key = "rotary%d" % first
    if key not in s:
        s[key] = k.Rotary(s["step"], first=first, layout=s["case"]["layout"], scale=s["gain"])
    return s[key]


def _cache(s):
    import compressed_sparse_attention_score_b200 as k
    if "cache" not in s:
        c = s["case"]
        more = ({"seq_stride": s["per"]} if s["table"] is None else
                {"num_slots": s["planes"][0].shape[0], "page_table": s["table"], "page_size": c["page"]})
        s["cache"] = k.GlobalKVCache(c["B"], c["ratio"], planes=tuple(s["planes"]), num_entries=s["num_entries"], **more)
    return s["cache"]


def _run_own(s):
    import compressed_sparse_attention_score_b200 as k
    c, op = s["case"], s["case"]["op"]
    if op == "rotate":
        return k.csa2_rotate(s["x"], s["pos"], _rotary(s, c["first"]), inverse=c["inverse"], out=s["out"])
    if op == "window":
        k.csa2_pack_swa_rotary(s["x"], s["pos"], s["codes"], s["scale"], _rotary(s, D - c["rot"]), err=s["err"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    if op == "prefix":
        W = c["window"]
        if "ws" not in s:
            s["ws"] = torch.empty(max(1, k.csa2_prefix_workspace_size(c["B"], c["Q"], s["most"])), dtype=torch.uint8, device=DEV)
        k.csa2_prefix_attn(s["q"], s["q_pos"], _cache(s), s["tau"], s["most"], c["prefix"],
                           swa_codes=s["codes"] if W else None, swa_scale=s["scale"] if W else None, window=W or 128,
                           o=s["o"], lse=s["lse"], ws=s["ws"], err=s["err"])
        return {"o": s["o"], "lse": s["lse"]}
    kv, ix = _rotary(s, D - c["rot"]), _rotary(s, DI - c["rot"])
    if op == "append":
        k.csa2_append_kv_rotary(s["lat_kv"], s["lat_ix"], s["pos"], _cache(s), kv, ix, stage=s["stage"],
                                kv_hat=s["kv_hat"], ix_hat=s["ix_hat"], err=s["err"])
    else:
        k.csa2_pack_kv_rotary(s["lat_kv"], s["lat_ix"], s["first_entry"], _cache(s), kv, ix, kv_hat=s["kv_hat"],
                              ix_hat=s["ix_hat"], err=s["err"])
    return _cache_outputs(s)


def _cache_outputs(s):
    kv, sc, ix, ex = s["planes"]
    got = {"kv": s["kv_hat"], "ix": s["ix_hat"], "kv_codes": kv, "kv_scales": sc.view(torch.float8_e4m3fn),
           "ix_codes": ix, "ix_exponents": ex, "num_entries": s["num_entries"]}
    return got if s.get("stage") is None else {**got, "stage": s["stage"]}


# ------------------------------------------------------------------------------------ the plain form
def _angles(pos, step):
    """cos and sin of pos x step turns (fp64): the product wraps modulo 2^64, which is modulo one turn."""
    turn = (pos.to(torch.int64)[..., None] * step).to(torch.float64) * 2.0 ** -64
    return torch.cos(2 * math.pi * turn), torch.sin(2 * math.pi * turn)


def _turn(x, cos, sin, first, layout, gain):
    """x (any float type) with the pairs of dims first .. first + 2 n - 1 turned, in x's own type."""
    n = cos.shape[-1]
    y = x.clone()
    part = x[..., first:first + 2 * n]
    a, b = (part[..., 0::2], part[..., 1::2]) if layout == "interleaved" else (part[..., :n], part[..., n:])
    u, v = (a * cos - b * sin) * gain, (a * sin + b * cos) * gain
    y[..., first:first + 2 * n] = torch.stack((u, v), -1).flatten(-2) if layout == "interleaved" else torch.cat((u, v), -1)
    return y


def _turn64(x, cos, sin, first, layout, gain):
    """fp32 x turned in fp64 and rounded once: values next to a border between two codes stay on their side."""
    y = x.clone()
    w = slice(first, first + 2 * cos.shape[-1])
    y[..., w] = _turn(x[..., w].double(), cos, sin, 0, layout, gain).float()
    return y


def _nearest_e2m1(y):
    """e2m1 codes of y: nearest magnitude, ties to the even code, a zero result without its sign."""
    m = y.abs()
    i = torch.zeros_like(m, dtype=torch.uint8)
    i = (i + (m > BORDERS[0]) + (m >= BORDERS[1]) + (m > BORDERS[2]) + (m >= BORDERS[3]) + (m > BORDERS[4])
         + (m >= BORDERS[5]) + (m > BORDERS[6])).to(torch.uint8)
    return i | (((y < 0) & (i > 0)).to(torch.uint8) << 3)


def _pairs(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _encode_main(x):
    """fp32 [.., 512] -> 256 code bytes and 32 E4M3 scale bytes (amax / 6 of each 16 values)."""
    blocks = x.unflatten(-1, (32, 16))
    e = (blocks.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = e.float()[..., None]
    codes = torch.where(s > 0, _nearest_e2m1(blocks / torch.where(s > 0, s, 1.0)), 0).to(torch.uint8)
    return _pairs(codes.flatten(-2)), e.view(torch.uint8)


def _encode_index(x):
    """fp32 [.., 128] -> 64 code bytes and 4 E8M0 bytes (2^ceil(log2(amax / 6)) of each 32 values)."""
    blocks = x.unflatten(-1, (4, 32))
    q = blocks.abs().amax(-1) / 6.0
    m, e = torch.frexp(q)
    ex = torch.where(q > 0, torch.where(m == 0.5, e - 1, e), -127).clamp(-127, 127)
    codes = torch.where(q[..., None] > 0, _nearest_e2m1(blocks / torch.ldexp(torch.ones_like(q), ex)[..., None]), 0)
    return _pairs(codes.to(torch.uint8).flatten(-2)), (ex + 127).to(torch.uint8)


def _e2m1_values(codes):
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)[both.int()]


def _decode_main(codes, scales):
    return (_e2m1_values(codes).unflatten(-1, (32, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _decode_index(codes, ex):
    s = torch.ldexp(torch.ones_like(ex, dtype=torch.float32), ex.int() - 127)
    return (_e2m1_values(codes).unflatten(-1, (4, 32)) * s[..., None]).flatten(-2)


def _slot(s, b, n):
    """Physical slots of entries n of the sequences b."""
    if s["table"] is None:
        return b * s["per"] + n
    page = s["case"]["page"]
    return s["table"][b, n // page].long() * page + n % page


def _entries(s, x, xi, n):
    """Entries n from pooled fp32 values: turned at their first token's position and quantised.  Returns the
    bytes of the four planes and the values that they stand for."""
    c = s["case"]
    cos, sin = _angles(n * c["ratio"], s["step"])
    kv, sc = _encode_main(_turn64(x, cos, sin, D - c["rot"], c["layout"], s["gain"]))
    ix, ex = _encode_index(_turn64(xi, cos, sin, DI - c["rot"], c["layout"], s["gain"]))
    return [kv, sc, ix, ex], [_decode_main(kv, sc).bfloat16(), _decode_index(ix, ex).bfloat16()]


def _pool(x, r):
    """[.., r, width] fp32 summed with weight 1 / r, from the first token to the last."""
    y = x[..., 0, :] * (1.0 / r)
    for t in range(1, r):
        y = y + x[..., t, :] * (1.0 / r)
    return y


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "rotate":
        cos, sin = (t.float()[:, None] for t in _angles(s["pos"], s["step"]))
        y = _turn(s["x"].float(), cos, -sin if c["inverse"] else sin, c["first"], c["layout"], s["gain"])
        return y.to(NAMED[c["out"]])
    if op == "prefix":
        return _prefix_plain(s)
    if op == "window":
        R, T = c["R"], c["T"]  # only the last R tokens stay in the ring
        x, pos = s["x"][:, max(0, T - R):].float(), s["pos"][:, max(0, T - R):].long()
        y = _turn64(x, *_angles(pos, s["step"]), D - c["rot"], c["layout"], s["gain"])
        sc = y.abs().amax(-1) / 448.0
        codes = torch.where(sc[..., None] > 0, y / torch.where(sc > 0, sc, 1.0)[..., None], 0.0).to(torch.float8_e4m3fn)
        codes = codes.view(torch.uint8)
        b = torch.arange(c["B"], device=DEV)[:, None].expand_as(pos)
        s["codes"][b, pos % R] = torch.where((codes & 127) == 0, 0, codes)
        s["scale"][b, pos % R] = sc
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    r, B = c["ratio"], c["B"]
    if op == "pack":
        n = c["T"] // r
        x, xi = (_pool(t[:, :n * r].float().unflatten(1, (n, r)), r) for t in (s["lat_kv"], s["lat_ix"]))
        e = s["first_entry"].long()[:, None] + torch.arange(n, device=DEV)
        rows, hats = _entries(s, x, xi, e)
        at = _slot(s, torch.arange(B, device=DEV)[:, None], e)
        for plane, new in zip(s["planes"] + [s["kv_hat"].view(-1, D), s["ix_hat"].view(-1, DI)], rows + hats):
            plane[at if new.dtype == torch.uint8 else torch.arange(B * n, device=DEV).view(B, n)] = new
        return _cache_outputs(s)
    # append: the token joins its group's staged tokens; a complete group makes an entry
    pos, b = s["pos"].long(), torch.arange(B, device=DEV)
    e, done = pos // r, pos % r == r - 1
    kv, ix = s["lat_kv"].float(), s["lat_ix"].float()
    if r > 1:
        s["stage"][b, pos % r] = torch.cat((kv, ix), -1)
        kv, ix = _pool(s["stage"][..., :D], r), _pool(s["stage"][..., D:], r)
    rows, hats = _entries(s, kv, ix, e)
    at = _slot(s, b, e)
    for plane, new in zip(s["planes"], rows):
        plane[at] = torch.where(done[:, None], new, plane[at])
    for hat, new in zip((s["kv_hat"], s["ix_hat"]), hats):
        hat.copy_(torch.where(done[:, None], new, hat))
    s["num_entries"].copy_(torch.maximum(s["num_entries"], torch.where(done, e + 1, 0)))
    return _cache_outputs(s)


def _prefix_plain(s):
    c = s["case"]
    B, Q, S, r, W, own_n = c["B"], c["Q"], c["prefix"], c["ratio"], c["window"], c["most_own"]
    kv, sc = s["planes"][0], s["planes"][1]
    pos = s["q_pos"].long()
    seen = torch.minimum(s["num_entries"].long()[:, None], (pos + 1).clamp(min=0) // r)[:, :, None, None]
    q = s["q"].float() * s["tau"]
    b = torch.arange(B, device=DEV)
    at = _slot(s, torch.zeros(S, dtype=torch.long, device=DEV), torch.arange(S, device=DEV))
    shared = _decode_main(kv[at], sc[at])
    n = S + torch.arange(own_n, device=DEV)
    at = _slot(s, b[:, None], n.expand(B, own_n))
    tail = _decode_main(kv[at], sc[at])
    parts = [torch.where(torch.arange(S, device=DEV) < seen, q @ shared.T, -math.inf),
             torch.where(n < seen, torch.einsum("bqhd,bnd->bqhn", q, tail), -math.inf)]
    if W:
        t = pos[..., None] - (W - 1) + torch.arange(W, device=DEV)
        ring = t.clamp(min=0) % s["R"]
        near = s["codes"].view(torch.float8_e4m3fn)[b[:, None, None], ring].float() * s["scale"][b[:, None, None], ring][..., None]
        parts.append(torch.where((t >= 0)[:, :, None], torch.einsum("bqhd,bqnd->bqhn", q, near), -math.inf))
    x = torch.cat(parts, -1)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = e[..., :S] @ shared + torch.einsum("bqhn,bnd->bqhd", e[..., S:S + own_n], tail)
    if W:
        o = o + torch.einsum("bqhn,bqnd->bqhd", e[..., S + own_n:], near)
    o = torch.where(total > 0, o / total, 0.0)
    return {"o": o.to(NAMED[c["out"]]), "lse": (m + torch.log(total))[..., 0]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------ what a pass has to do
def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "rotate":
        n = c["tokens"] * c["heads"]
        return {"bytes": n * c["dim"] * (size[c["x"]] + size[c["out"]]) + 4 * c["tokens"], "flops": 3 * n * c["rot"]}
    if op == "window":
        n = c["B"] * min(c["T"], c["R"])
        return {"bytes": n * (D * size[c["x"]] + D + 8), "flops": n * (3 * c["rot"] + 3 * D)}
    entry = 288 + 68 + 2 * (D + DI)  # the four planes and the values they stand for
    if op == "pack":
        n = c["B"] * (c["T"] // c["ratio"])
        return {"bytes": n * (c["ratio"] * (D + DI) * size[c["x"]] + entry), "flops": n * (c["ratio"] + 4) * (D + DI)}
    if op == "append":
        r = c["ratio"]
        done = 0.5 + 0.5 / r  # of the sequences, about
        stage = 0 if r == 1 else 4 * (D + DI) * (1 + done * (r - 1))
        return {"bytes": c["B"] * ((D + DI) * size[c["x"]] + stage + done * entry), "flops": c["B"] * done * (r + 4) * (D + DI)}
    rows, tail = c["B"] * c["Q"], c["most_own"] / 2
    return {"bytes": (c["prefix"] + c["B"] * tail) * 288 + c["B"] * c["window"] * 516
            + rows * H * (D * (2 + size[c["out"]]) + 4), "flops": 4 * rows * H * D * (c["prefix"] + tail + c["window"])}


# ------------------------------------------------------------------------------------ the definition, in 64 bits
def _nearest(x, bits, least, most):
    """x to the nearest number of `bits` fraction bits (ties to even), exponents from `least`, at most `most`."""
    _, e = torch.frexp(x)
    quantum = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=least) - bits)
    return (torch.round(x / quantum) * quantum).clamp(-most, most)


def _exact_turn(x, pos, s, first, back=False):
    """Pairs of x as complex numbers times e^(2 pi i turn); the turn from the step's two 32-bit halves."""
    c = s["case"]
    step = s["step"]
    hi, lo = (step >> 32) & 0xFFFFFFFF, step & 0xFFFFFFFF
    p = pos.long()[..., None]
    turn = (((p * hi) & 0xFFFFFFFF).double() + (p * lo).double() * 2.0 ** -32) * 2.0 ** -32
    w = torch.polar(torch.full_like(turn, s["gain"]), 2 * math.pi * turn)
    w = w.conj() if back else w
    n = step.numel()
    part = x[..., first:first + 2 * n].double()
    pairs = part.unflatten(-1, (n, 2)) if c["layout"] == "interleaved" else part.unflatten(-1, (2, n)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    y = x.double().clone()
    y[..., first:first + 2 * n] = (z if c["layout"] == "interleaved" else z.transpose(-1, -2)).flatten(-2)
    return y


def _exact_entries(s, x, xi, pos):
    c = s["case"]
    x = _exact_turn(x, pos, s, D - c["rot"]).unflatten(-1, (32, 16))
    sc = _nearest(x.abs().amax(-1, keepdim=True) / 6, 3, -6, 448.0)
    kv = _nearest(x / torch.where(sc > 0, sc, 1.0), 1, 0, 6.0) * sc
    xi = _exact_turn(xi, pos, s, DI - c["rot"]).unflatten(-1, (4, 32))
    m, e = torch.frexp(xi.abs().amax(-1, keepdim=True) / 6)
    si = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    return kv.flatten(-2), (_nearest(xi / si, 1, 0, 6.0) * si).flatten(-2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    c = case
    if op == "rotate":
        return _exact_turn(s["x"], s["pos"][:, None].expand(c["tokens"], c["heads"]), s, c["first"], c["inverse"])
    if op == "window":
        codes, scale = s["codes"].double(), s["scale"].double()
        keep = slice(max(0, c["T"] - c["R"]), None)
        y = _exact_turn(s["x"][:, keep], s["pos"][:, keep], s, D - c["rot"])
        sc = (y.abs().amax(-1) / 448).float().double()  # as it is stored; the quotient is an fp32 one too
        for b in range(c["B"]):
            codes[b, s["pos"][b, keep].long() % c["R"]] = _nearest((y[b] / sc[b, :, None]).float().double(), 3, -6, 448.0)
            scale[b, s["pos"][b, keep].long() % c["R"]] = sc[b]
        return {"codes": codes, "scale": scale}
    nothing = {k: None for k in ("kv_codes", "kv_scales", "ix_codes", "ix_exponents", "num_entries")}
    if op in ("pack", "append"):
        r = c["ratio"]
        if op == "pack":
            n = c["T"] // r
            x, xi = (t[:, :n * r].double().unflatten(1, (n, r)).mean(2) for t in (s["lat_kv"], s["lat_ix"]))
            kv, ix = _exact_entries(s, x, xi, (c["first_entry"] + torch.arange(n, device=DEV)).expand(c["B"], n) * r)
            return {"kv": kv, "ix": ix, **nothing}
        new, p = torch.cat((s["lat_kv"], s["lat_ix"]), -1).double(), s["pos"].long()
        group = s["stage"].double().clone() if r > 1 else new[:, None]
        group[torch.arange(c["B"], device=DEV), p % r] = new
        x = group.mean(1)
        kv, ix = _exact_entries(s, x[:, :D], x[:, D:], p // r * r)
        done = (p % r == r - 1)[:, None]
        return {"kv": kv * done, "ix": ix * done, "stage": None, **nothing}
    return _exact_prefix(s)


def _exact_prefix(s):
    c = s["case"]
    codes, scales = s["planes"][0], s["planes"][1]
    o = torch.zeros((c["B"], c["Q"], H, D), dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["Q"], H), -math.inf, dtype=torch.float64, device=DEV)

    def values(b, n):
        if s["table"] is None:
            at = torch.arange(n.start, n.stop, device=DEV) + b * s["per"]
        else:
            i = torch.arange(n.start, n.stop, device=DEV)
            at = s["table"][b].long()[torch.div(i, c["page"], rounding_mode="floor")] * c["page"] + i % c["page"]
        k = codes[at].int()
        k = torch.stack((k % 16, k // 16), -1).flatten(1)
        e, m = (k // 2) % 4, (k % 2).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1).double()) * torch.where(k >= 8, -1.0, 1.0)
        return v * scales[at].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)

    shared = values(0, range(0, c["prefix"]))
    for b in range(c["B"]):
        count = int(s["num_entries"][b])
        all_of = torch.cat((shared, values(b, range(c["prefix"], count))))
        for i in range(c["Q"]):
            p = int(s["q_pos"][b, i])
            if p < 0:
                continue
            keys = all_of[:min(count, (p + 1) // c["ratio"])]
            if c["window"]:
                at = torch.arange(max(0, p - c["window"] + 1), p + 1, device=DEV) % s["R"]
                near = s["codes"][b, at].view(torch.float8_e4m3fn).double() * s["scale"][b, at].double()[:, None]
                keys = torch.cat((keys, near))
            if len(keys):
                x = s["q"][b, i].double() @ keys.T * s["tau"]
                lse[b, i] = torch.logsumexp(x, -1)
                o[b, i] = torch.softmax(x, -1) @ keys
    return {"o": o, "lse": lse}
