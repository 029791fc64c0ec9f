"""The operators around a KV cache held in 4 bits, as a serving step calls them.

Four operators, each with a plain form in elementary torch operations:

* ``qk``     RMS norm of every query and key head, then the rotary position
             embedding (half or interleaved layout, a part of the head, plain,
             linear, llama3 or yarn frequencies).
* ``append`` keys and values quantised to 4 bits as they are written into a
             paged cache, and read back at the same slots.
* ``read``   rows of a 4-bit paged cache read back to bf16, for a list of slots.
* ``attn``   causal grouped-query attention over a 4-bit paged cache: sequences
             with one or a few new tokens, prompt chunks, and both in one batch.

A 4-bit cache array is ``[num_blocks, n_kv, tile]`` bytes; a tile holds 16
tokens of one KV head: 4-bit e2m1 codes (``CODE`` bytes) and one e4m3 scale for
16 neighbouring elements of a token.  ``_places`` gives where the code and the
scale of (token, element) lie.  A value is code * scale * (a power of two for
the whole cache).
"""

import math

import torch

own = False

BLOCK = 16
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LLAMA3 = (8.0, 1.0, 4.0, 8192)       # factor, low_freq_factor, high_freq_factor, original positions
YARN = (4.0, 32.0, 1.0, 32768)       # factor, beta_fast, beta_slow, original positions
LINEAR = (4.0, 0.0, 0.0, 0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step's queries and keys: a Qwen3-MoE layer (32 query and 4 key heads), 64 sequences
        {"name": "qk_decode_64", "op": "qk", "tokens": 64, "nq": 32, "nkv": 4, "d": 128, "rot": 128, "inter": False,
         "scaling": "none", "theta": 1e7, "norm": True, "maxpos": 4096},
        # a prompt of 8 x 4096 tokens through the 70B layer's heads with llama3 frequencies
        {"name": "qk_prefill_32768", "op": "qk", "tokens": 32768, "nq": 64, "nkv": 8, "d": 128, "rot": 128,
         "inter": False, "scaling": "llama3", "theta": 5e5, "norm": True, "maxpos": 131072},
        # half of a 64-wide head rotated, interleaved pairs, yarn at far positions, an odd token count
        {"name": "qk_partial_1021", "op": "qk", "tokens": 1021, "nq": 8, "nkv": 2, "d": 64, "rot": 32, "inter": True,
         "scaling": "yarn", "theta": 1e4, "norm": True, "maxpos": 131072},
        # the new token of each of 128 sequences
        {"name": "append_decode_128", "op": "append", "tokens": 128, "nkv": 8, "d": 128, "skip": 0, "kexp": 0,
         "vexp": -2},
        # a prompt of 8 x 4096 tokens written at once
        {"name": "append_prefill_32768", "op": "append", "tokens": 32768, "nkv": 8, "d": 128, "skip": 0, "kexp": 0,
         "vexp": -2},
        # an odd number of cached rows of 64-wide heads, some of them padding (slot -1)
        {"name": "read_5003", "op": "read", "tokens": 5003, "nkv": 2, "d": 64, "skip": 7, "kexp": 1, "vexp": -3},
        # a whole long context handed on to another worker in bf16
        {"name": "read_131072", "op": "read", "tokens": 131072, "nkv": 8, "d": 128, "skip": 0, "kexp": 0, "vexp": 0},
        # the smallest call: one sequence, one token, a short context
        {"name": "attn_one_777", "op": "attn", "nq": 8, "nkv": 2, "d": 64, "dec": 1, "dec_new": 1, "dec_lo": 777,
         "dec_hi": 777, "pre": 0, "pre_new": 0, "pre_ctx": 0, "kexp": 0, "vexp": 0},
        # the 70B layer's decode batch: 128 sequences, contexts of 512 to 8192
        {"name": "attn_decode_128", "op": "attn", "nq": 64, "nkv": 8, "d": 128, "dec": 128, "dec_new": 1,
         "dec_lo": 512, "dec_hi": 8192, "pre": 0, "pre_new": 0, "pre_ctx": 0, "kexp": 0, "vexp": -2},
        # four sequences at up to 128K tokens, two draft tokens each to verify
        {"name": "attn_long_4", "op": "attn", "nq": 32, "nkv": 4, "d": 128, "dec": 4, "dec_new": 2, "dec_lo": 49152,
         "dec_hi": 131072, "pre": 0, "pre_new": 0, "pre_ctx": 0, "kexp": 0, "vexp": 0},
        # the 70B stack's batch: 32 decode sequences beside two prompt chunks of 2048 tokens
        {"name": "attn_mixed_70b", "op": "attn", "nq": 64, "nkv": 8, "d": 128, "dec": 32, "dec_new": 1,
         "dec_lo": 1024, "dec_hi": 16384, "pre": 2, "pre_new": 2048, "pre_ctx": 0, "kexp": 0, "vexp": -2},
        # odd chunks of 64-wide heads after an odd cached prefix
        {"name": "attn_chunk_64", "op": "attn", "nq": 8, "nkv": 2, "d": 64, "dec": 3, "dec_new": 1, "dec_lo": 65,
         "dec_hi": 2100, "pre": 3, "pre_new": 421, "pre_ctx": 1033, "kexp": 1, "vexp": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "append", "read", "attn", "attn", "attn"])
    nkv, group, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128, 128])
    if op == "qk":
        return {"op": op, "tokens": _log(rng, 1, 16384), "nq": nkv * group, "nkv": nkv, "d": d,
                "rot": rng.choice([16, 32, 48, 64] if d == 64 else [32, 64, 96, 128]), "inter": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "llama3", "yarn"]), "theta": rng.choice([1e4, 5e5, 1e7]),
                "norm": rng.random() < 0.75, "maxpos": rng.choice([1024, 131072, 1000000])}
    if op != "attn":
        return {"op": op, "tokens": _log(rng, 1, 32768), "nkv": nkv, "d": d, "skip": rng.choice([0, 0, 3, 11]),
                "kexp": rng.randint(-4, 4), "vexp": rng.randint(-6, 2)}
    dec, ctx = _log(rng, 1, 96), _log(rng, 1, 32768)
    while dec * ctx * nkv > 2_000_000:
        dec = max(1, dec // 2)
        ctx = ctx if dec > 1 else ctx // 2
    pre, new, before = rng.choice([0, 0, 1, 2, 3]), _log(rng, 2, 2000), rng.choice([0, 17, _log(rng, 1, 2000)])
    while pre * new * (new + before) * nkv * group * d > 2e10:
        new = new // 2
    return {"op": op, "nq": nkv * group, "nkv": nkv, "d": d, "dec": dec, "dec_new": rng.choice([1, 1, 1, 2, 3]),
            "dec_lo": max(3, ctx // rng.choice([1, 2, 8])), "dec_hi": max(3, ctx), "pre": pre,
            "pre_new": new if pre else 0, "pre_ctx": before if pre else 0,
            "kexp": rng.randint(-3, 3), "vexp": rng.randint(-4, 2)}


def _spread(n, lo, hi):
    """n lengths over [lo, hi], the same for every seed: work() has to know them."""
    return [lo + int((hi - lo) * ((0.5 + i * 0.6180339887) % 1.0)) if n > 1 else hi for i in range(n)]


def _lens(c):
    """(new tokens, total length) of every sequence: the decode group, then the prompt chunks."""
    return ([(min(c["dec_new"], n), n) for n in _spread(c["dec"], c["dec_lo"], c["dec_hi"])],
            [(c["pre_new"], c["pre_ctx"] + c["pre_new"])] * c["pre"])


def work(c):
    row = c["nkv"] * c["d"]
    if c["op"] == "qk":
        heads = c["nq"] + c["nkv"]
        return {"bytes": 4 * c["tokens"] * heads * c["d"] + 4 * c["tokens"] + 4 * c["d"],
                "flops": c["tokens"] * heads * (4 * c["d"] * c["norm"] + 3 * c["rot"])}
    if c["op"] in ("append", "read"):
        kept = c["tokens"] - (c["tokens"] // c["skip"] if c["skip"] else 0)
        quant, bf16 = 2 * row * kept * 9 // 16, 4 * row * kept
        if c["op"] == "read":
            return {"bytes": quant + bf16 + 4 * c["tokens"], "flops": 4 * row * kept}
        # read k and v, write the cache; read it again, write what it holds
        return {"bytes": 2 * quant + 2 * bf16 + 8 * c["tokens"], "flops": 12 * row * kept}
    byte, flop = 0, 0
    for new, total in _lens(c)[0] + _lens(c)[1]:
        byte += 2 * row * total * 9 // 16 + 4 * (-(-total // BLOCK)) + 4 * new * c["nq"] * c["d"]
        flop += 4 * c["nq"] * c["d"] * sum(range(total - new + 1, total + 1))
    return {"bytes": byte, "flops": flop}


# ---------------------------------------------------------------------------
# the 4-bit format
# ---------------------------------------------------------------------------
def _places(d, value, dev):
    """(byte of the code, its shift, byte of the scale) in a tile for every (token, element), flat [16 * d].

    Keys: token rows of d / 2 bytes.  Values: the lane order of the matrix
    instruction that contracts over tokens.  Element 2i is the low half of its
    byte."""
    key, e = torch.arange(BLOCK, device=dev)[:, None], torch.arange(d, device=dev)[None, :]
    half, row, grp = key // 8, key % 8, e // 16
    if value:
        w = d // 8
        code = half * 4 * d + ((e // w) * 4 + row // 2) * w + (key % 2) * (w // 2) + (e % w) // 2
        scale = (grp * 4 + row // 2) * 4 + half * 2 + key % 2
    else:
        per = d // 64
        code = key * (d // 2) + e // 2
        scale = (row * 4 + grp // per) * 2 * per + half * per + grp % per
    scale = scale + 8 * d
    return code.reshape(-1), ((e % 2) * 4).expand(BLOCK, d).reshape(-1), scale.reshape(-1)


def _tile_bytes(d):
    return 9 * d


def _decode(tiles, d, value, scale):
    """tiles [n, 9 d] uint8 -> [n, 16, d] fp32 values."""
    code, shift, at = _places(d, value, tiles.device)
    nib = (tiles.index_select(1, code) >> shift.to(torch.uint8)) & 15
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=tiles.device)
    s = tiles[:, 8 * d:].contiguous().view(torch.float8_e4m3fn).float().index_select(1, at - 8 * d)
    return (grid[nib.int()] * s * scale).view(-1, BLOCK, d)


def _quantise(x, scale):
    """x [..., d] bf16 -> (codes [..., d] uint8, scales [..., d / 16] uint8 bits).

    NaN counts as zero.  The scale of 16 neighbours is e4m3(amax / 6), the code
    the nearest of the grid (ties to the even code).  In 64 bits: values next to
    a border."""
    x = torch.nan_to_num(x.double() / scale, nan=0.0, posinf=math.inf, neginf=-math.inf)
    g = x.reshape(*x.shape[:-1], -1, 16)
    s8 = (g.abs().amax(-1) / 6).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    s = s8.double()[..., None]
    y = torch.where(s > 0, g.abs() / torch.where(s > 0, s, 1.0), 0.0)
    code = (y > 0.25).byte() + (y >= 0.75).byte() + (y > 1.25).byte() + (y >= 1.75).byte() + (y > 2.5).byte() \
        + (y >= 3.5).byte() + (y > 5.0).byte()
    code = code + 8 * (torch.signbit(g) & (s > 0)).byte()
    return code.reshape(x.shape), s8.view(torch.uint8)


def _store(cache, slots, x, d, value, scale):
    """x [n, n_kv, d] written at slots [n] of cache [blocks, n_kv, 9 d] (slots < 0 skipped)."""
    keep = slots >= 0
    slots, x = slots[keep].long(), x[keep]
    code, s = _quantise(x, scale)
    at, _, sat = _places(d, value, x.device)
    blk, tok = slots // BLOCK, slots % BLOCK
    heads = torch.arange(x.shape[1], device=x.device)[None, :, None]
    at = at.view(BLOCK, d)[tok][:, None, 0::2]
    sat = sat.view(BLOCK, d)[tok][:, None, 0::16]
    cache[blk[:, None, None], heads, at] = code[..., 0::2] | (code[..., 1::2] << 4)
    cache[blk[:, None, None], heads, sat] = s


def _rows(cache, slots, d, value, scale):
    """[n, n_kv, d] fp32 of the rows at slots [n] (all >= 0)."""
    slots = slots.long()
    at, shift, sat = (t.view(BLOCK, d)[slots % BLOCK][:, None] for t in _places(d, value, cache.device))
    heads = torch.arange(cache.shape[1], device=cache.device)[None, :, None]
    blk = (slots // BLOCK)[:, None, None]
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=cache.device)
    nib = (cache[blk, heads, at] >> shift.to(torch.uint8)) & 15
    return grid[nib.int()] * cache[blk, heads, sat].view(torch.float8_e4m3fn).float() * scale


# ---------------------------------------------------------------------------
# rotary frequencies
# ---------------------------------------------------------------------------
def _frequencies(c, dev):
    """[rot / 2] fp64 radians a position, and the factor on cos and sin."""
    rot, theta = c["rot"], c["theta"]
    inv = theta ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=dev) / rot)
    if c["scaling"] == "linear":
        return inv / LINEAR[0], 1.0
    if c["scaling"] == "llama3":
        f, low, high, orig = LLAMA3
        turns = orig * inv / (2 * math.pi)
        s = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        return (1 - s) * inv / f + s * inv, 1.0
    if c["scaling"] == "yarn":
        f, fast, slow, orig = YARN
        def at(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64, device=dev) - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    return inv, 1.0


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _keys(g, n, nkv, d):
    """Keys as a layer makes them: a few channels of every head far larger than the others."""
    big = 1.0 + 6.0 * (torch.rand(nkv, d, generator=g, device="cuda") > 0.95)
    return (_normal(g, n, nkv, d) * big).bfloat16()


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] == "qk":
        t, nq, nkv, d = c["tokens"], c["nq"], c["nkv"], c["d"]
        rows = _normal(g, t, nq + 2 * nkv, d).bfloat16()  # a projection's output, [q; k; v] a token
        st = {"op": "qk", "c": c, "q": rows[:, :nq], "k": rows[:, nq:nq + nkv], "eps": 1e-6,
              "pos": torch.randint(0, c["maxpos"], (t,), generator=g, device="cuda", dtype=torch.int32),
              "qw": (1 + 0.2 * _normal(g, d)).bfloat16() if c["norm"] else None,
              "kw": (1 + 0.2 * _normal(g, d)).bfloat16() if c["norm"] else None}
        st["q_out"], st["k_out"] = torch.empty_like(st["q"], memory_format=torch.contiguous_format), \
            torch.empty_like(st["k"], memory_format=torch.contiguous_format)
        if own:
            from llama_decoder_layer_gb300 import binding as lb
            scaling = {"none": None, "linear": {"rope_type": "linear", "factor": LINEAR[0]},
                       "llama3": {"rope_type": "llama3", "factor": LLAMA3[0], "low_freq_factor": LLAMA3[1],
                                  "high_freq_factor": LLAMA3[2], "original_max_position_embeddings": LLAMA3[3]},
                       "yarn": {"rope_type": "yarn", "factor": YARN[0], "beta_fast": YARN[1], "beta_slow": YARN[2],
                                "original_max_position_embeddings": YARN[3]}}[c["scaling"]]
            st["cfg"] = lb.QkNormRopeConfig(nq, nkv, d, rotary_dim=c["rot"], interleaved=c["inter"],
                                            rms_eps=st["eps"], rope_theta=c["theta"], rope_scaling=scaling)
        return st
    d, nkv = c["d"], c["nkv"]
    ks, vs = 2.0 ** c["kexp"], 2.0 ** c["vexp"]
    if c["op"] in ("append", "read"):
        n = c["tokens"]
        blocks = -(-n // BLOCK) * 5 // 4 + 2
        slots = torch.randperm(blocks, generator=g, device="cuda")[:-(-n // BLOCK), None] * BLOCK
        slots = (slots + torch.arange(BLOCK, device="cuda")).reshape(-1)[:n].int()  # block by block, as tables give them
        if c["skip"]:
            slots[c["skip"] - 1::c["skip"]] = -1
        k, v = _keys(g, n, nkv, d) * ks, (_normal(g, n, nkv, d) * vs).bfloat16()
        st = {"op": c["op"], "d": d, "slots": slots, "ks": ks, "vs": vs,
              "kc": torch.zeros(blocks, nkv, _tile_bytes(d), dtype=torch.uint8, device="cuda"),
              "vc": torch.zeros(blocks, nkv, _tile_bytes(d), dtype=torch.uint8, device="cuda"),
              "k_out": torch.zeros(n, nkv, d, dtype=torch.bfloat16, device="cuda"),
              "v_out": torch.zeros(n, nkv, d, dtype=torch.bfloat16, device="cuda")}
        if c["op"] == "append":
            st["k"], st["v"] = k, v
        else:
            _store(st["kc"], slots, k, d, False, ks)
            _store(st["vc"], slots, v, d, True, vs)
        return st
    nq, groups = c["nq"], _lens(c)
    seqs = groups[0] + groups[1]
    nblk = [-(-t // BLOCK) for _, t in seqs]
    blocks = sum(nblk) + 8
    perm = torch.randperm(blocks, generator=g, device="cuda").int()
    table = torch.full((len(seqs), max(nblk)), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max(nblk), device="cuda") < torch.tensor(nblk, device="cuda")[:, None]] = perm[:sum(nblk)]
    # slots that no token was written to hold whatever the memory held
    kc, vc = (torch.randint(0, 256, (blocks, nkv, _tile_bytes(d)), generator=g, device="cuda", dtype=torch.uint8)
              for _ in range(2))
    total = torch.tensor([t for _, t in seqs], device="cuda")
    at = torch.arange(int(total.max()), device="cuda").expand(len(seqs), -1)
    slots = (table.gather(1, at // BLOCK) * BLOCK + at % BLOCK)[at < total[:, None]]
    _store(kc, slots, _keys(g, slots.numel(), nkv, d) * ks, d, False, ks)
    _store(vc, slots, (_normal(g, slots.numel(), nkv, d) * vs).bfloat16(), d, True, vs)
    q_lens = [n for n, _ in seqs]
    pos = [p for n, t in seqs for p in range(t - n, t)]
    start = [sum(q_lens[:b]) for b in range(len(q_lens) + 1)]
    i32 = dict(dtype=torch.int32, device="cuda")
    q = (_normal(g, start[-1], nq, d)).bfloat16()
    st = {"op": "attn", "c": c, "kc": kc, "vc": vc, "q": q, "table": table, "ks": ks, "vs": vs,
          "pos": torch.tensor(pos, **i32), "lens": torch.tensor([t for _, t in seqs], **i32),
          "start": torch.tensor(start, **i32), "out": torch.empty(start[-1], nq * d, dtype=torch.bfloat16, device="cuda")}
    if own:
        from llama_decoder_layer_gb300 import binding as lb
        st["cfg"] = lb.LayerConfig(nq * d, nq, nkv, d, 4 * nq * d, 1e-5, 1e4)
        st["batch"] = lb.Batch(st["pos"], st["start"], st["lens"], table, blocks, max(q_lens), max(t for _, t in seqs))
        st["prefill_blocks"] = lb.prefill_blocks(q_lens, [t for _, t in seqs], nq // nkv)
        st["ws"] = lb.alloc_workspace(lb.paged_attention_q4_workspace_size(
            st["cfg"], start[-1], len(seqs), st["batch"].max_seq_len, st["prefill_blocks"]))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "qk":
        return _qk(st["c"], st["q"], st["qw"], st["pos"], st["eps"]), _qk(st["c"], st["k"], st["kw"], st["pos"], st["eps"])
    if st["op"] == "attn":
        return _attend(st)
    if st["op"] == "append":
        _store(st["kc"], st["slots"], st["k"], st["d"], False, st["ks"])
        _store(st["vc"], st["slots"], st["v"], st["d"], True, st["vs"])
    keep = st["slots"] >= 0
    st["k_out"][keep] = _rows(st["kc"], st["slots"][keep], st["d"], False, st["ks"]).bfloat16()
    st["v_out"][keep] = _rows(st["vc"], st["slots"][keep], st["d"], True, st["vs"]).bfloat16()
    return st["k_out"], st["v_out"]


def _run_own(st):
    from llama_decoder_layer_gb300 import binding as lb
    if st["op"] == "qk":
        lb.qk_norm_rope(st["cfg"], st["qw"], st["kw"], st["pos"], st["q"], st["k"], st["q_out"], st["k_out"])
        return st["q_out"], st["k_out"]
    if st["op"] == "attn":
        lb.paged_attention_q4(st["cfg"], st["batch"], st["q"], st["kc"], st["vc"], st["out"], st["ws"],
                              k_scale=st["ks"], v_scale=st["vs"], prefill_blocks=st["prefill_blocks"])
        return st["out"]
    if st["op"] == "append":
        lb.kv_cache_write_q4(st["k"], st["v"], st["slots"], st["kc"], st["vc"], k_scale=st["ks"], v_scale=st["vs"])
    lb.kv_cache_read_q4(st["kc"], st["vc"], st["slots"], st["k_out"], st["v_out"], k_scale=st["ks"], v_scale=st["vs"])
    return st["k_out"], st["v_out"]


def _qk(c, x, w, pos, eps):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    inv, factor = _frequencies(c, x.device)
    angle = pos.double()[:, None] * inv  # far positions
    cos, sin = (angle.cos() * factor).float()[:, None], (angle.sin() * factor).float()[:, None]
    r = c["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :r // 2], x[..., r // 2:r])
    out = x.clone()
    if c["inter"]:
        out[..., 0:r:2], out[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        out[..., :r // 2], out[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    return out.bfloat16()


def _group(st, first, n, t0):
    """The attention of sequences [first, first + n), the same number of new tokens each, from token t0 on."""
    c = st["c"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    new = (c["dec_new"] if first == 0 and c["dec"] else c["pre_new"]) if n else 0
    if n == 0:
        return st["q"].new_zeros(0, nq * d), t0
    total = st["lens"][first:first + n]
    blocks = -(-max(t for _, t in (_lens(c)[0] if first == 0 and c["dec"] else _lens(c)[1])) // BLOCK)
    table = st["table"][first:first + n, :blocks].clamp(min=0).long()

    def rows(cache, value, scale):
        x = _decode(cache[table].reshape(-1, _tile_bytes(d)), d, value, scale)
        x = x.view(n, blocks, nkv, BLOCK, d).transpose(1, 2).reshape(n, nkv, blocks * BLOCK, d)
        there = torch.arange(blocks * BLOCK, device=x.device) < total[:, None]
        return torch.where(there[:, None, :, None], x, 0.0)

    q = st["q"][t0:t0 + n * new].float().view(n, new, nkv, nq // nkv, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(n, nkv, -1, d)
    s = q @ rows(st["kc"], False, st["ks"]).transpose(-1, -2) / math.sqrt(d)
    s = s.view(n, nkv, nq // nkv, new, -1)
    seen = torch.arange(s.shape[-1], device=s.device) <= st["pos"][t0:t0 + n * new].view(n, 1, 1, new, 1)
    s = torch.where(seen, s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.view(n, nkv, -1, p.shape[-1]) @ rows(st["vc"], True, st["vs"])
    o = o.view(n, nkv, nq // nkv, new, d).permute(0, 3, 1, 2, 4).reshape(n * new, nq * d)
    return o.bfloat16(), t0 + n * new


def _attend(st):
    a, t0 = _group(st, 0, st["c"]["dec"], 0)
    b, _ = _group(st, st["c"]["dec"], st["c"]["pre"], t0)
    return torch.cat([a, b])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(cache, block, token, d, value, scale):
    """One [n, d] fp64 array for n (block, token) pairs of one head, from the bits of the format."""
    e = torch.arange(d, device=cache.device)
    half, low, w = token[:, None] >> 3, token[:, None] & 7, d // 8
    if value:
        byte = half * 4 * d + ((e // w) * 4 + (low >> 1)) * w + (low & 1) * (w >> 1) + ((e % w) >> 1)
        where = ((e >> 4) * 4 + (low >> 1)) * 4 + half * 2 + (low & 1)
    else:
        byte = token[:, None] * (d >> 1) + (e >> 1)
        per = d // 64
        where = (low * 4 + (e >> 4) // per) * (2 * per) + half * per + (e >> 4) % per
    raw = cache[block[:, None], byte].long()
    nib = torch.where(e % 2 == 1, raw >> 4, raw & 15)
    ee, m = (nib >> 1) & 3, nib & 1
    mag = torch.where(ee > 0, (1.0 + 0.5 * m) * torch.exp2((ee - 1).double()), 0.5 * m)
    sb = cache[block[:, None], 8 * d + where].long()
    se, sm = (sb >> 3) & 15, sb & 7
    s = torch.where(se > 0, (1.0 + sm / 8.0) * torch.exp2((se - 7).double()), sm / 512.0)
    return torch.where(nib >= 8, -mag, mag) * s * scale


def _exact_store(x, scale):
    """The values that a 4-bit row of x [..., d] stands for, in fp64."""
    g = x.double().reshape(*x.shape[:-1], -1, 16) / scale
    top = g.abs().amax(-1, keepdim=True) / 6.0
    e = (torch.frexp(top.clamp(min=2.0 ** -6)).exponent - 1).double()  # e4m3: four bits, exponents from -6
    s = (torch.round(top / torch.exp2(e - 3)) * torch.exp2(e - 3)).clamp(max=448.0)
    y = torch.where(s > 0, g / torch.where(s > 0, s, 1.0), 0.0)
    a = y.abs()
    ulp = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))  # e2m1: two bits
    return (torch.sign(y) * (torch.round(a / ulp) * ulp).clamp(max=6.0) * s * scale).reshape(x.shape)


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "qk":
        return _exact_qk(c, st["q"], st["qw"], st), _exact_qk(c, st["k"], st["kw"], st)
    if c["op"] in ("append", "read"):
        keep = st["slots"] >= 0
        outs = []
        for name, value, scale in (("k", False, st["ks"]), ("v", True, st["vs"])):
            out = torch.zeros(st["k_out"].shape, dtype=torch.float64, device="cuda")
            if c["op"] == "append":
                out[keep] = _exact_store(st[name][keep], scale)
            else:
                slots = st["slots"][keep].long()
                for h in range(c["nkv"]):
                    out[keep, h] = _exact_rows(st[name + "c"][:, h], slots // BLOCK, slots % BLOCK, c["d"], value, scale)
            outs.append(out)
        return tuple(outs)
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    out = torch.zeros(st["q"].shape[0], nq, d, dtype=torch.float64, device="cuda")
    t0, seqs = 0, _lens(c)[0] + _lens(c)[1]
    for b, (new, total) in enumerate(seqs):
        at = torch.arange(total, device="cuda")
        block, token = st["table"][b].long()[at // BLOCK], at % BLOCK
        for h in range(nkv):
            k = _exact_rows(st["kc"][:, h], block, token, d, False, st["ks"])
            v = _exact_rows(st["vc"][:, h], block, token, d, True, st["vs"])
            heads = slice(h * (nq // nkv), (h + 1) * (nq // nkv))
            x = st["q"][t0:t0 + new, heads].double().reshape(-1, d)
            s = (x @ k.T) * d ** -0.5
            last = st["pos"][t0:t0 + new].long().repeat_interleave(nq // nkv)
            s = s.masked_fill(at[None] > last[:, None], -math.inf)
            out[t0:t0 + new, heads] = ((s - s.logsumexp(-1, keepdim=True)).exp() @ v).view(new, -1, d)
        t0 += new
    return out.view(-1, nq * d)


def _exact_frequencies(c):
    """Radians a position of each rotated pair, by the rules one pair at a time."""
    found = []
    for i in range(c["rot"] // 2):
        f = math.exp(-math.log(c["theta"]) * 2 * i / c["rot"])
        if c["scaling"] == "linear":
            f = f / LINEAR[0]
        elif c["scaling"] == "llama3":
            by, low, high, orig = LLAMA3
            wave = 2 * math.pi / f
            if wave > orig / low:
                f = f / by
            elif wave >= orig / high:
                smooth = (orig / wave - low) / (high - low)
                f = (1 - smooth) * f / by + smooth * f
        elif c["scaling"] == "yarn":
            by, fast, slow, orig = YARN
            first, last = (c["rot"] / 2 * math.log(orig / (2 * math.pi * b), c["theta"]) for b in (fast, slow))
            first, last = max(0, math.floor(first)), min(c["rot"] - 1, math.ceil(last))
            kept = 1.0 - min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            f = f * kept + f / by * (1.0 - kept)
        found.append(f)
    return found


def _exact_qk(c, x, w, st):
    x = x.double()
    if w is not None:
        x = x / (x.square().sum(-1, keepdim=True) / c["d"] + st["eps"]).sqrt() * w.double()
    r, i = c["rot"], torch.arange(c["rot"] // 2, device=x.device)
    freq, factor = torch.tensor(_exact_frequencies(c), dtype=torch.float64, device=x.device), 1.0
    if c["scaling"] == "yarn":
        factor = 1.0 + math.log(YARN[0]) / 10
    turn = torch.polar(torch.full((x.shape[0], r // 2), factor, dtype=torch.float64, device=x.device),
                       st["pos"].double()[:, None] * freq)[:, None]
    first, second = (2 * i, 2 * i + 1) if c["inter"] else (i, i + r // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out
