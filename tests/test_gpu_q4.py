"""The operators around the 4-bit KV cache on the GPU, against their plain
64-bit forms: quantised rows bit for bit, the head norm with rotation and the
attention within the rounding of their types.

Tolerances.  A bf16 result is rounded once: 2^-8 of its size (half a step).
* norm and rotation: before that, fp32 arithmetic on values of size |a| + |b|
  (the pair): the sum of 128 squares, rsqrt, three products and the angle (2^-21
  radian) stay below 2^-18 of that size.
* attention: a weight p is used with a relative error eps_p: 2^-11 where it is
  stored as fp16, 2^-8 as bf16 (a prompt's path), and the scores' fp32 error, at
  most 2^-12 for |score| < 2^9 with sums of 128 products, so the result is off
  by at most 2^-8 |o| + 2 (eps_p + 2^-12) sum p |v| (numerator and denominator).
  fp16 weights are stored as 2^(s - m + 6), m a maximum that is never above the
  largest score s_max: the largest weight is at least 2^6, and one below fp16's
  normal range is off by up to half its smallest number, 2^-25, which is 2^-31 of
  the largest.  The largest, normalised, is at most 1, so this adds at most 2^-31
  sum |v| over the keys seen.
"""

import numpy as np
import pytest
import torch

import q4_reference as R
from llama_decoder_layer_gb300 import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ok():
    st, detail = lb.get_device_error()
    assert st == lb.LLAMA_OK, (lb.status_string(st), detail)


def guard():
    assert lb.get_device_error()[0] == lb.LLAMA_ERR_DEVICE_GUARD


def f64(t):
    return t.detach().double().cpu().numpy()


def caches(blocks, nkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, 256, (2, blocks, nkv, lb.kv_cache_q4_tile_bytes(d)), generator=g, dtype=torch.uint8)
    return t[0].to(DEV), t[1].to(DEV)


# ---------------------------------------------------------------------------
# writing and reading the cache
# ---------------------------------------------------------------------------
def hard_rows(n, nkv, d, seed, g):
    """bf16 rows that meet the quantisation's borders: exact ties, equal values, tiny and huge groups, zeros, both
    signs, infinities and NaN."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, nkv, d // 16, 16)) * 2.0 ** r.integers(-14, 12, (n, nkv, d // 16, 1))
    kind = r.integers(0, 8, (n, nkv, d // 16))
    grid = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    tie = grid[r.integers(0, len(grid), x.shape)] * np.where(r.random(x.shape) < 0.5, -1, 1)
    tie[..., 0] = 6.0
    x = np.where(kind[..., None] == 0, tie * 2.0 ** r.integers(-6, 8, kind.shape)[..., None], x)
    x = np.where(kind[..., None] == 1, 0.0, x)
    x = np.where(kind[..., None] == 2, x[..., :1], x)  # all equal
    odd = r.random(x.shape) < 0.05
    x = np.where((kind[..., None] == 3) & odd, np.inf, x)
    x = np.where((kind[..., None] == 4) & odd, np.nan, x)
    x = np.where(kind[..., None] == 5, x * 2.0 ** -12, x)
    return (torch.from_numpy(x.reshape(n, nkv, d)) * g).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,nkv", [(1, 1), (5, 3), (16, 8), (37, 2), (300, 5), (9, 64), (40, 33), (3, 70), (5300, 8), (20011, 3)])
@pytest.mark.parametrize("kexp,vexp", [(0, 0), (-5, 3)])
def test_write_and_read_bit_for_bit(d, T, nkv, kexp, vexp):
    blocks = T // 16 + 4
    kg, vg = 2.0 ** kexp, 2.0 ** vexp
    k, v = hard_rows(T, nkv, d, T + d, kg), hard_rows(T, nkv, d, T + d + 1, vg)
    slots = torch.randperm(blocks * 16, generator=torch.Generator().manual_seed(T))[:T].int()
    slots[2::5] = -1
    kc, vc = caches(blocks, nkv, d)
    want = [kc.cpu().numpy().copy(), vc.cpu().numpy().copy()]
    lb.kv_cache_write_q4(k.to(DEV), v.to(DEV), slots.to(DEV), kc, vc, kg, vg)
    for tiles, x, g, is_v in ((want[0], k, kg, False), (want[1], v, vg, True)):
        R.pack_rows(tiles, slots.tolist(), *R.quantise(f64(x), g), d, is_v)
    # every byte, those of other tokens included
    assert np.array_equal(kc.cpu().numpy(), want[0])
    assert np.array_equal(vc.cpu().numpy(), want[1])
    ko = torch.full((T, nkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vo = torch.full((T, nkv, d), 9.0, dtype=torch.bfloat16, device=DEV)
    lb.kv_cache_read_q4(kc, vc, slots.to(DEV), ko, vo, kg, vg)
    ok()
    keep = slots.numpy() >= 0
    for out, tiles, g, is_v, old in ((ko, want[0], kg, False, 7.0), (vo, want[1], vg, True, 9.0)):
        out = f64(out)
        assert np.all(out[~keep] == old)
        assert np.array_equal(out[keep], R.cache_rows(tiles, slots.numpy()[keep], d, is_v, g))


def test_write_from_and_read_into_columns_of_wider_rows():
    T, nq, nkv, d = 21, 8, 2, 64
    rows = torch.randn(T, nq + 2 * nkv, d, device=DEV).bfloat16()
    k, v = rows[:, nq:nq + nkv], rows[:, nq + nkv:]
    slots = torch.randperm(64, device=DEV)[:T].int()
    a, b = caches(4, nkv, d), caches(4, nkv, d)
    lb.kv_cache_write_q4(k, v, slots, *a)
    lb.kv_cache_write_q4(k.contiguous(), v.contiguous(), slots, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = torch.full((T, nq + 2 * nkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
    lb.kv_cache_read_q4(*a, slots, wide[:, nq:nq + nkv], wide[:, nq + nkv:])
    ko, vo = torch.empty_like(k.contiguous()), torch.empty_like(v.contiguous())
    lb.kv_cache_read_q4(*a, slots, ko, vo)
    ok()
    assert torch.equal(wide[:, nq:nq + nkv], ko) and torch.equal(wide[:, nq + nkv:], vo)
    assert bool((wide[:, :nq] == 3.0).all())


def test_bad_slots_are_reported_and_left():
    T, nkv, d, blocks = 6, 2, 128, 3
    k = torch.randn(T, nkv, d, device=DEV).bfloat16()
    kc, vc = caches(blocks, nkv, d)
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.tensor([48, 1 << 30, 2 ** 31 - 1, -1, -(2 ** 31), 5], dtype=torch.int32, device=DEV)
    lb.kv_cache_write_q4(k, k, slots, kc, vc)
    guard()
    only = torch.tensor([5], dtype=torch.int32, device=DEV)
    lb.kv_cache_write_q4(k[5:], k[5:], only, k0, v0)
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    out = torch.full((T, nkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lb.kv_cache_read_q4(kc, vc, slots, out, out.clone())
    guard()
    assert bool((out[:5] == 7.0).all()) and not bool((out[5] == 7.0).all())


def test_a_slot_may_be_read_more_than_once():
    kc, vc = caches(2, 3, 64)
    one = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    k1, v1 = (torch.empty(1, 3, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k9, v9 = (torch.empty(50, 3, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kw = torch.randn(1, 3, 64, device=DEV).bfloat16()
    lb.kv_cache_write_q4(kw, kw, one, kc, vc)
    lb.kv_cache_read_q4(kc, vc, one, k1, v1)
    lb.kv_cache_read_q4(kc, vc, one.expand(50).contiguous(), k9, v9)
    ok()
    assert torch.equal(k9, k1.expand(50, -1, -1)) and torch.equal(v9, v1.expand(50, -1, -1))


# ---------------------------------------------------------------------------
# norm and rotation of the heads
# ---------------------------------------------------------------------------
LLAMA3 = {"rope_type": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
          "original_max_position_embeddings": 8192}
YARN = {"rope_type": "yarn", "factor": 4.0, "original_max_position_embeddings": 32768}


def check_qk(got, x, w, pos, cfg):
    rot = cfg.head_dim if cfg.rotary_dim is None else cfg.rotary_dim
    want, size = R.norm_rope(f64(x), None if w is None else f64(w), pos.cpu().numpy(), rot, cfg.interleaved,
                             np.float32(cfg.rms_eps).astype(np.float64), cfg.rope_theta, cfg.rope_scaling)
    err = np.abs(f64(got) - want)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size
    assert np.all(err <= tol), float(np.max(err - tol))


@pytest.mark.parametrize("T", [1, 7, 200])
@pytest.mark.parametrize("nq,nkv,d,rot", [(8, 2, 64, 64), (1, 1, 128, 128), (32, 4, 128, 128), (5, 1, 64, 16),
                                          (6, 3, 128, 48), (2, 2, 64, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scaling", [None, {"rope_type": "linear", "factor": 4.0}, LLAMA3, YARN])
def test_norm_rope(T, nq, nkv, d, rot, inter, scaling):
    g = torch.Generator(device=DEV).manual_seed(T + nq + rot)
    rows = (torch.randn(T, nq + 2 * nkv, d, generator=g, device=DEV) * 3).bfloat16()
    q, k = rows[:, :nq], rows[:, nq:nq + nkv]
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    pos[0] = 0
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g, device=DEV)).bfloat16() for _ in range(2))
    cfg = lb.QkNormRopeConfig(nq, nkv, d, rot, inter, 1e-5, 1e6, scaling)
    for a, b in ((qw, kw), (None, kw), (None, None)):
        qo, ko = (torch.empty(T, n, d, dtype=torch.bfloat16, device=DEV) for n in (nq, nkv))
        lb.qk_norm_rope(cfg, a, b, pos if rot else None, q, k, qo, ko)
        ok()
        check_qk(qo, q, a, pos, cfg)
        check_qk(ko, k, b, pos, cfg)
    # in place, inside the merged rows; the values between stay
    v = rows[:, nq + nkv:].clone()
    lb.qk_norm_rope(cfg, qw, kw, pos, q, k, q, k)
    qo2, ko2 = torch.empty_like(qo), torch.empty_like(ko)
    rows2 = (torch.randn(T, nq + 2 * nkv, d, generator=torch.Generator(device=DEV).manual_seed(T + nq + rot),
                         device=DEV) * 3).bfloat16()
    lb.qk_norm_rope(cfg, qw, kw, pos, rows2[:, :nq], rows2[:, nq:nq + nkv], qo2, ko2)
    ok()
    assert torch.equal(rows[:, :nq], qo2) and torch.equal(rows[:, nq:nq + nkv], ko2)
    assert torch.equal(rows[:, nq + nkv:], v)


def test_norm_rope_far_positions():
    # the angle's error: 2^-24 of a revolution and the position times 2^-48
    pos = torch.tensor([(1 << 24) - 1, (1 << 24) + 1, 123456789, 2 ** 31 - 1, -5], dtype=torch.int32, device=DEV)
    q = torch.randn(5, 4, 64, device=DEV).bfloat16()
    k = torch.randn(5, 1, 64, device=DEV).bfloat16()
    cfg = lb.QkNormRopeConfig(4, 1, 64, rope_theta=1e4)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    lb.qk_norm_rope(cfg, None, None, pos, q, k, qo, ko)
    ok()
    want, size = R.norm_rope(f64(q), None, pos.cpu().numpy(), 64, False, 0.0, 1e4, None)
    assert np.all(np.abs(f64(qo) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -18 + 2.0 ** 31 * 2.0 ** -48 * 8) * size)


def test_norm_rope_of_zero_and_huge_rows():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.full((2, 1, 128), 2.0 ** 50, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    cfg = lb.QkNormRopeConfig(4, 1, 128)
    pos = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    lb.qk_norm_rope(cfg, w, w, pos, q, k, q, k)
    ok()
    assert bool((q == 0).all())
    check_qk(k, torch.full((2, 1, 128), 2.0 ** 50, dtype=torch.bfloat16), w, pos, cfg)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Case:
    """A batch of (new tokens, total length) sequences over random 4-bit caches; slots past a sequence's end hold
    random bytes, NaN scales among them."""

    def __init__(self, seqs, nq, nkv, d, seed=0, kg=1.0, vg=1.0, extra_tokens=0, qmul=1.0, bound=0):
        r = np.random.default_rng(seed)
        self.seqs, self.nq, self.nkv, self.d, self.kg, self.vg = seqs, nq, nkv, d, kg, vg
        nblk = [-(-t // 16) for _, t in seqs]
        blocks = sum(nblk) + 3
        perm = r.permutation(blocks)
        self.table = np.full((len(seqs), max(nblk)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(nblk):
            self.table[b, :n] = perm[at:at + n]
            at += n
        tiles = r.integers(0, 256, (2, blocks, nkv, 9 * d), dtype=np.uint8)
        slots = np.concatenate([[self.table[b][j // 16] * 16 + j % 16 for j in range(t)]
                                for b, (_, t) in enumerate(seqs)]).astype(np.int64)
        for i, (g, is_v) in enumerate(((kg, False), (vg, True))):
            x = r.standard_normal((len(slots), nkv, d)) * g
            x[..., :3] *= 1 if is_v else 6
            R.pack_rows(tiles[i], slots, *R.quantise(x, g), d, is_v)
        self.tiles = tiles
        self.qsl = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        self.pos = np.concatenate([np.arange(t - n, t) for n, t in seqs] + [np.zeros(extra_tokens)]).astype(np.int32)
        T = len(self.pos)
        self.q = torch.from_numpy(r.standard_normal((T, nq, d)) * qmul).to(torch.bfloat16)
        self.cfg = lb.LayerConfig(nq * d, nq, nkv, d, 4 * nq * d, 1e-5, 1e4)
        t32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)  # noqa: E731
        self.batch = lb.Batch(t32(self.pos), t32(self.qsl), t32([t for _, t in seqs]), t32(self.table), blocks,
                              max(n for n, _ in seqs), max(bound, max(t for _, t in seqs)))
        self.pre = lb.prefill_blocks([n for n, _ in seqs], [t for _, t in seqs], nq // nkv)
        self.kc, self.vc = (torch.from_numpy(t).to(DEV) for t in tiles)
        self.qd = self.q.to(DEV)
        self.ws = lb.alloc_workspace(lb.paged_attention_q4_workspace_size(
            self.cfg, T, len(seqs), self.batch.max_seq_len, self.pre))
        self.out = torch.full((T, nq * d), 5.0, dtype=torch.bfloat16, device=DEV)

    def run(self, **kw):
        a = dict(batch=self.batch, q=self.qd, out=self.out, ws=self.ws, pre=self.pre)
        a.update(kw)
        lb.paged_attention_q4(self.cfg, a["batch"], a["q"], self.kc, self.vc, a["out"], a["ws"], self.kg, self.vg,
                              a["pre"])
        return a["out"]

    def check(self, out=None):
        T = int(self.qsl[-1])
        got = f64(self.out if out is None else out).reshape(-1, self.nq, self.d)
        want, spread, flat = R.attention(f64(self.q)[:T], self.pos, self.qsl, self.table, self.tiles[0], self.tiles[1],
                                   self.kg, self.vg)
        new = np.concatenate([np.full(n, n) for n, _ in self.seqs])
        eps_p = np.where((new > 1) & (new * (self.nq // self.nkv) > 16), 2.0 ** -8, 2.0 ** -11)[:, None, None]
        err = np.abs(got[:T] - want)
        tol = 2.0 ** -8 * np.abs(want) + 2 * (eps_p + 2.0 ** -12) * spread + 2.0 ** -31 * flat
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(err)))
        assert np.all(got[T:] == 5.0)  # rows behind the last sequence


HEADS = [(8, 2, 64), (64, 8, 128), (1, 1, 128), (16, 1, 64), (5, 1, 128), (12, 2, 128), (24, 2, 64), (3, 3, 64)]


# max_seq_len, the bound the caller gives: up to 1024 a (sequence, KV head) stays whole, above it may be split
BOUNDS = [0, 5000]


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("nq,nkv,d", HEADS)
def test_attention_one_token_each(nq, nkv, d, bound):
    c = Case([(1, n) for n in (1, 2, 15, 16, 17, 33, 64, 65, 100, 257, 530)], nq, nkv, d, seed=d + nq, bound=bound)
    c.run()
    ok()
    c.check()


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("nq,nkv,d", HEADS)
def test_attention_a_few_new_tokens(nq, nkv, d, bound):
    c = Case([(n, n + p) for n, p in ((2, 0), (3, 14), (1, 40), (2, 301), (4, 77), (16, 5))], nq, nkv, d, seed=d + nq,
             bound=bound)
    c.run()
    ok()
    c.check()


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("nq,nkv,d", HEADS)
def test_attention_prompts_and_single_tokens_in_one_batch(nq, nkv, d, bound):
    c = Case([(1, 70), (33, 33), (1, 1), (70, 201), (17, 18), (2, 400), (129, 130), (1, 300)], nq, nkv, d, seed=nq,
             bound=bound)
    c.run()
    ok()
    c.check()


@pytest.mark.parametrize("nq,nkv,d", HEADS)
@pytest.mark.parametrize("seqs", [[(70, 900), (1, 60), (33, 400), (18, 131)], [(20, 5000)], [(600, 1300), (2, 9)]])
def test_attention_few_prompt_rows_over_many_keys(nq, nkv, d, seqs):
    # (head shapes off the tensor-memory kernel: the keys of a tile split over several CTAs, some without any)
    c = Case(seqs, nq, nkv, d, seed=nq + d)
    c.run()
    ok()
    c.check()


@pytest.mark.parametrize("nq,nkv,d,lens", [(32, 4, 128, (20000, 3, 9000)), (8, 8, 64, (30001,)), (64, 8, 128, (5000, 1))])
def test_attention_long_contexts(nq, nkv, d, lens):
    c = Case([(1, n) for n in lens], nq, nkv, d, seed=3)
    c.run()
    ok()
    c.check()


def test_attention_many_short_sequences():
    r = np.random.default_rng(5)
    c = Case([(1, int(n)) for n in r.integers(1, 60, 700)], 8, 2, 64, seed=6)
    c.run()
    ok()
    c.check()


@pytest.mark.parametrize("kexp,vexp,qmul", [(-6, 5, 1.0), (4, -9, 2.0 ** -40), (0, 0, 3e-38), (-3, 0, 30.0)])
def test_attention_scales_and_query_sizes(kexp, vexp, qmul):
    c = Case([(1, 90), (2, 45), (40, 60)], 16, 2, 128, seed=8, kg=2.0 ** kexp, vg=2.0 ** vexp, qmul=qmul)
    c.run()
    ok()
    c.check()


def test_attention_when_one_key_takes_all_the_weight():
    # scores far apart: the running maximum jumps late, early keys lose all weight
    c = Case([(1, 700), (1, 64)], 8, 1, 128, seed=9, kg=16.0, qmul=2.0)
    c.run()
    ok()
    c.check()


def test_rows_behind_the_last_sequence_stay():
    for seqs in ([(1, 40), (1, 3)], [(1, 40), (50, 60)]):
        c = Case(seqs, 8, 2, 64, extra_tokens=5)
        c.run()
        ok()
        c.check()


@pytest.mark.parametrize("bound", BOUNDS)
def test_a_sequence_without_new_tokens_is_passed_over(bound):
    c = Case([(1, 40), (0, 77), (1, 3), (0, 5), (20, 31), (0, 16)], 8, 2, 64, bound=bound)
    c.run()
    ok()
    c.check()


@pytest.mark.parametrize("bound", BOUNDS)
def test_bad_positions_lengths_and_blocks_are_reported(bound):
    for new in (1, 30):
        for what in ("past", "negative", "long", "blocks"):
            c = Case([(new, 40), (new, 100), (new, 60)], 8, 2, 128, seed=11, bound=bound)
            if what == "past":
                c.batch.positions[c.qsl[2] - 1] = 100
            elif what == "negative":
                c.batch.positions[c.qsl[1]:c.qsl[2]] = -1
            elif what == "long":
                c.batch.seq_lens[1] = 100000
                c.batch.positions[c.qsl[2] - 1] = 99999
            else:
                c.batch.block_table[1, 2] = 1 << 20
            c.run()
            guard()
            # the other sequences' rows are right
            got, want = f64(c.out).reshape(-1, 8, 128), R.attention(
                f64(c.q), c.pos, c.qsl, c.table, c.tiles[0], c.tiles[1], 1.0, 1.0)[0]
            rest = np.r_[0:c.qsl[1], c.qsl[2]:c.qsl[3]]
            assert np.abs(got[rest] - want[rest]).max() < 0.05 * np.abs(want).max(), (new, what)


@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 64), (8, 2, 128), (5, 1, 128)])
@pytest.mark.parametrize("new,at", [(30, 7), (300, 299)])
def test_one_negative_position_in_a_longer_sequence(nq, nkv, d, new, at):
    c = Case([(1, 40), (new, new + 17), (1, 60)], nq, nkv, d, seed=20)
    c.batch.positions[1 + at] = -1
    c.run()
    guard()
    got = f64(c.out).reshape(-1, nq, d)
    want, spread, flat = R.attention(f64(c.q), c.pos, c.qsl, c.table, c.tiles[0], c.tiles[1], 1.0, 1.0)
    rest = np.delete(np.arange(len(c.pos)), 1 + at)
    tol = 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -8 + 2.0 ** -12) * spread + 2.0 ** -31 * flat
    assert np.all((np.abs(got - want) <= tol)[rest])


def test_too_few_prefill_blocks_are_reported():
    c = Case([(1, 40), (50, 60), (20, 100)], 8, 2, 128, seed=12)
    c.run(pre=4)  # room for the first prompt (4 blocks), not for the second (7)
    guard()
    got = f64(c.out).reshape(-1, 8, 128)
    want, spread, _ = R.attention(f64(c.q), c.pos, c.qsl, c.table, c.tiles[0], c.tiles[1], 1.0, 1.0)
    assert np.all(np.abs(got - want)[:51] <= 2.0 ** -8 * np.abs(want[:51]) + 2.0 ** -6 * spread[:51])
    assert np.all(got[51:] == 5.0)


@pytest.mark.parametrize("many", [300, 700])
def test_prompts_among_many_sequences(many):
    r = np.random.default_rng(23)
    seqs = [(1, int(n)) for n in r.integers(1, 40, many)]
    for at, s in ((3, (40, 77)), (many // 2, (18, 18)), (many - 2, (33, 300)), (many, (70, 71))):
        seqs.insert(at, s)
    c = Case(seqs, 8, 2, 64, seed=24)
    c.run()
    ok()
    c.check()


def test_prompts_without_prefill_blocks_are_reported():
    c = Case([(1, 40), (50, 60), (2, 9)], 8, 2, 128, seed=25)
    c.run(pre=0)
    guard()
    got = f64(c.out).reshape(-1, 8, 128)
    want, spread, _ = R.attention(f64(c.q), c.pos, c.qsl, c.table, c.tiles[0], c.tiles[1], 1.0, 1.0)
    rest = np.r_[0:1, 51:53]
    assert np.all(np.abs(got - want)[rest] <= 2.0 ** -8 * np.abs(want[rest]) + 2.0 ** -9 * spread[rest])
    assert np.all(got[1:51] == 5.0)


def test_same_result_on_every_run_and_on_another_stream():
    c = Case([(1, 3000), (1, 17), (33, 500), (2, 999), (1, 1200)], 32, 4, 128, seed=13)
    a = c.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            c.ws.random_(0, 255)  # nothing in the workspace has to be set
            assert torch.equal(c.run(out=torch.full_like(a, 5.0)), a)
    torch.cuda.current_stream().wait_stream(s)
    ok()
    c.check(a)


@pytest.mark.parametrize("bound", BOUNDS)
def test_captured_and_replayed_with_new_lengths(bound):
    c = Case([(1, 900), (1, 40), (1, 333)], 8, 2, 128, seed=14, bound=bound)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens in ((900, 40, 333), (1, 40, 32), (513, 2, 333)):
        c.seqs = [(1, n) for n in lens]
        c.pos = np.array([n - 1 for n in lens], dtype=np.int32)
        c.batch.positions.copy_(torch.from_numpy(c.pos))
        c.batch.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.out.fill_(5.0)
        g.replay()
        ok()
        c.check()


@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 64), (16, 2, 128), (5, 1, 128)])
def test_a_chunk_over_many_keys_replayed_with_new_lengths(nq, nkv, d):
    # more and fewer key tiles than parts, and parts without a key
    c = Case([(40, 3000), (1, 40), (40, 2500)], nq, nkv, d, seed=22)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens in ((3000, 40, 2500), (40, 1, 41), (130, 17, 2500), (2999, 33, 65)):
        c.seqs = [(40, lens[0]), (1, lens[1]), (40, lens[2])]
        c.pos = np.concatenate([np.arange(t - n, t) for n, t in c.seqs]).astype(np.int32)
        c.batch.positions.copy_(torch.from_numpy(c.pos))
        c.batch.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.out.fill_(5.0)
        c.ws.random_(0, 255)
        g.replay()
        ok()
        c.check()


def test_a_mixed_batch_captured_and_replayed():
    # the decode kernels' side stream joins the capture
    c = Case([(1, 900), (40, 77), (1, 40), (3, 333)], 8, 2, 128, seed=16)
    want = c.run().clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
        c.run()
    for _ in range(3):
        c.out.fill_(5.0)
        g.replay()
        ok()
        assert torch.equal(c.out, want)
    c.check()


@pytest.mark.parametrize("captured", [False, True])
def test_the_cache_written_right_behind_a_mixed_batch(captured):
    # the write starts while the batch's last kernels end, those of the side stream too, and must not reach the cache
    c = Case([(1, 900), (40, 77), (1, 40), (200, 333), (3, 50)], 32, 4, 128, seed=19)
    slots = torch.from_numpy(np.concatenate([[c.table[b][j // 16] * 16 + j % 16 for j in range(t)]
                                             for b, (_, t) in enumerate(c.seqs)]).astype(np.int32)).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(19)
    rows = [torch.randn(len(slots), 4, 128, generator=g, device=DEV).bfloat16() for _ in range(4)]
    outs = [torch.empty_like(c.out) for _ in range(4)]

    def write(i):
        lb.kv_cache_write_q4(rows[2 * i], rows[2 * i + 1], slots, c.kc, c.vc)

    def chain():
        for n in range(4):
            write(n % 2)
            c.run(out=outs[n])

    want = []
    for i in range(2):
        write(i)
        torch.cuda.synchronize()
        want.append(c.run().clone())
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        chain = graph.replay
    for _ in range(5):
        for o in outs:
            o.fill_(5.0)
        chain()
        ok()
        for n in range(4):
            assert torch.equal(outs[n], want[n % 2]), n


def test_calls_back_to_back_on_two_streams():
    # each with a workspace of its own, many calls in flight
    a = Case([(1, 2000), (1, 70)], 16, 2, 128, seed=17)
    b = Case([(1, 3000), (2, 500)], 8, 2, 64, seed=18)
    wa, wb = a.run().clone(), b.run().clone()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(40):
        with torch.cuda.stream(s):
            a.run()
        with torch.cuda.stream(t):
            b.run()
    torch.cuda.synchronize()
    ok()
    assert torch.equal(a.out, wa) and torch.equal(b.out, wb)


def test_caches_over_four_gigabytes():
    # block numbers whose byte offsets pass 32 bits
    nkv, d = 8, 128
    blocks = (1 << 32) // (nkv * 9 * d) + 40
    kc = torch.zeros(blocks, nkv, 9 * d, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    small = Case([(1, 100), (40, 70)], 64, nkv, d, seed=15)
    shift = blocks - small.batch.num_blocks
    kc[shift:], vc[shift:] = small.kc, small.vc
    k2, v2 = (torch.empty(64, nkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k1, v1 = torch.empty_like(k2), torch.empty_like(v2)
    slots = torch.from_numpy(np.array([small.table[0][j // 16] * 16 + j % 16 for j in range(64)], np.int32)).to(DEV)
    lb.kv_cache_read_q4(small.kc, small.vc, slots, k1, v1)
    lb.kv_cache_read_q4(kc, vc, slots + shift * 16, k2, v2)
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
    a = small.run().clone()
    small.kc, small.vc = kc, vc
    small.batch.num_blocks = blocks
    small.batch.block_table[small.batch.block_table >= 0] += shift
    assert torch.equal(small.run(), a)
    w = torch.randn(64, nkv, d, device=DEV).bfloat16()
    lb.kv_cache_write_q4(w, w, slots + shift * 16, kc, vc)
    lb.kv_cache_read_q4(kc, vc, slots + shift * 16, k2, v2)
    ok()
    assert (k2 - w).abs().max() < 1.0  # half a step of the largest group's scale (amax 5 / 6, 2 / 2 codes)
    assert int(kc[:shift].max()) == 0


# ---------------------------------------------------------------------------
# together: a step's projections to its attention output
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 64), (32, 4, 128)])
def test_prompt_then_tokens_through_all_of_them(nq, nkv, d):
    cfg = lb.LayerConfig(nq * d, nq, nkv, d, 4 * nq * d, 1e-5, 1e4)
    rope = lb.QkNormRopeConfig(nq, nkv, d, rms_eps=1e-6, rope_theta=1e6)
    g = torch.Generator(device=DEV).manual_seed(21)
    kg, vg = 1.0, 0.25
    lens0, blocks = [37, 5, 80], 16
    table = torch.randperm(blocks, generator=g, device=DEV)[:15].view(3, 5).int()
    shape = (blocks, nkv, lb.kv_cache_q4_tile_bytes(d))
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() for _ in range(2))
    tiles = [np.zeros(shape, np.uint8), np.zeros(shape, np.uint8)]
    seen = [0, 0, 0]
    for new in (lens0[:2] + [79], [1, 1, 1], [2, 1, 0]):
        T = sum(new)
        pos = torch.tensor([p for s, n in zip(seen, new) for p in range(s, s + n)], dtype=torch.int32, device=DEV)
        seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device=DEV)
        seen = [s + n for s, n in zip(seen, new)]
        qsl = torch.tensor([0, new[0], new[0] + new[1], T], dtype=torch.int32, device=DEV)
        slots = (table[seq, (pos // 16).long()] * 16 + pos % 16).int()
        rows = torch.randn(T, nq + 2 * nkv, d, generator=g, device=DEV).bfloat16()
        q, k, v = rows[:, :nq], rows[:, nq:nq + nkv], rows[:, nq + nkv:] * vg
        q_in, k_in = q.clone(), k.clone()
        qd = torch.empty(T, nq, d, dtype=torch.bfloat16, device=DEV)
        lb.qk_norm_rope(rope, qw, kw, pos, q, k, qd, k)
        lb.kv_cache_write_q4(k, v, slots, kc, vc, kg, vg)
        batch = lb.Batch(pos, qsl, torch.tensor(seen, dtype=torch.int32, device=DEV), table, blocks, max(new), max(seen))
        pre = lb.prefill_blocks(new, seen, nq // nkv)
        out = torch.empty(T, nq * d, dtype=torch.bfloat16, device=DEV)
        ws = lb.alloc_workspace(lb.paged_attention_q4_workspace_size(cfg, T, 3, max(seen), pre))
        lb.paged_attention_q4(cfg, batch, qd, kc, vc, out, ws, kg, vg, pre)
        ok()
        check_qk(qd, q_in, qw, pos, rope)
        check_qk(k, k_in, kw, pos, rope)
        R.pack_rows(tiles[0], slots.tolist(), *R.quantise(f64(k), kg), d, False)
        R.pack_rows(tiles[1], slots.tolist(), *R.quantise(f64(v), vg), d, True)
        assert np.array_equal(kc.cpu().numpy(), tiles[0]) and np.array_equal(vc.cpu().numpy(), tiles[1])
        want, spread, flat = R.attention(f64(qd), pos.tolist(), qsl.tolist(), table.tolist(), tiles[0], tiles[1], kg, vg)
        err = np.abs(f64(out).reshape(T, nq, d) - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -8 + 2.0 ** -12) * spread + 2.0 ** -31 * flat)
