"""Plain 64-bit forms of the operators around the 4-bit KV cache, for the tests:
the stored format one value at a time, attention over the values it stands for,
and the norm and rotation of query and key heads."""

from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every finite non-negative e4m3 number, by its bits
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest_even(x, grid):
    """Index of the entry of an increasing grid nearest to each x >= 0; of two
    equally near ones the even index; past the end the last."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    take_lo = (below < above) | ((below == above) & (lo % 2 == 0))
    return np.where(np.isinf(x), len(grid) - 1, np.where(take_lo, lo, hi))


def quantise(x, g):
    """x [..., d] -> (codes [..., d] 0..15, scale bits [..., d/16]) by the definition."""
    x = np.where(np.isnan(x), 0.0, np.asarray(x, dtype=np.float64)) / g
    grp = x.reshape(*x.shape[:-1], -1, 16)
    s8 = nearest_even(np.abs(grp).max(-1) / 6.0, E4M3)
    s = E4M3[s8][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, np.abs(grp) / s, 0.0)
    code = nearest_even(y, E2M1) + 8 * (np.signbit(grp) & (s > 0))
    return code.reshape(x.shape).astype(np.uint8), s8.astype(np.uint8)


def value(code, s8, g):
    """The values that codes [..., d] and scale bits [..., d/16] stand for."""
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    return v * np.repeat(E4M3[s8], 16, axis=-1) * g


def code_place(d, k, e, is_v):
    if not is_v:
        return k * (d // 2) + e // 2
    w = d // 8
    return (k // 8) * 4 * d + ((e // w) * 4 + (k % 8) // 2) * w + (k % 2) * (w // 2) + (e % w) // 2


def scale_place(d, k, s, is_v):
    if is_v:
        return 8 * d + (s * 4 + (k % 8) // 2) * 4 + (k // 8) * 2 + k % 2
    p = d // 64
    return 8 * d + ((k % 8) * 4 + s // p) * 2 * p + (k // 8) * p + s % p


def unpack_tiles(tiles, d, is_v):
    """tiles [..., 9d] uint8 -> (codes [..., 16, d], scale bits [..., 16, d/16])."""
    at = np.array([[code_place(d, k, e, is_v) for e in range(d)] for k in range(16)])
    sat = np.array([[scale_place(d, k, s, is_v) for s in range(d // 16)] for k in range(16)])
    b = tiles[..., at]
    return np.where(np.arange(d) % 2 == 1, b >> 4, b & 15), tiles[..., sat]


def pack_rows(tiles, slots, code, s8, d, is_v):
    """Rows (codes [n, n_kv, d], scale bits [n, n_kv, d/16]) at slots >= 0 of tiles [blocks, n_kv, 9d], in place."""
    slots = np.asarray(slots, dtype=np.int64)
    keep = slots >= 0
    b, k = slots[keep] // 16, slots[keep] % 16
    code, s8 = code[keep], s8[keep]
    heads = np.arange(tiles.shape[1])[None, :]
    for e in range(0, d, 2):
        tiles[b[:, None], heads, code_place(d, k, e, is_v)[:, None]] = code[:, :, e] | (code[:, :, e + 1] << 4)
    for s in range(d // 16):
        tiles[b[:, None], heads, scale_place(d, k, s, is_v)[:, None]] = s8[:, :, s]


def cache_rows(tiles, slots, d, is_v, g):
    """[n, n_kv, d] values at slots."""
    code, s8 = unpack_tiles(tiles[np.asarray(slots) // 16], d, is_v)
    n = np.arange(len(slots))
    k = np.asarray(slots) % 16
    return value(code[n, :, k], s8[n, :, k], g)


def attention(q, positions, qsl, block_table, k_tiles, v_tiles, kg, vg):
    """q [T, nq, d] fp64 -> (out, sum p |v|, sum |v| over the keys seen), [T, nq, d] each."""
    T, nq, d = q.shape
    nkv = k_tiles.shape[1]
    out, spread, flat = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(qsl) - 1):
        if qsl[b + 1] == qsl[b]:
            continue
        n = max(int(positions[t]) for t in range(qsl[b], qsl[b + 1])) + 1
        slots = np.array([block_table[b][j // 16] * 16 + j % 16 for j in range(n)])
        k = torch.from_numpy(np.repeat(cache_rows(k_tiles, slots, d, False, kg), nq // nkv, axis=1))
        v = torch.from_numpy(np.repeat(cache_rows(v_tiles, slots, d, True, vg), nq // nkv, axis=1))
        x = torch.from_numpy(q[qsl[b]:qsl[b + 1]])
        s = torch.einsum("thd,jhd->thj", x, k) / math.sqrt(d)
        seen = torch.arange(n)[None] <= torch.as_tensor(np.asarray(positions[qsl[b]:qsl[b + 1]]))[:, None]
        p = torch.softmax(torch.where(seen[:, None], s, -math.inf), -1)
        out[qsl[b]:qsl[b + 1]] = torch.einsum("thj,jhd->thd", p, v).numpy()
        spread[qsl[b]:qsl[b + 1]] = torch.einsum("thj,jhd->thd", p, v.abs()).numpy()
        flat[qsl[b]:qsl[b + 1]] = torch.einsum("tj,jhd->thd", seen.double(), v.abs()).numpy()
    return out, spread, flat


def frequencies(rot, theta, scaling):
    """(radians a position of each pair, factor on cosine and sine)."""
    out, s = [], scaling or {}
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        kind = s.get("rope_type")
        if kind == "linear":
            f /= s["factor"]
        elif kind == "llama3":
            lam, orig = 2 * math.pi / f, s["original_max_position_embeddings"]
            lo, hi = s["low_freq_factor"], s["high_freq_factor"]
            if lam > orig / lo:
                f /= s["factor"]
            elif lam >= orig / hi:
                a = (orig / lam - lo) / (hi - lo)
                f = (1 - a) * f / s["factor"] + a * f
        elif kind == "yarn":
            orig = s["original_max_position_embeddings"]
            at = [rot * math.log(orig / (2 * math.pi * b)) / (2 * math.log(theta))
                  for b in (s.get("beta_fast", 32.0), s.get("beta_slow", 1.0))]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            a = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f / s["factor"] * a + f * (1 - a)
        out.append(f)
    factor = 1.0
    if s.get("rope_type") == "yarn":
        factor = s.get("attention_factor", 0.1 * math.log(s["factor"]) + 1.0)
    return np.array(out), factor


def norm_rope(x, w, positions, rot, interleaved, eps, theta, scaling):
    """x [T, h, d] fp64 -> (y, |a| + |b| of each element's pair before the rotation)."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    size = np.abs(y)
    if rot:
        f, factor = frequencies(rot, theta, scaling)
        ang = np.asarray(positions, dtype=np.float64)[:, None, None] * f
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a] = factor * (ya * np.cos(ang) - yb * np.sin(ang))
        y[..., b] = factor * (yb * np.cos(ang) + ya * np.sin(ang))
        size[..., a] = size[..., b] = factor * (np.abs(ya) + np.abs(yb))
    return y, size
