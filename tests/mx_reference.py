"""Microscaled matrices in 64 bits on the CPU: the formats, their rounding and
their layout, from the definitions in include/llama_layer.h."""

from __future__ import annotations

import numpy as np

NVFP4, FP4, FP8 = 1, 2, 3
GROUP = {NVFP4: 16, FP4: 32, FP8: 32}
TOP = {NVFP4: 6.0, FP4: 6.0, FP8: 448.0}
STEP = {NVFP4: 64, FP4: 64, FP8: 32}  # elements that one tensor-core instruction contracts


def e4m3_table() -> np.ndarray:
    b = np.arange(128)
    e, m = b >> 3, b & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    v[127] = np.nan
    return np.concatenate([v, -v])


def e2m1_table() -> np.ndarray:
    v = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    return np.concatenate([v, -v])


E4M3, E2M1 = e4m3_table(), e2m1_table()
E8M0 = np.append(2.0 ** (np.arange(255.0) - 127), np.nan)


def nearest(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the nearest of an ascending table of non-negative numbers, ties to the even index, saturating."""
    i = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo, hi = table[i - 1], table[i]
    mid = (lo + hi) / 2
    return np.where((x > mid) | ((x == mid) & (i % 2 == 0)), i, i - 1)


def scale_bytes(top: np.ndarray, fmt: int, g: float) -> np.ndarray:
    """The scale byte of groups whose largest |x| is top (NaN or infinity: the NaN scale)."""
    bad = ~np.isfinite(top)
    t = np.where(bad, 0.0, top)
    if fmt == NVFP4:
        return np.where(bad, 127, nearest(t / (6.0 * g), E4M3[:127]))
    b = np.searchsorted(E8M0[:255] * TOP[fmt], t)  # the first power of two with t <= top * 2^e
    return np.where(bad, 255, np.minimum(b, 254))


def scale_value(b: np.ndarray, fmt: int) -> np.ndarray:
    return E4M3[b] if fmt == NVFP4 else E8M0[b]


def round_codes(y: np.ndarray, fmt: int) -> np.ndarray:
    """y to the nearest code values (signed)."""
    t = E4M3[:127] if fmt == FP8 else E2M1[:8]
    return np.copysign(t[nearest(np.abs(y), t)], y)


def quantise(x: np.ndarray, fmt: int, g: float):
    """(values of the codes [rows, cols], scale bytes [rows, groups]); codes of NaN groups are 0."""
    rows, cols = x.shape
    y = x.reshape(rows, -1, GROUP[fmt])
    with np.errstate(invalid="ignore"):
        top = np.abs(y).max(-1)
    b = scale_bytes(top, fmt, g)
    s = np.nan_to_num(scale_value(b, fmt))[..., None] * g
    q = np.where(s > 0, np.where(np.isfinite(y), y, 0.0) / np.where(s > 0, s, 1.0), 0.0)
    q = np.where(np.isfinite(top)[..., None], round_codes(q, fmt), 0.0)
    return q.reshape(rows, cols), b


def values(q: np.ndarray, b: np.ndarray, fmt: int, g: float) -> np.ndarray:
    return (q.reshape(*b.shape, GROUP[fmt]) * (scale_value(b, fmt) * g)[..., None]).reshape(q.shape)


def code_values(codes: np.ndarray, fmt: int) -> np.ndarray:
    if fmt == FP8:
        return E4M3[codes]
    out = np.empty((codes.shape[0], codes.shape[1] * 2))
    out[:, 0::2], out[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    return out


def scale_place(r, s, groups: int):
    return ((r // 128) * (-(-groups // 4)) + s // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + s % 4


def scale_places(rows: int, groups: int) -> np.ndarray:
    return scale_place(np.arange(rows)[:, None], np.arange(groups)[None, :], groups)


def pack(q: np.ndarray, b: np.ndarray, fmt: int, fill: int = 0):
    """(codes, scales) bytes of code values and scale bytes; padded rows of the scales hold `fill`."""
    if fmt == FP8:
        codes = nearest(np.abs(q), E4M3[:127]) + 128 * np.signbit(q)
    else:
        n = nearest(np.abs(q), E2M1[:8]) + 8 * np.signbit(q)
        codes = n[:, 0::2] | (n[:, 1::2] << 4)
    rows, groups = b.shape
    padded = -(-groups // 4) * 4
    scales = np.full(-(-rows // 128) * padded * 128, fill, np.uint8)
    full = np.zeros((rows, padded), np.uint8)
    full[:, :groups] = b
    scales[scale_places(rows, padded)] = full
    return codes.astype(np.uint8), scales


def check_quantised(codes, scales, want, slack, fmt: int, g: float) -> None:
    """Stored rows against 64-bit results that are known to within `slack` (>= 0, of want's shape): each scale lies
    between those of the least and the greatest largest element, each code between the roundings of the least and the
    greatest quotient.  With slack 0 both are exact."""
    rows, cols = want.shape
    groups = cols // GROUP[fmt]
    b = scales[scale_places(rows, groups)].astype(int)
    a = np.abs(want).reshape(rows, groups, -1)
    sl = np.broadcast_to(slack, want.shape).reshape(a.shape)
    lo, hi = scale_bytes((a - sl).max(-1).clip(min=0), fmt, g), scale_bytes((a + sl).max(-1), fmt, g)
    assert np.all((lo <= b) & (b <= hi)), np.argwhere((lo > b) | (b > hi))[:5]
    s = (scale_value(b, fmt) * g)[..., None]
    safe = np.where(s > 0, s, 1.0)
    w = want.reshape(a.shape)
    low, high = (np.where(s > 0, round_codes(x / safe, fmt), 0.0) for x in (w - sl, w + sl))
    q = code_values(codes, fmt).reshape(a.shape)
    bad = (q < low) | (q > high)
    assert not bad.any(), (np.argwhere(bad)[:5], q[bad][:5], low[bad][:5], high[bad][:5])
