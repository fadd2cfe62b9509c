"""Plain 64-bit forms (numpy) of the operators on the rows' contents, written from
the formulas: e4m3 by its fields, rows by their layout, softmax attention, the
row writer and rotary positions. Test infrastructure only."""

from __future__ import annotations

import math

import numpy as np

LATENT, GROUP, ROPE, LATENT_ROW = 512, 128, 64, 656


def e4m3_table() -> np.ndarray:
    """The value of every e4m3 code (S EEEE FFF, bias 7; 0x7f and 0xff are NaN)."""
    out = np.empty(256, np.float64)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = (f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if c & 127 == 127 else (-v if c & 128 else v)
    return out


E4M3 = e4m3_table()


def e4m3_nearest(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values, ties to the even code, values beyond 448 to 448, NaN to
    0x7f (either NaN code compares equal to it by value)."""
    x = np.asarray(x, np.float64)
    pos = E4M3[:127]                                  # ascending
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0)), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 127, code | np.where(np.signbit(x), 128, 0))
    return code.astype(np.uint8)


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f32_at(rows: np.ndarray, at: int, n: int) -> np.ndarray:
    return np.ascontiguousarray(rows[..., at:at + 4 * n]).view("<f4").astype(np.float64)


def latent_kv(rows: np.ndarray):
    """(keys [..., 576], values [..., 512]) of latent rows [..., 656]."""
    lat = E4M3[rows[..., :LATENT]].reshape(*rows.shape[:-1], LATENT // GROUP, GROUP)
    lat = (lat * f32_at(rows, LATENT + 2 * ROPE, LATENT // GROUP)[..., None]).reshape(*rows.shape[:-1], LATENT)
    rope = bf16_values(np.ascontiguousarray(rows[..., LATENT:LATENT + 2 * ROPE]).view("<u2"))
    return np.concatenate([lat, rope], -1), lat


def heads_kv(rows: np.ndarray, kv_heads: int, dim: int, block: int):
    """(keys, values [..., kv_heads, block, dim], tokens in use [...]) of heads rows."""
    part = kv_heads * block * dim
    sc = f32_at(rows, 2 * part, 2 * kv_heads).reshape(*rows.shape[:-1], 2, kv_heads, 1, 1)
    kv = E4M3[rows[..., :2 * part]].reshape(*rows.shape[:-1], 2, kv_heads, block, dim) * sc
    at = 2 * part + 8 * kv_heads
    count = np.ascontiguousarray(rows[..., at:at + 4]).view("<i4")[..., 0]
    return kv[..., 0, :, :, :], kv[..., 1, :, :, :], np.clip(count, 0, block)


def attention(q: np.ndarray, keys: np.ndarray, values: np.ndarray, scale: float):
    """One set: q [heads][w], keys and values [tokens][...] -> (out, lse, mag, reach): mag is the
    sum of weight x |value| and reach the largest sum of |q key| x |scale| of a logit, which
    bound the errors of the sums."""
    heads = q.shape[0]
    if keys.shape[0] == 0:
        z = np.zeros((heads, values.shape[-1]))
        return z, np.full(heads, -math.inf), z, np.zeros(heads)
    s = (q @ keys.T) * scale
    top = s.max(-1, keepdims=True)
    w = np.exp(s - top)
    tot = w.sum(-1, keepdims=True)
    w /= tot
    reach = ((np.abs(q) @ np.abs(keys).T) * abs(scale)).max(-1)
    return w @ values, (top + np.log(tot))[:, 0], w @ np.abs(values), reach


def turn(x: np.ndarray, positions: np.ndarray, sections, theta: float, interleaved: bool, inverse: bool = False):
    """x [tokens][..., dim] turned by positions [tokens][axes]."""
    dim = x.shape[-1]
    half = dim // 2
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = positions[:, axis].astype(np.float64) * theta ** (-2.0 * np.arange(half) / dim)
    ang = ang.reshape(ang.shape[0], *([1] * (x.ndim - 2)), half) * (-1.0 if inverse else 1.0)
    c, s = np.cos(ang), np.sin(ang)
    out = np.empty_like(x)
    i0, i1 = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, half), slice(half, None))
    a, b = x[..., i0], x[..., i1]
    out[..., i0] = a * c - b * s
    out[..., i1] = a * s + b * c
    return out


def pack_scale(x: np.ndarray) -> np.ndarray:
    """fp32 scales over the last axis of x (fp32 values)."""
    a = np.where(np.isfinite(x), np.abs(x), 0).astype(np.float32).max(-1)
    return np.maximum(a / np.float32(448), np.float32(2.0 ** -126))
