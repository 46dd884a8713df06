"""Paged-cache operators (oracle; test infrastructure): position rotation with
append, the 4-bit cache, attention with a sliding window and sinks.

Definitions:
  * rotation over the pairs (i, j) of the first dim channels: y_i = x_i cos -
    x_j sin, y_j = x_j cos + x_i sin, each product and sum rounded to fp32, the
    result to bf16 (nearest, ties to even);
  * 4-bit group of 128 or 64 channels: z = fp16(min) (a zero as +0), s = fp16(fl32(fl32(max -
    min) / 15)), code = clamp(rint(fl32(fl32(x - z) / s)), 0, 15), 0 where s is 0,
    of bf16 values saturated to +-65504 with NaN as 0; a code stands for s code + z;
  * the query at position p sees the tokens t <= p with t < sinks or t > p -
    window (window < 0: all t <= p); o = softmax(scale q k^T) v, 0 where it sees
    none; float64.
"""
from __future__ import annotations

import numpy as np

PAGE, D = 64, 128


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """bf16 bit patterns of fp32 values, nearest even (finite values)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def rotate(bits: np.ndarray, table: np.ndarray, pos: np.ndarray, interleaved: bool) -> np.ndarray:
    """bf16 bits [rows][heads][128] rotated by table[pos] (fp32 [rows][dim])."""
    x = bf16_values(bits)
    dim = table.shape[1]
    cos, sin = table[pos][:, None, :dim // 2], table[pos][:, None, dim // 2:]
    i = np.arange(0, dim, 2) if interleaved else np.arange(dim // 2)
    j = i + 1 if interleaved else i + dim // 2
    a, b = x[..., i], x[..., j]
    out = np.array(bits, copy=True)
    out[..., i] = bf16_bits((a * cos).astype(np.float32) - (b * sin).astype(np.float32))
    out[..., j] = bf16_bits((b * cos).astype(np.float32) + (a * sin).astype(np.float32))
    return out


def quantise4(bits: np.ndarray, group: int):
    """Codes uint8 [..., 128] and fp16 {s, z} [..., 128 / group, 2] of bf16 bits [..., 128]."""
    x = bf16_values(bits)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-65504), np.float32(65504)))
    x = x.reshape(*x.shape[:-1], D // group, group)
    mn, mx = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    z = (mn + np.float32(0)).astype(np.float16)          # a zero is +0
    s = ((mx - mn).astype(np.float32) / np.float32(15)).astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = ((x - z.astype(np.float32)).astype(np.float32) / s.astype(np.float32)).astype(np.float32)
        code = np.where(s == 0, 0, np.clip(np.rint(t), 0, 15)).astype(np.uint8)
    return code.reshape(bits.shape), np.concatenate([s, z], -1)


def dequantise4(code: np.ndarray, meta: np.ndarray) -> np.ndarray:
    """float64 values s code + z."""
    m = meta.astype(np.float64)
    group = D // m.shape[-2]
    c = code.reshape(*code.shape[:-1], D // group, group).astype(np.float64)
    return (c * m[..., :1] + m[..., 1:]).reshape(code.shape)


def record_bytes(group: int) -> int:
    return 2 * PAGE * D // 2 + 2 * PAGE * 4 * (D // group)


def put4(rec: np.ndarray, which: int, slot: int, code: np.ndarray, meta: np.ndarray) -> None:
    """Store one token's 128 codes and {s, z} pairs into a record (uint8 [record])."""
    at = which * PAGE * D // 2 + slot * D // 2
    rec[at:at + D // 2] = code[0::2] | (code[1::2] << 4)
    m = np.ascontiguousarray(meta, np.float16).reshape(-1).view(np.uint8)
    at = PAGE * D + which * PAGE * m.size + slot * m.size
    rec[at:at + m.size] = m


def seen(pos: int, window: int, sinks: int) -> np.ndarray:
    t = np.arange(pos + 1)
    return t if window < 0 else t[(t < sinks) | (t > pos - window)]


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, pos: int, window: int, sinks: int, scale: float, kmag=None,
           vmag=None):
    """One query row [128] at position pos against k, v [tokens][128], float64: out [128], log-sum-exp,
    and the magnitudes that rounding errors go by: sum p vmag [128] and scale max_t sum |q| kmag
    (kmag, vmag [tokens][128]: what is added up for a key or value, |k| and |v| unless given)."""
    kmag = np.abs(k) if kmag is None else kmag
    vmag = np.abs(v) if vmag is None else vmag
    t = seen(pos, window, sinks)
    if len(t) == 0:
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    x = scale * (k[t] @ q)
    m = x.max()
    p = np.exp(x - m)
    s = p.sum()
    return (p / s) @ v[t], m + np.log(s), (p / s) @ vmag[t], scale * (kmag[t] @ np.abs(q)).max()
