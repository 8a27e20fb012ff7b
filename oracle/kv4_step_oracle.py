"""Plain CPU reference of what surrounds the attention over the 4-bit latent
cache: norm and rotation of the tokens that are written, page digests and page
selection.

It shares no code with the CUDA path.  Roundings that belong to the definition
are made in numpy's float32; everything else is float64 or whole numbers.
"""

from __future__ import annotations

import numpy as np

from . import kv4_oracle as ko
from .mlaqp_oracle import bf16_to_f64

DIM = ko.LATENT + ko.ROPE
EXP_MIN, EXP_MAX, EXP_NONE = -60, 60, 255
DIGEST_BYTES = 1168


def normalise(latent_bits: np.ndarray, weight_bits, eps: float) -> np.ndarray:
    """BF16 bits [T,512] -> float32 values that are quantised."""
    x = bf16_to_f64(latent_bits)
    if weight_bits is None:
        return x.astype(np.float32)
    with np.errstate(all="ignore"):
        mean = (x * x).sum(1, keepdims=True).astype(np.float32) / np.float32(ko.LATENT)
        r = np.float32(1.0) / np.sqrt(mean + np.float32(eps))
        return x.astype(np.float32) * r * bf16_to_f64(weight_bits).astype(np.float32)


def rotate(part_bits: np.ndarray, angles: np.ndarray, halves: bool) -> np.ndarray:
    """BF16 bits [..,64], angles [..,64] (32 cosines, 32 sines) -> float64."""
    v, angles = bf16_to_f64(part_bits), angles.astype(np.float64)
    first = np.arange(32) if halves else 2 * np.arange(32)
    second = first + 32 if halves else first + 1
    out = np.empty_like(v)
    cos, sin = angles[..., :32], angles[..., 32:]
    out[..., first] = v[..., first] * cos - v[..., second] * sin
    out[..., second] = v[..., second] * cos + v[..., first] * sin
    return out


def codes_and_scales(y: np.ndarray):
    """float32 [512] -> (code bytes [256], scale bytes [16]) of the token."""
    row, scales = np.zeros(256, dtype=np.uint8), np.zeros(16, dtype=np.uint8)
    for j in range(ko.LATENT // ko.BLOCK):
        codes, scales[j] = ko.quantise_block(y[ko.BLOCK * j: ko.BLOCK * (j + 1)].astype(np.float64))
        for i, c in enumerate(codes):
            mb, mbit, sb, sbit = ko.code_place(ko.BLOCK * j + i)
            row[mb] |= (int(c) & 7) << mbit
            row[sb] |= (int(c) >> 3) << sbit
    return row, scales


def _bounds(v: np.ndarray):
    """Values [tokens, channels] -> (largest, smallest, exponent byte)."""
    zeros = np.zeros(v.shape[1], dtype=np.int64)
    if not np.isfinite(v).all():
        return zeros, zeros, EXP_NONE
    e = EXP_MIN
    while np.abs(v).max() > 127.0 * 2.0 ** e:
        e += 1
    if e > EXP_MAX:
        return zeros, zeros, EXP_NONE
    return np.ceil(v.max(0) / 2.0 ** e).astype(np.int64), np.floor(v.min(0) / 2.0 ** e).astype(np.int64), e + 127


def digest(keys: np.ndarray) -> np.ndarray:
    """float64 [P,576], the tokens of a page -> its 1168 bytes."""
    lat, rope = _bounds(keys[:, :ko.LATENT]), _bounds(keys[:, ko.LATENT:])
    out = np.zeros(DIGEST_BYTES, dtype=np.uint8)
    out[:1152] = np.concatenate([lat[0], lat[1], rope[0], rope[1]]).astype(np.int8).view(np.uint8)
    out[1152], out[1153] = lat[2], rope[2]
    return out


def query_sums(q: np.ndarray):
    """float64 [H,576] -> (up, down, f): whole numbers per channel and the power of two."""
    if not np.isfinite(q).all():
        return np.zeros(DIM, dtype=np.int64), np.zeros(DIM, dtype=np.int64), 0
    f = -100
    while np.abs(q).max() > 2047.0 * 2.0 ** f:
        f += 1
    qi = np.rint(q * 2.0 ** -f).astype(np.int64)
    return np.maximum(qi, 0).sum(0), np.minimum(qi, 0).sum(0), f


def scores(q: np.ndarray, digests: np.ndarray) -> np.ndarray:
    """q float64 [H,576], digests uint8 [n,1168] -> float32 [n]."""
    up, down, _ = query_sums(q)
    v = np.ascontiguousarray(digests[:, :1152]).view(np.int8).astype(np.int64)
    lat = v[:, :512] @ up[:512] + v[:, 512:1024] @ down[:512]
    rope = v[:, 1024:1088] @ up[512:] + v[:, 1088:1152] @ down[512:]
    e = digests[:, 1152:1154].astype(np.int64)
    power = np.exp2(np.minimum(e, 254) - 127.0).astype(np.float32)
    power[e == 0] = 0.0  # (no digest has it: a float's bits without an exponent)
    s = lat.astype(np.float32) * power[:, 0] + rope.astype(np.float32) * power[:, 1]
    s[(e == EXP_NONE).any(1) | np.isnan(s)] = np.inf
    return s


def select(q: np.ndarray, digests: np.ndarray, row, n: int, page_size: int, k: int, first: int, last: int):
    """Pages (their numbers, in order) and visible tokens in them, of one query token that sees n tokens."""
    if n <= 0:
        return [], 0
    pages = -(-n // page_size)
    take = list(range(pages))
    if pages > k:
        between = range(first, pages - last)
        good = [0 <= row[j] < len(digests) for j in between]
        s = scores(q, digests[[row[j] if ok else 0 for j, ok in zip(between, good)]]) if len(good) else []
        # a page out of range scores least of all
        order = sorted(range(len(good)), key=lambda i: (not good[i], -float(s[i]) if good[i] else 0.0, i))
        take = list(range(first)) + sorted(first + i for i in order[:k - first - last]) + list(range(pages - last, pages))
    return [int(row[j]) for j in take], (len(take) - 1) * page_size + n - (pages - 1) * page_size
