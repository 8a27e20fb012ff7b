"""Plain CPU reference of the paged 4-bit latent cache: its codes, the
attention over it in float64, and the page operations as Python loops.

It shares no code with the CUDA path.  Latents and rope elements come and go
as BF16 bit patterns (uint16); a layer's cache is a uint8 array
[num_pages, page_bytes].
"""

from __future__ import annotations

import numpy as np

from .mlaqp_oracle import bf16_to_f64

LATENT = 512
ROPE = 64
BLOCK = 32
TOKEN_BYTES = 400
SCALE_MIN, SCALE_MAX, SCALE_NAN = 87, 167, 255
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise_block(v: np.ndarray):
    """32 float64 values -> (codes 0..15, scale byte)."""
    if not np.isfinite(v).all():
        return np.zeros(BLOCK, dtype=np.uint8), SCALE_NAN
    amax = np.abs(v).max()
    s = SCALE_MIN
    while s < SCALE_MAX and amax > 7.0 * 2.0 ** (s - 127):
        s += 1
    codes = np.empty(BLOCK, dtype=np.uint8)
    for i, x in enumerate(v):
        y = abs(x) / 2.0 ** (s - 127)
        d = np.abs(E2M1 - y)
        near = np.flatnonzero(d == d.min())
        c = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]  # ties to the even code
        codes[i] = c | (8 if np.signbit(x) else 0)
    return codes, s


def scale_value(s: int) -> float:
    return float("nan") if s == SCALE_NAN else 2.0 ** (min(max(int(s), SCALE_MIN), SCALE_MAX) - 127)


def code_place(n: int):
    """Latent n of a token -> (byte of the 256, bit of its magnitude, byte and bit of its sign)."""
    j, i = divmod(n, BLOCK)
    word, e = divmod(i, 8)
    if j & 4:
        word = (word + 2) % 4
    at = 16 * j + 4 * word
    sign = 8 * e + 7 if e < 4 else 8 * (e - 4) + 3
    return at + (4 * e) // 8, (4 * e) % 8, at + sign // 8, sign % 8


def write_token(page: np.ndarray, page_size: int, pos: int, latent_bits: np.ndarray, rope_bits: np.ndarray):
    row = page[256 * pos: 256 * (pos + 1)]
    row[:] = 0
    vals = bf16_to_f64(latent_bits)
    for j in range(LATENT // BLOCK):
        codes, s = quantise_block(vals[BLOCK * j: BLOCK * (j + 1)])
        page[384 * page_size + 16 * pos + j] = s
        for i, c in enumerate(codes):
            mb, mbit, sb, sbit = code_place(BLOCK * j + i)
            row[mb] |= (int(c) & 7) << mbit
            row[sb] |= (int(c) >> 3) << sbit
    rope = page[256 * page_size + 128 * pos: 256 * page_size + 128 * (pos + 1)].view(np.uint16).reshape(8, 8)
    for c in range(8):
        rope[c ^ (pos & 7)] = rope_bits[8 * c: 8 * c + 8]


_PLACE = np.array([code_place(n) for n in range(LATENT)])


def read_tokens(cache: np.ndarray, page_size: int, slots) -> np.ndarray:
    """float64 [T,576] of the cached tokens at `slots`."""
    out = np.zeros((len(slots), LATENT + ROPE))
    for t, slot in enumerate(slots):
        page, pos = cache[slot // page_size], slot % page_size
        row = page[256 * pos: 256 * (pos + 1)].astype(np.int64)
        mag = E2M1[(row[_PLACE[:, 0]] >> _PLACE[:, 1]) & 7]
        sign = 1.0 - 2.0 * ((row[_PLACE[:, 2]] >> _PLACE[:, 3]) & 1)
        sc = np.array([scale_value(s) for s in page[384 * page_size + 16 * pos: 384 * page_size + 16 * (pos + 1)]])
        out[t, :LATENT] = mag * sign * np.repeat(sc, BLOCK)
        rope = page[256 * page_size + 128 * pos: 256 * page_size + 128 * (pos + 1)].view(np.uint16).reshape(8, 8)
        out[t, LATENT:] = bf16_to_f64(rope[np.arange(8) ^ (pos & 7)].reshape(-1))
    return out


def attend(q: np.ndarray, keys: np.ndarray, softmax_scale: float):
    """q float64 [R,576], keys float64 [n,576] (all visible) -> x [R,512], lse [R]."""
    if keys.shape[0] == 0:
        return np.zeros((q.shape[0], LATENT)), np.full(q.shape[0], -np.inf)
    s = q @ keys.T * softmax_scale
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    tot = e.sum(1, keepdims=True)
    return (e @ keys[:, :LATENT]) / tot, (top + np.log(tot))[:, 0]


class Tables:
    """Block table, lengths and counts with the page operations on them."""

    def __init__(self, num_seqs, stride, num_pages, page_size):
        self.table = np.full((num_seqs, stride), -1, dtype=np.int32)
        self.lens = np.zeros(num_seqs, dtype=np.int32)
        self.ref = np.zeros(num_pages, dtype=np.int32)
        self.page_size = page_size

    def _free(self):
        return [int(p) for p in np.flatnonzero(self.ref == 0)]

    def _pages(self, n):
        return -(-int(n) // self.page_size)

    def extend(self, seqs, new_tokens, max_new):
        """Item i takes the free pages behind what the items before it ask for."""
        P, free, asked = self.page_size, self._free(), 0
        slots = np.full((len(seqs), max_new), -1, dtype=np.int32)
        for i, (s, k) in enumerate(zip(seqs, new_tokens)):
            if not (0 <= s < len(self.lens)) or not (0 <= k <= max_new) or \
                    self.lens[s] + k > self.table.shape[1] * P:
                continue
            if k and self.lens[s] % P and not 0 <= self.table[s, self.lens[s] // P] < len(self.ref):
                continue
            have, end = self._pages(self.lens[s]), self._pages(self.lens[s] + k)
            first, asked = asked, asked + end - have
            if end > have and asked > len(free):
                continue
            for j in range(have, end):
                self.table[s, j] = free[first + j - have]
                self.ref[self.table[s, j]] = 1
            for t in range(k):
                at = self.lens[s] + t
                slots[i, t] = self.table[s, at // P] * P + at % P
            self.lens[s] += k
        return slots

    def fork(self, parents, children, caches):
        """caches: list of layers [num_pages, page_bytes], changed in place."""
        P, free, asked = self.page_size, self._free(), 0
        before = self.lens.copy()  # lengths count as they were before the call
        for p, c in zip(parents, children):
            if not (0 <= p < len(before)) or not (0 <= c < len(before)) or p == c or before[c] != 0:
                continue
            held = self.table[p, :self._pages(before[p])]
            if ((held < 0) | (held >= len(self.ref))).any():
                continue
            full, tail = divmod(int(before[p]), P)
            if tail:
                asked += 1
                if asked > len(free):
                    continue
                new = free[asked - 1]
                self.table[c, full] = new
                self.ref[new] = 1
                for layer in caches:
                    a, b = layer[self.table[p, full]], layer[new]
                    for off, row in ((0, 256), (256 * P, 128), (384 * P, 16)):
                        b[off: off + row * tail] = a[off: off + row * tail]
            for j in range(full):
                self.table[c, j] = self.table[p, j]
                self.ref[self.table[p, j]] += 1
            self.lens[c] = before[p]

    def release(self, seqs):
        for s in seqs:
            if not 0 <= self.lens[s] <= self.table.shape[1] * self.page_size:
                continue
            for j in range(self._pages(self.lens[s])):
                self.ref[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = 0

    def compact(self, caches):
        n = int((self.ref != 0).sum())
        holes = [p for p in range(n) if self.ref[p] == 0]
        movers = [p for p in range(n, len(self.ref)) if self.ref[p] != 0]
        for a, b in zip(movers, holes):
            for layer in caches:
                layer[b] = layer[a]
            self.ref[b], self.ref[a] = self.ref[a], 0
            self.table[self.table == a] = b
        return n
