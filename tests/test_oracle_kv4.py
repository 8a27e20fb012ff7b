"""Pins of the 4-bit cache's CPU reference: codes, layout, scale rule,
attention and page operations on cases worked out by hand or by brute force."""

import numpy as np
import pytest

import oracle
from oracle import kv4_oracle as ko


def _bits(x):
    return oracle.f64_to_bf16_rne(np.asarray(x, dtype=np.float64))


def test_every_code_place_is_used_once():
    mags, signs = set(), set()
    for n in range(512):
        mb, mbit, sb, sbit = ko.code_place(n)
        for b in range(3):
            mags.add((mb, mbit + b))
        signs.add((sb, sbit))
    assert len(mags) == 1536 and len(signs) == 512 and not (mags & signs)
    assert mags | signs == {(b, i) for b in range(256) for i in range(8)}


def test_word_layout_of_one_block():
    # Block 0, word 0: magnitudes in nibble order, signs of elements 0..3 at
    # bits 7, 15, 23, 31 and of 4..7 at bits 3, 11, 19, 27.
    assert ko.code_place(0) == (0, 0, 0, 7)
    assert ko.code_place(1) == (0, 4, 1, 7)
    assert ko.code_place(3) == (1, 4, 3, 7)
    assert ko.code_place(4) == (2, 0, 0, 3)
    assert ko.code_place(7) == (3, 4, 3, 3)
    # block 4 (j & 4) holds its words 2, 3 first
    assert ko.code_place(128)[0] == 64 + 8
    assert ko.code_place(128 + 16)[0] == 64


@pytest.mark.parametrize("amax,byte", [
    (6.0, 127), (7.0, 127), (7.03125, 128), (8.0, 128), (3.5, 126), (3.515625, 127), (1.75, 125), (0.0, 87),
    (2.0 ** -60, 87), (2.0 ** 60, 167),
])
def test_scale_rule(amax, byte):
    v = np.zeros(32)
    v[7] = -amax
    codes, s = ko.quantise_block(v)
    assert s == byte
    if amax == 7.0:
        assert codes[7] == 15  # saturates at 6, half a step away


def test_ties_go_to_the_even_code():
    v = np.zeros(32)
    v[0] = 6.0
    for x, c in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (-0.25, 8), (5.03125, 7)):
        v[1] = x
        codes, s = ko.quantise_block(v)
        assert s == 127 and codes[1] == c, x


def test_non_finite_block_reads_as_nan():
    for bad in (np.nan, np.inf, -np.inf):
        v = np.ones(32)
        v[3] = bad
        codes, s = ko.quantise_block(v)
        assert s == 255 and not codes.any()


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
def test_write_then_read(page_size):
    rng = np.random.default_rng(page_size)
    cache = np.full((3, 400 * page_size), 0xA5, dtype=np.uint8)
    for pos in (0, 1, page_size - 1):
        lat = rng.standard_normal(512) * np.exp2(rng.integers(-6, 6, 512 // 32)).repeat(32)
        rope = rng.standard_normal(64)
        ko.write_token(cache[1], page_size, pos, _bits(lat), _bits(rope))
        got = ko.read_tokens(cache, page_size, [page_size + pos])[0]
        latq = oracle.bf16_to_f64(_bits(lat))
        for j in range(16):
            blk = latq[32 * j: 32 * j + 32]
            top = np.abs(blk).max()
            step = 2.0 ** np.ceil(np.log2(top / 7.0))
            assert np.abs(got[32 * j: 32 * j + 32] - blk).max() <= step  # half of the coarsest step, 2
        np.testing.assert_array_equal(got[512:], oracle.bf16_to_f64(_bits(rope)))
    assert (cache[0] == 0xA5).all() and (cache[2] == 0xA5).all()


def test_attention_against_brute_force():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 576)), rng.standard_normal((5, 576))
    x, lse = ko.attend(q, k, 0.1)
    for r in range(2):
        w = [np.exp(0.1 * float(sum(q[r, c] * k[t, c] for c in range(576)))) for t in range(5)]
        np.testing.assert_allclose(lse[r], np.log(sum(w)), rtol=1e-12)
        np.testing.assert_allclose(x[r], sum(w[t] * k[t, :512] for t in range(5)) / sum(w), rtol=1e-10)
    x, lse = ko.attend(q, k[:0], 0.1)
    assert not x.any() and np.isneginf(lse).all()


def test_page_operations_by_hand():
    t = ko.Tables(4, 4, 8, 16)
    caches = [np.zeros((8, 6400), dtype=np.uint8)]
    slots = t.extend([0, 2], [20, 16], 20)
    assert t.table[0, :2].tolist() == [0, 1] and t.table[2, 0] == 2
    assert slots[0, 16] == 16 and slots[1, 15] == 47 and slots[1, 16] == -1
    caches[0][1, :] = 7
    t.fork([0, 2], [1, 3], caches)
    assert t.table[1, :2].tolist() == [0, 3] and t.table[3, 0] == 2
    assert t.ref.tolist() == [2, 1, 2, 1, 0, 0, 0, 0] and t.lens.tolist() == [20, 20, 16, 16]
    assert caches[0][3, :1024].tolist() == [7] * 1024 and not caches[0][3, 1024:4096].any()
    t.release([0])
    assert t.ref.tolist() == [1, 0, 2, 1, 0, 0, 0, 0]
    assert t.compact(caches) == 3
    assert t.ref.tolist() == [1, 1, 2, 0, 0, 0, 0, 0] and t.table[1, :2].tolist() == [0, 1]
    assert caches[0][1, 0] == 7
