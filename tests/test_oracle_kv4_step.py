"""Pins of the oracle of norm, rotation, digests and page selection (CPU only)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import kv4_oracle as ko
from oracle import kv4_step_oracle as so


def _bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _keys(rng, n):
    """Values that a cache can hold."""
    rows = _bits(np.concatenate([rng.standard_normal((n, 512)) * 3, rng.standard_normal((n, 64))], 1))
    cache = np.zeros((1, 400 * 128), dtype=np.uint8)
    for t in range(n):
        ko.write_token(cache[0], 128, t, rows[t, :512], rows[t, 512:])
    return ko.read_tokens(cache, 128, range(n))


def test_norm_is_the_formula_and_keeps_the_rows_without_a_weight():
    rng = np.random.default_rng(0)
    x, w = _bits(rng.standard_normal((5, 512)) * 4), _bits(rng.standard_normal(512))
    v = oracle.bf16_to_f64(x)
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-5) * oracle.bf16_to_f64(w)
    # mean, sum, root, reciprocal (halves of the first two's errors), two products: 5 roundings of 2^-24
    assert np.abs(so.normalise(x, w, 1e-5) - want).max() <= 5 * 2.0 ** -24 * np.abs(want).max()
    assert np.array_equal(so.normalise(x, None, 1e-5), v)


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_by_a_right_angle_and_its_length(halves):
    rng = np.random.default_rng(1)
    bits = _bits(rng.standard_normal((3, 64)))
    v = oracle.bf16_to_f64(bits)
    quarter = np.concatenate([np.zeros(32), np.ones(32)])
    out = so.rotate(bits, np.tile(quarter, (3, 1)), halves)
    a, b = (slice(0, 32), slice(32, 64)) if halves else (slice(0, None, 2), slice(1, None, 2))
    assert np.array_equal(out[:, a], -v[:, b]) and np.array_equal(out[:, b], v[:, a])
    phi = rng.uniform(0, 6, (3, 32))
    out = so.rotate(bits, np.concatenate([np.cos(phi), np.sin(phi)], 1), halves)
    np.testing.assert_allclose(out[:, a] ** 2 + out[:, b] ** 2, v[:, a] ** 2 + v[:, b] ** 2, rtol=1e-12)


def test_tokens_as_the_cache_oracle_writes_them():
    rng = np.random.default_rng(2)
    x = _bits(rng.standard_normal((4, 512)) * np.array([[1e-3], [1], [50], [0]]))
    for t in range(4):
        page = np.zeros(400 * 16, dtype=np.uint8)
        ko.write_token(page, 16, 3, x[t], _bits(np.zeros(64)))
        row, scales = so.codes_and_scales(so.normalise(x[t:t + 1], None, 0.0)[0])
        assert np.array_equal(row, page[768:1024]) and np.array_equal(scales, page[6144 + 48:6144 + 64])


def test_digest_bounds_every_token_within_a_step():
    rng = np.random.default_rng(3)
    keys = _keys(rng, 32)
    d = so.digest(keys)
    v = d[:1152].view(np.int8).astype(np.float64)
    for part, hi, lo, e in ((keys[:, :512], v[:512], v[512:1024], d[1152]), (keys[:, 512:], v[1024:1088], v[1088:], d[1153])):
        step = 2.0 ** (int(e) - 127)
        assert (hi * step >= part.max(0)).all() and (hi * step < part.max(0) + step).all()
        assert (lo * step <= part.min(0)).all() and (lo * step > part.min(0) - step).all()
        assert np.abs(part).max() > 127 * step / 2  # the smallest step there is
    assert (d[1154:] == 0).all()


@pytest.mark.parametrize("value,byte", [(0.0, 67), (127.0, 127), (127.0078125, 128), (2.0 ** -80, 67), (127 * 2.0 ** 60, 187),
                                        (128 * 2.0 ** 60, 255), (np.inf, 255), (np.nan, 255)])
def test_digest_exponents(value, byte):
    keys = np.zeros((16, 576))
    keys[3, 570] = -value
    d = so.digest(keys)
    assert d[1152] == 67 and d[1153] == byte
    if byte == 255:
        assert not d[1024:1152].any()


def test_scores_bound_the_sum_of_the_heads_scores():
    rng = np.random.default_rng(4)
    for H in (1, 8, 16):
        keys = _keys(rng, 16)
        q = rng.standard_normal((H, 576)) * np.exp(rng.standard_normal((H, 1)))
        up, down, f = so.query_sums(q)
        assert np.abs(q).max() <= 2047 * 2.0 ** f < 2 * np.abs(q).max() * (1 + 2.0 ** -10)
        # half a step of q times the keys is what rounding q can take away; the score's own roundings 2^-23 of it
        slack = 0.5 * 2.0 ** f * H * np.abs(keys).sum(1).max()
        bound = float(so.scores(q, so.digest(keys)[None])[0]) * 2.0 ** f
        assert bound * (1 + 2.0 ** -20) + slack >= (q @ keys.T).sum(0).max()


def test_selection_takes_first_last_and_best_and_ties_to_the_lowest():
    P = 16
    digests = np.zeros((12, 1168), dtype=np.uint8)
    digests[:, 1152:1154] = 127
    q = np.zeros((1, 576))
    q[0, 0] = 1.0
    best = [0, 9, 3, 7, 3, 9, 9, 1, 2, 5, 0, 0]
    digests[:, 0] = best
    row = list(range(12))
    assert so.select(q, digests, row, 12 * P, P, 5, 1, 1) == ([0, 1, 5, 6, 11], 5 * P)
    assert so.select(q, digests, row, 12 * P - 3, P, 4, 1, 1) == ([0, 1, 5, 11], 4 * P - 3)
    assert so.select(q, digests, row, 12 * P, P, 3, 1, 2) == ([0, 10, 11], 3 * P)
    assert so.select(q, digests, row, 11 * P + 1, P, 12, 1, 1) == (row, 11 * P + 1)
    assert so.select(q, digests, row, 0, P, 4, 1, 1) == ([], 0)
    row[5] = 99  # out of range
    assert so.select(q, digests, row, 12 * P, P, 5, 1, 1)[0] == [0, 1, 3, 6, 11]
