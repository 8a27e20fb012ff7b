"""Attention over the 4-bit cache where its arithmetic can be told to a token:
every visible token counts once wherever the work is cut, and probabilities
keep FP16's 11 bits.

Tolerances, from the number formats:
  every token once   with queries of zero all weights are 1/n and every code
                     and sum is exact in FP32, so x is off by its rounding to
                     BF16 alone: half a step, 2^-8 |x|.  lse is ln n: 1e-5.
  probabilities      2^-11 sum_t p |K| for FP16 probabilities; 2^-14 sum_t p |K|
                     covers the scores (sums of four products, a factor of log2 e
                     rounded to FP32) and exp.  |x| is a small part of that sum
                     here, so 2^-9 |x| beside it is enough for BF16.
  small query elements  each up to half of a step of 2^-20 of the row's largest
                     off, so a score by dS = 2^-21 largest scale sum |K|, a
                     probability by a factor of exp(+-2 dS), lse by dS.
  small p beside large scales  2^-8 |x| for BF16, 2^-11 and 2^-14 as above, and
                     half of a step of 2^-28 of the largest p 2^s for each
                     token, times codes of up to 6.
"""

import numpy as np
import pytest

from oracle import kv4_oracle as ko
from test_gpu_kv4_attend import Case, _bits, _device_status, _ok

pytestmark = pytest.mark.gpu


def _one_column_a_token(rng, T):
    """Token t holds 1.0 in latent 37 t mod 512 and nothing else."""
    r = np.zeros((T, 576), dtype=np.float32)
    t = np.arange(T)
    r[t, 37 * t % 512] = 1.0
    return _bits(r)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,H", [(1, 16), (1, 5), (2, 16), (7, 8)])
@pytest.mark.parametrize("lens", [[20000], [9000, 40, 5000], [40001, 129], [127, 128, 129, 383, 385], [3000] * 9])
def test_every_token_counts_once(cuda_device, lens, q_len, H, dtype):
    c = Case(lens, P=64, q_len=q_len, H=H, dtype=dtype, rows=_one_column_a_token, q=lambda rng, M, H: np.zeros((M, H, 576)))
    _device_status()
    _ok(c.run())
    x, lse = c.outputs()
    assert _device_status() == 0
    first = 0
    for b, length in enumerate(lens):
        for i in range(q_len):
            n = length - (q_len - 1 - i)
            count = np.bincount(37 * (first + np.arange(n)) % 512, minlength=512)
            want = count / n
            assert count.max() < 2 ** 7  # so that a token more or less shows beside 2^-8 of its column
            m = b * q_len + i
            assert (np.abs(x[m] - want) <= 2.0 ** -8 * want).all(), (b, i)
            assert (np.abs(lse[m] - np.log(n)) <= 1e-5).all(), (b, i)
        first += length


def balanced(lens, H, q_len, seed):
    """Rows and queries of sequences in which token 0 and all others, p times
    as likely each, nearly cancel, so that x shows the error of p; (rows, q)."""
    def rows(rng, T):
        r = np.zeros((T, 576))
        r[:, :512], r[:, 512:516] = -4.0, 1.0
        at = np.concatenate([[0], np.cumsum(lens)[:-1]])
        r[at, :512], r[at, 512:516] = 4.0, 0.0
        return _bits(r)

    def q(rng, M, H):
        others = np.repeat(np.array(lens, dtype=np.float64) - 1, q_len)
        delta = np.log(others)[:, None] + np.random.default_rng(seed).uniform(-0.1, 0.1, (M, H))
        v = np.zeros((M, H, 576))
        v[:, :, 512:516] = -delta[:, :, None] * np.array([0.5, 0.25, 0.15, 0.1])
        return v

    return rows, q


def balanced_bound(q, keys):
    x, lse = ko.attend(q, keys, 1.0)
    p = np.exp(q @ keys.T - lse[:, None])
    return x, 2.0 ** -9 * np.abs(x) + (2.0 ** -11 + 2.0 ** -14) * (p @ np.abs(keys[:, :512]))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 2])
def test_probabilities_keep_eleven_bits(cuda_device, q_len, dtype):
    lens = list(range(4, 129, 3))  # one tile each: a sequence is not cut, so p is what the tile holds
    rows, q = balanced(lens, 16, q_len, 5)
    c = Case(lens, P=64, q_len=q_len, H=16, dtype=dtype, rows=rows, q=q, scale=1.0)
    _ok(c.run())
    x, _ = c.outputs()
    for b in range(len(lens)):
        keys = c.keys(b)
        for i in range(q_len):
            m = b * q_len + i
            want, bound = balanced_bound(c.q[m], keys[:len(keys) - (q_len - 1 - i)])
            err = np.abs(x[m] - want)
            assert (err <= bound).all(), f"sequence {b} token {i}: off by {(err / bound).max()} of the bound"


@pytest.mark.parametrize("rope_top", [0.0, 2.0 ** 42])
def test_query_elements_far_below_the_largest_of_their_row(cuda_device, rope_top):
    # the largest meets latents of zero, so the small ones make the score
    def rows(rng, T):
        r = np.zeros((T, 576))
        r[:, :512] = rng.choice([-6, -4, -3, -2, -1.5, -1, -0.5, 0.5, 1, 1.5, 2, 3, 4, 6], (T, 512))
        r[:, :32] = 0.0
        return _bits(r)

    def q(rng, M, H):
        v = rng.choice([-1, 1], (M, H, 576)) * rng.uniform(1, 2, (M, H, 576)) * 2.0 ** -rng.integers(10, 25, (M, H, 576))
        v[:, :, :32] = 0.0
        v[:, :, 7] = 1.0
        v[:, :, 512:] = rope_top
        return v

    scale = 32.0
    c = Case([200, 33, 128], P=64, H=16, rows=rows, q=q, scale=scale, seed=12)
    _ok(c.run())
    x, lse = c.outputs()
    for b in range(3):
        keys = c.keys(b)
        wx, wl = ko.attend(c.q[b], keys, scale)
        p = np.exp(c.q[b] @ keys.T * scale - wl[:, None])
        ds = 2.0 ** -21 * max(1.0, 2.0 ** -40 * rope_top) * scale * np.abs(keys[:, :512]).sum(1).max()
        assert ds < 0.25 and np.ptp(c.q[b] @ keys.T * scale, axis=1).min() > 4 * ds  # the scores are told apart
        bound = 2.0 ** -9 * np.abs(wx) + (2.0 ** -11 + 2.0 ** -14 + np.expm1(2 * ds)) * (p @ np.abs(keys[:, :512]))
        assert (np.abs(x[b] - wx) <= bound).all(), b
        assert (np.abs(lse[b] - wl) <= ds + 1e-5).all(), b


def test_small_probabilities_beside_large_scales(cuda_device):
    # two tokens: the second is the likelier one, the first's latents are up
    # to 2^30 times as large; they share no latent
    octaves = list(range(0, 31))

    def rows(rng, T):
        r = np.zeros((T, 576))
        r[0::2, :256] = 6.0 * 2.0 ** np.array(octaves)[:, None]
        r[1::2, 256:512] = rng.choice([-6, -4, -3, -2, 2, 3, 4, 6], (T // 2, 256))
        r[1::2, 512] = 1.0
        return _bits(r)

    def q(rng, M, H):
        v = np.zeros((M, H, 576))
        v[:, :, 512] = rng.uniform(1, 6, (M, H))
        return v

    c = Case([2] * len(octaves), P=16, H=16, rows=rows, q=q, scale=1.0, seed=13)
    _ok(c.run())
    x, lse = c.outputs()
    for b, k in enumerate(octaves):
        keys = c.keys(b)
        wx, wl = ko.attend(c.q[b], keys, 1.0)
        p = np.exp(c.q[b] @ keys.T - wl[:, None])
        largest = np.maximum(p[:, 0] * 2.0 ** k, p[:, 1])
        bound = (2.0 ** -8 * np.abs(wx) + (2.0 ** -11 + 2.0 ** -14) * (p @ np.abs(keys[:, :512]))
                 + 2.0 ** -29 * 6.0 * largest[:, None])
        assert (np.abs(x[b] - wx) <= bound).all(), k
        assert (np.abs(lse[b] - wl) <= 1e-5).all(), k
