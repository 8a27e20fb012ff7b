"""Attention over the 4-bit cache where its arithmetic can be told to a token:
every visible token counts once wherever the work is cut, and probabilities
keep FP16's 11 bits.

Tolerances, from the number formats:
  every token once   with queries of zero all weights are 1/n and every code
                     and sum is exact in FP32, so x is off by its rounding to
                     BF16 alone: 2^-9 |x|, doubled.  lse is ln n: 1e-5.
  probabilities      2^-9 |x| for BF16, and 2^-11 sum_t p |K| for FP16
                     probabilities; 2^-14 sum_t p |K| covers the scores (sums
                     of four products, a factor of log2 e rounded to FP32) and
                     exp.
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
