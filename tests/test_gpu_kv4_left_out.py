"""What the device finds out of range is left out, reported, and nothing else
changes: pages of the attention."""

import numpy as np
import pytest

import mla_decode_query_gb300 as mq
from test_gpu_kv4_attend import Case, _device_status, _ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,H", [(1, 16), (3, 5), (3, 11)])
@pytest.mark.parametrize("n", [1, 10, 32, 128, 129, 700, 20000])
def test_a_row_whose_pages_are_all_bad_is_an_empty_row(cuda_device, n, q_len, H, dtype):
    # one tile (a CTA writes the row), several (the join does)
    c = Case([n, 60, n], P=32, q_len=q_len, H=H, dtype=dtype, seed=n)
    c.dev_table[0] = -1
    c.dev_table[2] = 10 ** 6
    _device_status()
    _ok(c.run())
    x, lse = c.outputs()
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    for b in (0, 2):
        rows = slice(b * q_len, (b + 1) * q_len)
        assert not x[rows].any() and np.isneginf(lse[rows]).all(), b
    keys = c.keys(1)
    for i in range(q_len):
        m = q_len + i
        c.compare(x[m], lse[m], c.q[m], keys[:60 - (q_len - 1 - i)], f"intact, token {i}")


@pytest.mark.parametrize("n", [33, 129, 5000])
def test_only_the_last_query_token_sees_a_good_page(cuda_device, n):
    # the last token alone lies on a good page
    n = n // 16 * 16 + 1
    c = Case([n], P=16, q_len=2, H=8)
    c.dev_table[0, :n // 16] = -1
    _device_status()
    _ok(c.run())
    x, lse = c.outputs()
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    assert not x[0].any() and np.isneginf(lse[0]).all()
    c.compare(x[1], lse[1], c.q[1], c.keys(0)[n - 1:], "last token")


def test_a_nan_beside_bad_pages_still_spoils_its_row(cuda_device):
    # the only page that is there holds a NaN, before and behind bad ones
    for where in (0, 2, 4):
        c = Case([5 * 128], P=128, H=8, seed=where)
        c.dev_table[0, [p for p in range(5) if p != where]] = -1
        c.cache.buf[c.table[0, where], 384 * 128:] = 255
        _ok(c.run())
        x, lse = c.outputs()
        assert np.isnan(x).all() and np.isnan(lse).all()
    _device_status()
