"""What the device finds out of range is left out, reported, and nothing else
changes: pages of the attention, parents of a fork, lengths of a
release, the page that an extension goes on in, table entries of a compaction."""

import numpy as np
import pytest
import torch

import mla_decode_query_gb300 as mq
from test_gpu_kv4_attend import Case, _device_status, _ok
from test_gpu_kv4_pages import Pool, _i32

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


class Rows(Pool):
    """A pool whose tables are written to on the device behind the oracle's back."""

    def put(self, seq, j, page):
        self.table[seq, j] = page
        self.o.table[seq, j] = page


@pytest.mark.parametrize("bad", [-1, 40, 1 << 26, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("at", [0, 2, 3])
def test_a_fork_from_a_row_with_a_bad_page_is_left_out(cuda_device, at, bad):
    # three full pages and a tail; the items around it go through, with the
    # pages that they would get without it
    p = Rows(8, 6, 40, 16)
    p.extend([0, 1, 2], [53, 20, 37], 53)
    p.put(0, at, bad)
    _device_status()
    before = p.table.clone()
    _ok(mq.mlaqp_kv4_fork(*p.tables(), _i32([1, 0, 2, 0]), _i32([3, 4, 5, 6]), 4, *p.pool(), p.ws, p.ws.numel()))
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    p.o.fork([1, 0, 2, 0], [3, 4, 5, 6], p.caches)
    assert p.o.lens.tolist() == [53, 20, 37, 20, 0, 37, 0, 0]
    p.check()
    assert torch.equal(p.table[[4, 6]], before[[4, 6]])


def test_a_fork_of_full_pages_only_checks_them_all(cuda_device):
    p = Rows(4, 80, 100, 16)
    p.extend([0], [64 * 16], 64 * 16)
    p.put(0, 63, 100)
    _device_status()
    _ok(mq.mlaqp_kv4_fork(*p.tables(), _i32([0]), _i32([1]), 1, *p.pool(), p.ws, p.ws.numel()))
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    p.check()
    p.put(0, 63, p.o.table[0, 0])
    p.put(0, 64, -1)  # behind its length: not looked at
    p.fork([0], [1])
    assert _device_status() == 0
    p.check()


@pytest.mark.parametrize("length", [-1, -2 ** 31, 6 * 16 + 1, 2 ** 31 - 1])
def test_a_release_of_a_bad_length_is_left_out(cuda_device, length):
    p = Pool(4, 6, 20, 16)
    p.extend([0, 1, 2], [40, 16, 5], 40)
    p.lens[1] = length
    p.o.lens[1] = length
    _device_status()
    _ok(mq.mlaqp_kv4_release(*p.tables(), _i32([0, 1, 1, 2]), 4))
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    p.o.release([0, 1, 1, 2])
    assert p.o.lens.tolist() == [0, length, 0, 0]
    p.check()


@pytest.mark.parametrize("bad", [-1, 20, 1 << 28, 2 ** 31 - 1])
def test_an_extension_of_a_bad_page_is_left_out(cuda_device, bad):
    p = Rows(5, 4, 20, 16)
    p.extend([0, 1, 2, 3], [18, 16, 3, 18], 18)
    p.put(0, 1, bad)
    p.put(1, 0, bad)  # full: what is added begins a page of its own
    p.put(3, 0, bad)  # not the page that goes on
    _device_status()
    slots = torch.full((5, 20), 77, dtype=torch.int32, device="cuda")
    _ok(mq.mlaqp_kv4_extend(*p.tables(), _i32([0, 1, 2, 3, 4]), _i32([20, 2, 14, 1, 16]), 5, slots, 20))
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    got = slots.cpu().numpy()
    assert (got[0] == -1).all()
    np.testing.assert_array_equal(got, p.o.extend([0, 1, 2, 3, 4], [20, 2, 14, 1, 16], 20))
    assert p.o.lens.tolist() == [18, 18, 17, 19, 16]
    p.check()
    p.extend([0], [0], 1)  # nothing added: nothing to write to
    assert _device_status() == 0
    p.check()


@pytest.mark.parametrize("left", [-1, 0, 3])
@pytest.mark.parametrize("bad", [15, 19, 20, 2 ** 31 - 1])
def test_an_entry_that_no_live_page_stands_for_stays_in_a_compaction(cuda_device, bad, left):
    # whatever an earlier call left in the workspace
    p = Rows(5, 4, 20, 16)
    p.extend([0, 1, 2, 3], [40, 33, 3, 48], 48)
    p.release([1])  # pages 3, 4, 5 are free: 7, 8 and 9 move there, 10..19 are free
    p.put(2, 0, bad)
    p.o.ref[6] = 0
    p.ref[6] = 0
    p.ws.view(torch.int32).fill_(left)
    _device_status()
    p.compact()
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    assert p.o.table[2, 0] == bad
    p.check()
