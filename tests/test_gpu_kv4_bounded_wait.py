"""The attention kernel's waits are bounded: with any one of the hand-overs
between its warps never taking place, the call ends, the device status says
so, and the calls behind it are right (the kernel had let its copies and
products land and given its tensor memory back)."""

import numpy as np
import pytest
import torch

import mla_decode_query_gb300 as mq
from test_gpu_kv4_attend import Case, _device_status, _ok

pytestmark = pytest.mark.gpu

LIMIT = 2_000_000  # 2 ms
STAGES = 13
LATER = (2, 5, 7, 9, 13)  # hand-overs that a CTA of one tile does not wait for


def _held(c, held, limit=LIMIT):
    return mq.mlaqp_debug_kv4_attend_bounded_wait(
        c.dev_q, c.q_stride, c.dtype, c.q_scale, *c.cache.args(), c.dev_table, c.table.shape[1], c.table.shape[0],
        c.dev_lens, c.dev_seqs, c.B, c.q_len, c.H, c.scale, c.x, c.x_stride, c.lse, c.ws, c.ws.numel(), limit, held)


def _check_every_stage(c, stages):
    _device_status()
    _ok(c.run())
    x, lse = c.outputs()
    assert _device_status() == 0
    for held in stages:
        _ok(_held(c, held))
        torch.cuda.synchronize()
        assert _device_status() & mq.MLAQP_DEVSTATUS_WAIT_TIMEOUT, held
        for _ in range(2):
            c.x.fill_(0x5A5A)
            c.lse.fill_(123.0)
            _ok(c.run())
            again = c.outputs()
            np.testing.assert_array_equal(again[0], x, err_msg=f"after {held}")
            np.testing.assert_array_equal(again[1], lse, err_msg=f"after {held}")
            assert _device_status() == 0, held
    # nothing held: the limit alone changes nothing
    _ok(_held(c, 0, 10 ** 9))
    again = c.outputs()
    np.testing.assert_array_equal(again[0], x)
    np.testing.assert_array_equal(again[1], lse)
    assert _device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,H", [(1, 16), (2, 16)])
def test_one_tile(cuda_device, q_len, H, dtype):
    c = Case([60], q_len=q_len, H=H, dtype=dtype)
    _ok(c.run())
    c.check()
    # 32 rows with BF16 queries copy a tile in four units, more than there are places
    later = [h for h in LATER if h != 2 or q_len == 1 or dtype == "e4m3"]
    _check_every_stage(c, [h for h in range(1, STAGES + 1) if h not in later])
    # the others are not waited for
    for held in later:
        _ok(_held(c, held, 10 ** 8))
        c.check()
        assert _device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,H,B", [(1, 16, 200), (2, 16, 120)])
def test_several_tiles_and_sequences_a_cta(cuda_device, q_len, H, B, dtype):
    rng = np.random.default_rng(B)
    c = Case([int(n) for n in rng.integers(300, 700, B)], P=32, q_len=q_len, H=H, dtype=dtype, seed=B)
    _check_every_stage(c, range(1, STAGES + 1))
    x, lse = c.outputs()
    for b in (0, 57, B - 1):
        keys = c.keys(b)
        m = (b + 1) * q_len - 1
        c.compare(x[m], lse[m], c.q[m], keys, f"sequence {b}")
