"""Page digests and page selection at the ends of their arguments' ranges, against
the CPU oracle.  Digests, tables and lengths are whole numbers and equal."""

import numpy as np
import pytest
import torch

from test_gpu_kv4_select import BAD_INDEX, Digests, Select, _query, _rand_cache, _rand_digests

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("max_new", [2 ** 31 - 1, 10 ** 6])
def test_more_new_tokens_than_a_row_holds(cuda_device, P, max_new):
    rng = np.random.default_rng(P)
    c = _rand_cache(rng, 12, P)
    table = rng.permutation(12).reshape(3, 4)
    d = Digests(c, P, table, [4 * P, 3 * P + 5, P - 1])
    d.run([0, 1, 2], [max_new, P + 6, max_new], max_new)
    d.check([*table[0], table[1, 1], table[1, 2]])


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_pages_of_many_sequences(cuda_device, P):
    """So many candidates that two warps have a page: special values in pages that 20 sequences share."""
    rng = np.random.default_rng(60 + P)
    pages = 48
    c = _rand_cache(rng, pages, P)
    codes, scales = c[:, :256 * P].reshape(pages, P, 16, 16), c[:, 384 * P:].reshape(pages, P, 16)
    rope = c[:, 256 * P:384 * P].view(np.uint16).reshape(pages, P, 64)
    for j in range(0, 30, 6):
        t, block = rng.integers(0, P), rng.integers(0, 16)
        scales[j, t, block] = 255                                   # a NaN block
        rope[j + 1, t, rng.integers(0, 64)] = (0x7F80, 0xFF80, 0x7FC1)[j % 3]
        scales[j + 2] = rng.integers(87, 168, (P, 16))
        scales[j + 3, t, block], codes[j + 3, t, block] = 165, 0     # the largest scale stands over zeros
        codes[j + 4] = 0
        codes[j + 4, t, block, 3] = 0x70                            # one value in the page
        rope[j + 5] = 0
        rope[j + 5, t, j] = 0xBF80
    d = Digests(c, P, np.tile(np.arange(pages), (20, 1)), [pages * P] * 20)
    d.run(range(20), [pages * P] * 20, pages * P)
    d.check(range(pages))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_len,k,first,last", [(1, 3, 1, 2), (4, 6, 2, 4), (1, 40, 20, 20), (3, 5, 1, 2)])
@pytest.mark.parametrize("pages", [60, 3000])
def test_pages_out_of_range_are_reported_whether_or_not_there_is_a_choice(cuda_device, pages, q_len, k, first, last, e4m3):
    """Also where the first and the last pages are all that is taken."""
    rng = np.random.default_rng(pages + k)
    q_dev, q = _query(rng, 2 * q_len, 8, e4m3)
    table = np.stack([rng.permutation(pages) for _ in range(2)])
    s = Select(_rand_digests(rng, pages), 16, table, [pages * 16, pages * 16 - 5], q_dev, q, e4m3)
    s.run(2, q_len, k, first, last)
    for row, at, bad in ((0, first, -1), (1, pages - last - 1, pages), (1, pages // 2, 2 ** 31 - 1)):
        s.table[:] = table
        s.table[row, at] = bad
        s.t.copy_(torch.from_numpy(s.table))
        s.run(2, q_len, k, first, last, status=BAD_INDEX)
    # pages that are taken anyway are the attention's to report
    s.table[:] = table
    s.table[0, 0], s.table[1, -1] = -1, pages
    s.t.copy_(torch.from_numpy(s.table))
    s.run(2, q_len, k, first, last)
