"""GPU parity of the 4-bit cache's page operations with the oracle's loops:
tables, counts, lengths, slots and page contents are equal."""

import numpy as np
import pytest
import torch

import mla_decode_query_gb300 as mq
from oracle import kv4_oracle as ko

pytestmark = pytest.mark.gpu


def _ok(st):
    assert st == mq.MLAQP_OK, mq.mlaqp_last_error()


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _device_status():
    st, word = mq.mlaqp_device_status(reset=True)
    _ok(st)
    return word


class Pool:
    """Tables and layers on the device beside the oracle's."""

    def __init__(self, num_seqs, stride, num_pages, P, layers=2, interleaved=False, seed=0, pad=0):
        self.o = ko.Tables(num_seqs, stride, num_pages, P)
        rng = np.random.default_rng(seed)
        page = 400 * P
        self.caches = [rng.integers(0, 256, (num_pages, page), dtype=np.uint8) for _ in range(layers)]
        self.layers, self.interleaved, self.pad = layers, interleaved, pad
        if interleaved:
            self.buf = torch.full((num_pages, layers, page + pad), 0xA5, dtype=torch.uint8, device="cuda")
            self.page_stride, self.layer_stride = layers * (page + pad), page + pad
        else:
            self.buf = torch.full((layers, num_pages, page + pad), 0xA5, dtype=torch.uint8, device="cuda")
            self.page_stride, self.layer_stride = page + pad, num_pages * (page + pad)
        for l, c in enumerate(self.caches):
            self._layer(l)[:, :page] = torch.from_numpy(c).cuda()
        self.table, self.lens, self.ref = _i32(self.o.table), _i32(self.o.lens), _i32(self.o.ref)
        self.ws = torch.full((mq.mlaqp_kv4_pages_workspace(num_pages, 64),), 0xFF, dtype=torch.uint8, device="cuda")
        self.n_live = _i32([-7])

    def _layer(self, l):
        return self.buf[:, l] if self.interleaved else self.buf[l]

    def tables(self):
        return (self.table, self.table.shape[1], self.table.shape[0], self.lens, self.ref, self.ref.numel(),
                self.o.page_size)

    def pool(self):
        return self.buf, self.page_stride, self.layer_stride, self.layers

    def extend(self, seqs, new, max_new):
        slots = torch.full((len(seqs), max_new), 77, dtype=torch.int32, device="cuda")
        _ok(mq.mlaqp_kv4_extend(*self.tables(), _i32(seqs), _i32(new), len(seqs), slots, max_new))
        np.testing.assert_array_equal(slots.cpu().numpy(), self.o.extend(seqs, new, max_new))

    def fork(self, parents, children):
        _ok(mq.mlaqp_kv4_fork(*self.tables(), _i32(parents), _i32(children), len(parents), *self.pool(), self.ws,
                              self.ws.numel()))
        self.o.fork(parents, children, self.caches)

    def release(self, seqs):
        _ok(mq.mlaqp_kv4_release(*self.tables(), _i32(seqs), len(seqs)))
        self.o.release(seqs)

    def compact(self):
        _ok(mq.mlaqp_kv4_compact(*self.tables(), *self.pool(), self.n_live, self.ws, self.ws.numel()))
        assert self.n_live.item() == self.o.compact(self.caches)

    def check(self, contents=True):
        torch.cuda.synchronize()
        np.testing.assert_array_equal(self.ref.cpu().numpy(), self.o.ref)
        np.testing.assert_array_equal(self.lens.cpu().numpy(), self.o.lens)
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.o.table)
        if contents:
            page = 400 * self.o.page_size
            for l, c in enumerate(self.caches):
                got = self._layer(l).cpu().numpy()
                np.testing.assert_array_equal(got[:, :page], c)
                assert (got[:, page:] == 0xA5).all()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_random_life_of_a_pool(cuda_device, P, interleaved):
    p = Pool(24, 6, 70, P, layers=3, interleaved=interleaved, seed=P, pad=16)
    rng = np.random.default_rng(P + 1)
    _device_status()
    for step in range(40):
        live = [int(s) for s in np.flatnonzero(p.o.lens > 0)]
        empty = [int(s) for s in np.flatnonzero(p.o.lens == 0)]
        free = int((p.o.ref == 0).sum())
        what = rng.integers(0, 4)
        if what == 0 or not live:
            seqs = [int(s) for s in rng.permutation(24)[:rng.integers(1, 9)]]
            new = [int(k) for k in rng.integers(0, 2 * P, len(seqs))]
            new = [min(k, 6 * P - int(p.o.lens[s])) for s, k in zip(seqs, new)]
            while seqs and sum(-(-k // P) + 1 for k in new) > free:
                seqs, new = seqs[:-1], new[:-1]
            if seqs:
                p.extend(seqs, new, 2 * P)
        elif what == 1 and empty and free >= 8:
            n = min(len(empty), 1 + int(rng.integers(0, 8)))
            p.fork([int(live[i]) for i in rng.integers(0, len(live), n)], empty[:n])
        elif what == 2:
            p.release([int(s) for s in rng.permutation(live)[:rng.integers(1, max(2, len(live) // 2))]])
        else:
            p.compact()
        p.check(contents=step % 5 == 4)
    p.compact()
    p.check()
    assert _device_status() == 0


def test_extension_by_many_pages_and_none(cuda_device):
    p = Pool(5, 600, 2500, 16, layers=1)
    p.extend([0, 1, 2], [0, 9600, 1], 9600)
    p.extend([2, 0, 3], [5, 17, 8000], 8000)
    p.extend([2, 4], [10, 0], 10)
    p.check()


def test_many_list_items(cuda_device):
    p = Pool(3000, 2, 6000, 16, layers=1)
    p.extend(list(range(0, 2000)), [1 + i % 20 for i in range(2000)], 20)
    p.check(contents=False)
    p.ws = torch.empty(mq.mlaqp_kv4_pages_workspace(6000, 1000), dtype=torch.uint8, device="cuda")
    p.fork([(7 * i) % 2000 for i in range(1000)], list(range(2000, 3000)))
    p.check()
    p.release(list(range(0, 3000, 2)))
    p.compact()
    p.check()


@pytest.mark.parametrize("pages,live", [(1, 1), (1, 0), (31, 17), (32, 32), (33, 1), (64, 0), (1025, 500), (40000, 33333)])
def test_compact_counts(cuda_device, pages, live):
    p = Pool(7, pages, pages, 16, layers=1, seed=pages)
    rng = np.random.default_rng(pages + live)
    order = rng.permutation(pages)[:live]
    for k, pg in enumerate(order):
        s = k % 7
        p.o.table[s, k // 7] = pg
        p.o.ref[pg] = 1
        p.o.lens[s] = 16 * (k // 7 + 1)
    p.table, p.lens, p.ref = _i32(p.o.table), _i32(p.o.lens), _i32(p.o.ref)
    if pages <= 1025:
        p.compact()
        p.check()
    else:  # the oracle's loops are too slow: its rule in numpy
        _ok(mq.mlaqp_kv4_compact(*p.tables(), *p.pool(), p.n_live, p.ws, p.ws.numel()))
        old = p.o.ref.copy()
        holes, movers = np.flatnonzero(old[:live] == 0), live + np.flatnonzero(old[live:])
        remap = np.arange(pages)
        remap[movers] = holes
        t = p.o.table
        np.testing.assert_array_equal(p.table.cpu().numpy(), np.where(t >= 0, remap[t], t))
        ref = p.ref.cpu().numpy()
        assert (ref[:live] == 1).all() and not ref[live:].any() and p.n_live.item() == live
        want = p.caches[0].copy()
        want[holes] = p.caches[0][movers]
        np.testing.assert_array_equal(p.buf[0].cpu().numpy()[:, :6400], want)


def test_out_of_pages_leaves_the_sequence_as_it_was(cuda_device):
    p = Pool(6, 8, 5, 16)
    _device_status()
    p.extend([0, 1, 2], [40, 60, 3], 60)  # three pages, then four (not there), then one behind them
    assert _device_status() == mq.MLAQP_DEVSTATUS_OUT_OF_PAGES
    p.check()
    assert p.o.lens.tolist() == [40, 0, 0, 0, 0, 0]
    p.fork([0, 0, 0], [1, 2, 3])  # two free pages for three tails
    assert _device_status() == mq.MLAQP_DEVSTATUS_OUT_OF_PAGES
    p.check()
    assert p.o.lens.tolist() == [40, 40, 40, 0, 0, 0]
    p.extend([0], [8], 8)  # fills the last page: none needed
    assert _device_status() == 0
    p.check()


def test_bad_items_are_left_out_and_reported(cuda_device):
    p = Pool(4, 3, 20, 16)
    _device_status()
    p.extend([0, 9, -1, 1, 2], [10, 3, 3, 49, 11], 10)  # two sequences out of range, a row too short, over max_new
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    p.check()
    p.fork([0, 0, 5, 0, 1], [1, 0, 2, 4, 2])  # a child that is its parent, a parent and a child out of range
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    p.check()
    p.fork([0], [1])  # not empty any more
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    p.check()
    _ok(mq.mlaqp_kv4_release(*p.tables(), _i32([7, 0, 0]), 3))  # out of range, and one listed twice
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    p.o.release([0])
    p.check()


@pytest.mark.parametrize("P,layers", [(16, 1), (128, 3)])
def test_copy_pages(cuda_device, P, layers):
    p = Pool(1, 1, 12, P, layers=layers, pad=32)
    _device_status()
    src, dst = [3, 3, 7, -1, 5, 12], [0, 1, 11, 4, -2, 6]
    _ok(mq.mlaqp_kv4_copy_pages(*p.pool(), 12, P, _i32(src), _i32(dst), len(src)))
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX  # page 12
    for c in p.caches:
        c[0] = c[1] = c[3]
        c[11] = c[7]
    p.check()


def test_beam_step_in_a_graph(cuda_device):
    p = Pool(8, 6, 60, 16, layers=2)
    p.extend([0, 1, 2], [33, 16, 40], 40)
    par, chi, gone, one = _i32([0, 2, 2]), _i32([3, 4, 5]), _i32([0, 1]), _i32([1, 1, 1])
    slots = torch.empty(3, 1, dtype=torch.int32, device="cuda")
    _ok(mq.mlaqp_kv4_prewarm())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _ok(mq.mlaqp_kv4_fork(*p.tables(), par, chi, 3, *p.pool(), p.ws, p.ws.numel()))
        _ok(mq.mlaqp_kv4_release(*p.tables(), gone, 2))
        _ok(mq.mlaqp_kv4_extend(*p.tables(), chi, one, 3, slots, 1))
    g.replay()
    p.o.fork([0, 2, 2], [3, 4, 5], p.caches)
    p.o.release([0, 1])
    np.testing.assert_array_equal(slots.cpu().numpy(), p.o.extend([3, 4, 5], [1, 1, 1], 1))
    p.check()


@pytest.mark.parametrize("pages", [5, 127, 4099, 33000, 140001])
@pytest.mark.parametrize("offset", [0, 1])
def test_counts_of_any_alignment(cuda_device, pages, offset):
    # free pages are found wherever the counts begin and however many there are
    p = Pool(4, pages, pages, 16, layers=0)
    rng = np.random.default_rng(pages)
    p.o.ref[:] = rng.integers(0, 2, pages) * rng.integers(1, 1 << 30, pages)
    at = torch.zeros(pages + offset, dtype=torch.int32, device="cuda")
    p.ref = at[offset:]
    p.ref.copy_(_i32(p.o.ref))
    free = int((p.o.ref == 0).sum())
    take = [free // 3, 0, free // 2]
    p.extend([2, 1, 0], [16 * n for n in take], 1 + 16 * max(take))
    p.check(contents=False)
    assert _device_status() == 0
