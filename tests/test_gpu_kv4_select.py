"""GPU parity of page digests and page selection with the CPU oracle, and of the
whole sparse step with float64.

Digests, tables and lengths are whole numbers and equal.  The sparse step's
attention is held to the bounds of test_gpu_kv4_attend.py over the pages taken.
"""

import numpy as np
import pytest
import torch

import mla_decode_query_gb300 as mq
from oracle import kv4_oracle as ko
from oracle import kv4_step_oracle as so

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
BAD_INDEX = mq.MLAQP_DEVSTATUS_BAD_INDEX


def _ok(st):
    assert st == mq.MLAQP_OK, mq.mlaqp_last_error()


def _device_status():
    st, word = mq.mlaqp_device_status(reset=True)
    _ok(st)
    return word


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _rand_cache(rng, pages, P, pad=0):
    """Bytes of a cache: any codes, scales of a spread of sizes, finite rope elements."""
    c = rng.integers(0, 256, (pages, 400 * P + pad), dtype=np.uint8)
    rope = (rng.standard_normal((pages, 64 * P)) * np.exp(rng.standard_normal((pages, 1)))).astype(np.float32)
    c[:, 256 * P:384 * P] = (rope.view(np.uint32) >> 16).astype(np.uint16).view(np.uint8).reshape(pages, 128 * P)
    c[:, 384 * P:400 * P] = rng.integers(120, 131, (pages, 16 * P))
    return c


# --------------------------------------------------------------------------
# Digests
# --------------------------------------------------------------------------

class Digests:
    def __init__(self, cache, P, table, lens, pad=0):
        self.host, self.P = cache, P
        self.cache = torch.from_numpy(cache).cuda()
        self.table, self.lens = np.asarray(table, dtype=np.int32), np.asarray(lens, dtype=np.int32)
        self.stride = 1168 + pad
        self.out = torch.full((len(cache), self.stride), 0x5A, dtype=torch.uint8, device="cuda")

    def run(self, seqs, new, max_new, status=0, stream=None):
        table = _i32(self.table)
        _ok(mq.mlaqp_kv4_digest(self.cache, self.cache.stride(0), len(self.host), self.P, table, table.stride(0),
                                len(self.table), _i32(self.lens), _i32(seqs), _i32(new), len(seqs), max_new, self.out,
                                self.stride, stream=stream))
        torch.cuda.synchronize()
        assert _device_status() == status

    def check(self, pages):
        want = np.full((len(self.host), self.stride), 0x5A, dtype=np.uint8)
        for p in pages:
            want[p, :1168] = so.digest(ko.read_tokens(self.host, self.P, range(p * self.P, (p + 1) * self.P)))
        np.testing.assert_array_equal(self.out.cpu().numpy(), want)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_pages_that_have_filled_up(cuda_device, P):
    rng = np.random.default_rng(P)
    cache = _rand_cache(rng, 24, P, pad=48)
    order = rng.permutation(24)
    table = np.full((5, 6), -1)
    lens = [3 * P, 4 * P - 1, 2 * P + 1, 0, P]
    at = 0
    for s, n in enumerate(lens):
        k = -(-n // P)
        table[s, :k] = order[at:at + k]
        at += k
    for new, want in (([1, 1, 1, 0, 1], [(0, 2), (4, 0)]),
                      ([0, 0, 0, 0, 0], []),
                      ([P, P, P, 3, P + 5], [(0, 2), (1, 2), (2, 1), (4, 0)]),   # more than there is: all of it
                      ([2 * P + 1, 3 * P - 1, 1, 0, 0], [(0, 0), (0, 1), (0, 2), (1, 1), (1, 2)]),
                      ([2 * P, 3 * P, 2, P + 1, 0], [(0, 1), (0, 2), (1, 0), (1, 1), (1, 2), (2, 1)])):
        d = Digests(cache, P, table, lens, pad=32)
        d.run([0, 1, 2, 3, 4], new, 4 * P)
        d.check([table[s, j] for s, j in want])
    d = Digests(cache, P, table, lens)
    d.run([2, 0], [2 * P, 1], 2 * P)  # a list in another order
    d.check([table[2, 0], table[2, 1], table[0, 2]])


def test_special_values(cuda_device):
    rng = np.random.default_rng(1)
    P = 16
    c = _rand_cache(rng, 14, P)
    scale, rope = slice(384 * P, 400 * P), slice(256 * P, 384 * P)
    c[0, :256 * P] = 0                                   # all latents zero
    c[1, rope] = 0
    c[2, 384 * P + 5] = 255                              # a NaN block
    c[3, rope.start:rope.start + 2] = 0x80, 0x7F         # an infinity
    c[4, rope.start + 126:rope.start + 128] = 0x01, 0xFF  # a NaN
    c[5, scale] = 87                                     # the smallest latents there are
    c[6, scale] = 167                                    # the largest
    c[7, scale] = rng.integers(0, 255, 16 * P)           # scale bytes out of range read as the nearer end
    c[8, rope] = np.tile(np.array([1, 0], dtype=np.uint8), 64 * P)        # BF16's smallest number
    c[9, rope] = np.tile(np.array([0x7F, 0x7F], dtype=np.uint8), 64 * P)  # its largest: no exponent for it
    c[10, rope] = np.tile(np.array([0xFE, 0x60], dtype=np.uint8), 64 * P)  # 127 * 2^60
    c[11, rope] = np.tile(np.array([0xFF, 0x60], dtype=np.uint8), 64 * P)  # the number above it
    c[12, rope] = np.tile(np.array([0x00, 0x80], dtype=np.uint8), 64 * P)  # -0
    d = Digests(c, P, np.arange(14).reshape(1, 14), [14 * P])
    d.run([0], [14 * P], 14 * P)
    d.check(range(14))
    got = d.out.cpu().numpy()
    assert got[2, 1152] == 255 and got[3, 1153] == 255 and got[4, 1153] == 255 and got[9, 1153] == 255
    assert got[10, 1153] == 187 and got[11, 1153] == 255


@pytest.mark.parametrize("P", [16, 64, 128])
def test_scales_far_apart(cuda_device, P):
    """Values many octaves below the page's largest scale byte, and pages whose largest scale byte stands over small
    codes or none."""
    rng = np.random.default_rng(10 + P)
    c = _rand_cache(rng, 9, P)
    codes, scales = c[:, :256 * P].reshape(9, P, 16, 16), c[:, 384 * P:].reshape(9, P, 16)
    scales[0] = rng.integers(90, 140, (P, 16))            # every octave
    scales[1] = rng.integers(87, 168, (P, 16))
    scales[2] = 100                                       # one block far above all others
    scales[2, P // 2, 5] = 130
    scales[3] = 117                                       # 13 and 14 octaves
    scales[3, 0], scales[3, 1, ::2] = 130, 116
    scales[4] = 120                                       # the largest scale stands over zeros
    scales[4, 3, 7], codes[4, 3, 7] = 160, 0
    codes[5] &= 0x99                                      # magnitudes 0 and 0.5 only, and signs
    codes[6] = rng.choice([0, 0x88, 0x08, 0x80], codes[6].shape)  # zeros of either sign
    codes[7] &= 0xBB                                      # at most 1.5
    scales[8], codes[8] = rng.integers(87, 168, (P, 16)), 0
    scales[8, 1, 2], codes[8, 1, 2, 3] = 88, 0x55         # all that is not zero lies far below
    d = Digests(c, P, np.arange(9).reshape(1, 9), [9 * P])
    d.run([0], [9 * P], 9 * P)
    d.check(range(9))


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_few_and_many_pages(cuda_device, P, few):
    """The same pages in a call that can fill a few pages and in one that can fill thousands."""
    rng = np.random.default_rng(40 + P)
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
    d = Digests(c, P, np.arange(pages).reshape(1, pages), [pages * P])
    d.run([0], [pages * P], pages * P if few else 5000 * P)
    d.check(range(pages))


def test_what_is_out_of_range_is_left_out(cuda_device):
    rng = np.random.default_rng(2)
    P = 16
    c = _rand_cache(rng, 9, P)
    table = np.array([[0, 1, 2], [3, 9, 4], [5, -1, 6], [7, 8, 0]])
    lens = [3 * P, 3 * P, 3 * P, 2 * P]
    d = Digests(c, P, table, lens)
    d.run([0, 4, -1, 1, 2], [P, P, P, 3 * P, 3 * P], 3 * P, status=BAD_INDEX)
    d.check([2, 3, 4, 5, 6])
    d = Digests(c, P, table, [-1, 3 * P + 1, 3 * P, 2 * P])
    d.run([0, 1, 3], [P, P, P], 3 * P, status=BAD_INDEX)
    d.check([8])
    d = Digests(c, P, table, lens)
    d.run([0, 3, 1], [-1, P + 1, P], P, status=BAD_INDEX)  # new tokens out of range
    d.check([4])
    d = Digests(c, P, table, [2 ** 31 - 1, 3 * P, 3 * P, 2 * P])
    d.run([0, 3], [P, 1], P, status=BAD_INDEX)
    d.check([8])


def test_shared_pages_many_sequences_and_another_stream(cuda_device):
    rng = np.random.default_rng(3)
    P = 32
    c = _rand_cache(rng, 40, P)
    table = np.concatenate([np.tile(np.arange(2), (1500, 1)), rng.integers(2, 40, (1500, 1))], 1)
    d = Digests(c, P, table, [3 * P] * 1500)
    d.run(rng.permutation(1500), [3 * P] * 1500, 3 * P, stream=torch.cuda.Stream())
    d.check(sorted(set(table.reshape(-1))))


def test_a_list_longer_than_is_looked_up_at_once(cuda_device):
    rng = np.random.default_rng(4)
    P, seqs = 16, 50000
    c = _rand_cache(rng, 40, P)
    table = rng.integers(0, 38, (seqs, 1))
    table[0], table[-1] = 38, 39
    new = np.ones(seqs, dtype=int)
    new[1:-1:3] = 0
    d = Digests(c, P, table, [P] * seqs)
    d.run(np.arange(seqs), new, P)
    d.check(range(40))


# --------------------------------------------------------------------------
# Selection
# --------------------------------------------------------------------------

def _rand_digests(rng, pages, stride=1168):
    d = np.full((pages, stride), 0xA5, dtype=np.uint8)
    v = np.sort(rng.integers(-127, 128, (2, pages, 576)), 0).astype(np.int8).view(np.uint8)
    d[:, :512], d[:, 512:1024], d[:, 1024:1088], d[:, 1088:1152] = v[1][:, :512], v[0][:, :512], v[1][:, 512:], v[0][:, 512:]
    d[:, 1152:1154] = 127 + rng.integers(-1, 2, (pages, 2))
    d[:, 1154:1168] = 0
    return d


def _query(rng, M, H, e4m3, pad=0):
    """(device tensor [M, 576 H + pad], float64 [M,H,576])"""
    q = torch.from_numpy((rng.standard_normal((M, H, 576)) * np.exp(rng.standard_normal((M, 1, 1)))).astype(np.float32))
    q = q.to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    dev = torch.zeros(M, 576 * H + pad, dtype=q.dtype, device="cuda")
    dev[:, :576 * H] = q.reshape(M, -1).cuda()
    return dev, q.float().double().numpy()


class Select:
    def __init__(self, digests, P, table, lens, q_dev, q_host, e4m3=False):
        self.digests, self.P = digests, P
        self.table, self.lens = np.asarray(table, dtype=np.int32), np.asarray(lens, dtype=np.int32)
        self.q_dev, self.q, self.e4m3 = q_dev, q_host, e4m3
        self.d = torch.from_numpy(digests).cuda()
        self.t, self.l = _i32(self.table), _i32(self.lens)

    def run(self, B, q_len, k, first, last, seqs=None, pad=0, status=0, stream=None):
        M, H = B * q_len, self.q.shape[1]
        sel = torch.full((M, k + pad), -9, dtype=torch.int32, device="cuda")
        lens = torch.full((M + 1,), -9, dtype=torch.int32, device="cuda")
        n = mq.mlaqp_kv4_select_workspace(B, q_len, self.table.shape[1], len(self.digests))
        ws = torch.full((n + 16,), 0xEE, dtype=torch.uint8, device="cuda")
        rows = None if seqs is None else _i32(seqs)
        _ok(mq.mlaqp_kv4_select(self.q_dev, self.q_dev.stride(0), "e4m3" if self.e4m3 else "bf16", self.d, self.d.stride(0),
                                len(self.digests), self.P, self.t, self.t.stride(0), len(self.table), self.l, rows, B, q_len,
                                H, k, first, last, sel, k + pad, lens, ws, n, stream=stream))
        torch.cuda.synchronize()
        assert _device_status() == status
        got, got_lens = sel.cpu().numpy(), lens.cpu().numpy()
        assert got_lens[M] == -9 and (got[:, k:] == -9).all() and (ws[n:] == 0xEE).all()
        for m in range(M):
            b, i = divmod(m, q_len)
            s = b if seqs is None else seqs[b]
            good = 0 <= s < len(self.table) and 0 <= self.lens[s] <= min(self.table.shape[1], len(self.digests)) * self.P
            want, n = ([], 0) if not good else so.select(self.q[m], self.digests, self.table[s],
                                                         int(self.lens[s]) - (q_len - 1 - i), self.P, k, first, last)
            assert got_lens[m] == n, (m, got_lens[m], n)
            assert list(got[m, :k]) == want + [-1] * (k - len(want)), m
        return sel, lens


def _tables(rng, lens, P, pages, width=None):
    width = width or max(-(-max(lens) // P), 1)
    t = np.full((len(lens), width), -1)
    for s, n in enumerate(lens):
        k = -(-n // P)
        t[s, :k] = rng.permutation(pages)[:k]
    return t


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("P,q_len,H,k,first,last", [
    (16, 1, 16, 8, 1, 2), (32, 4, 11, 9, 2, 1), (64, 1, 1, 1, 0, 1), (128, 16, 8, 5, 0, 5), (16, 3, 5, 40, 3, 3),
    (64, 2, 16, 7, 6, 1), (16, 1, 13, 300, 0, 1)])
def test_selection(cuda_device, P, q_len, H, k, first, last, e4m3):
    rng = np.random.default_rng(P + q_len + H)
    B = min(12, 256 // q_len)
    pages = 400
    lens = [int(n) for n in rng.integers(1, 390 * P, B)]
    lens[:8] = [0, 1, P, P * k, P * k + 1, P * (k + 1) - 1 if k < 389 else 5, q_len - 1, 399 * P + 1][:len(lens)]
    q_dev, q = _query(rng, B * q_len, H, e4m3, pad=32)
    s = Select(_rand_digests(rng, pages, 1168 + 16), P, _tables(rng, lens, P, pages, 405), lens, q_dev, q, e4m3)
    s.run(B, q_len, k, first, last, pad=3)


@pytest.mark.parametrize("pages,k", [(257, 2), (1025, 64), (5000, 700), (20011, 33), (40009, 3000)])
def test_one_long_sequence(cuda_device, pages, k):
    rng = np.random.default_rng(pages)
    q_dev, q = _query(rng, 2, 16, False)
    s = Select(_rand_digests(rng, pages), 16, rng.permutation(pages)[None], [pages * 16 - 3], q_dev, q)
    s.run(1, 2, k, 1, 1)


def test_many_query_tokens_of_few_sequences(cuda_device):
    rng = np.random.default_rng(20)
    lens = [int(n) for n in rng.integers(600 * 16, 900 * 16, 40)]
    seqs = [int(x) for x in rng.integers(0, 40, 256)]  # a sequence may occur several times
    q_dev, q = _query(rng, 256, 16, True)
    s = Select(_rand_digests(rng, 1000), 16, _tables(rng, lens, 16, 1000), lens, q_dev, q, True)
    s.run(256, 1, 20, 1, 2, seqs=seqs)
    s.run(16, 16, 20, 1, 2, seqs=seqs[:16])


@pytest.mark.parametrize("distinct", [1, 2, 5])
def test_equal_scores_go_to_the_first(cuda_device, distinct):
    rng = np.random.default_rng(21)
    d = _rand_digests(rng, distinct)[rng.integers(0, distinct, 700)]
    q_dev, q = _query(rng, 3, 7, False)
    s = Select(d, 16, np.stack([rng.permutation(700) for _ in range(3)]), [700 * 16, 650 * 16, 30], q_dev, q)
    for k in (2, 3, 50, 351, 649):
        s.run(3, 1, k, 0, 1)


def test_scores_next_to_each_other(cuda_device):
    """Scores that differ in the last bit of the integer sum, over all magnitudes and both signs."""
    rng = np.random.default_rng(22)
    d = np.zeros((900, 1168), dtype=np.uint8)
    d[:, 1152:1154] = 127
    d[:, :512] = 127
    d[:, 0] = rng.integers(-127, 128, 900).astype(np.int8).view(np.uint8)
    d[:, 512:1024] = 0x81  # -127
    d[300:600, 1152] = rng.integers(67, 188, 300)
    d[600:, :1024] = d[600:, :1024] ^ 0xFF
    q = np.ones((2, 16, 576))
    q[1] = -1
    q[:, 0, 0] = 2.0 ** -9
    dev = torch.from_numpy(q.reshape(2, -1)).to(torch.bfloat16).cuda()
    s = Select(d, 16, np.stack([rng.permutation(900)] * 2), [900 * 16] * 2, dev, q)
    for k in (3, 20, 400, 800):
        s.run(2, 1, k, 1, 1)


def test_largest_sums_stay_whole(cuda_device):
    """All of q at its largest, all bounds at theirs: 512 * 16 * 2047 * 127 is just below 2^31."""
    d = np.zeros((40, 1168), dtype=np.uint8)
    d[:, 1152:1154] = 127
    d[:, :512], d[:, 1024:1088] = 127, 127
    d[:, 512:1024], d[:, 1088:1152] = 0x81, 0x81
    d[:, 0] = np.arange(40) + 88
    q = np.full((1, 16, 576), 2040.0)  # BF16 below 2047
    dev = torch.from_numpy(q.reshape(1, -1)).to(torch.bfloat16).cuda()
    for sign in (1, -1):
        s = Select(d, 16, np.arange(40)[None], [40 * 16], sign * dev, sign * q)
        s.run(1, 1, 5, 1, 1)


def test_unknown_digests_nan_queries_and_tiny_ones(cuda_device):
    rng = np.random.default_rng(23)
    d = _rand_digests(rng, 100)
    d[[5, 40, 77], 1152] = 255
    d[[9, 41], 1153] = 255
    q = rng.standard_normal((7, 4, 576))
    q[1, 2, 3] = np.nan
    q[2, 0, 575] = np.inf
    q[3] = 0
    q[4] *= 2.0 ** -120
    q[5] *= 2.0 ** 100
    q[6] = 2.0 ** -133
    dev = torch.from_numpy(q.astype(np.float32).reshape(7, -1)).to(torch.bfloat16).cuda()
    host = dev.double().cpu().numpy().reshape(7, 4, 576)
    s = Select(d, 32, np.stack([rng.permutation(100) for _ in range(7)]), [100 * 32 - 1] * 7, dev, host)
    for k in (3, 6, 8, 60):
        s.run(7, 1, k, 1, 1)
    e = torch.from_numpy(np.nan_to_num(q[:4]).clip(-400, 400).astype(np.float32)).to(torch.float8_e4m3fn).reshape(4, -1).cuda()
    e.view(torch.uint8)[1, 700] = 0x7F  # NaN
    e.view(torch.uint8)[2, 701] = 0xFF
    s = Select(d, 32, s.table[:4], [100 * 32 - 1] * 4, e, e.float().double().cpu().numpy().reshape(4, 4, 576), True)
    s.run(4, 1, 6, 1, 1)


@pytest.mark.parametrize("pages,k", [(300, 20), (1000, 500), (5000, 40)])
def test_digests_that_were_never_written(cuda_device, pages, k):
    """Any bytes: scores that are no numbers count as unknown pages do, and nothing is written beside the rows."""
    rng = np.random.default_rng(pages)
    d = rng.integers(0, 256, (pages, 1168), dtype=np.uint8)
    d[::3] = 0xFF
    d[1::3, 1152:1154] = 254  # sums of infinities of both signs
    q_dev, q = _query(rng, 3, 16, False)
    s = Select(d, 16, np.stack([rng.permutation(pages) for _ in range(3)]), [pages * 16] * 3, q_dev, q)
    with np.errstate(all="ignore"):
        s.run(3, 1, k, 1, 1, pad=5)


def test_what_is_out_of_range(cuda_device):
    rng = np.random.default_rng(24)
    d = _rand_digests(rng, 60)
    table = np.stack([rng.permutation(60) for _ in range(5)])
    table[0, [4, 20]] = 60, -3            # least of all scores
    table[1, [0, 59]] = 99, -1            # taken without a look: written as they are
    q_dev, q = _query(rng, 5, 8, False)
    s = Select(d, 16, table, [60 * 16] * 5, q_dev, q)
    s.run(5, 1, 59, 1, 1, status=BAD_INDEX)
    s.run(5, 1, 7, 1, 1, status=BAD_INDEX)
    s = Select(d, 16, table[2:], [60 * 16] * 3, q_dev, q)
    s.run(5, 1, 7, 1, 1, seqs=[0, 3, 1, -1, 2], status=BAD_INDEX)
    s = Select(d, 16, table[2:], [-1, 60 * 16 + 1, 2 ** 31 - 1], q_dev[:3], q[:3])
    s.run(3, 1, 7, 1, 1, status=BAD_INDEX)


def test_streams_and_graph_replay(cuda_device):
    rng = np.random.default_rng(25)
    lens = [int(n) for n in rng.integers(1, 300 * 32, 9)]
    q_dev, q = _query(rng, 9, 16, False)
    s = Select(_rand_digests(rng, 320), 32, _tables(rng, lens, 32, 320, 300), lens, q_dev, q)
    s.run(9, 1, 10, 1, 1, stream=torch.cuda.Stream())
    # two calls at once, each with its own workspace and outputs
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    n = mq.mlaqp_kv4_select_workspace(9, 1, s.table.shape[1], 320)
    torch.cuda.synchronize()
    for st in streams:
        sel, ln, ws = (torch.empty(9, 10, dtype=torch.int32, device="cuda"), torch.empty(9, dtype=torch.int32, device="cuda"),
                       torch.empty(n, dtype=torch.uint8, device="cuda"))
        outs.append((sel, ln, ws))
    torch.cuda.synchronize()
    args = lambda o: (s.q_dev, 576 * 16, "bf16", s.d, 1168, 320, 32, s.t, s.t.stride(0), 9, s.l, None, 9, 1, 16, 10, 1, 1,
                      o[0], 10, o[1], o[2], n)
    for _ in range(20):
        for st, o in zip(streams, outs):
            _ok(mq.mlaqp_kv4_select(*args(o), stream=st))
    torch.cuda.synchronize()
    want, want_lens = s.run(9, 1, 10, 1, 1)
    for sel, ln, _ in outs:
        assert torch.equal(sel, want) and torch.equal(ln, want_lens[:9])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _ok(mq.mlaqp_kv4_select(*args(outs[0])))
    lens = [int(n) for n in rng.integers(1, 300 * 32, 9)]
    s.lens[:] = lens
    s.table[:] = _tables(rng, lens, 32, 320, s.table.shape[1])
    s.t.copy_(_i32(s.table)), s.l.copy_(_i32(lens))
    q2, s.q = _query(rng, 9, 16, False)
    s.q_dev.copy_(q2)
    g.replay()
    torch.cuda.synchronize()
    want, want_lens = s.run(9, 1, 10, 1, 1)
    assert torch.equal(outs[0][0], want) and torch.equal(outs[0][1], want_lens[:9])


def test_offsets_beyond_32_bits(cuda_device):
    rng = np.random.default_rng(26)
    P, pages, far = 16, 70, 1 << 26
    c = _rand_cache(rng, pages, P)
    big = torch.empty(2, pages, far, dtype=torch.uint8, device="cuda")
    table = rng.permutation(pages)[None]
    d = Digests(c, P, table, [pages * P])
    d.cache, d.out, d.stride = big[0, :, :400 * P], big[1, :, :1168], far
    d.cache.copy_(torch.from_numpy(c))
    d.run([0], [pages * P], pages * P)
    digests = d.out.cpu().numpy()
    for p in range(pages):
        np.testing.assert_array_equal(digests[p], so.digest(ko.read_tokens(c, P, range(p * P, p * P + P))))
    q_dev, q = _query(rng, 1, 16, False)
    s = Select(digests, P, table, [pages * P], q_dev, q)
    s.d = d.out
    s.run(1, 1, 9, 1, 1)


# --------------------------------------------------------------------------
# Together: decode steps of a layer with a cache that grows
# --------------------------------------------------------------------------

@pytest.mark.parametrize("P,q_len,H,e4m3,graph", [(16, 1, 16, False, False), (16, 3, 11, True, False), (32, 1, 8, False, True)])
def test_sparse_decode_steps(cuda_device, P, q_len, H, e4m3, graph):
    """extend -> append_rope -> digest -> mlaqp_run -> select -> attend, step after step."""
    g = torch.Generator(device="cuda").manual_seed(P + q_len)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    B, pages, row, k, first, last = 5, 200, 36, 7, 1, 2
    M = B * q_len
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = torch.zeros(pages, 400 * P, dtype=torch.uint8, device="cuda")
    digests = torch.full((pages, 1168), 0xFF, dtype=torch.uint8, device="cuda")
    table, lens, refs = torch.full((B, row), -1, **i32), torch.zeros(B, **i32), torch.zeros(pages, **i32)
    tables = (table, row, B, lens, refs, pages, P)
    seqs, weight = torch.arange(B, **i32), rand(512)
    phi = torch.rand(1024, 32, generator=g, device="cuda") * 6
    angles = torch.cat([torch.cos(phi), torch.sin(phi)], 1)
    pool = (cache, cache.stride(0), pages, P)

    def write(rows, q_pe, counts, most):
        """Grow the sequences, write the tokens (padded to `most` a sequence) and rotate their queries in place."""
        pos = (lens[:, None] + torch.arange(most, **i32)).reshape(-1).int()
        slots = torch.empty(B, most, **i32)
        _ok(mq.mlaqp_kv4_extend(*tables, seqs, counts, B, slots, most))
        heads = 0 if q_pe is None else H
        _ok(mq.mlaqp_kv4_append_rope(rows, 576, weight, 1e-6, rows[:, 512:], 576, q_pe, heads * 64, 64, q_pe, heads * 64, 64, heads,
                                     pos, angles, 1024, "halves", *pool, slots, B * most))
        _ok(mq.mlaqp_kv4_digest(*pool, table, row, B, lens, seqs, counts, B, most, digests, 1168))

    prompts = torch.tensor([0, 1, 12 * P, 20 * P - 1, 30 * P + 2], **i32)
    write(rand(B * 31 * P, 576), None, prompts, 31 * P)
    w = rand(H, 128, 512) / 128 ** 0.5
    q = torch.empty(M, H * 576, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device="cuda")
    q_scale = torch.tensor([0.05], device="cuda") if e4m3 else None
    kind = "e4m3" if e4m3 else "bf16"
    sel, sel_lens = torch.empty(M, k, **i32), torch.empty(M, **i32)
    x, lse = torch.empty(M, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(M, H, device="cuda")
    ws = torch.empty(mq.mlaqp_kv4_select_workspace(B, q_len, row, pages), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(mq.mlaqp_kv4_attend_workspace(M, 1, H), dtype=torch.uint8, device="cuda")
    fresh = torch.full((B,), q_len, **i32)
    rows, q_nope, q_pe = rand(M, 576), rand(M, H, 128), rand(M, H, 64)

    def step():
        write(rows, q_pe, fresh, q_len)
        _ok(mq.mlaqp_run(q_nope, q_pe, w, None, q, 576 * H, q_scale, M, H, "bf16", kind))
        _ok(mq.mlaqp_kv4_select(q, 576 * H, kind, digests, 1168, pages, P, table, row, B, lens, None, B, q_len, H, k, first, last,
                                sel, k, sel_lens, ws, ws.numel()))
        _ok(mq.mlaqp_kv4_attend(q, 576 * H, kind, q_scale, *pool, sel, k, M, sel_lens, None, M, 1, H, SCALE, x, 512 * H, lse, ws2,
                                ws2.numel()))

    captured = None
    if graph:
        _ok(mq.mlaqp_prewarm(H, M, "bf16", kind)), _ok(mq.mlaqp_kv4_prewarm()), _ok(mq.mlaqp_kv4_step_prewarm())
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    for n in range(P + 3):
        rows.copy_(rand(M, 576)), q_nope.copy_(rand(M, H, 128)), q_pe.copy_(rand(M, H, 64))
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        if n % 5 and n < P:
            continue
        assert _device_status() == 0
        host, dig, tab, ln = cache.cpu().numpy(), digests.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy()
        got, got_lens = sel.cpu().numpy(), sel_lens.cpu().numpy()
        qd = q.float().double().cpu().numpy().reshape(M, H, 576)
        for m in range(M):
            b, i = divmod(m, q_len)
            seen = int(ln[b]) - (q_len - 1 - i)
            full = [so.digest(ko.read_tokens(host, P, range(p * P, p * P + P))) for p in tab[b, :ln[b] // P]]
            for j, page in enumerate(tab[b, :ln[b] // P]):
                assert np.array_equal(dig[page], full[j])
            want, total = so.select(qd[m], dig, tab[b], seen, P, k, first, last)
            assert list(got[m]) == want + [-1] * (k - len(want)) and got_lens[m] == total
            keys = ko.read_tokens(host, P, [want[t // P] * P + t % P for t in range(total)])
            qm = qd[m] * float(q_scale) if e4m3 else qd[m]
            sx, sl = ko.attend(qm, keys, SCALE)
            s = qm @ keys.T * SCALE
            p = np.exp(s - sl[:, None])
            bound = 2.0 ** -8 * np.abs(sx) + 2.0 ** -8 * (p @ np.abs(keys[:, :512]))
            assert (np.abs(x[m].double().cpu().numpy() - sx) <= bound).all(), (n, m)
            size = (np.abs(qm) @ np.abs(keys).T).max(1) * SCALE
            assert (np.abs(lse[m].double().cpu().numpy() - sl) <= 2.0 ** -15 * size + 1e-5).all(), (n, m)
