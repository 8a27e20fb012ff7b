"""GPU parity of the 4-bit cache's append, gather and attention against the
CPU oracle in float64.

Append and gather are exact.  Attention tolerances, per output:
  x    2^-8 |x|             the BF16 rounding (2^-9) with a factor of two
       + 2^-8 sum_t p |K|   probabilities held to 8 bits or more (2^-9 each,
                            all of one sign at worst) and score errors below
                            2^-9 in the exponent
  lse  FP32 sums of 576 products, 2^-15 of the largest sum of magnitudes
       (576 roundings of 2^-24, all of one sign), plus 1e-5 for exp and log.
"""

import numpy as np
import pytest
import torch

import mla_decode_query_gb300 as mq
import oracle
from helpers import to_device, to_host_bits
from oracle import kv4_oracle as ko

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _ok(st):
    assert st == mq.MLAQP_OK, mq.mlaqp_last_error()


def _device_status():
    st, word = mq.mlaqp_device_status(reset=True)
    _ok(st)
    return word


class Cache:
    """A one-layer cache in a buffer poisoned with 0xFF (NaN scales, NaN rope)."""

    def __init__(self, num_pages, page_size, page_stride=None):
        self.P, self.n = page_size, num_pages
        self.stride = page_stride or 400 * page_size
        self.buf = torch.full((num_pages, self.stride), 0xFF, dtype=torch.uint8, device="cuda")

    def host(self):
        return self.buf.cpu().numpy()[:, :400 * self.P].copy()

    def args(self):
        return self.buf, self.stride, self.n, self.P

    def append(self, rows, slots, stream=None):
        """rows: uint16 bits [T,576]"""
        t = to_device(rows)
        s = torch.tensor(np.asarray(slots), dtype=torch.int32, device="cuda")
        _ok(mq.mlaqp_kv4_append(t, 576, t[:, 512:], 576, *self.args(), s, len(slots), stream=stream))
        torch.cuda.synchronize()


def _rows(rng, T, spread=0.5):
    lat = rng.standard_normal((T, 512)) * np.exp(spread * rng.standard_normal(512))
    return _bits(np.concatenate([lat, rng.standard_normal((T, 64))], 1))


def _special_rows(rng):
    """Values on ties and range ends, zero blocks, negative zeros, tiny and huge blocks, NaN and Inf blocks."""
    rows = oracle.bf16_to_f64(_rows(rng, 24)).astype(np.float64)
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    rows[0, :32] = np.concatenate([grid, -grid])
    rows[0, 32:64] = np.concatenate([grid, -grid]) * 2.0 ** -9
    rows[1, :32] = 0.0
    rows[1, 32:64] = -0.0
    rows[2, :] = 0.0
    rows[3, :64] = 2.0 ** -70
    rows[4, 64:96] = 2.0 ** 55
    rows[5, 7] = np.nan
    rows[6, 40] = np.inf
    rows[7, 511] = -np.inf
    rows[8, 512:] = np.nan
    rows[9, :32] *= 2.0 ** 30
    rows[9, 32:64] *= 2.0 ** -30
    rows[10, :32] = 7.0
    rows[11, :32] = 7.03125
    return _bits(rows)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_append_writes_the_oracles_bytes(cuda_device, P):
    rng = np.random.default_rng(P)
    rows = np.concatenate([_special_rows(rng), _rows(rng, 30)])
    c = Cache(5, P, 400 * P + 48)
    want = c.host()
    slots = rng.permutation(5 * P)[:len(rows)]
    slots[4] = -1
    for r, s in zip(rows, slots):
        if s >= 0:
            ko.write_token(want[s // P], P, s % P, r[:512], r[512:])
    _device_status()
    c.append(rows, slots)
    assert _device_status() == 0
    np.testing.assert_array_equal(c.host(), want)
    assert (c.buf.cpu().numpy()[:, 400 * P:] == 0xFF).all()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 131])
def test_append_takes_strided_views(cuda_device, T):
    P, rng = 64, np.random.default_rng(T)
    rows = _rows(rng, T)
    c = Cache(3, P)
    lat = torch.full((T, 528), 0x7FC0, dtype=torch.int16, device="cuda")
    pe = torch.full((T, 72), 0x7FC0, dtype=torch.int16, device="cuda")
    lat[:, 8:520] = to_device(rows[:, :512])
    pe[:, 8:] = to_device(rows[:, 512:])
    slots = rng.permutation(3 * P)[:T].astype(np.int32)
    s = to_device(slots.view(np.uint8).reshape(-1, 4)).view(torch.int32)
    _ok(mq.mlaqp_kv4_append(lat[:, 8:], 528, pe[:, 8:], 72, *c.args(), s, T))
    want = np.full((3, 400 * P), 0xFF, dtype=np.uint8)
    for r, at in zip(rows, slots):
        ko.write_token(want[at // P], P, at % P, r[:512], r[512:])
    np.testing.assert_array_equal(c.host(), want)


@pytest.mark.parametrize("P", [16, 128])
def test_gather_reads_the_oracles_values(cuda_device, P):
    rng = np.random.default_rng(100 + P)
    rows = np.concatenate([_special_rows(rng), _rows(rng, 20)])
    c = Cache(4, P, 400 * P + 16)
    slots = rng.permutation(4 * P)[:len(rows)]
    c.append(rows, slots)
    ask = np.concatenate([slots, [-1, slots[0], -5]]).astype(np.int32)
    out = torch.full((len(ask), 592), 0x5A5A, dtype=torch.int16, device="cuda")
    _device_status()
    _ok(mq.mlaqp_kv4_gather(*c.args(), torch.from_numpy(ask).cuda(), len(ask), out, 592))
    got = to_host_bits(out, np.uint16)
    assert _device_status() == 0 and (got[:, 576:] == 0x5A5A).all()
    want = np.zeros((len(ask), 576))
    want[ask >= 0] = ko.read_tokens(c.host(), P, ask[ask >= 0])
    np.testing.assert_array_equal(oracle.bf16_to_f64(got[:, :576]), want)


def test_slots_out_of_range_are_left_out_and_reported(cuda_device):
    P, rng = 32, np.random.default_rng(5)
    rows = _rows(rng, 3)
    c = Cache(2, P)
    _device_status()
    c.append(rows, [2 * P, 3, 2 ** 31 - 1])
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    want = np.full((2, 400 * P), 0xFF, dtype=np.uint8)
    ko.write_token(want[0], P, 3, rows[1, :512], rows[1, 512:])
    np.testing.assert_array_equal(c.host(), want)
    out = torch.full((2, 576), 0x5A5A, dtype=torch.int16, device="cuda")
    _ok(mq.mlaqp_kv4_gather(*c.args(), torch.tensor([2 * P, 3], dtype=torch.int32, device="cuda"), 2, out, 576))
    got = oracle.bf16_to_f64(to_host_bits(out, np.uint16))
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    assert not got[0].any()
    np.testing.assert_array_equal(got[1], ko.read_tokens(want, P, [3])[0])


def _layout(rng, lens, P, spare=2):
    """Shuffled pages of sequences: (table, slots per sequence, number of pages)."""
    need = [-(-n // P) for n in lens]
    perm = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -1, dtype=np.int32)
    slots, at = [], 0
    for b, (n, k) in enumerate(zip(lens, need)):
        table[b, :k] = perm[at:at + k]
        t = np.arange(n)
        slots.append(table[b, t // P].astype(np.int64) * P + t % P)
        at += k
    return table, slots, sum(need) + spare


class Case:
    """Sequences in a cache, queries, and the oracle's answer."""

    def __init__(self, lens, P=64, q_len=1, H=16, dtype="bf16", seed=0, page_stride=None, rows=None, q=None,
                 q_pad=0, x_pad=0, seqs=None, scale=SCALE):
        rng = np.random.default_rng(seed)
        self.lens, self.P, self.q_len, self.H, self.dtype, self.scale = lens, P, q_len, H, dtype, scale
        self.table, self.slots, pages = _layout(rng, lens, P)
        self.cache = Cache(pages, P, page_stride)
        every = np.concatenate(self.slots).astype(np.int64)
        self.rows = _rows(rng, len(every)) if rows is None else rows(rng, len(every))
        if len(every):
            self.cache.append(self.rows, every)
        self.seqs = seqs
        self.B = len(lens) if seqs is None else len(seqs)
        M = self.B * q_len
        qv = rng.standard_normal((M, H, 576)) if q is None else q(rng, M, H)
        self.q_stride = 576 * H + q_pad
        if dtype == "bf16":
            bits = _bits(qv)
            self.q = oracle.bf16_to_f64(bits)
            self.dev_q = torch.full((M, self.q_stride), 0x7FC0, dtype=torch.int16, device="cuda")
            self.dev_q[:, :576 * H] = to_device(bits).reshape(M, -1)
            self.q_scale = None
        else:
            qs = np.float32(0.037)
            codes = torch.from_numpy((qv / qs).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.q = codes.float().numpy().astype(np.float64) * float(qs)
            self.dev_q = torch.full((M, self.q_stride), 0x7F, dtype=torch.uint8, device="cuda")
            self.dev_q[:, :576 * H] = codes.view(torch.uint8).reshape(M, -1).cuda()
            self.q_scale = torch.tensor([qs], device="cuda")
        self.x_stride = 512 * H + x_pad
        self.x = torch.full((M, self.x_stride), 0x5A5A, dtype=torch.int16, device="cuda")
        self.lse = torch.full((M, H), 123.0, device="cuda")
        n = mq.mlaqp_kv4_attend_workspace(self.B, q_len, H)
        assert n >= 0, mq.mlaqp_last_error()
        self.ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        self.dev_table = torch.from_numpy(self.table).cuda()
        self.dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dev_seqs = None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device="cuda")

    def run(self, stream=None, lse=True):
        return mq.mlaqp_kv4_attend(
            self.dev_q, self.q_stride, self.dtype, self.q_scale, *self.cache.args(), self.dev_table,
            self.table.shape[1], self.table.shape[0], self.dev_lens, self.dev_seqs, self.B, self.q_len, self.H, self.scale,
            self.x, self.x_stride, self.lse if lse else None, self.ws, self.ws.numel(), stream=stream)

    def outputs(self):
        torch.cuda.synchronize()
        x = to_host_bits(self.x, np.uint16)
        assert (x[:, 512 * self.H:] == 0x5A5A).all(), "written between the rows"
        return (oracle.bf16_to_f64(x[:, :512 * self.H]).reshape(-1, self.H, 512),
                self.lse.cpu().numpy().astype(np.float64))

    def keys(self, b):
        s = b if self.seqs is None else self.seqs[b]
        return ko.read_tokens(self.cache.host() if not hasattr(self, "_host") else self._host, self.P, self.slots[s])

    def check(self):
        x, lse = self.outputs()
        self._host = self.cache.host()
        for b in range(self.B):
            keys = self.keys(b)
            for i in range(self.q_len):
                n = max(0, len(keys) - (self.q_len - 1 - i))
                m = b * self.q_len + i
                self.compare(x[m], lse[m], self.q[m], keys[:n], f"sequence {b} token {i} of {n}")

    def compare(self, x, lse, q, keys, where, small_blocks=None):
        wx, wl = ko.attend(q, keys, self.scale)
        if keys.shape[0] == 0:
            assert not x.any() and np.isneginf(lse).all(), where
            return
        p = np.exp(q @ keys.T * self.scale - wl[:, None])
        bound = 2.0 ** -8 * np.abs(wx) + 2.0 ** -8 * (p @ np.abs(keys[:, :512])) + 1e-30
        if small_blocks is not None:  # the tokens' largest block scales
            bound = bound + 2.0 ** -16 * (p @ small_blocks)[:, None]
        err = np.abs(x - wx)
        assert (err <= bound).all(), f"{where}: x off by {np.nanmax(err / bound)} of its bound"
        lb = 2.0 ** -15 * self.scale * (np.abs(q) @ np.abs(keys).T).max(1) + 1e-5
        assert (np.abs(lse - wl) <= lb).all(), f"{where}: lse off by {np.nanmax(np.abs(lse - wl) / lb)} of its bound"


LENS = {
    "short": [0, 1, 2, 15, 16, 17, 31, 33],
    "tiles": [63, 64, 65, 127, 128, 129, 255, 256, 257],
    "mixed": [1, 700, 0, 129, 1500, 3, 384],
}


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("name", sorted(LENS))
def test_lengths_and_page_sizes(cuda_device, name, P):
    c = Case(LENS[name], P=P, seed=P)
    _device_status()
    _ok(c.run())
    c.check()
    assert _device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("H", [1, 5, 8, 11, 16])
@pytest.mark.parametrize("q_len", [1, 2, 3, 4])
def test_heads_and_query_lengths(cuda_device, q_len, H, dtype):
    c = Case([1, 2, 130, 3, 260], P=32, q_len=q_len, H=H, dtype=dtype, seed=10 * H + q_len, q_pad=32, x_pad=24)
    _ok(c.run())
    c.check()


@pytest.mark.parametrize("q_len,B,H", [(16, 3, 16), (16, 2, 11), (7, 4, 8), (1, 256, 16), (2, 128, 8)])
def test_row_counts_up_to_the_domain(cuda_device, q_len, B, H):
    rng = np.random.default_rng(q_len)
    c = Case([int(n) for n in rng.integers(0, 90, B)], P=16, q_len=q_len, H=H, seed=q_len)
    _ok(c.run())
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_long_sequence_is_split_and_joined(cuda_device, dtype):
    for lens in ([20000], [9000, 40, 5000]):
        c = Case(lens, P=64, H=16, dtype=dtype, seed=len(lens))
        _ok(c.run())
        c.check()


def test_peaked_softmax_and_long_tail(cuda_device):
    # One key far above the rest, late in the sequence, then many equal keys
    # at a distance: the running maximum jumps, and what lies far below the
    # maximum still adds up.
    def rows(rng, T):
        r = np.tile(rng.standard_normal((1, 576)), (T, 1))
        r[:, :512] *= np.where(rng.random((T, 512)) < 0.5, 1, -1)
        r[T // 2] = 4.0
        return _bits(r)

    def q(rng, M, H):
        v = 0.02 * rng.standard_normal((M, H, 576))
        v += 0.05 * np.arange(H)[None, :, None] / H
        return v

    c = Case([3000], P=64, rows=rows, q=q, scale=0.5)
    _ok(c.run())
    c.check()


def test_token_scales_of_very_different_size(cuda_device):
    def rows(rng, T):
        r = rng.standard_normal((T, 576))
        r[:, :512] *= 2.0 ** rng.integers(-20, 3, T)[:, None]
        r[:, :512] *= (2.0 ** rng.integers(-12, 1, (T, 16))).repeat(32, 1)
        r[::7, :512] = 0.0
        return _bits(r)

    for lens in ([300], [7], [1, 1]):
        c = Case(lens, P=32, rows=rows, seed=4)
        _ok(c.run())
        c.check()


def test_all_zero_latents(cuda_device):
    def rows(rng, T):
        r = rng.standard_normal((T, 576))
        r[:, :512] = 0.0
        return _bits(r)

    c = Case([200, 3], rows=rows)
    _ok(c.run())
    c.check()


@pytest.mark.parametrize("mag", [2.0 ** -30, 2.0 ** -10, 2.0 ** 12])
def test_query_magnitudes(cuda_device, mag):
    # rows whose elements span many octaves: the large ones carry the score
    def q(rng, M, H):
        return mag * rng.standard_normal((M, H, 576)) * 2.0 ** rng.integers(-12, 1, (M, H, 576))

    c = Case([150, 33], q=q, scale=min(1.0 / mag, 2.0 ** 20) * SCALE, seed=3)
    _ok(c.run())
    c.check()


def test_nan_and_infinity_stay_where_they_are_visible(cuda_device):
    def rows(rng, T):
        r = oracle.bf16_to_f64(_rows(rng, T))
        r[10, 5] = np.nan      # sequence 0, a latent
        r[40 + 20, 520] = np.nan  # sequence 1, a rope element
        r[80 + 39, 3] = np.inf  # sequence 2, the last token: seen by its last query token only
        return _bits(r)

    c = Case([40, 40, 40, 40], P=16, q_len=2, H=8, rows=rows, seed=9)
    _ok(c.run())
    x, lse = c.outputs()
    for b, nan_rows in ((0, (0, 1)), (1, (0, 1)), (2, (1,)), (3, ())):
        for i in range(2):
            if i in nan_rows:
                assert np.isnan(x[2 * b + i]).all() and np.isnan(lse[2 * b + i]).all()
            else:
                assert not np.isnan(x[2 * b + i]).any()
                c.compare(x[2 * b + i], lse[2 * b + i], c.q[2 * b + i], c.keys(b)[:39 + i], f"{b},{i}")


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("col", [17, 530])
def test_non_finite_query_spoils_its_own_row_only(cuda_device, value, col):
    def q(rng, M, H):
        v = rng.standard_normal((M, H, 576))
        v[1, 3, col] = value
        return v

    c = Case([200, 150], H=8, q=q, seed=2)
    _ok(c.run())
    x, lse = c.outputs()
    assert np.isnan(x[1, 3]).all()
    x[1, 3], lse[1, 3], c.q[1, 3] = x[1, 2], lse[1, 2], c.q[1, 2]
    for b in range(2):
        c.compare(x[b], lse[b], c.q[b], c.keys(b), f"sequence {b}")


def test_sequences_by_index_and_no_lse(cuda_device):
    c = Case([50, 0, 300, 129], seqs=[3, 0, 2, 3, 1], P=32, H=11)
    _ok(c.run(lse=False))
    x, lse = c.outputs()
    assert (lse == 123.0).all()
    _ok(c.run())
    c.check()
    np.testing.assert_array_equal(x, c.outputs()[0])


def test_bad_pages_lengths_and_sequences_are_reported(cuda_device):
    c = Case([64, 64, 64, 64], P=32, H=8)
    c.dev_table[1, 1] = 10 ** 6
    c.dev_table[2, 0] = -1
    c.dev_lens[3] = 65  # beyond the table row
    _device_status()
    _ok(c.run())
    x, lse = c.outputs()
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    c.compare(x[0], lse[0], c.q[0], c.keys(0), "intact")
    c.compare(x[1], lse[1], c.q[1], c.keys(1)[:32], "second page out of range")
    c.compare(x[2], lse[2], c.q[2], c.keys(2)[32:], "first page none")
    c.compare(x[3], lse[3], c.q[3], c.keys(3)[:0], "length beyond its row")
    c = Case([40, 50], P=16, H=8, seqs=[1, 7, -1])
    _ok(c.run())
    x, lse = c.outputs()
    assert _device_status() == mq.MLAQP_DEVSTATUS_BAD_INDEX
    c.compare(x[0], lse[0], c.q[0], c.keys(0), "intact")
    for b in (1, 2):
        assert not x[b].any() and np.isneginf(lse[b]).all()


def test_offsets_past_32_bits(cuda_device):
    # pages 1 MB apart, 5000 of them: the sequences' pages lie anywhere in 5 GB
    P, stride, pages = 16, 1 << 20, 5000
    rng = np.random.default_rng(8)
    buf = torch.empty(pages * stride, dtype=torch.uint8, device="cuda")
    rows = _rows(rng, 300)
    chosen = np.concatenate([[4999, 0, 4200], rng.permutation(np.arange(1, 4000))[:16]]).astype(np.int32)
    t = np.arange(300)
    slots = (chosen[t // P] * P + t % P).astype(np.int32)
    dev = to_device(rows)
    _ok(mq.mlaqp_kv4_append(dev, 576, dev[:, 512:], 576, buf, stride, pages, P, torch.from_numpy(slots).cuda(), 300))
    out = torch.empty(300, 576, dtype=torch.int16, device="cuda")
    _ok(mq.mlaqp_kv4_gather(buf, stride, pages, P, torch.from_numpy(slots).cuda(), 300, out, 576))
    host = np.zeros((1, 400 * P * 20), dtype=np.uint8)
    small = np.zeros((19, 400 * P), dtype=np.uint8)
    for k, r in enumerate(rows):
        ko.write_token(small[k // P], P, k % P, r[:512], r[512:])
    keys = ko.read_tokens(small, P, t)
    np.testing.assert_array_equal(oracle.bf16_to_f64(to_host_bits(out, np.uint16)), keys)
    del host
    c = Case([300], P=P, H=16)
    c.dev_table = torch.from_numpy(chosen[None, :]).cuda()
    c.table = chosen[None, :]
    c.cache.buf, c.cache.stride, c.cache.n = buf, stride, pages
    _ok(c.run())
    x, lse = c.outputs()
    c.compare(x[0], lse[0], c.q[0], keys, "far pages")


def test_same_bits_every_time_and_on_another_stream(cuda_device):
    c = Case([5000, 100, 2111], P=64, H=16)
    _ok(c.run())
    first = c.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        c.x.fill_(0x5A5A)
        c.ws.fill_(0xFF)
        s.wait_stream(torch.cuda.current_stream())
        _ok(c.run(stream=s))
        s.synchronize()
        again = c.outputs()
        np.testing.assert_array_equal(first[0], again[0])
        np.testing.assert_array_equal(first[1], again[1])


def test_graph_replay_follows_lengths_and_cache(cuda_device):
    c = Case([700, 90, 4000], P=64, H=8, q_len=2)
    _ok(mq.mlaqp_kv4_prewarm())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _ok(c.run())
    g.replay()
    c.check()
    c.slots = [c.slots[0][:3], c.slots[1][:0], c.slots[2][:2500]]
    c.dev_lens.copy_(torch.tensor([3, 0, 2500], dtype=torch.int32))
    g.replay()
    c.check()


def test_workspace_is_required(cuda_device):
    c = Case([10])
    n = mq.mlaqp_kv4_attend_workspace(1, 1, 16)
    for ws, nb in ((None, n), (c.ws[8:], n), (c.ws, n - 1)):
        keep = c.ws
        st = mq.mlaqp_kv4_attend(c.dev_q, c.q_stride, "bf16", None, *c.cache.args(), c.dev_table, 1, 1, c.dev_lens, None,
                                 1, 1, 16, SCALE, c.x, c.x_stride, None, ws, nb)
        assert st == mq.MLAQP_ERR_INVALID_ARG
        assert keep is c.ws


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_projection_to_attention_to_v_up(cuda_device, dtype):
    """A layer's decode step: projection -> append -> attention -> V up-projection on one stream."""
    from mla_decode_query_gb300 import inputs
    H, B, P = 16, 5, 64
    d = inputs.make_layer(7, H, "mxfp8", m_max=B)
    dv = inputs.make_v_layer(8, H, "bf16", m_max=B)
    qs = np.float32(0.03) if dtype == "e4m3" else None
    c = Case([130, 1, 64, 500, 65], P=P, H=H, dtype=dtype, seed=1)
    w, ws = to_device(d["weight"]), to_device(d["weight_scale"])
    qn, qp = to_device(d["q_nope"]), to_device(d["q_pe"])
    if dtype == "e4m3":
        c.q_scale = torch.tensor([qs], device="cuda")
    y = torch.zeros(B, H, 128, dtype=torch.int16, device="cuda")
    wv = to_device(dv["weight"])
    _ok(mq.mlaqp_run_pdl(qn, qp, w, ws, c.dev_q, c.q_stride, c.q_scale, B, H, "mxfp8", dtype))
    _ok(c.run())
    _ok(mq.mlaqp_v_up_run(c.x, c.x_stride, 512, wv, None, y, 128 * H, B, H, "bf16", pdl=1))
    torch.cuda.synchronize()
    if dtype == "bf16":
        c.q = oracle.bf16_to_f64(to_host_bits(c.dev_q, np.uint16)).reshape(B, H, 576)
    else:
        c.q = oracle.e4m3_to_f64(to_host_bits(c.dev_q, np.uint8)).reshape(B, H, 576) * float(qs)
    c.check()
    _, acc = oracle.mla_v_up(to_host_bits(c.x, np.uint16).reshape(B, H, 512), dv["weight"], None, "bf16")
    got = oracle.bf16_to_f64(to_host_bits(y, np.uint16))
    assert (np.abs(got - acc) <= 1e-2 * np.abs(acc) + 1e-3).all()


@pytest.mark.parametrize("fill", [0, 5, 6, 86, 168, 254])
def test_bytes_behind_a_sequence_are_never_used(cuda_device, fill):
    # whatever byte stands in the scales behind the last token
    c = Case([1, 100, 130], P=32, H=8, q_len=2, seed=fill)
    c.cache.buf.fill_(fill)
    c.cache.append(c.rows, np.concatenate(c.slots))
    _ok(c.run())
    c.check()


def _largest_scale(c, b):
    """2^(s_t-127) of a sequence's tokens."""
    host = c.cache.host()
    at = c.slots[b]
    byte = [host[t // c.P, c.P * 384 + t % c.P * 16:][:16].max() for t in at]
    return np.array([ko.scale_value(v) for v in byte])


def test_scale_bytes_out_of_range_read_as_the_nearest(cuda_device):
    c = Case([70, 140], P=64, H=8, seed=21)
    page = c.table[0, 0]
    scales = c.cache.buf[page, 64 * 384:64 * 400].view(64, 16)
    scales[3, 2], scales[4, 15], scales[5, :], scales[6, 1:] = 0, 86, 5, 12
    page = c.table[1, 1]
    scales = c.cache.buf[page, 64 * 384:64 * 400].view(64, 16)
    scales[9, 4], scales[10, :] = 168, 254
    _ok(c.run())
    x, lse = c.outputs()
    for b in range(2):
        c.compare(x[b], lse[b], c.q[b], c.keys(b), f"sequence {b}", small_blocks=_largest_scale(c, b))


def test_blocks_far_below_the_largest_of_their_token(cuda_device):
    # octaves between the blocks of a token, up to the 80 that the cache holds
    def rows(rng, T):
        r = rng.standard_normal((T, 576))
        r[:, :512] *= (2.0 ** rng.integers(-38, 38, (T, 16))).repeat(32, 1)
        return _bits(r)

    c = Case([1] * 40, P=16, H=3, rows=rows, seed=6, scale=2.0 ** -40)
    _ok(c.run())
    x, lse = c.outputs()
    for b in range(40):
        c.compare(x[b], lse[b], c.q[b], c.keys(b), f"sequence {b}", small_blocks=_largest_scale(c, b))
