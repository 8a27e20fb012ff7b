"""GPU parity of mlaqp_kv4_append_rope with the CPU oracle.

The latents' codes and scales are equal: the mean of squares is the FP32 number
next to the exact one, and what follows it is rounded to FP32 step by step in
both.  Rotated elements, per output: 2^-8 of it for its rounding to BF16 (half a
step), and 3 roundings of 2^-24 (two products, a sum; fewer where they are fused)
of |a cos| + |b sin|, plus half of BF16's smallest step, 2^-134.
"""

import numpy as np
import pytest
import torch

import mla_decode_query_gb300 as mq
import oracle
from helpers import to_device, to_host_bits
from oracle import kv4_oracle as ko
from oracle import kv4_step_oracle as so

pytestmark = pytest.mark.gpu

POSITIONS = 300
EPS = 1e-6


def _bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _ok(st):
    assert st == mq.MLAQP_OK, mq.mlaqp_last_error()


def _device_status():
    st, word = mq.mlaqp_device_status(reset=True)
    _ok(st)
    return word


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _angles(rng):
    a = rng.uniform(0, 2 * np.pi, (POSITIONS, 32))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _close(got_bits, part_bits, angles, halves):
    want = so.rotate(part_bits, angles, halves)
    # |a cos| + |b sin| and |b cos| + |a sin|: the larger of what rotating the magnitudes by +-|angle| gives
    turn = np.abs(angles)
    back = np.concatenate([turn[..., :32], -turn[..., 32:]], -1)
    size = np.maximum(so.rotate(part_bits & 0x7FFF, turn, halves), so.rotate(part_bits & 0x7FFF, back, halves))
    got = oracle.bf16_to_f64(got_bits)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -24 * size + 2.0 ** -134).all()


class Case:
    """T tokens with their inputs on both sides; the cache is poisoned with 0xA5."""

    def __init__(self, T, H, P, rng, norm=True, halves=False, pages=None):
        self.T, self.H, self.P, self.halves = T, H, P, halves
        self.pages = pages or -(-T // P) + 2
        self.latent = _bits(rng.standard_normal((T, 512)) * np.exp(rng.standard_normal((T, 1))))
        self.k_pe = _bits(rng.standard_normal((T, 64)))
        self.q = _bits(rng.standard_normal((T, H, 64))) if H else np.zeros((T, 0, 64), dtype=np.uint16)
        self.weight = _bits(np.exp(0.5 * rng.standard_normal(512))) if norm else None
        self.angles = _angles(rng)
        self.pos = rng.integers(0, POSITIONS, T)
        self.slots = rng.permutation(self.pages * P)[:T]
        self.cache = torch.full((self.pages, 400 * P + 32), 0xA5, dtype=torch.uint8, device="cuda")
        self.dev = dict(latent=to_device(self.latent), k_pe=to_device(self.k_pe), angles=torch.from_numpy(self.angles).cuda(),
                        weight=None if self.weight is None else to_device(self.weight), pos=_i32(self.pos),
                        slots=_i32(self.slots))
        self.q_in = to_device(self.q) if H else None
        self.q_out = torch.full((T, H, 64), 0x7777, dtype=torch.int16, device="cuda") if H else None

    def run(self, eps=EPS, stream=None, status=0):
        d, H = self.dev, self.H
        _ok(mq.mlaqp_kv4_append_rope(
            d["latent"], 512, d["weight"], eps, d["k_pe"], 64, self.q_in, 64 * H, 64, self.q_out, 64 * H, 64, H, d["pos"],
            d["angles"], POSITIONS, "halves" if self.halves else "interleaved", self.cache, self.cache.stride(0),
            self.pages, self.P, d["slots"], self.T, stream=stream))
        torch.cuda.synchronize()
        assert _device_status() == status

    def check(self, eps=EPS):
        got = self.cache.cpu().numpy()
        want = np.full_like(got, 0xA5)
        P = self.P
        y = so.normalise(self.latent, self.weight, eps)
        keys, places = [], []
        for t in range(self.T):
            if not (0 <= self.pos[t] < POSITIONS and 0 <= self.slots[t] < self.pages * P):
                continue
            page, at = want[self.slots[t] // P], self.slots[t] % P
            page[256 * at: 256 * at + 256], page[384 * P + 16 * at: 384 * P + 16 * at + 16] = so.codes_and_scales(y[t])
            row = got[self.slots[t] // P][256 * P + 128 * at: 256 * P + 128 * at + 128]
            keys.append(np.ascontiguousarray(row).view(np.uint16).reshape(8, 8)[np.arange(8) ^ (at & 7)].reshape(-1))
            places.append(t)
            page[256 * P + 128 * at: 256 * P + 128 * at + 128] = row
        np.testing.assert_array_equal(got, want)  # and nothing else was written
        if places:
            _close(np.stack(keys), self.k_pe[places], self.angles[self.pos[places]], self.halves)
        if self.H:
            out = to_host_bits(self.q_out, np.uint16)
            left = (self.pos < 0) | (self.pos >= POSITIONS)
            assert (out[left] == 0x7777).all()
            _close(out[~left], self.q[~left], np.repeat(self.angles[self.pos[~left]][:, None], self.H, 1), self.halves)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T,H,P,norm", [(1, 1, 16, True), (1, 16, 128, False), (7, 8, 64, True), (9, 11, 32, True),
                                        (33, 16, 16, True), (5, 17, 64, True), (3, 128, 64, False), (8, 4, 16, True),
                                        (130, 0, 64, True), (2, 31, 32, False)])
def test_tokens_and_queries(cuda_device, T, H, P, norm, halves):
    c = Case(T, H, P, np.random.default_rng(T * 1000 + H), norm, halves)
    c.run()
    c.check()


def test_without_norm_the_codes_are_the_plain_appends(cuda_device):
    c = Case(40, 0, 32, np.random.default_rng(5), norm=False)
    c.run()
    plain = torch.full_like(c.cache, 0xA5)
    _ok(mq.mlaqp_kv4_append(c.dev["latent"], 512, c.dev["k_pe"], 64, plain, plain.stride(0), c.pages, 32, c.dev["slots"], 40))
    for page, want in zip(c.cache.cpu().numpy(), plain.cpu().numpy()):
        assert np.array_equal(page[:256 * 32], want[:256 * 32]) and np.array_equal(page[384 * 32:], want[384 * 32:])


@pytest.mark.parametrize("halves", [False, True])
def test_tokens_that_are_left_out(cuda_device, halves):
    c = Case(12, 5, 16, np.random.default_rng(6), halves=halves)
    c.slots[[1, 4]] = -1, -(1 << 31)
    c.slots[7] = c.pages * 16
    c.pos[[2, 4, 8]] = -1, 3, -(1 << 31)
    c.pos[9] = POSITIONS
    c.dev["slots"], c.dev["pos"] = _i32(c.slots), _i32(c.pos)
    c.run(status=mq.MLAQP_DEVSTATUS_BAD_INDEX)
    c.check()
    c = Case(4, 5, 16, np.random.default_rng(6), halves=halves)  # padding alone is not reported
    c.slots[[1, 2]] = -1
    c.pos[[2, 3]] = -1
    c.dev["slots"], c.dev["pos"] = _i32(c.slots), _i32(c.pos)
    c.run()
    c.check()


@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e4])
def test_special_latents(cuda_device, eps):
    rng = np.random.default_rng(7)
    c = Case(12, 0, 16, rng)
    v = oracle.bf16_to_f64(c.latent).astype(np.float32)
    v[0] = 0.0                      # with eps 0: 0 * infinity
    v[1] = -0.0
    v[2, 5] = np.nan                # all NaN
    v[3, 40] = np.inf               # r = 0: that block NaN, the others zero
    v[4] *= 2.0 ** 70               # squares beyond FP32: zeros
    v[5] *= 2.0 ** -60              # squares below its normal range
    v[6] = 0.0
    v[6, 511] = 2.0 ** -20
    v[7, :256] *= 2.0 ** 30         # parts of very different size
    v[8] = 1.0
    v[9, ::2] = 2.0 ** 12
    c.latent = _bits(v)
    c.dev["latent"] = to_device(c.latent)
    # below FP32's normal range squares lose bits of their own: not compared there with eps = 0
    if eps == 0.0:
        c.latent[5] = c.latent[8]
        c.dev["latent"] = to_device(c.latent)
    c.run(eps)
    with np.errstate(all="ignore"):
        c.check(eps)


def test_sums_of_squares_at_the_end_of_fp32(cuda_device):
    c = Case(6, 0, 16, np.random.default_rng(21))
    v = np.zeros((6, 512), dtype=np.float32)
    v[0] = 1.25 * 2.0 ** 59     # sum 1.5625 * 2^127
    v[1] = 1.5 * 2.0 ** 59      # sum 2.25 * 2^127: r = 0
    v[2, 77] = 1.375 * 2.0 ** 63
    v[3, 77] = 1.5 * 2.0 ** 63  # r = 0
    v[4, ::2] = 1.5 * 2.0 ** 59
    v[5] = np.where(np.arange(512) < 256, 1.25 * 2.0 ** 59, 2.0 ** 20)
    c.latent = _bits(v)
    c.dev["latent"] = to_device(c.latent)
    c.run()
    c.check()


def test_one_buffer_for_everything_rotated_in_place(cuda_device):
    rng = np.random.default_rng(8)
    T, H, P, row = 20, 11, 32, 11 * 192 + 576 + 24
    c = Case(T, H, P, rng)
    buf = _bits(rng.standard_normal((T, row)))
    buf[:, H * 192:H * 192 + 512], buf[:, H * 192 + 512:H * 192 + 576] = c.latent, c.k_pe
    heads = buf[:, :H * 192].reshape(T, H, 192)
    heads[:, :, 128:] = c.q
    dev = to_device(buf)
    lat = dev[:, H * 192:]
    q = dev[:, 128:]
    d = c.dev
    _ok(mq.mlaqp_kv4_append_rope(lat, row, d["weight"], EPS, lat[:, 512:], row, q, row, 192, q, row, 192, H, d["pos"],
                                 d["angles"], POSITIONS, "interleaved", c.cache, c.cache.stride(0), c.pages, P,
                                 d["slots"], T))
    torch.cuda.synchronize()
    after = to_host_bits(dev, np.uint16)
    part = after[:, :H * 192].reshape(T, H, 192)[:, :, 128:]
    c.q_out = to_device(np.ascontiguousarray(part))
    c.check()
    after[:, :H * 192].reshape(T, H, 192)[:, :, 128:] = c.q
    np.testing.assert_array_equal(after, buf)  # nothing beside the parts has changed


def test_broadcast_rows_and_padded_outputs(cuda_device):
    rng = np.random.default_rng(9)
    c = Case(6, 3, 16, rng)
    c.latent[:], c.k_pe[:], c.q[:] = c.latent[:1], c.k_pe[:1], c.q[:1, :1]
    out = torch.full((6, 3 * 80 + 8), 0x7777, dtype=torch.int16, device="cuda")
    d = c.dev
    _ok(mq.mlaqp_kv4_append_rope(to_device(c.latent[0]), 0, d["weight"], EPS, to_device(c.k_pe[0]), 0, to_device(c.q[0, 0]), 0, 0,
                                 out, 3 * 80 + 8, 80, 3, d["pos"], d["angles"], POSITIONS, 0, c.cache, c.cache.stride(0),
                                 c.pages, 16, d["slots"], 6))
    torch.cuda.synchronize()
    c.q_out = out[:, :240].reshape(6, 3, 80)[:, :, :64].contiguous()
    c.check()
    assert (out[:, 240:] == 0x7777).all() and (out[:, :240].reshape(6, 3, 80)[:, :, 64:] == 0x7777).all()


def test_graph_replay_with_other_inputs_and_another_stream(cuda_device):
    rng = np.random.default_rng(10)
    _ok(mq.mlaqp_kv4_step_prewarm())
    c = Case(17, 16, 64, rng)
    side = torch.cuda.Stream()
    c.run(stream=side)
    c.check()
    g = torch.cuda.CUDAGraph()
    d = c.dev
    with torch.cuda.graph(g):
        _ok(mq.mlaqp_kv4_append_rope(
            d["latent"], 512, d["weight"], EPS, d["k_pe"], 64, c.q_in, 1024, 64, c.q_out, 1024, 64, 16, d["pos"], d["angles"],
            POSITIONS, 0, c.cache, c.cache.stride(0), c.pages, 64, d["slots"], 17))
    other = Case(17, 16, 64, np.random.default_rng(11))
    for name in ("latent", "k_pe", "weight", "pos", "slots", "angles"):
        d[name].copy_(other.dev[name])
    c.q_in.copy_(other.q_in)
    c.cache.fill_(0xA5)
    g.replay()
    torch.cuda.synchronize()
    other.cache, other.q_out = c.cache, c.q_out
    other.check()


def test_offsets_beyond_32_bits(cuda_device):
    """A pool of more than 4 GB, tokens at both of its ends."""
    P, pages = 128, 90000
    c = Case(6, 2, P, np.random.default_rng(12), pages=2)
    cache = torch.empty(pages, 400 * P, dtype=torch.uint8, device="cuda")
    for page in (0, pages - 1):
        cache[page].fill_(0xA5)
    slots = np.array([0, 5, P - 1, (pages - 1) * P, (pages - 1) * P + 77, pages * P - 1])
    d = c.dev
    _ok(mq.mlaqp_kv4_append_rope(d["latent"], 512, d["weight"], EPS, d["k_pe"], 64, c.q_in, 128, 64, c.q_out, 128, 64, 2, d["pos"],
                                 d["angles"], POSITIONS, 0, cache, cache.stride(0), pages, P, _i32(slots), 6))
    torch.cuda.synchronize()
    c.cache.fill_(0xA5)
    c.cache[0, :400 * P], c.cache[1, :400 * P] = cache[0], cache[pages - 1]
    c.slots = np.array([0, 5, P - 1, P, P + 77, 2 * P - 1])
    c.check()
