"""Decoding over the paged 4-bit latent cache, with this library's operators alone.

A few sequences get their prompts, one of them is forked (a beam, or two
samples of one prompt), all are decoded for some steps, the losing one is
released and the pool compacted.  A decode step of a layer is

    mlaqp_run -> mlaqp_kv4_append -> mlaqp_kv4_attend -> mlaqp_v_up_run

with mlaqp_kv4_extend once for all layers before it.  Nothing is read back
by the host in between: lengths, tables and slots live on the device.

Weights and activations are random; the projections around these operators
(q, kv and o) are left out, a model has them.

    PYTHONPATH=. python examples/kv4_decode_step.py
"""

from __future__ import annotations

import torch

import mla_decode_query_gb300 as mq

H, K = 16, 128                 # heads, nope dim
LAYERS, PAGE, PAGES = 2, 64, 96
SEQS, ROW = 8, 32              # rows of the block table, pages a row
SCALE = (K + 64) ** -0.5


def int32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    """A cache of all layers, its tables and what the calls want as workspace."""

    def __init__(self, batch):
        page_bytes = mq.mlaqp_kv4_page_bytes(PAGE)
        self.cache = torch.zeros(LAYERS, PAGES, page_bytes, dtype=torch.uint8, device="cuda")
        self.table = torch.full((SEQS, ROW), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(SEQS, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.live = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.tables = (self.table, ROW, SEQS, self.lens, self.refs, PAGES, PAGE)
        self.layers = (self.cache, page_bytes, self.cache.stride(0), LAYERS)
        self.work = torch.empty(max(mq.mlaqp_kv4_pages_workspace(PAGES, SEQS), mq.mlaqp_kv4_attend_workspace(batch, 1, H)),
                                dtype=torch.uint8, device="cuda")
        mq.check(mq.mlaqp_kv4_prewarm())

    def layer(self, i):
        return self.cache[i], self.cache.stride(1), PAGES, PAGE

    def extend(self, seqs, counts, max_new):
        slots = torch.empty(len(seqs), max_new, dtype=torch.int32, device="cuda")
        mq.check(mq.mlaqp_kv4_extend(*self.tables, seqs, counts, len(seqs), slots, max_new))
        return slots

    def append(self, i, rows, slots):  # rows: [T,576], latents and rope side by side
        mq.check(mq.mlaqp_kv4_append(rows, rows.stride(0), rows[:, 512:], rows.stride(0), *self.layer(i), slots,
                                     slots.numel()))

    def attend(self, i, q, seqs, x, lse):
        mq.check(mq.mlaqp_kv4_attend(q, q.stride(0), "bf16", None, *self.layer(i), self.table, ROW, SEQS, self.lens,
                                     seqs, len(seqs), 1, H, SCALE, x, x.stride(0), lse, self.work, self.work.numel()))

    def gather(self, i, slots):
        out = torch.empty(slots.numel(), 576, dtype=torch.bfloat16, device="cuda")
        mq.check(mq.mlaqp_kv4_gather(*self.layer(i), slots, slots.numel(), out, 576))
        return out


def run(steps=6, seed=0):
    """The largest difference of the last step's attention from float64, relative to its largest output."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    w_uk = [rand(H, K, 512) / K ** 0.5 for _ in range(LAYERS)]
    w_uv = [rand(H, 512, 128) / 512 ** 0.5 for _ in range(LAYERS)]
    pool = Pool(batch=4)

    # prompts of sequences 0..2
    prompts = (130, 64, 17)
    slots = pool.extend(int32(0, 1, 2), int32(*prompts), max(prompts))  # -1 behind the shorter ones
    for i in range(LAYERS):
        pool.append(i, rand(slots.numel(), 576), slots)

    # sequence 3 continues sequence 0 on its own: full pages shared, the last one copied
    mq.check(mq.mlaqp_kv4_fork(*pool.tables, int32(0), int32(3), 1, *pool.layers, pool.work, pool.work.numel()))

    seqs, ones = int32(0, 1, 2, 3), int32(1, 1, 1, 1)
    M = len(seqs)
    q = torch.empty(M, H * 576, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(M, H * 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(M, H, device="cuda")
    out = torch.empty(M, H * 128, dtype=torch.bfloat16, device="cuda")
    for _ in range(steps):
        slots = pool.extend(seqs, ones, 1)
        for i in range(LAYERS):
            mq.check(mq.mlaqp_run(rand(M, H, K), rand(M, H, 64), w_uk[i], None, q, 576 * H, None, M, H, "bf16", "bf16"))
            pool.append(i, rand(M, 576), slots)
            pool.attend(i, q, seqs, x, lse)
            mq.check(mq.mlaqp_v_up_run(x, 512 * H, 512, w_uv[i], None, out, 128 * H, M, H, "bf16"))

    # sequence 0 lost: its pages go (the shared ones stay with 3), the pool closes up
    mq.check(mq.mlaqp_kv4_release(*pool.tables, int32(0), 1))
    mq.check(mq.mlaqp_kv4_compact(*pool.tables, *pool.layers, pool.live, pool.work, pool.work.numel()))

    # the last layer's attention again, over the moved pages, against float64
    pool.attend(LAYERS - 1, q, seqs, x, lse)  # sequence 0 sees nothing now
    status, word = mq.mlaqp_device_status(reset=True)
    mq.check(status)
    assert word == 0, f"device status {word}"
    assert int(pool.live) == int((pool.refs > 0).sum()) and not pool.refs[int(pool.live):].any()
    assert not x[0].any() and torch.isneginf(lse[0]).all()
    worst = 0.0
    for b in range(1, M):
        n = int(pool.lens[b])
        t = torch.arange(n, device="cuda")
        keys = pool.gather(LAYERS - 1, (pool.table[b, t // PAGE] * PAGE + t % PAGE).int()).double()
        p = torch.softmax(SCALE * q[b].view(H, 576).double() @ keys.T, dim=-1)
        want = p @ keys[:, :512]
        worst = max(worst, ((x[b].view(H, 512).double() - want).abs().max() / want.abs().max()).item())
    return worst


if __name__ == "__main__":
    print(f"attention off by {run():.1e} of its largest output")
