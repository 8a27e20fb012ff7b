"""Measured operators: what a decode step over the paged 4-bit latent cache needs around its attention.

`append` normalises latents, rotates the key parts and the queries' parts by
their positions and writes the tokens into the cache (read back, as the values
that the cache stands for).  `digest` takes the bounds of every channel over
the tokens of each page that has filled up.  `sparse` selects pages for every
query token by those bounds and attends over the selected ones.

With `own` false every operator runs in its plain form, elementary torch
operations in 32 bits (64 for integer sums and the mean of squares); with
`own` true it is the library's call.

A cached token is 512 latents as E2M1 codes with an E8M0 scale byte per 32,
and 64 rope elements in BF16.  A page of P tokens holds three planes, codes
[P][256 bytes], rope [P][128 bytes] and scales [P][16 bytes].  A page's digest
is 1168 bytes: 512 upper bounds of the latents, 512 lower ones, 64 upper and 64
lower ones of the rope elements (8-bit integers), an exponent byte for each of
the two parts, zeros.
"""

import math
import random

import torch

own = False

LATENT = 512
ROPE = 64
DIM = LATENT + ROPE
BLOCK = 32
NBLOCK = LATENT // BLOCK
TOKEN_BYTES = LATENT // 2 + 2 * ROPE + NBLOCK
DIGEST_BYTES = 2 * DIM + 16
SCALE_MIN, SCALE_MAX = 87, 167
EXP_MIN, EXP_MAX, EXP_NONE = -60, 60, 255
SOFTMAX_SCALE = 1.0 / math.sqrt(192.0)  # nope dim 128 + rope dim 64
POSITIONS = 131072
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the tokens of one decode step of a full batch
        dict(name="append_decode", op="append", T=64, H=16, page=64, style="interleaved", norm=True),
        # a short prompt of a model that splits its rotated halves and normalises elsewhere, odd head count, small pages
        dict(name="append_halves", op="append", T=1027, H=11, page=16, style="halves", norm=False),
        # a long prompt with its queries
        dict(name="append_prompt", op="append", T=16385, H=16, page=32, style="interleaved", norm=True),
        # speculative decoding: a few tokens of every sequence, some of them fill a page
        dict(name="digest_step", op="digest", seqs=32, new=17, max_len=4000, page=16),
        # prompts that have just been written
        dict(name="digest_prompt", op="digest", seqs=16, new=4096, max_len=4097, page=64),
        # a few short conversations, most of them within what is selected anyway: latency alone
        dict(name="sparse_short", op="sparse", B=4, q_len=1, H=16, min_len=50, max_len=3000, page=64, k=24, first=1,
             last=2, q="bf16"),
        # an ordinary batch
        dict(name="sparse_b48_8k", op="sparse", B=48, q_len=1, H=16, min_len=2000, max_len=8191, page=64, k=24, first=1,
             last=2, q="bf16"),
        # multi-token prediction, odd head count, small pages
        dict(name="sparse_b16_mtp", op="sparse", B=16, q_len=4, H=11, min_len=900, max_len=9100, page=16, k=64, first=1,
             last=4, q="e4m3"),
        # one long document on a model split over its heads
        dict(name="sparse_b1_128k", op="sparse", B=1, q_len=1, H=8, min_len=131071, max_len=131071, page=128, k=32,
             first=1, last=1, q="bf16"),
        # a full server: many long contexts, E4M3 queries as the projection writes them
        dict(name="sparse_b64_32k", op="sparse", B=64, q_len=1, H=16, min_len=16000, max_len=32768, page=64, k=32,
             first=1, last=2, q="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "digest", "sparse", "sparse", "sparse"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        return dict(op=op, T=_log_int(rng, 1, 16384), H=rng.choice([8, 11, 16]), page=page,
                    style=rng.choice(["interleaved", "halves"]), norm=rng.random() < 0.7)
    if op == "digest":
        seqs = _log_int(rng, 1, 64)
        new = _log_int(rng, page, 65536 // seqs)
        return dict(op=op, seqs=seqs, new=new, max_len=new + rng.randint(0, 2000), page=page)
    b = _log_int(rng, 1, 64)
    top = _log_int(rng, 1, min(131072, 1500000 // b))
    q_len = rng.choice([1, 1, 1, 2, 3, 4])
    if b * q_len > 64:
        q_len = 1
    last = rng.randint(1, 4)
    first = rng.randint(0, 2)
    most = max(first + last, min(2048 // page, 131072 // (b * q_len * page)))
    return dict(op=op, B=b, q_len=q_len, H=rng.choice([8, 11, 16]), min_len=rng.randint(1, top), max_len=top, page=page,
                k=rng.randint(first + last, most), first=first, last=last, q=rng.choice(["bf16", "e4m3"]))


def _layout_rng(case):
    """Sizes that belong to the case, the same for every seed."""
    return random.Random("|".join(f"{k}={case[k]}" for k in sorted(case) if k != "name"))


def _lens(case):
    r = _layout_rng(case)
    if case["op"] == "digest":
        return [r.randint(case["new"], case["max_len"]) for _ in range(case["seqs"])]
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["B"])]
    lens[r.randrange(case["B"])] = case["max_len"]
    return lens


def _filled(case):
    """Pages that fill up with the last `new` tokens of each sequence."""
    P = case["page"]
    return sum(n // P - (n - case["new"]) // P for n in _lens(case))


def work(case):
    op, P = case["op"], case["page"]
    if op == "append":
        T, H = case["T"], case["H"]
        # latents and keys in, codes out and in again, rows out; queries in and out; angles, position and slot
        per = 2 * DIM + 2 * TOKEN_BYTES + 2 * DIM + 2 * 2 * H * ROPE + 4 * ROPE + 12
        return {"bytes": T * per, "flops": T * (5 * LATENT + 3 * ROPE * (H + 1))}
    if op == "digest":
        pages = _filled(case)
        return {"bytes": pages * (P * TOKEN_BYTES + DIGEST_BYTES + 4), "flops": pages * P * 3 * DIM}
    H, q_len = case["H"], case["q_len"]
    rows = case["B"] * q_len
    qb = DIM * (2 if case["q"] == "bf16" else 1)
    scored = attended = bounds = 0
    for n in _lens(case):
        middle = 0
        for i in range(q_len):
            seen = max(0, n - (q_len - 1 - i))
            pages = -(-seen // P)
            if pages > case["k"]:
                middle = max(middle, pages - case["first"] - case["last"])
                bounds += pages - case["first"] - case["last"]
            attended += seen if pages <= case["k"] else (case["k"] - 1) * P + seen - (pages - 1) * P
        scored += middle
    return {"bytes": scored * (DIGEST_BYTES + 4) + attended * TOKEN_BYTES
            + rows * (H * (qb + 2 * LATENT + 4) + 4 * case["k"] + 4) + 4 * case["B"],
            "flops": 2 * bounds * 2 * DIM + 2 * attended * H * (DIM + LATENT)}


# ---------------------------------------------------------------------------
# The cache's layout and codes, in elementary operations
# ---------------------------------------------------------------------------

def _quantise(lat):
    """[T,512] floats -> E2M1 codes [T,512] (sign 8, magnitude 0..7) and scale bytes [T,16]."""
    blk = lat.float().reshape(-1, NBLOCK, BLOCK)
    bits = blk.abs().amax(-1).contiguous().view(torch.int32)
    byte = torch.clamp(((bits + 0x1FFFFF) >> 23) - 2, SCALE_MIN, SCALE_MAX)
    y = blk * torch.exp2((127 - byte).float()).unsqueeze(-1)
    a = y.abs()
    mag = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
           + (a >= 3.5).int() + (a > 5.0).int())
    return (mag + 8 * torch.signbit(blk).int()).reshape(-1, LATENT), byte


def _swap_halves(word):
    odd = ((torch.arange(NBLOCK, device=word.device) & 4) != 0)[:, None]
    return torch.where(odd, word.roll(2, -1), word)


def _element_bits(device):
    """Bit of the magnitude and of the sign of each of a word's eight elements."""
    e = torch.arange(8, device=device)
    return 4 * e, torch.where(e < 4, 8 * e + 7, 8 * (e - 4) + 3)


def _pack_codes(code):
    """Codes [T,512] -> bytes [T,256]: 32-bit words of eight elements; blocks with bit 2 of their number set hold
    their two 8-byte halves in swapped order."""
    c = code.reshape(-1, NBLOCK, 4, 8).long()
    mag, sign = _element_bits(code.device)
    word = _swap_halves((((c & 7) << mag) + ((c >> 3) << sign)).sum(-1))
    out = (word.unsqueeze(-1) >> torch.arange(0, 32, 8, device=code.device)) & 255
    return out.to(torch.uint8).reshape(-1, LATENT // 2)


def _unpack_codes(raw):
    """Bytes [T,256] -> signed code values [T,512] in 32-bit floats."""
    word = _swap_halves(raw.contiguous().view(torch.int32).reshape(-1, NBLOCK, 4)).unsqueeze(-1)
    at, sign = _element_bits(raw.device)
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=raw.device)
    v = mags[((word >> at.int()) & 7).long()]
    return torch.where(((word >> sign.int()) & 1) != 0, -v, v).reshape(-1, LATENT)


def _rope_at(page, pos):
    """Byte offsets [T,8,16] of a token's rope row within its page: chunk c lies at place c ^ (pos & 7)."""
    chunk = torch.arange(8, device=pos.device) ^ (pos & 7)[:, None]
    return 256 * page + (pos * 128)[:, None, None] + 16 * chunk[:, :, None] + torch.arange(16, device=pos.device)


def _store(cache, page, slots, code, byte, rope):
    pg, pos = slots // page, slots % page
    ar = torch.arange(256, device=cache.device)
    cache[pg[:, None], (pos * 256)[:, None] + ar] = _pack_codes(code)
    cache[pg[:, None, None], _rope_at(page, pos)] = rope.contiguous().view(torch.uint8).reshape(-1, 8, 16)
    cache[pg[:, None], 384 * page + (pos * 16)[:, None] + ar[:16]] = byte.to(torch.uint8)


def _load(cache, page, slots):
    """Tokens at `slots` as 32-bit floats: latents [T,512], rope [T,64]."""
    pg, pos = slots // page, slots % page
    ar = torch.arange(256, device=cache.device)
    code = cache[pg[:, None], (pos * 256)[:, None] + ar]
    rope = cache[pg[:, None, None], _rope_at(page, pos)].reshape(-1, 128).view(torch.bfloat16).float()
    byte = cache[pg[:, None], 384 * page + (pos * 16)[:, None] + ar[:16]].float()
    lat = _unpack_codes(code).reshape(-1, NBLOCK, BLOCK) * torch.exp2(byte - 127.0).unsqueeze(-1)
    return lat.reshape(-1, LATENT), rope


def _bounds(values, top):
    """Outward integers of values [n,2,c] (largest, smallest) on the grid 2^e, and the exponent byte [n]."""
    bits = values.abs().amax((1, 2)).contiguous().view(torch.int32)
    e = torch.clamp(((bits + 0x01FFFF) >> 23) - 127 - 6, min=EXP_MIN)
    y = values * torch.exp2(-e.float())[:, None, None]
    known = e <= EXP_MAX
    out = torch.stack([torch.ceil(y[:, 0]), torch.floor(y[:, 1])], 1)
    out = torch.where(known[:, None, None], out, torch.zeros_like(out))
    return out.to(torch.int8).reshape(values.shape[0], 2 * top), torch.where(known, e + 127, EXP_NONE)


def _digest_rows(cache, page, pages):
    """Digests [n,1168] of full pages."""
    n = pages.numel()
    slots = (pages[:, None] * page + torch.arange(page, device=cache.device)).reshape(-1)
    lat, rope = _load(cache, page, slots)
    lat, rope = lat.reshape(n, page, LATENT), rope.reshape(n, page, ROPE)
    lat_q, lat_e = _bounds(torch.stack([lat.amax(1), lat.amin(1)], 1), LATENT)
    rope_q, rope_e = _bounds(torch.stack([rope.amax(1), rope.amin(1)], 1), ROPE)
    tail = torch.zeros(n, 16, dtype=torch.uint8, device=cache.device)
    tail[:, 0], tail[:, 1] = lat_e.to(torch.uint8), rope_e.to(torch.uint8)
    return torch.cat([lat_q.view(torch.uint8), rope_q.view(torch.uint8), tail], 1)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _fill(cache, page, slots, g):
    """Cached context: latents as a normalised down-projection leaves them (a spread of channel gains) about what their
    page deals with, and rotated keys.  Returns the pages' topics."""
    gain = torch.exp(0.4 * torch.randn(LATENT, generator=g, device="cuda"))
    topics = 0.7 * torch.randn(cache.shape[0], LATENT, generator=g, device="cuda") * gain
    for i in range(0, slots.numel(), 65536):
        s = slots[i:i + 65536]
        lat = torch.randn(s.numel(), LATENT, generator=g, device="cuda") * gain + topics[s // page]
        code, byte = _quantise(lat)
        _store(cache, page, s, code, byte, torch.randn(s.numel(), ROPE, generator=g, device="cuda").to(torch.bfloat16))
    return topics


def _paged_slots(lens, page, g, spare=3):
    """A table of shuffled pages for sequences of these lengths: (table, pages, slots of every token in order)."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    slots, at = [], 0
    for b, (n, k) in enumerate(zip(lens, need)):
        table[b, :k] = perm[at:at + k]
        t = torch.arange(n, device="cuda")
        slots.append(perm[at:at + k].long()[t // page] * page + t % page)
        at += k
    return table, total, torch.cat(slots)


def _angles():
    """cos and sin of the 32 frequencies at every position, [POSITIONS,64]."""
    f = 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
    a = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def prepare(case, seed):
    g = _gen(seed)
    return {"append": _prepare_append, "digest": _prepare_digest, "sparse": _prepare_sparse}[case["op"]](case, g)


def _prepare_append(case, g):
    T, H, page = case["T"], case["H"], case["page"]
    _, pages, slots = _paged_slots([T], page, g)
    rows = torch.randn(T, DIM, generator=g, device="cuda") * torch.exp(0.3 * torch.randn(T, 1, generator=g, device="cuda"))
    weight = torch.exp(0.4 * torch.randn(LATENT, generator=g, device="cuda")).to(torch.bfloat16)
    if T <= 256:  # one token of each sequence
        pos = torch.randint(0, POSITIONS, (T,), generator=g, device="cuda")
    else:  # a prompt, from somewhere on
        pos = torch.randint(0, POSITIONS - T, (1,), generator=g, device="cuda") + torch.arange(T, device="cuda")
    return dict(case=case, cache=torch.full((pages, TOKEN_BYTES * page), 255, dtype=torch.uint8, device="cuda"),
                slots=slots.int(), rows=rows.to(torch.bfloat16), weight=weight if case["norm"] else None,
                pos=pos.int(), cos_sin=_angles(),
                # the projection's [T,H,192] output: the last 64 of each head are the rotated part
                q=torch.randn(T, H, 192, generator=g, device="cuda").to(torch.bfloat16),
                q_pe=torch.empty(T, H, ROPE, dtype=torch.bfloat16, device="cuda"),
                out=torch.empty(T, DIM, dtype=torch.bfloat16, device="cuda"))


def _prepare_digest(case, g):
    lens, page = _lens(case), case["page"]
    table, pages, slots = _paged_slots(lens, page, g)
    cache = torch.full((pages, TOKEN_BYTES * page), 127, dtype=torch.uint8, device="cuda")
    _fill(cache, page, slots, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(case=case, cache=cache, table=table, lens=torch.tensor(lens, **i32),
                seqs=torch.arange(case["seqs"], **i32), new=torch.full((case["seqs"],), case["new"], **i32),
                digests=torch.zeros(pages, DIGEST_BYTES, dtype=torch.uint8, device="cuda"))


def _prepare_sparse(case, g):
    B, q_len, H, page, k = case["B"], case["q_len"], case["H"], case["page"], case["k"]
    M = B * q_len
    lens = _lens(case)
    table, pages, slots = _paged_slots(lens, page, g)
    cache = torch.full((pages, TOKEN_BYTES * page), 127, dtype=torch.uint8, device="cuda")
    topics = _fill(cache, page, slots, g)
    digests = torch.cat([_digest_rows(cache, page, torch.arange(i, min(i + 2048, pages), device="cuda"))
                         for i in range(0, pages, 2048)])
    q = torch.randn(B, q_len, H, DIM, generator=g, device="cuda")
    # half of the heads ask for what one of the sequence's pages deals with
    pick = torch.floor(torch.rand(B, generator=g, device="cuda") * ((torch.tensor(lens, device="cuda") + page - 1) // page))
    q[:, :, ::2, :LATENT] += topics[table[torch.arange(B, device="cuda"), pick.long()].long()][:, None, None]
    q = q.reshape(M, H, DIM)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=case, cache=cache, digests=digests, table=table, lens=torch.tensor(lens, **i32),
             q_scale=None, sel=torch.empty(M, k, **i32), sel_lens=torch.empty(M, **i32),
             x=torch.empty(M, H, LATENT, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(M, H, dtype=torch.float32, device="cuda"))
    if case["q"] == "bf16":
        s["q"] = q.to(torch.bfloat16)
    else:
        s["q_scale"] = torch.tensor([0.02], device="cuda")
        s["q"] = (q / s["q_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
    if own:
        import mla_decode_query_gb300 as mq
        n = mq.mlaqp_kv4_select_workspace(B, q_len, table.shape[1], pages)
        s["select_ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        n = mq.mlaqp_kv4_attend_workspace(M, 1, H)
        s["attend_ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    table = _OWN if own else _PLAIN
    return table[op](state)


def _rotate(v, angles, style):
    """[T,n,64] rotated by the angles [T,64] of the tokens."""
    cos, sin = angles[:, None, :32], angles[:, None, 32:]
    v = v.float()
    if style == "interleaved":
        a, b = v[..., 0::2], v[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = v[..., :32], v[..., 32:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append_plain(s):
    case, page, slots = s["case"], s["case"]["page"], s["slots"].long()
    angles = s["cos_sin"][s["pos"].long()]
    lat = s["rows"][:, :LATENT].float()
    if s["weight"] is not None:
        mean = (lat.double() ** 2).mean(-1, keepdim=True).float()
        lat = lat * (1.0 / torch.sqrt(mean + EPS)) * s["weight"].float()
    code, byte = _quantise(lat)
    key = _rotate(s["rows"][:, None, LATENT:], angles, case["style"])[:, 0].to(torch.bfloat16)
    _store(s["cache"], page, slots, code, byte, key)
    s["q_pe"].copy_(_rotate(s["q"][..., 128:], angles, case["style"]).to(torch.bfloat16))
    lat, rope = _load(s["cache"], page, slots)
    return {"rows": torch.cat([lat, rope], 1).to(torch.bfloat16), "q_pe": s["q_pe"]}


def _append_own(s):
    import mla_decode_query_gb300 as mq
    case, rows, cache, q, q_pe = s["case"], s["rows"], s["cache"], s["q"], s["q_pe"]
    T, H, page = case["T"], case["H"], case["page"]
    mq.check(mq.mlaqp_kv4_append_rope(
        rows, DIM, s["weight"], EPS, rows[:, LATENT:], DIM, q[..., 128:], H * 192, 192, q_pe, H * ROPE, ROPE, H, s["pos"],
        s["cos_sin"], POSITIONS, case["style"], cache, cache.stride(0), cache.shape[0], page, s["slots"], T))
    mq.check(mq.mlaqp_kv4_gather(cache, cache.stride(0), cache.shape[0], page, s["slots"], T, s["out"], DIM))
    return {"rows": s["out"], "q_pe": q_pe}


def _digest_plain(s):
    page, lens = s["case"]["page"], s["lens"].long()
    j = torch.arange(s["table"].shape[1], device=lens.device)
    end = (j + 1) * page
    filled = (end <= lens[:, None]) & (end > (lens - s["new"])[:, None])
    pages = s["table"][filled].long()
    s["digests"][pages] = _digest_rows(s["cache"], page, pages)
    return {"digests": s["digests"]}


def _digest_own(s):
    import mla_decode_query_gb300 as mq
    case, cache, table, digests = s["case"], s["cache"], s["table"], s["digests"]
    mq.check(mq.mlaqp_kv4_digest(cache, cache.stride(0), cache.shape[0], case["page"], table, table.stride(0),
                                 table.shape[0], s["lens"], s["seqs"], s["new"], case["seqs"], case["new"], digests,
                                 digests.stride(0)))
    return {"digests": digests}


def _select_plain(s):
    """Block table [M,k] and lengths [M] of the selected pages."""
    case = s["case"]
    B, q_len, H, page, k = case["B"], case["q_len"], case["H"], case["page"], case["k"]
    first, last, M = case["first"], case["last"], case["B"] * case["q_len"]
    q = s["q"].float()
    bits = q.abs().amax((1, 2)).contiguous().view(torch.int32)
    f = torch.clamp(((bits + 0x1FFF) >> 23) - 127 - 10, min=-100)
    qi = torch.round(q * torch.exp2(-f.float())[:, None, None]).double()
    up, down = qi.clamp(min=0).sum(1).reshape(B, q_len, DIM), qi.clamp(max=0).sum(1).reshape(B, q_len, DIM)
    d = s["digests"][s["table"].clamp(min=0).long()]  # [B,W,1168]
    v = d[..., :2 * DIM].view(torch.int8).double()
    hi, lo, rhi, rlo = v.split([LATENT, LATENT, ROPE, ROPE], -1)
    e = d[..., 2 * DIM:2 * DIM + 2].double()
    lat = up[..., :LATENT] @ hi.transpose(1, 2) + down[..., :LATENT] @ lo.transpose(1, 2)
    rope = up[..., LATENT:] @ rhi.transpose(1, 2) + down[..., LATENT:] @ rlo.transpose(1, 2)
    power = torch.exp2(e.clamp(max=EXP_MAX + 127) - 127).float()[:, None]
    score = lat.float() * power[..., 0] + rope.float() * power[..., 1]
    none = (e == EXP_NONE).any(-1)[:, None].expand_as(score)
    score = torch.where(none, torch.full_like(score, float("inf")), score).reshape(M, -1)
    i = torch.arange(q_len, device=q.device)
    n = (s["lens"].long()[:, None] - (q_len - 1 - i)).clamp(min=0).reshape(M, 1)
    pages = (n + page - 1) // page
    j = torch.arange(score.shape[1], device=q.device)
    middle = (j >= first) & (j < pages - last)
    order = torch.sort(torch.where(middle, score, torch.full_like(score, float("-inf"))), dim=1,
                       descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order).contiguous())
    chosen = torch.where(middle & (pages > k), rank < k - first - last, j < pages)
    at = torch.sort(torch.where(chosen, j, score.shape[1]), 1).values[:, :k]
    rows = s["table"].repeat_interleave(q_len, 0)
    got = torch.where(at < score.shape[1], rows.gather(1, at.clamp(max=score.shape[1] - 1)), -1)
    s["sel"].fill_(-1)
    s["sel"][:, :got.shape[1]] = got
    s["sel_lens"].copy_(torch.where(pages > 0, (pages.clamp(max=k) - 1) * page + n - (pages - 1) * page, 0)[:, 0])


def _sparse_plain(s):
    case = s["case"]
    H, page, k, M = case["H"], case["page"], case["k"], case["B"] * case["q_len"]
    _select_plain(s)
    t = torch.arange(k * page, device=s["q"].device)
    slots = s["sel"].long().clamp(min=0)[:, t // page] * page + t % page
    lat, rope = _load(s["cache"], page, slots.reshape(-1))
    lat, rope = lat.reshape(M, -1, LATENT), rope.reshape(M, -1, ROPE)
    q = s["q"].float()
    if s["q_scale"] is not None:
        q = q * s["q_scale"]
    sc = (q[..., :LATENT] @ lat.transpose(1, 2) + q[..., LATENT:] @ rope.transpose(1, 2)) * SOFTMAX_SCALE
    seen = (t < s["sel_lens"][:, None])[:, None].expand_as(sc)
    sc = torch.where(seen, sc, torch.full_like(sc, float("-inf")))
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(sc - top)
    total = p.sum(-1, keepdim=True)
    x = torch.where(total > 0, (p @ lat) / total, torch.zeros_like(total))
    return {"table": s["sel"], "lens": s["sel_lens"], "x": x.to(torch.bfloat16), "lse": (top + torch.log(total))[..., 0]}


def _sparse_own(s):
    import mla_decode_query_gb300 as mq
    case, q, cache, table, digests = s["case"], s["q"], s["cache"], s["table"], s["digests"]
    B, q_len, H, page, k = case["B"], case["q_len"], case["H"], case["page"], case["k"]
    M, ws = B * q_len, s["select_ws"]
    mq.check(mq.mlaqp_kv4_select(q, H * DIM, case["q"], digests, digests.stride(0), cache.shape[0], page, table,
                                 table.stride(0), table.shape[0], s["lens"], None, B, q_len, H, k, case["first"],
                                 case["last"], s["sel"], k, s["sel_lens"], ws, ws.numel()))
    ws = s["attend_ws"]
    mq.check(mq.mlaqp_kv4_attend(q, H * DIM, case["q"], s["q_scale"], cache, cache.stride(0), cache.shape[0], page,
                                 s["sel"], k, M, s["sel_lens"], None, M, 1, H, SOFTMAX_SCALE, s["x"], H * LATENT, s["lse"],
                                 ws, ws.numel()))
    return {"table": s["sel"], "lens": s["sel_lens"], "x": s["x"], "lse": s["lse"]}


_PLAIN = dict(append=_append_plain, digest=_digest_plain, sparse=_sparse_plain)
_OWN = dict(append=_append_own, digest=_digest_own, sparse=_sparse_own)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(cache, page, slots):
    """Cached rows [T,576] in 64 bits, read byte by byte from the format."""
    rows = cache[slots // page]
    pos = slots % page
    n = torch.arange(LATENT, device=rows.device)
    j, i = n // BLOCK, n % BLOCK
    word, e = i // 8, i % 8
    stored = torch.where((j & 4) != 0, word ^ 2, word)
    base = (pos * 256)[:, None] + 16 * j + 4 * stored
    pick = lambda at: torch.gather(rows, 1, at).long()
    mag = (pick(base + e // 2) >> (4 * (e % 2))) & 7
    sign = (pick(base + e % 4) >> torch.where(e < 4, 7, 3)) & 1
    exponent, mantissa = mag >> 1, mag & 1
    v = torch.where(exponent > 0, torch.exp2((exponent - 1).double()) * (1.0 + 0.5 * mantissa), 0.5 * mantissa.double())
    byte = torch.gather(rows, 1, 384 * page + (pos * 16)[:, None] + j).double()
    v = v * (1.0 - 2.0 * sign) * torch.exp2(byte - 127.0)
    c = torch.arange(ROPE, device=rows.device)
    at = 256 * page + (pos * 128)[:, None] + 16 * ((c // 8) ^ (pos & 7)[:, None]) + 2 * (c % 8)
    bits = (torch.gather(rows, 1, at).int() | (torch.gather(rows, 1, at + 1).int() << 8)) << 16
    return torch.cat([v, bits.view(torch.float32).double()], 1)


def _exact_append(case, s):
    lat = s["rows"][:, :LATENT].double()
    if case["norm"]:
        lat = lat * torch.rsqrt((lat * lat).sum(1, keepdim=True) / LATENT + EPS) * s["weight"].double()
    lat = lat.reshape(-1, NBLOCK, BLOCK)
    top = lat.abs().amax(-1, keepdim=True)
    # the smallest power of two with top <= 7 * scale
    e = torch.ceil(torch.log2(torch.clamp(top / 7.0, min=1e-30)))
    e = torch.where(top > 7.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 7.0 * torch.exp2(e - 1), e - 1, e)
    scale = torch.exp2(e.clamp(SCALE_MIN - 127, SCALE_MAX - 127))
    y = lat / scale
    # E2M1 step: 0.5 below 2, 1 below 4, 2 from there; torch.round takes ties to even multiples of the step
    step = torch.where(y.abs() < 2.0, 0.5, torch.where(y.abs() < 4.0, 1.0, 2.0)).double()
    v = torch.clamp(torch.round(y / step) * step, -6.0, 6.0) * scale
    turn = torch.complex(s["cos_sin"][s["pos"].long(), :32].double(), s["cos_sin"][s["pos"].long(), 32:].double())

    def rotated(z):  # [T,n,64], the pairs as complex numbers
        z = z.double()
        halves = case["style"] == "halves"
        a, b = (z[..., :32], z[..., 32:]) if halves else (z[..., 0::2], z[..., 1::2])
        z = torch.complex(a, b) * turn[:, None]
        return torch.cat([z.real, z.imag], -1) if halves else torch.view_as_real(z).flatten(-2)

    key = rotated(s["rows"][:, None, LATENT:])[:, 0]
    return {"rows": torch.cat([v.reshape(-1, LATENT), key], 1), "q_pe": rotated(s["q"][:, :, 128:])}


def exact(case, seed):
    op = case["op"]
    if op == "digest":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "append":
        return _exact_append(case, s)
    B, q_len, H, page, k = case["B"], case["q_len"], case["H"], case["page"], case["k"]
    first, last = case["first"], case["last"]
    q = s["q"].double() if s["q_scale"] is None else s["q"].float().double()
    q = q.reshape(B, q_len, H, DIM)
    x = torch.zeros(B, q_len, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, q_len, H), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        digest = s["digests"][s["table"][b].clamp(min=0).long()]
        v = digest[:, :2 * DIM].view(torch.int8).double()
        hi, lo = torch.cat([v[:, :512], v[:, 1024:1088]], 1), torch.cat([v[:, 512:1024], v[:, 1088:1152]], 1)
        for i in range(q_len):
            seen = n - (q_len - 1 - i)
            if seen <= 0:
                continue
            pages = -(-seen // page)
            take = list(range(pages))
            if pages > k:
                a = q[b, i].abs().max().item()
                f = math.frexp(a)[1] - 11 if a > 0 else 0  # a = m * 2^(f + 11), m in [1/2,1)
                f += 1 if a > 2047 * 2.0 ** f else 0
                qi = torch.round(q[b, i] * 2.0 ** -f)
                up, down = qi.clamp(min=0).sum(0), qi.clamp(max=0).sum(0)
                parts = hi * up + lo * down
                # the two sums, whole numbers, and the score are 32-bit floats by definition: a tie there is a tie
                score = (parts[:, :LATENT].sum(1).float() * torch.exp2(digest[:, 1152].float() - 127)
                         + parts[:, LATENT:].sum(1).float() * torch.exp2(digest[:, 1153].float() - 127)).tolist()
                best = sorted(range(first, pages - last), key=lambda j: (-score[j], j))[:k - first - last]
                take = list(range(first)) + sorted(best) + list(range(pages - last, pages))
            at = torch.tensor([j * page for j in take], device="cuda")[:, None] + torch.arange(page, device="cuda")
            at = at.reshape(-1)
            at = at[at < seen]
            slots = s["table"][b].long()[at // page] * page + at % page
            key = torch.cat([_exact_rows(s["cache"], page, slots[c:c + 8192]) for c in range(0, slots.numel(), 8192)])
            query = q[b, i] if s["q_scale"] is None else q[b, i] * s["q_scale"].double()
            sc = query @ key.T * SOFTMAX_SCALE
            lse[b, i] = torch.logsumexp(sc, 1)
            x[b, i] = torch.exp(sc - lse[b, i][:, None]) @ key[:, :LATENT]
    return {"table": None, "lens": None, "x": x.reshape(B * q_len, H, LATENT), "lse": lse.reshape(B * q_len, H)}
