"""Measured operators: the paged 4-bit latent cache and what works on it.

One cached token of one layer is 512 latents held as E2M1 codes with an E8M0
scale byte per 32, and 64 rope elements in BF16: 400 bytes.  A page of P
tokens holds three planes, codes [P][256 bytes], rope [P][128 bytes] and
scales [P][16 bytes], laid out as `_pack_codes` and `_rope_chunks` say.

Operators: `attend` (MLA decode attention over the cached tokens of each
sequence), `append` / `gather` (write tokens into the cache, read them back)
and the page operations (`beam`: fork, release and extend of a beam step;
`compact`: move the live pages to the front).

With `own` false every operator runs in its plain form, elementary torch
operations in 32 bits; with `own` true it is the library's call.
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
SCALE_MIN, SCALE_MAX, SCALE_NAN = 87, 167, 255
SOFTMAX_SCALE = 1.0 / math.sqrt(192.0)  # nope dim 128 + rope dim 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the first tokens of a single conversation: latency alone
        dict(name="attend_one_short", op="attend", B=1, q_len=1, H=16, min_len=200, max_len=200, page=64, q="bf16"),
        # a mixed batch of ordinary requests, every length from a few tokens up
        dict(name="attend_b32_mixed", op="attend", B=32, q_len=1, H=16, min_len=5, max_len=8191, page=64, q="bf16"),
        # multi-token prediction, odd head count (six-way split), small pages
        dict(name="attend_b16_mtp", op="attend", B=16, q_len=4, H=11, min_len=900, max_len=4100, page=16, q="e4m3"),
        # one long document on a model split eight ways over its heads
        dict(name="attend_b1_128k", op="attend", B=1, q_len=1, H=8, min_len=131071, max_len=131071, page=128, q="bf16"),
        # a full server: many long contexts, E4M3 queries as the projection writes them
        dict(name="attend_b64_32k", op="attend", B=64, q_len=1, H=16, min_len=16000, max_len=32768, page=64, q="e4m3"),
        # one decode step's tokens written and read back
        dict(name="append_decode", op="append", T=32, page=64),
        # a long prompt written chunk after chunk
        dict(name="append_prompt", op="append", T=16385, page=32),
        # cached context read back for a prompt that continues it
        dict(name="gather_context", op="gather", T=65536, page=64),
        # a beam step of one request
        dict(name="beam_small", op="beam", seqs=8, forks=2, layers=4, pages=96, max_len=500, page=64),
        # a beam step of a batch over a model's layers
        dict(name="beam_batch", op="beam", seqs=96, forks=48, layers=32, pages=768, max_len=420, page=64),
        # a small pool tidied after a request ended
        dict(name="compact_small", op="compact", pages=200, live=77, layers=4, seqs=9, page=16),
        # a model's whole pool tidied, half of it live
        dict(name="compact_pool", op="compact", pages=1024, live=512, layers=32, seqs=64, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "gather", "beam", "compact"])
    page = rng.choice([16, 32, 64, 128])
    if op == "attend":
        b = _log_int(rng, 1, 64)
        top = _log_int(rng, 1, min(131072, 1500000 // b))
        q_len = rng.choice([1, 1, 1, 2, 3, 4])
        if q_len > 1 and b * top > 600000:
            q_len = 1
        return dict(op=op, B=b, q_len=q_len, H=rng.choice([8, 11, 16]), min_len=rng.randint(1, top), max_len=top,
                    page=page, q=rng.choice(["bf16", "e4m3"]))
    if op in ("append", "gather"):
        return dict(op=op, T=_log_int(rng, 1, 16384 if op == "append" else 65536), page=page)
    layers = _log_int(rng, 1, 32)
    if op == "beam":
        seqs = _log_int(rng, 2, 96)
        max_len = rng.randint(1, 400)
        per = -(-max_len // page) + 1
        forks = rng.randint(1, max(1, min(64, seqs // 2)))
        return dict(op=op, seqs=seqs, forks=forks, layers=layers, pages=seqs * per + forks + rng.randint(0, 64),
                    max_len=max_len, page=page)
    pages = _log_int(rng, 16, 65536 // page)
    return dict(op=op, pages=pages, live=rng.randint(1, pages), layers=layers, seqs=rng.randint(1, 64), page=page)


def _layout_rng(case):
    """Sizes that belong to the case, the same for every seed."""
    return random.Random("|".join(f"{k}={case[k]}" for k in sorted(case) if k != "name"))


def _lens(case):
    r = _layout_rng(case)
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["B"])]
    lens[r.randrange(case["B"])] = case["max_len"]
    return lens


def _beam_layout(case):
    """Lengths of the live sequences, (parent, child) pairs and the sequences
    that end: children go to empty slots behind the live ones."""
    r = _layout_rng(case)
    live = case["seqs"] - min(case["forks"], case["seqs"] // 2)
    lens = [r.randint(1, case["max_len"]) for _ in range(live)]
    children = list(range(live, live + min(case["forks"], case["seqs"] - live)))
    parents = [r.randrange(live) for _ in children]
    ends = sorted(r.sample(range(live), max(1, live // 3)))
    return lens, parents, children, ends


def _live_pages(case):
    r = _layout_rng(case)
    return sorted(r.sample(range(case["pages"]), case["live"]))


def work(case):
    op, page = case["op"], case["page"]
    if op == "attend":
        rows = case["B"] * case["q_len"] * case["H"]
        lens = _lens(case)
        qb = DIM * (2 if case["q"] == "bf16" else 1)
        pages = sum(-(-n // page) for n in lens)
        visible = sum(max(0, n - i) for n in lens for i in range(case["q_len"]))
        return {"bytes": sum(lens) * TOKEN_BYTES + rows * (qb + 2 * LATENT + 4) + 4 * pages + 4 * case["B"],
                "flops": 2 * visible * case["H"] * (DIM + LATENT)}
    if op == "append":
        return {"bytes": case["T"] * 2 * (2 * DIM + TOKEN_BYTES + 4), "flops": 3 * case["T"] * LATENT}
    if op == "gather":
        return {"bytes": case["T"] * (2 * DIM + TOKEN_BYTES + 4), "flops": case["T"] * LATENT}
    if op == "beam":
        lens, parents, children, ends = _beam_layout(case)
        tails = sum(lens[p] % page for p in parents)
        held = sum(-(-lens[s] // page) for s in parents + ends)
        return {"bytes": 2 * tails * TOKEN_BYTES * case["layers"] + 16 * held, "flops": held}
    moved = sum(1 for p in _live_pages(case) if p >= case["live"])
    return {"bytes": 2 * moved * page * TOKEN_BYTES * case["layers"] + 8 * case["pages"] + 8 * case["live"],
            "flops": case["pages"]}


# ---------------------------------------------------------------------------
# The cache's layout and codes, in elementary operations
# ---------------------------------------------------------------------------

def _magnitudes(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def _quantise(lat):
    """[T,512] floats -> E2M1 codes [T,512] (sign 8, magnitude 0..7) and scale bytes [T,16]."""
    blk = lat.float().reshape(-1, NBLOCK, BLOCK)
    bits = blk.abs().amax(-1).contiguous().view(torch.int32)
    bad = (~torch.isfinite(blk)).any(-1)
    byte = torch.clamp(((bits + 0x1FFFFF) >> 23) - 2, SCALE_MIN, SCALE_MAX)
    y = blk * torch.exp2((127 - byte).float()).unsqueeze(-1)
    a = y.abs()
    mag = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
           + (a >= 3.5).int() + (a > 5.0).int())
    code = mag + 8 * torch.signbit(blk).int()
    code = torch.where(bad.unsqueeze(-1), torch.zeros_like(code), code)
    byte = torch.where(bad, torch.full_like(byte, SCALE_NAN), byte)
    return code.reshape(-1, LATENT), byte


def _pack_codes(code):
    """Codes [T,512] -> bytes [T,256].  A 32-bit word holds eight elements: the
    magnitude of element e in bits 4e..4e+2, the sign of e < 4 in bit 8e+7 and
    of e >= 4 in bit 8(e-4)+3.  Odd groups of four blocks hold each block's two
    8-byte halves in swapped order."""
    c = code.reshape(-1, NBLOCK, 4, 8).long()
    word = torch.zeros(c.shape[:-1], dtype=torch.int64, device=code.device)
    for e in range(8):
        word += (c[..., e] & 7) << (4 * e)
        word += (c[..., e] >> 3) << (8 * e + 7 if e < 4 else 8 * (e - 4) + 3)
    word = _swap_halves(word)
    out = torch.stack([(word >> (8 * i)) & 255 for i in range(4)], -1)
    return out.to(torch.uint8).reshape(-1, LATENT // 2)


def _swap_halves(word):
    w = word.clone()
    odd = [j for j in range(NBLOCK) if j & 4]
    w[:, odd] = word[:, odd][:, :, [2, 3, 0, 1]]
    return w


def _unpack_codes(raw):
    """Bytes [T,256] -> signed code values [T,512] in 32-bit floats."""
    b = raw.reshape(-1, NBLOCK, 4, 4).int()
    word = _swap_halves(b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16) | (b[..., 3] << 24))
    e = torch.arange(8, device=raw.device, dtype=torch.int32)
    sign_bit = torch.where(e < 4, 8 * e + 7, 8 * (e - 4) + 3)
    w = word.unsqueeze(-1)
    mag = _magnitudes(raw.device)[((w >> (4 * e)) & 7).long()]
    return torch.where(((w >> sign_bit) & 1) != 0, -mag, mag).reshape(-1, LATENT)


def _rope_chunks(pos):
    """Where the eight 16-byte chunks of a token's rope row lie in its 128 bytes."""
    return torch.arange(8, device=pos.device).unsqueeze(0) ^ (pos & 7).unsqueeze(1)


def _store(cache, page, slots, code, byte, rope):
    """Write tokens into one layer's pages [pages, 400*page]; negative slots are left out."""
    keep = slots >= 0
    slots, code, byte, rope = slots[keep], code[keep], byte[keep], rope[keep]
    pg, pos = slots // page, slots % page
    ar = torch.arange
    dev = cache.device
    cache[pg[:, None], (pos * 256)[:, None] + ar(256, device=dev)] = _pack_codes(code)
    r8 = rope.contiguous().view(torch.uint8).reshape(-1, 8, 16)
    at = 256 * page + (pos * 128)[:, None, None] + 16 * _rope_chunks(pos)[:, :, None] + ar(16, device=dev)
    cache[pg[:, None, None], at] = r8
    cache[pg[:, None], 384 * page + (pos * 16)[:, None] + ar(16, device=dev)] = byte.to(torch.uint8)


def _load(cache, page, slots):
    """Tokens at `slots` as 32-bit floats: latents [T,512], rope [T,64]."""
    pg, pos = slots // page, slots % page
    ar = torch.arange
    dev = cache.device
    code = cache[pg[:, None], (pos * 256)[:, None] + ar(256, device=dev)]
    at = 256 * page + (pos * 128)[:, None, None] + 16 * _rope_chunks(pos)[:, :, None] + ar(16, device=dev)
    rope = cache[pg[:, None, None], at].reshape(-1, 128).view(torch.bfloat16).float()
    byte = cache[pg[:, None], 384 * page + (pos * 16)[:, None] + ar(16, device=dev)].int()
    scale = torch.exp2((byte.clamp(SCALE_MIN, SCALE_MAX) - 127).float())
    scale = torch.where(byte == SCALE_NAN, torch.full_like(scale, float("nan")), scale)
    lat = _unpack_codes(code).reshape(-1, NBLOCK, BLOCK) * scale.unsqueeze(-1)
    return lat.reshape(-1, LATENT), rope


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(n, g):
    """Latents as a normalised down-projection leaves them (a spread of channel
    gains) and rotated keys, side by side as the projection writes them."""
    gain = torch.exp(0.4 * torch.randn(LATENT, generator=g, device="cuda"))
    lat = torch.randn(n, LATENT, generator=g, device="cuda") * gain
    rope = torch.randn(n, ROPE, generator=g, device="cuda")
    return torch.cat([lat, rope], 1).to(torch.bfloat16)


def _fill(cache, page, slots, g):
    for i in range(0, slots.numel(), 131072):
        s = slots[i:i + 131072]
        rows = _tokens(s.numel(), g)
        code, byte = _quantise(rows[:, :LATENT])
        _store(cache, page, s, code, byte, rows[:, LATENT:])


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


def prepare(case, seed):
    g = _gen(seed)
    return {"attend": _prepare_attend, "append": _prepare_rows, "gather": _prepare_rows, "beam": _prepare_beam,
            "compact": _prepare_compact}[case["op"]](case, g)


def _prepare_attend(case, g):
    B, q_len, H, page = case["B"], case["q_len"], case["H"], case["page"]
    M = B * q_len
    lens = _lens(case)
    table, pages, slots = _paged_slots(lens, page, g)
    cache = torch.full((pages, TOKEN_BYTES * page), 255, dtype=torch.uint8, device="cuda")
    _fill(cache, page, slots, g)
    q = torch.randn(M, H, DIM, generator=g, device="cuda")
    s = dict(case=case, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             host_lens=lens, q_scale=None)
    if case["q"] == "bf16":
        s["q"] = q.to(torch.bfloat16)
    else:
        s["q_scale"] = torch.tensor([0.02], device="cuda")
        s["q"] = (q / s["q_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
    if own:
        import mla_decode_query_gb300 as mq
        s["x"] = torch.empty(M, H, LATENT, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(M, H, dtype=torch.float32, device="cuda")
        n = mq.mlaqp_kv4_attend_workspace(B, q_len, H)
        s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return s


def _prepare_rows(case, g):
    T, page = case["T"], case["page"]
    _, pages, slots = _paged_slots([T], page, g)
    cache = torch.full((pages, TOKEN_BYTES * page), 255, dtype=torch.uint8, device="cuda")
    s = dict(case=case, cache=cache, slots=slots.int())
    if case["op"] == "gather":
        _fill(cache, page, slots, g)
    else:
        s["rows"] = _tokens(T, g)
    if own:
        s["out"] = torch.empty(T, DIM, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_beam(case, g):
    lens, parents, children, ends = _beam_layout(case)
    page, S = case["page"], case["seqs"]
    stride = -(-(case["max_len"] + 1) // page)
    num_pages = case["pages"]
    perm = torch.randperm(num_pages, generator=g, device="cuda").int()
    meta = torch.zeros(num_pages + S + S * stride, dtype=torch.int32, device="cuda")
    ref, slens, table = _split_meta(meta, num_pages, S, stride)
    table.fill_(-1)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = perm[at:at + k]
        slens[b] = n
        at += k
    ref[perm[:at].long()] = 1
    cache = torch.randint(0, 256, (case["layers"], num_pages, TOKEN_BYTES * page), generator=g, device="cuda",
                          dtype=torch.uint8)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=case, cache=cache, before=meta.clone(), meta=meta, stride=stride,
             parents=torch.tensor(parents, **i32), children=torch.tensor(children, **i32), ends=torch.tensor(ends, **i32),
             ones=torch.ones(len(children), **i32), slots=torch.empty(len(children), 1, **i32))
    if own:
        import mla_decode_query_gb300 as mq
        n = mq.mlaqp_kv4_pages_workspace(num_pages, max(len(children), 1))
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


def _prepare_compact(case, g):
    page, num_pages, S = case["page"], case["pages"], case["seqs"]
    live = _live_pages(case)
    stride = -(-len(live) // S) + 1
    meta = torch.zeros(num_pages + S + S * stride, dtype=torch.int32, device="cuda")
    ref, slens, table = _split_meta(meta, num_pages, S, stride)
    table.fill_(-1)
    order = torch.tensor(live, dtype=torch.int32, device="cuda")[torch.randperm(len(live), generator=g, device="cuda")]
    rows = torch.arange(len(live), device="cuda") % S
    cols = torch.arange(len(live), device="cuda") // S
    table[rows, cols] = order
    ref[order.long()] = 1
    slens += torch.bincount(rows, minlength=S).int() * page
    cache = torch.randint(0, 256, (case["layers"], num_pages, TOKEN_BYTES * page), generator=g, device="cuda",
                          dtype=torch.uint8)
    s = dict(case=case, cache=cache, before=meta.clone(), meta=meta, stride=stride)
    if own:
        import mla_decode_query_gb300 as mq
        s["ws"] = torch.empty(mq.mlaqp_kv4_pages_workspace(num_pages, 1), dtype=torch.uint8, device="cuda")
        s["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return s


def _split_meta(meta, num_pages, S, stride):
    return meta[:num_pages], meta[num_pages:num_pages + S], meta[num_pages + S:].view(S, stride)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    table = _OWN if own else _PLAIN
    return table[op](state)


def _attend_plain(s):
    case = s["case"]
    B, q_len, H, page = case["B"], case["q_len"], case["H"], case["page"]
    q = s["q"].float()
    if s["q_scale"] is not None:
        q = q * s["q_scale"]
    q = q.reshape(B, q_len * H, DIM)
    x = torch.zeros(B, q_len * H, LATENT, device=q.device)
    lse = torch.full((B, q_len * H), float("-inf"), device=q.device)
    for b, n in enumerate(s["host_lens"]):
        if n <= 0:
            continue
        t = torch.arange(n, device=q.device)
        lat, rope = _load(s["cache"], page, s["table"][b].long()[t // page] * page + t % page)
        sc = (q[b, :, :LATENT] @ lat.T + q[b, :, LATENT:] @ rope.T) * SOFTMAX_SCALE
        seen = n - (q_len - 1 - torch.arange(q_len, device=q.device)).repeat_interleave(H)
        sc = torch.where(t[None, :] < seen[:, None], sc, torch.full_like(sc, float("-inf")))
        top = sc.amax(1, keepdim=True)
        top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
        p = torch.exp(sc - top)
        total = p.sum(1, keepdim=True)
        x[b] = torch.where(total > 0, (p @ lat) / total, torch.zeros_like(x[b])) if q_len > 1 else (p @ lat) / total
        lse[b] = (top + torch.log(total)).squeeze(1)
    return {"x": x.reshape(B * q_len, H, LATENT).to(torch.bfloat16), "lse": lse.reshape(B * q_len, H)}


def _attend_own(s):
    import mla_decode_query_gb300 as mq
    case, q, cache, table = s["case"], s["q"], s["cache"], s["table"]
    mq.check(mq.mlaqp_kv4_attend(
        q, case["H"] * DIM, case["q"], s["q_scale"], cache, cache.stride(0), cache.shape[0], case["page"], table,
        table.stride(0), table.shape[0], s["lens"], None, case["B"], case["q_len"], case["H"], SOFTMAX_SCALE, s["x"],
        case["H"] * LATENT, s["lse"], s["ws"], s["ws"].numel()))
    return {"x": s["x"], "lse": s["lse"]}


def _append_plain(s):
    page = s["case"]["page"]
    slots = s["slots"].long()
    code, byte = _quantise(s["rows"][:, :LATENT])
    _store(s["cache"], page, slots, code, byte, s["rows"][:, LATENT:])
    return _gather_plain(s)


def _gather_plain(s):
    lat, rope = _load(s["cache"], s["case"]["page"], s["slots"].long())
    return {"rows": torch.cat([lat, rope], 1).to(torch.bfloat16)}


def _append_own(s):
    import mla_decode_query_gb300 as mq
    rows, cache, page = s["rows"], s["cache"], s["case"]["page"]
    mq.check(mq.mlaqp_kv4_append(rows, DIM, rows[:, LATENT:], DIM, cache, cache.stride(0), cache.shape[0], page,
                                 s["slots"], s["case"]["T"]))
    return _gather_own(s)


def _gather_own(s):
    import mla_decode_query_gb300 as mq
    cache, page = s["cache"], s["case"]["page"]
    mq.check(mq.mlaqp_kv4_gather(cache, cache.stride(0), cache.shape[0], page, s["slots"], s["case"]["T"], s["out"],
                                 DIM))
    return {"rows": s["out"]}


def _beam_outputs(s, ref, lens, table):
    return {"ref_count": ref, "lens": lens, "table": table, "slots": s["slots"], "cache": s["cache"]}


def _beam_plain(s):
    case = s["case"]
    page, cache = case["page"], s["cache"]
    s["meta"].copy_(s["before"])
    ref, lens, table = _split_meta(s["meta"], case["pages"], case["seqs"], s["stride"])
    par, chi, ends = s["parents"].long(), s["children"].long(), s["ends"].long()
    cols = torch.arange(s["stride"], device=cache.device)
    # fork: share the full pages, copy the tokens of a partly filled last page into a new one
    plen = lens[par]
    full, tail = plen // page, plen % page
    rows = torch.where(cols < full[:, None], table[par], torch.full_like(table[par], -1))
    shared = rows[rows >= 0].long()
    has = (tail > 0).nonzero().squeeze(1)
    fresh = (ref == 0).nonzero().squeeze(1)[:has.numel()]
    src = table[par[has], full[has].long()].long()
    rows[has, full[has].long()] = fresh.int()
    ref.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    ref[fresh] = 1
    table[chi] = rows
    lens[chi] = plen
    at = torch.arange(TOKEN_BYTES * page, device=cache.device)
    pos = torch.where(at < 256 * page, at // 256,
                      torch.where(at < 384 * page, (at - 256 * page) // 128, (at - 384 * page) // 16))
    cache[:, fresh] = torch.where(pos < tail[has][:, None], cache[:, src], cache[:, fresh])
    # release the sequences that end
    gone = table[ends]
    gone = gone[gone >= 0].long()
    ref.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[ends] = -1
    lens[ends] = 0
    # extend the children by one token
    clen = lens[chi]
    new = (clen % page == 0).nonzero().squeeze(1)
    fresh = (ref == 0).nonzero().squeeze(1)[:new.numel()]
    ref[fresh] = 1
    table[chi[new], (clen[new] // page).long()] = fresh.int()
    s["slots"][:, 0] = table[chi, (clen // page).long()] * page + clen % page
    lens[chi] = clen + 1
    return _beam_outputs(s, ref, lens, table)


def _beam_own(s):
    import mla_decode_query_gb300 as mq
    case, cache, ws = s["case"], s["cache"], s["ws"]
    s["meta"].copy_(s["before"])
    ref, lens, table = _split_meta(s["meta"], case["pages"], case["seqs"], s["stride"])
    n, S, P = s["children"].numel(), case["seqs"], case["pages"]
    mq.check(mq.mlaqp_kv4_fork(table, s["stride"], S, lens, ref, P, case["page"], s["parents"], s["children"], n, cache,
                               cache.stride(1), cache.stride(0), case["layers"], ws, ws.numel()))
    mq.check(mq.mlaqp_kv4_release(table, s["stride"], S, lens, ref, P, case["page"], s["ends"], s["ends"].numel()))
    mq.check(mq.mlaqp_kv4_extend(table, s["stride"], S, lens, ref, P, case["page"], s["children"], s["ones"], n,
                                 s["slots"], 1))
    return _beam_outputs(s, ref, lens, table)


def _compact_plain(s):
    case, cache = s["case"], s["cache"]
    s["meta"].copy_(s["before"])
    ref, lens, table = _split_meta(s["meta"], case["pages"], case["seqs"], s["stride"])
    live = ref > 0
    n = live.sum()
    idx = torch.arange(case["pages"], device=cache.device)
    dst = (~live & (idx < n)).nonzero().squeeze(1)
    src = (live & (idx >= n)).nonzero().squeeze(1)
    cache[:, dst] = cache[:, src]
    remap = idx.clone()
    remap[src] = dst
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()].int(), table))
    ref[dst] = ref[src]
    ref[src] = 0
    return {"ref_count": ref, "table": table, "n_live": n.int().reshape(1), "cache": cache}


def _compact_own(s):
    import mla_decode_query_gb300 as mq
    case, cache, ws = s["case"], s["cache"], s["ws"]
    s["meta"].copy_(s["before"])
    ref, lens, table = _split_meta(s["meta"], case["pages"], case["seqs"], s["stride"])
    mq.check(mq.mlaqp_kv4_compact(table, s["stride"], case["seqs"], lens, ref, case["pages"], case["page"], cache,
                                  cache.stride(1), cache.stride(0), case["layers"], s["n_live"], ws, ws.numel()))
    return {"ref_count": ref, "table": table, "n_live": s["n_live"], "cache": cache}


_PLAIN = dict(attend=_attend_plain, append=_append_plain, gather=_gather_plain, beam=_beam_plain,
              compact=_compact_plain)
_OWN = dict(attend=_attend_own, append=_append_own, gather=_gather_own, beam=_beam_own, compact=_compact_own)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(s, slots):
    """Cached rows [T,576] in 64 bits, read byte by byte from the format."""
    page = s["case"]["page"]
    rows = s["cache"][slots // page]
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
    v = v * (1.0 - 2.0 * sign) * torch.exp2(byte.clamp(SCALE_MIN, SCALE_MAX) - 127.0)
    v = torch.where(byte == SCALE_NAN, torch.full_like(v, float("nan")), v)
    c = torch.arange(ROPE, device=rows.device)
    at = 256 * page + (pos * 128)[:, None] + 16 * ((c // 8) ^ (pos & 7)[:, None]) + 2 * (c % 8)
    bits = (torch.gather(rows, 1, at).int() | (torch.gather(rows, 1, at + 1).int() << 8)) << 16
    return torch.cat([v, bits.view(torch.float32).double()], 1)


def _exact_quantised(rows):
    """Rows as the cache stands for them: each block of 32 on the grid of its scale."""
    lat = rows[:, :LATENT].double().reshape(-1, NBLOCK, BLOCK)
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
    return torch.cat([v.reshape(-1, LATENT), rows[:, LATENT:].double()], 1)


def exact(case, seed):
    op = case["op"]
    if op in ("beam", "compact"):
        return None  # whole numbers and copied bytes
    s = prepare(case, seed)
    if op == "append":
        return {"rows": _exact_quantised(s["rows"])}
    page = case["page"]
    if op == "gather":
        slots = s["slots"].long()
        return {"rows": torch.cat([_exact_rows(s, slots[i:i + 8192]) for i in range(0, slots.numel(), 8192)])}
    B, q_len, H = case["B"], case["q_len"], case["H"]
    q = s["q"].double() if s["q_scale"] is None else s["q"].float().double() * s["q_scale"].double()
    q = q.reshape(B, q_len, H, DIM)
    x = torch.zeros(B, q_len, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, q_len, H), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["host_lens"]):
        t = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[t // page] * page + t % page
        k = torch.cat([_exact_rows(s, slots[i:i + 8192]) for i in range(0, n, 8192)])
        for i in range(q_len):
            seen = n - (q_len - 1 - i)
            if seen <= 0:
                continue
            sc = q[b, i] @ k[:seen].T * SOFTMAX_SCALE
            lse[b, i] = torch.logsumexp(sc, 1)
            x[b, i] = torch.exp(sc - lse[b, i][:, None]) @ k[:seen, :LATENT]
    return {"x": x.reshape(B * q_len, H, LATENT), "lse": lse.reshape(B * q_len, H)}
