"""Refusals of append_rope, digest and select: every check that needs no device
returns its status before any CUDA call (no GPU needed)."""

import pytest

import mla_decode_query_gb300 as mq

A = 1 << 24  # fake, aligned device addresses, never dereferenced
INVALID, UNSUPPORTED = mq.MLAQP_ERR_INVALID_ARG, mq.MLAQP_ERR_UNSUPPORTED
NO_DEVICE = (mq.MLAQP_ERR_CUDA, UNSUPPORTED)  # what a call that passes every check gets here


def _rope(**kw):
    a = dict(latent=A, latent_token_stride=576, norm_weight=2 * A, norm_eps=1e-6, k_pe=A + 1024, k_pe_token_stride=576,
             q_pe=3 * A, q_token_stride=1024, q_head_stride=64, q_pe_out=4 * A, q_out_token_stride=1024,
             q_out_head_stride=64, H=16, positions=5 * A, cos_sin=6 * A, num_positions=4096, rope_style="interleaved",
             cache=8 * A, page_stride=25600, num_pages=16, page_size=64, slots=7 * A, T=3, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_append_rope(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=48), UNSUPPORTED),
    (dict(num_pages=0), INVALID),
    (dict(cache=None), INVALID),
    (dict(page_stride=25584), INVALID),
    (dict(rope_style=2), INVALID),
    (dict(H=-1), INVALID),
    (dict(H=129), UNSUPPORTED),
    (dict(T=-1), INVALID),
    (dict(num_positions=0), INVALID),
    (dict(latent=None), INVALID),
    (dict(k_pe=None), INVALID),
    (dict(positions=None), INVALID),
    (dict(cos_sin=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(latent=A + 8), INVALID),
    (dict(norm_weight=2 * A + 2), INVALID),
    (dict(cos_sin=6 * A + 4), INVALID),
    (dict(positions=5 * A + 2), INVALID),
    (dict(latent_token_stride=580), INVALID),
    (dict(k_pe_token_stride=-8), INVALID),
    (dict(norm_eps=-1e-6), INVALID),
    (dict(norm_eps=float("nan")), INVALID),
    (dict(norm_eps=float("inf")), INVALID),
    (dict(q_pe=None), INVALID),
    (dict(q_pe_out=None), INVALID),
    (dict(H=0), INVALID),                                # queries without heads
    (dict(q_pe=3 * A + 8), INVALID),
    (dict(q_pe_out=4 * A + 8), INVALID),
    (dict(q_token_stride=1028), INVALID),
    (dict(q_head_stride=-64), INVALID),
    (dict(q_out_head_stride=56), INVALID),
    (dict(q_out_token_stride=1016), INVALID),            # rows of 16 heads overlap
    (dict(q_pe_out=3 * A + 16), INVALID),                # overlaps q_pe, not the same view
    (dict(q_pe_out=3 * A, q_out_token_stride=2048), INVALID),
    (dict(q_pe_out=A), INVALID),                         # overlaps the latents
    (dict(q_pe_out=2 * A), INVALID),                     # the norm's weight
    (dict(q_pe_out=6 * A + 1024 * 1023), INVALID),       # the angles
    (dict(q_pe_out=8 * A), INVALID),                     # the cache
    (dict(q_pe=8 * A + 64), INVALID),
    (dict(slots=8 * A), INVALID),
    (dict(latent=8 * A), INVALID),
    (dict(cos_sin=8 * A - 4096), INVALID),
])
def test_append_rope_refusals(built_library, kw, code):
    assert _rope(**kw) == code
    assert mq.mlaqp_last_error() != ""


ROW = 16 * 192 + 576  # one projection output: 16 heads of 128 + 64, then latent and key part


@pytest.mark.parametrize("kw", [
    dict(),
    dict(q_pe_out=3 * A),                                              # in place
    dict(q_pe=None, q_pe_out=None, H=0),
    dict(norm_weight=None, norm_eps=float("nan")),                     # not used
    dict(T=1, q_out_token_stride=0, q_token_stride=0),
    dict(H=1, q_out_head_stride=0, q_out_token_stride=64),
    # everything a view into one buffer, the queries' parts rotated in place beside the latents
    dict(latent=A + 2 * 16 * 192, latent_token_stride=ROW, k_pe=A + 2 * (16 * 192 + 512), k_pe_token_stride=ROW,
         q_pe=A + 256, q_pe_out=A + 256, q_token_stride=ROW, q_out_token_stride=ROW, q_head_stride=192,
         q_out_head_stride=192),
])
def test_append_rope_passes_the_checks(built_library, kw):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert _rope(**kw) in NO_DEVICE


def test_views_into_one_buffer_that_do_share_bytes_are_refused(built_library):
    v = dict(latent_token_stride=ROW, k_pe_token_stride=ROW, k_pe=2 * A, q_token_stride=ROW, q_out_token_stride=ROW,
             q_head_stride=192, q_out_head_stride=192, q_pe=3 * A, norm_weight=None)
    for first in (256, 256 + 2 * ROW):      # the first token's row, or the second's
        for off in (0, 2 * (15 * 192 + 64) - 16, -1008):
            assert _rope(**v, q_pe_out=A + first, latent=A + 256 + off) == INVALID, (first, off)


def test_no_tokens_is_no_launch(built_library):
    assert _rope(T=0, latent=None, slots=None) == mq.MLAQP_OK


def _digest(**kw):
    a = dict(cache=8 * A, page_stride=6400, num_pages=64, page_size=16, block_table=A, block_table_stride=4, num_seqs=3,
             seq_lens=2 * A, seqs=3 * A, new_tokens=4 * A, n=2, max_new=5, digests=16 * A, digest_stride=1168, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_digest(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=8), UNSUPPORTED),
    (dict(num_pages=(1 << 20) + 1), UNSUPPORTED),
    (dict(cache=8 * A + 8), INVALID),
    (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID),
    (dict(block_table=A + 2), INVALID),
    (dict(block_table_stride=0), INVALID),
    (dict(num_seqs=0), INVALID),
    (dict(digests=None), INVALID),
    (dict(digests=16 * A + 8), INVALID),
    (dict(digest_stride=1152), INVALID),
    (dict(digest_stride=1176), INVALID),
    (dict(n=-1), INVALID),
    (dict(seqs=None), INVALID),
    (dict(new_tokens=4 * A + 1), INVALID),
    (dict(max_new=0), INVALID),
    (dict(digests=8 * A), INVALID),      # overlaps the cache
    (dict(digests=A - 1168 * 63), INVALID),
])
def test_digest_refusals(built_library, kw, code):
    assert _digest(**kw) == code
    assert mq.mlaqp_last_error() != ""


def test_digest_of_nothing_is_no_launch(built_library):
    assert _digest(n=0, seqs=None, new_tokens=None) == mq.MLAQP_OK


def _select(**kw):
    a = dict(q=A, q_token_stride=576 * 16, q_dtype="bf16", digests=16 * A, digest_stride=1168, num_pages=64, page_size=16,
             block_table=2 * A, block_table_stride=8, num_seqs=3, seq_lens=3 * A, seqs=None, B=3, q_len=1, H=16, k=4, first=1,
             last=1, sel_table=4 * A, sel_stride=4, sel_lens=5 * A, workspace=6 * A, workspace_bytes=96, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_select(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q_dtype=7), INVALID),
    (dict(H=0), UNSUPPORTED),
    (dict(H=17), UNSUPPORTED),
    (dict(q_len=0), UNSUPPORTED),
    (dict(q_len=17), UNSUPPORTED),
    (dict(B=-1), INVALID),
    (dict(B=257), UNSUPPORTED),
    (dict(B=1 << 30, q_len=16), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED),
    (dict(num_pages=0), INVALID),
    (dict(digests=None), INVALID),
    (dict(digest_stride=1160), INVALID),
    (dict(k=0), INVALID),
    (dict(k=(1 << 20) + 1, sel_stride=1 << 21), UNSUPPORTED),
    (dict(first=-1), INVALID),
    (dict(last=0), INVALID),
    (dict(first=2, last=3), INVALID),
    (dict(first=(1 << 31) - 1, last=(1 << 31) - 1), INVALID),
    (dict(sel_stride=3), INVALID),
    (dict(q=None), INVALID),
    (dict(sel_table=None), INVALID),
    (dict(sel_lens=None), INVALID),
    (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID),
    (dict(q=A + 8), INVALID),
    (dict(sel_table=4 * A + 2), INVALID),
    (dict(q_token_stride=576 * 16 - 8), INVALID),
    (dict(q_token_stride=576 * 16 + 4), INVALID),
    (dict(q_dtype="e4m3", q_token_stride=576 * 16 + 8), INVALID),
    (dict(num_seqs=2), INVALID),
    (dict(workspace=None), INVALID),
    (dict(workspace=6 * A + 8), INVALID),
    (dict(workspace_bytes=95), INVALID),
    (dict(sel_table=A), INVALID),             # overlaps q
    (dict(sel_lens=4 * A + 16), INVALID),     # overlaps sel_table
    (dict(workspace=16 * A), INVALID),        # overlaps the digests
    (dict(sel_table=2 * A), INVALID),         # the table it reads
])
def test_select_refusals(built_library, kw, code):
    assert _select(**kw) == code
    assert mq.mlaqp_last_error() != ""


def test_select_of_nothing_is_no_launch(built_library):
    assert _select(B=0, q=None, sel_table=None, workspace=None) == mq.MLAQP_OK


def test_select_workspace(built_library):
    assert mq.mlaqp_kv4_select_workspace(3, 1, 8, 64) == 96
    assert mq.mlaqp_kv4_select_workspace(16, 16, 1 << 31, 1 << 20) == 1 << 30
    assert mq.mlaqp_kv4_select_workspace(1, 3, 5, 64) == 64  # 60, whole 16 bytes
    for bad in ((-1, 1, 8, 64), (257, 1, 8, 64), (1, 17, 8, 64), (1, 1, 0, 64), (1, 1, 8, 0), (1, 1, 8, (1 << 20) + 1)):
        assert mq.mlaqp_kv4_select_workspace(*bad) == -1
        assert mq.mlaqp_last_error() != ""
