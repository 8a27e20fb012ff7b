"""What select and digest write may not lie over a row of the block table that they
read, the last one included (no GPU needed)."""

import pytest

import mla_decode_query_gb300 as mq

A = 1 << 24  # fake, aligned device addresses, never dereferenced
INVALID = mq.MLAQP_ERR_INVALID_ARG
NO_DEVICE = (mq.MLAQP_ERR_CUDA, mq.MLAQP_ERR_UNSUPPORTED)  # what a call that passes every check gets here
WIDTH = 12  # entries of a row


def _select(**kw):
    a = dict(q=A, q_token_stride=576 * 16, q_dtype="bf16", digests=16 * A, digest_stride=1168, num_pages=64, page_size=16,
             block_table=2 * A, block_table_stride=WIDTH, num_seqs=1, seq_lens=3 * A, seqs=None, B=1, q_len=1, H=16, k=4, first=1,
             last=1, sel_table=4 * A, sel_stride=4, sel_lens=5 * A, workspace=6 * A, workspace_bytes=48, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_select(**a)


def _digest(**kw):
    a = dict(cache=8 * A, page_stride=6400, num_pages=64, page_size=16, block_table=2 * A, block_table_stride=WIDTH, num_seqs=1,
             seq_lens=3 * A, seqs=4 * A, new_tokens=5 * A, n=1, max_new=5, digests=16 * A, digest_stride=1168, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_digest(**a)


@pytest.mark.parametrize("num_seqs", [1, 3])
@pytest.mark.parametrize("name,entry", [(name, entry) for name in ("sel_table", "sel_lens") for entry in (1, WIDTH - 1)]
                         + [("workspace", WIDTH - 4)])
def test_select_refuses_outputs_in_the_last_row(built_library, num_seqs, name, entry):
    at = 2 * A + 4 * (WIDTH * (num_seqs - 1) + entry)
    assert _select(num_seqs=num_seqs, **{name: at}) == INVALID
    assert "overlaps an input" in mq.mlaqp_last_error()


@pytest.mark.parametrize("num_seqs", [1, 3])
def test_digest_refuses_digests_in_the_last_row(built_library, num_seqs):
    for entry in (4, WIDTH - 1):  # of the last row, where the digests begin
        assert _digest(num_seqs=num_seqs, block_table=2 * A - 4 * (WIDTH * (num_seqs - 1) + entry), digests=2 * A) == INVALID
    assert "overlap an input" in mq.mlaqp_last_error()


def test_behind_the_last_row_is_free(built_library):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert _select(sel_table=2 * A + 4 * WIDTH) in NO_DEVICE
    # a sequence has no more pages than there are: entries beyond are not read, however wide the row
    assert _select(num_pages=8, block_table_stride=1 << 20, sel_table=2 * A + 4 * 8) in NO_DEVICE
    assert _digest(num_pages=8, block_table_stride=1 << 20, digests=2 * A + 4 * 8) in NO_DEVICE


def _attend(**kw):
    a = dict(q=A, q_token_stride=576 * 16, q_dtype="bf16", q_scale=None, cache=8 * A, page_stride=6400, num_pages=64, page_size=16,
             block_table=2 * A, block_table_stride=WIDTH, num_seqs=1, seq_lens=3 * A, seqs=None, B=1, q_len=1, H=16, softmax_scale=0.07,
             x=4 * A, x_token_stride=512 * 16, lse=5 * A, workspace=32 * A, workspace_bytes=1 << 24, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_attend(**a)


@pytest.mark.parametrize("num_seqs", [1, 3])
@pytest.mark.parametrize("name,entry", [("x", 4), ("x", WIDTH - 4), ("lse", 1), ("lse", WIDTH - 1), ("workspace", 4)])
def test_attend_refuses_outputs_in_the_last_row(built_library, num_seqs, name, entry):
    at = 2 * A + 4 * (WIDTH * (num_seqs - 1) + entry)
    assert _attend(num_seqs=num_seqs, **{name: at}) == INVALID
    assert "overlaps an input" in mq.mlaqp_last_error()


def test_attend_may_write_behind_the_last_row(built_library):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert _attend(x=2 * A + 4 * WIDTH) in NO_DEVICE
    assert _attend(num_pages=8, block_table_stride=1 << 20, x=2 * A + 4 * 8) in NO_DEVICE
