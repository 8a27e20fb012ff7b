"""Refusals of the 4-bit cache's entry points: every check that needs no
device returns its status before any CUDA call (no GPU needed)."""

import pytest

import mla_decode_query_gb300 as mq

A = 1 << 24  # fake, aligned device addresses, never dereferenced
INVALID, UNSUPPORTED = mq.MLAQP_ERR_INVALID_ARG, mq.MLAQP_ERR_UNSUPPORTED


def test_page_bytes(built_library):
    assert [mq.mlaqp_kv4_page_bytes(p) for p in (16, 32, 64, 128)] == [6400, 12800, 25600, 51200]
    assert mq.mlaqp_kv4_page_bytes(48) == 0 and mq.mlaqp_kv4_page_bytes(0) == 0


def _append(**kw):
    a = dict(latent=A, latent_token_stride=576, k_pe=A + 1024, k_pe_token_stride=576, cache=8 * A, page_stride=25600,
             num_pages=16, page_size=64, slots=4 * A, T=3, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_append(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=256), UNSUPPORTED),
    (dict(num_pages=0), INVALID),
    (dict(num_pages=(1 << 20) + 1), UNSUPPORTED),
    (dict(cache=None), INVALID),
    (dict(cache=8 * A + 8), INVALID),
    (dict(page_stride=25584), INVALID),
    (dict(page_stride=25608), INVALID),
    (dict(T=-1), INVALID),
    (dict(latent=None), INVALID),
    (dict(k_pe=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(slots=4 * A + 2), INVALID),
    (dict(latent=A + 8), INVALID),
    (dict(k_pe=A + 1026), INVALID),
    (dict(latent_token_stride=580), INVALID),
    (dict(k_pe_token_stride=-64), INVALID),
    (dict(latent=8 * A + 1024), INVALID),   # inside the cache
    (dict(slots=8 * A + 16), INVALID),
])
def test_append_refusals(built_library, kw, code):
    assert _append(**kw) == code
    assert mq.mlaqp_last_error() != ""


def _gather(**kw):
    a = dict(cache=8 * A, page_stride=6400, num_pages=16, page_size=16, slots=4 * A, T=3, out=A, out_token_stride=576,
             stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_gather(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=8), UNSUPPORTED),
    (dict(T=-2), INVALID),
    (dict(out=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(out=A + 4), INVALID),
    (dict(out_token_stride=568), INVALID),
    (dict(out_token_stride=580), INVALID),
    (dict(out=8 * A), INVALID),
    (dict(out=4 * A), INVALID),
])
def test_gather_refusals(built_library, kw, code):
    assert _gather(**kw) == code
    assert mq.mlaqp_last_error() != ""


def _attend(**kw):
    a = dict(q=A, q_token_stride=576 * 16, q_dtype="bf16", q_scale=None, cache=8 * A, page_stride=25600, num_pages=16,
             page_size=64, block_table=4 * A, block_table_stride=4, num_seqs=3, seq_lens=5 * A, seqs=None, B=3, q_len=1,
             H=16, softmax_scale=0.07, x=2 * A, x_token_stride=512 * 16, lse=3 * A, workspace=16 * A,
             workspace_bytes=1 << 26, stream=0)
    a.update(kw)
    return mq.mlaqp_kv4_attend(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q_dtype=5), INVALID),
    (dict(H=0), UNSUPPORTED),
    (dict(H=17), UNSUPPORTED),
    (dict(q_len=0), UNSUPPORTED),
    (dict(q_len=17), UNSUPPORTED),
    (dict(B=-1), INVALID),
    (dict(B=129, q_len=2), UNSUPPORTED),
    (dict(B=1 << 30, q_len=16), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED),
    (dict(cache=None), INVALID),
    (dict(q=None), INVALID),
    (dict(x=None), INVALID),
    (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID),
    (dict(q_scale=6 * A), INVALID),                    # BF16 takes none
    (dict(q_dtype="e4m3"), INVALID),                   # E4M3 needs one
    (dict(q=A + 8), INVALID),
    (dict(x=2 * A + 8), INVALID),
    (dict(lse=3 * A + 2), INVALID),
    (dict(block_table=4 * A + 1), INVALID),
    (dict(q_token_stride=576 * 16 - 8), INVALID),
    (dict(q_token_stride=576 * 16 + 4), INVALID),      # 8 bytes
    (dict(q_dtype="e4m3", q_scale=6 * A, q_token_stride=576 * 16 + 8), INVALID),
    (dict(x_token_stride=512 * 16 - 8), INVALID),
    (dict(x_token_stride=512 * 16 + 4), INVALID),
    (dict(num_seqs=0), INVALID),
    (dict(num_seqs=2), INVALID),                       # fewer rows than sequences
    (dict(block_table_stride=0), INVALID),
    (dict(softmax_scale=0.0), INVALID),
    (dict(softmax_scale=-1.0), INVALID),
    (dict(softmax_scale=float("nan")), INVALID),
    (dict(softmax_scale=float("inf")), INVALID),
    (dict(x=A + 1024), INVALID),                       # overlaps q
    (dict(lse=2 * A + 64), INVALID),                   # overlaps x
    (dict(workspace=8 * A + 64), INVALID),             # overlaps the cache
])
def test_attend_refusals(built_library, kw, code):
    assert _attend(**kw) == code
    assert mq.mlaqp_last_error() != ""


def _tables(**kw):
    a = dict(block_table=A, block_table_stride=8, num_seqs=4, seq_lens=2 * A, ref_count=3 * A, num_pages=64,
             page_size=16)
    a.update(kw)
    return a


TABLE_CASES = [
    (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID),
    (dict(ref_count=None), INVALID),
    (dict(ref_count=3 * A + 1), INVALID),
    (dict(block_table_stride=0), INVALID),
    (dict(num_seqs=0), INVALID),
    (dict(num_pages=0), INVALID),
    (dict(num_pages=(1 << 20) + 1), UNSUPPORTED),
    (dict(page_size=17), UNSUPPORTED),
    (dict(n=-1), INVALID),
]


@pytest.mark.parametrize("kw,code", TABLE_CASES + [
    (dict(seqs=None), INVALID), (dict(new_tokens=None), INVALID), (dict(max_new=0), INVALID), (dict(slots=None), INVALID),
])
def test_extend_refusals(built_library, kw, code):
    a = dict(_tables(), seqs=4 * A, new_tokens=5 * A, n=2, slots=6 * A, max_new=4, stream=0)
    a.update(kw)
    assert mq.mlaqp_kv4_extend(**a) == code
    assert mq.mlaqp_last_error() != ""


POOL = dict(cache=8 * A, page_stride=6400, layer_stride=6400 * 64, layers=3)
POOL_CASES = [
    (dict(cache=None), INVALID),
    (dict(cache=8 * A + 4), INVALID),
    (dict(page_stride=6384), INVALID),
    (dict(layers=0), INVALID),
    (dict(layer_stride=6400 * 64 - 16), INVALID),     # layers run into each other
    (dict(layer_stride=6400 * 64 + 8), INVALID),
    (dict(layer_stride=-16), INVALID),
]


@pytest.mark.parametrize("kw,code", TABLE_CASES + POOL_CASES + [
    (dict(parents=None), INVALID), (dict(children=5 * A + 2), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace=7 * A + 8), INVALID), (dict(workspace_bytes=16), INVALID),
])
def test_fork_refusals(built_library, kw, code):
    a = dict(_tables(), parents=4 * A, children=5 * A, n=2, **POOL, workspace=7 * A, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    assert mq.mlaqp_kv4_fork(**a) == code
    assert mq.mlaqp_last_error() != ""


@pytest.mark.parametrize("kw,code", TABLE_CASES + [(dict(seqs=None), INVALID)])
def test_release_refusals(built_library, kw, code):
    a = dict(_tables(), seqs=4 * A, n=2, stream=0)
    a.update(kw)
    assert mq.mlaqp_kv4_release(**a) == code


@pytest.mark.parametrize("kw,code", TABLE_CASES[:-1] + POOL_CASES + [
    (dict(n_live=None), INVALID), (dict(workspace=None), INVALID), (dict(workspace_bytes=64), INVALID),
])
def test_compact_refusals(built_library, kw, code):
    a = dict(_tables(), **POOL, n_live=6 * A, workspace=7 * A, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    assert mq.mlaqp_kv4_compact(**a) == code


@pytest.mark.parametrize("kw,code", POOL_CASES + [
    (dict(num_pages=0), INVALID), (dict(page_size=20), UNSUPPORTED), (dict(n=-1), INVALID), (dict(src=None), INVALID),
    (dict(dst=None), INVALID),
])
def test_copy_pages_refusals(built_library, kw, code):
    a = dict(POOL, num_pages=64, page_size=16, src=A, dst=2 * A, n=2, stream=0)
    a.update(kw)
    assert mq.mlaqp_kv4_copy_pages(**a) == code


def test_empty_calls_launch_nothing(built_library):
    assert _append(T=0, latent=None, slots=None) == mq.MLAQP_OK
    assert _gather(T=0, out=None) == mq.MLAQP_OK
    assert _attend(B=0, q=None, x=None) == mq.MLAQP_OK
    assert mq.mlaqp_kv4_release(**_tables(), seqs=None, n=0, stream=0) == mq.MLAQP_OK
    assert mq.mlaqp_kv4_copy_pages(**POOL, num_pages=64, page_size=16, src=None, dst=None, n=0, stream=0) == mq.MLAQP_OK


def test_workspace_domains(built_library):
    assert mq.mlaqp_kv4_pages_workspace(0, 1) == -1 and mq.mlaqp_kv4_pages_workspace(64, -1) == -1
    assert mq.mlaqp_kv4_pages_workspace(64, 4) >= 16
    assert mq.mlaqp_kv4_attend_workspace(1, 1, 17) == -1 and mq.mlaqp_kv4_attend_workspace(300, 1, 16) == -1


def test_interleaved_layers_are_accepted(built_library):
    # layer l of page p at p*page_stride + l*6400: the call passes every host
    # check; without a GPU it stops at the device query
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    a = dict(POOL, page_stride=3 * 6400, layer_stride=6400)
    assert mq.mlaqp_kv4_copy_pages(**a, num_pages=64, page_size=16, src=A, dst=2 * A, n=2, stream=0) == mq.MLAQP_ERR_CUDA


@pytest.mark.parametrize("limit,held", [(0, 0), (10 ** 9 + 1, 0), (1000, -1), (1000, 14)])
def test_bounded_wait_hook_refusals(built_library, limit, held):
    a = dict(q=A, q_token_stride=576 * 16, q_dtype="bf16", q_scale=None, cache=8 * A, page_stride=25600, num_pages=16,
             page_size=64, block_table=4 * A, block_table_stride=4, num_seqs=3, seq_lens=5 * A, seqs=None, B=3, q_len=1,
             H=16, softmax_scale=0.07, x=2 * A, x_token_stride=512 * 16, lse=3 * A, workspace=16 * A,
             workspace_bytes=1 << 26, stream=0)
    assert mq.mlaqp_debug_kv4_attend_bounded_wait(**a, wait_limit_ns=limit, held=held) == INVALID
    assert mq.mlaqp_last_error() != ""
