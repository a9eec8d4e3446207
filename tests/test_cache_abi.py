"""The page plan, the norms with the rotation and the 8-bit cache without a GPU: bad
arguments are refused before the device is touched."""
import pytest
import torch

import prefill_kda_chunk_gb300 as K
from prefill_kda_chunk_gb300 import build as B

A = 1 << 20  # an aligned fake address; validation fails before any dereference
M = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return K.lib()


def plan(**kw):
    args = dict(page_table=A, seq_lens=A + M, new_lens=A + 2 * M, release=A + 3 * M,
                free_pages=A + 4 * M, free_count=A + 5 * M, B=4, max_pages=8, pool=40, page_size=16,
                T=100, page_table_out=A + 6 * M, seq_lens_out=A + 7 * M, free_pages_out=A + 8 * M,
                free_count_out=A + 9 * M, cu_seqlens=A + 10 * M, positions=A + 11 * M,
                slots=A + 12 * M, stream=0)
    args.update(kw)
    return K.kda_page_plan(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(B=65537), "KDA_ERR_BAD_SHAPE"),
    (dict(page_size=0), "KDA_ERR_BAD_SHAPE"),
    (dict(max_pages=1 << 27), "KDA_ERR_BAD_SHAPE"),
    (dict(T=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(pool=1 << 31), "KDA_ERR_BAD_SHAPE"),
    (dict(seq_lens=0), "KDA_ERR_NULL_ARG"),
    (dict(page_table=0), "KDA_ERR_NULL_ARG"),
    (dict(free_count=0), "KDA_ERR_NULL_ARG"),
    (dict(slots=0), "KDA_ERR_NULL_ARG"),
    (dict(cu_seqlens=0), "KDA_ERR_NULL_ARG"),
    (dict(slots=A + 12 * M + 4), "KDA_ERR_MISALIGNED"),
    (dict(page_table=A + 2), "KDA_ERR_MISALIGNED"),
    (dict(page_table_out=A + 4), "KDA_ERR_ALIAS"),       # its input, but one entry on
    (dict(seq_lens_out=A + 2 * M), "KDA_ERR_ALIAS"),
    (dict(positions=A + 12 * M), "KDA_ERR_ALIAS"),
    (dict(cu_seqlens=A + 7 * M), "KDA_ERR_ALIAS"),
])
def test_plan_refusals(kw, code):
    assert plan(**kw) == K.STATUS_CODE[code]


def test_plan_in_place_is_not_an_alias():
    rc = plan(page_table_out=A, seq_lens_out=A + M, free_pages_out=A + 4 * M, free_count_out=A + 5 * M)
    assert rc not in (K.STATUS_CODE["KDA_ERR_ALIAS"], 0)   # (stopped by the device's checks)


def heads(**kw):
    args = dict(q=A, k=A + M, q_weight=A + 2 * M, k_weight=A + 3 * M, inv_freq=A + 4 * M,
                positions=A + 5 * M, T=16, Hq=4, Hk=2, D=64, R=32, q_stride=256, k_stride=128,
                eps=1e-6, flags=0, q_out=A + 6 * M, q_out_stride=256, k_out=A + 7 * M,
                k_out_stride=128, stream=0)
    args.update(kw)
    return K.kda_qk_norm_rope(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=2), "KDA_ERR_BAD_FLAGS"),
    (dict(D=96), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(R=24), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(R=80), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(R=-16), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(T=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(Hq=0), "KDA_ERR_BAD_SHAPE"),
    (dict(Hk=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(eps=-1.0), "KDA_ERR_BAD_SHAPE"),
    (dict(eps=float("nan")), "KDA_ERR_BAD_SHAPE"),
    (dict(q_stride=248), "KDA_ERR_BAD_SHAPE"),
    (dict(k_out_stride=64), "KDA_ERR_BAD_SHAPE"),
    (dict(q=0), "KDA_ERR_NULL_ARG"),
    (dict(k=0), "KDA_ERR_NULL_ARG"),
    (dict(inv_freq=0), "KDA_ERR_NULL_ARG"),
    (dict(positions=0), "KDA_ERR_NULL_ARG"),
    (dict(k_out=0), "KDA_ERR_NULL_ARG"),
    (dict(q=A + 8), "KDA_ERR_MISALIGNED"),
    (dict(k_stride=132), "KDA_ERR_MISALIGNED"),
    (dict(q_out=A + 16), "KDA_ERR_ALIAS"),
    (dict(q_out=A, q_out_stride=512), "KDA_ERR_ALIAS"),
    (dict(k_out=A + 6 * M), "KDA_ERR_ALIAS"),
    (dict(k_out=A), "KDA_ERR_ALIAS"),
])
def test_heads_refusals(kw, code):
    assert heads(**kw) == K.STATUS_CODE[code]


def test_heads_in_place_and_slices_are_not_aliases():
    codes = (K.STATUS_CODE["KDA_ERR_ALIAS"], 0)
    assert heads(q_out=A, k_out=A + M) not in codes
    fused = dict(q=A, k=A + 512, q_stride=512, k_stride=512)   # one buffer's rows
    assert heads(**fused) not in codes
    assert heads(q_out=A, k_out=A + 512, q_out_stride=512, k_out_stride=512, **fused) not in codes


def heads_backward(**kw):
    args = dict(q=A, k=A + M, q_weight=A + 2 * M, k_weight=A + 3 * M, inv_freq=A + 4 * M,
                positions=A + 5 * M, T=16, Hq=4, Hk=2, D=64, R=32, q_stride=256, k_stride=128,
                eps=1e-6, flags=2, dq_out=A + 6 * M, dq_out_stride=256, dk_out=A + 7 * M,
                dk_out_stride=128, dq=A + 8 * M, dq_stride=256, dk=A + 9 * M, dk_stride=128,
                dq_weight=A + 10 * M, dk_weight=A + 11 * M, stream=0)
    args.update(kw)
    return K.kda_qk_norm_rope_backward(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=4), "KDA_ERR_BAD_FLAGS"),
    (dict(D=32), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(dq_out_stride=255), "KDA_ERR_BAD_SHAPE"),
    (dict(dk_stride=120), "KDA_ERR_BAD_SHAPE"),
    (dict(dq_out=0), "KDA_ERR_NULL_ARG"),
    (dict(dk=0), "KDA_ERR_NULL_ARG"),
    (dict(dq_out=A + 6 * M + 4), "KDA_ERR_MISALIGNED"),
    (dict(dk_out_stride=130), "KDA_ERR_MISALIGNED"),
    (dict(dq_weight=A + 10 * M + 1), "KDA_ERR_MISALIGNED"),
    (dict(dq=A), "KDA_ERR_ALIAS"),
    (dict(dk=A + 6 * M), "KDA_ERR_ALIAS"),
    (dict(dk_weight=A + 10 * M), "KDA_ERR_ALIAS"),
    (dict(dq_weight=A + 2 * M), "KDA_ERR_ALIAS"),
])
def test_heads_backward_refusals(kw, code):
    assert heads_backward(**kw) == K.STATUS_CODE[code]


TOK = 2 * 128   # a token of a cache of two heads


def append(**kw):
    args = dict(k=A, v=A + M, k_cache=A + 2 * M, v_cache=A + 4 * M, k_scale=A + 6 * M,
                v_scale=A + 7 * M, page_table=A + 8 * M, seq_lens=A + 9 * M, cu_seqlens=A + 10 * M,
                T=20, B=3, Hkv=2, D=128, pages=8, page_size=16, max_pages=4, k_stride=256,
                v_stride=256, k_page_stride=16 * TOK, k_token_stride=TOK, k_head_stride=128,
                v_page_stride=16 * TOK, v_token_stride=TOK, v_head_stride=128, k_scale_stride=2,
                v_scale_stride=2, stream=0)
    args.update(kw)
    return K.kda_paged_append_fp8(**args)


BOTH = dict(v_cache=A + 2 * M + 16 * TOK, k_page_stride=32 * TOK, v_page_stride=32 * TOK)


@pytest.mark.parametrize("kw,code", [
    (dict(D=256), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(B=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(Hkv=0), "KDA_ERR_BAD_SHAPE"),
    (dict(T=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(T=1 << 30), "KDA_ERR_BAD_SHAPE"),
    (dict(cu_seqlens=0), "KDA_ERR_BAD_SHAPE"),                 # T is not B
    (dict(page_size=0), "KDA_ERR_BAD_SHAPE"),
    (dict(k_head_stride=64), "KDA_ERR_BAD_SHAPE"),             # heads overlap
    (dict(k_token_stride=0), "KDA_ERR_BAD_SHAPE"),
    (dict(v_page_stride=15 * TOK), "KDA_ERR_BAD_SHAPE"),
    (dict(v_page_stride=-16 * TOK), "KDA_ERR_BAD_SHAPE"),
    (dict(k_scale_stride=1), "KDA_ERR_BAD_SHAPE"),
    (dict(v_stride=128), "KDA_ERR_BAD_SHAPE"),
    (dict(k=0), "KDA_ERR_NULL_ARG"),
    (dict(v_cache=0), "KDA_ERR_NULL_ARG"),
    (dict(k_scale=0), "KDA_ERR_NULL_ARG"),
    (dict(page_table=0), "KDA_ERR_NULL_ARG"),
    (dict(k_cache=A + 2 * M + 8), "KDA_ERR_MISALIGNED"),
    (dict(k_page_stride=16 * TOK + 8), "KDA_ERR_MISALIGNED"),
    (dict(k_stride=260), "KDA_ERR_MISALIGNED"),
    (dict(v_scale=A + 7 * M + 2), "KDA_ERR_MISALIGNED"),
    (dict(v_cache=A + 2 * M), "KDA_ERR_ALIAS"),
    (dict(v_cache=A + 2 * M + 128), "KDA_ERR_ALIAS"),
    (dict(BOTH, v_cache=A + 2 * M + 15 * TOK), "KDA_ERR_ALIAS"),
    (dict(v_scale=A + 6 * M), "KDA_ERR_ALIAS"),
    (dict(k_scale=A + 2 * M), "KDA_ERR_ALIAS"),
    (dict(k=A + 4 * M), "KDA_ERR_ALIAS"),
])
def test_append_refusals(kw, code):
    assert append(**kw) == K.STATUS_CODE[code]


@pytest.mark.parametrize("kw", [
    BOTH,                                                      # keys beside values in a page
    dict(v_cache=A + 2 * M + 128, k_page_stride=32 * TOK, k_token_stride=2 * TOK, k_head_stride=256,
         v_page_stride=32 * TOK, v_token_stride=2 * TOK, v_head_stride=256),   # in a head
    dict(v_cache=A + 2 * M + 256, k_page_stride=32 * TOK, k_token_stride=2 * TOK, v_page_stride=32 * TOK,
         v_token_stride=2 * TOK),                              # in a token
    dict(k_token_stride=128, k_head_stride=16 * 128, v_token_stride=128, v_head_stride=16 * 128),
    dict(k_scale=A + 6 * M, v_scale=A + 6 * M + 8, k_scale_stride=4, v_scale_stride=4),
    dict(cu_seqlens=0, T=3),
])
def test_append_layouts_that_are_taken(kw):
    assert append(**kw) not in (0, *(K.STATUS_CODE["KDA_ERR_" + n] for n in (
        "ALIAS", "BAD_SHAPE", "MISALIGNED", "NULL_ARG")))


def decode(**kw):
    args = dict(q=A, k_cache=A + 2 * M, v_cache=A + 4 * M, k_scale=A + 6 * M, v_scale=A + 7 * M,
                page_table=A + 8 * M, seq_lens=A + 9 * M, B=3, Hq=8, Hkv=2, D=128, pages=8, page_size=16,
                max_pages=4, k_page_stride=16 * TOK, k_token_stride=TOK, k_head_stride=128,
                v_page_stride=16 * TOK, v_token_stride=TOK, v_head_stride=128, k_scale_stride=2,
                v_scale_stride=2, scale=1.0, out=A + 10 * M, lse=A + 11 * M, stream=0)
    args.update(kw)
    return K.kda_paged_decode_fp8(**args)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(D=0), "KDA_ERR_UNSUPPORTED_DIM"),
    (dict(B=-1), "KDA_ERR_BAD_SHAPE"),
    (dict(Hq=7), "KDA_ERR_BAD_SHAPE"),
    (dict(Hq=1), "KDA_ERR_BAD_SHAPE"),
    (dict(page_size=0), "KDA_ERR_BAD_SHAPE"),
    (dict(max_pages=1 << 28), "KDA_ERR_BAD_SHAPE"),
    (dict(k_page_stride=15 * TOK), "KDA_ERR_BAD_SHAPE"),
    (dict(q=0), "KDA_ERR_NULL_ARG"),
    (dict(v_scale=0), "KDA_ERR_NULL_ARG"),
    (dict(page_table=0), "KDA_ERR_NULL_ARG"),
    (dict(seq_lens=0), "KDA_ERR_NULL_ARG"),
    (dict(q=A + 8), "KDA_ERR_MISALIGNED"),
    (dict(v_token_stride=TOK + 8, v_page_stride=17 * TOK), "KDA_ERR_MISALIGNED"),
    (dict(out=A), "KDA_ERR_ALIAS"),
    (dict(lse=A + 10 * M), "KDA_ERR_ALIAS"),
    (dict(out=A + 2 * M + 1024), "KDA_ERR_ALIAS"),
])
def test_decode_refusals(kw, code):
    assert decode(**kw) == K.STATUS_CODE[code]


def test_empty_batches_are_no_ops():
    assert K.kda_qk_norm_rope(0, 0, 0, 0, 0, 0, 0, 4, 2, 64, 32, 256, 128, 1e-6, 0, 0, 256, 0, 128, 0) == 0
    assert heads_backward(T=0, q=0, k=0, dq_out=0, dk_out=0, dq=0, dk=0, dq_weight=0, dk_weight=0) == 0
    assert append(T=0, k=0, v=0) == 0
    assert append(B=0, T=0, seq_lens=0, page_table=0) == 0
    assert decode(B=0, q=0, out=0, lse=0, seq_lens=0, page_table=0) == 0


def test_python_front_refuses():
    """The binding's own checks, which need no library call."""
    bf, f8, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
    q, k = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, 1, 64, dtype=bf)
    table, lens = torch.zeros(4, 2, dtype=i32), torch.zeros(4, dtype=i32)
    with pytest.raises(ValueError):
        K.qk_norm_rope(q, k)                                   # not on a GPU
    with pytest.raises(ValueError):
        K.qk_norm_rope(q[0], None)
    with pytest.raises(ValueError):
        K.qk_norm_rope_backward(q, k, q, None)
    with pytest.raises(ValueError):
        K.page_plan(table, lens, lens, lens, lens[:1], 16, 4)
    with pytest.raises(ValueError):
        K.page_plan(table[0], lens, lens, lens, lens[:1], 16, 4)
    cache, scale = torch.zeros(3, 16, 1, 64).to(f8), torch.zeros(3, 1)
    with pytest.raises(ValueError):
        K.paged_append_fp8(k, k, cache, cache, scale, scale, table, lens)
    with pytest.raises(ValueError):
        K.paged_append_fp8(k, k, cache.to(bf), cache.to(bf), scale, scale, table, lens)
    with pytest.raises(ValueError):
        K.paged_decode_fp8(q, cache, cache, scale, scale, table, lens)
    with pytest.raises(ValueError):
        K.paged_decode_fp8(q, cache[0], cache[0], scale, scale, table, lens)
