"""Refusals of the operators before and after the TopK, on the host: every argument
check of the C entry points runs before CUDA is touched."""
import pytest

import row_wise_topk_b200 as T
from test_abi import header_define


def test_codes_have_texts_and_constants():
    for name in ("DSEL_ERR_SHAPE", "DSEL_ERR_OVERLAP"):
        assert getattr(T, name) == header_define(name)
        assert T.dsel_status_string(header_define(name)) != "unknown status"


def logits(**kw):
    a = dict(x=0x1000, dtype=T.DSEL_F32, rows=4, vocab=1000, x_stride=1000, tokens=0x900000, token_dtype=T.DSEL_I32,
             width=16, tokens_stride=16, prompt_len=None, total_len=None, repetition=None, frequency=None,
             presence=None, bias_offsets=None, bias_ids=None, bias_values=None, bias_count=0, mask=None,
             mask_stride=0, mask_count=0, mask_rows=None, out=0x800000, out_stride=1008, stream=None)
    a.update(kw)
    return T.lib.dsel_logits(*a.values())


@pytest.mark.parametrize("kw,err", [
    (dict(dtype=2), "DSEL_ERR_DTYPE"),
    (dict(rows=-1), "DSEL_ERR_ROWS"),
    (dict(rows=1 << 31), "DSEL_ERR_ROWS"),
    (dict(vocab=0), "DSEL_ERR_SHAPE"),
    (dict(vocab=(1 << 31) - 1), "DSEL_ERR_SHAPE"),
    (dict(x_stride=999), "DSEL_ERR_STRIDE"),
    (dict(out_stride=992), "DSEL_ERR_STRIDE"),
    (dict(out_stride=1004), "DSEL_ERR_STRIDE"),
    (dict(token_dtype=2), "DSEL_ERR_INDEX_DTYPE"),
    (dict(width=-1), "DSEL_ERR_SHAPE"),
    (dict(tokens_stride=15), "DSEL_ERR_STRIDE"),
    (dict(bias_count=-1), "DSEL_ERR_SHAPE"),
    (dict(bias_ids=0x5000), "DSEL_ERR_NULL"),
    (dict(bias_ids=0x5000, bias_offsets=0x6000), "DSEL_ERR_NULL"),
    (dict(mask=0x5000, mask_stride=31, mask_count=4), "DSEL_ERR_STRIDE"),
    (dict(mask=0x5000, mask_stride=32, mask_count=3), "DSEL_ERR_SHAPE"),
    (dict(mask_count=-1), "DSEL_ERR_SHAPE"),
    (dict(x=None), "DSEL_ERR_NULL"),
    (dict(out=None), "DSEL_ERR_NULL"),
    (dict(out=0x800008), "DSEL_ERR_ALIGN"),
    (dict(x=0x1002), "DSEL_ERR_ALIGN"),
    (dict(x=0x1001, dtype=T.DSEL_BF16), "DSEL_ERR_ALIGN"),
    (dict(out=0x1000), "DSEL_ERR_OVERLAP"),                                  # another stride than x
    (dict(x=0x800010, x_stride=1008), "DSEL_ERR_OVERLAP"),                   # not the same start
    (dict(x=0x800000, x_stride=1008, dtype=T.DSEL_BF16), "DSEL_ERR_OVERLAP"),
])
def test_logits_refusals(kw, err):
    assert logits(**kw) == header_define(err)


def test_logits_zero_rows_is_a_noop():
    assert logits(rows=0, x=None, out=None) == T.DSEL_OK


def score(**kw):
    a = dict(q=0x1000, dtype=T.DSEL_BF16, tokens=4, heads=8, dim=64, q_token_stride=512, q_head_stride=64,
             weights=0x2000, weights_stride=8, keys=0x3000, pages=10, page_size=16, page_stride=1024, key_stride=64,
             key_scale=None, scale_page_stride=0, table=0x4000, seqs=4, table_width=5, table_stride=5, seq_ids=None,
             end=0x5000, out=0x6000, out_dtype=T.DSEL_BF16, row_stride=80, stream=None)
    a.update(kw)
    return T.lib.dsel_index_score(*a.values())


@pytest.mark.parametrize("kw,err", [
    (dict(dtype=T.DSEL_F32), "DSEL_ERR_DTYPE"),
    (dict(dtype=4), "DSEL_ERR_DTYPE"),
    (dict(out_dtype=T.DSEL_F16), "DSEL_ERR_DTYPE"),
    (dict(tokens=-1), "DSEL_ERR_ROWS"),
    (dict(heads=0), "DSEL_ERR_SHAPE"),
    (dict(heads=129, weights_stride=129), "DSEL_ERR_SHAPE"),
    (dict(dim=48), "DSEL_ERR_SHAPE"),
    (dict(dim=160), "DSEL_ERR_SHAPE"),
    (dict(page_size=0), "DSEL_ERR_SHAPE"),
    (dict(pages=-1), "DSEL_ERR_SHAPE"),
    (dict(seqs=3), "DSEL_ERR_SHAPE"),            # neither one sequence nor one for each query
    (dict(row_stride=72), "DSEL_ERR_STRIDE"),
    (dict(row_stride=0), "DSEL_ERR_STRIDE"),
    (dict(row_stride=(1 << 31) - 65536), "DSEL_ERR_STRIDE"),
    (dict(q_head_stride=32), "DSEL_ERR_STRIDE"),
    (dict(q_head_stride=68), "DSEL_ERR_STRIDE"),     # not 16 bytes
    (dict(q_token_stride=516), "DSEL_ERR_STRIDE"),
    (dict(key_stride=68), "DSEL_ERR_STRIDE"),
    (dict(page_stride=1028), "DSEL_ERR_STRIDE"),
    (dict(weights_stride=7), "DSEL_ERR_STRIDE"),
    (dict(table_stride=4), "DSEL_ERR_STRIDE"),
    (dict(q=None), "DSEL_ERR_NULL"),
    (dict(weights=None), "DSEL_ERR_NULL"),
    (dict(end=None), "DSEL_ERR_NULL"),
    (dict(q=0x1008), "DSEL_ERR_ALIGN"),
    (dict(keys=0x3008), "DSEL_ERR_ALIGN"),
    (dict(out=0x6008), "DSEL_ERR_ALIGN"),
])
def test_score_refusals(kw, err):
    assert score(**kw) == header_define(err)


def test_score_zero_tokens_is_a_noop():
    assert score(tokens=0, q=None, out=None, seqs=0) == T.DSEL_OK


def attn(**kw):
    a = dict(q=0x1000, dtype=T.DSEL_BF16, tokens=4, q_heads=8, kv_heads=2, dim=64, q_token_stride=512,
             q_head_stride=64, k=0x2000, v=0x3000, pages=10, page_size=16, k_page_stride=2048, k_row_stride=128,
             k_head_stride=64, v_page_stride=2048, v_row_stride=128, v_head_stride=64, table=0x4000, seqs=4,
             table_width=5, table_stride=5, seq_ids=None, end=0x5000, indices=0x6000, index_dtype=T.DSEL_I32, take=7,
             idx_token_stride=7, idx_head_stride=0, block=16, scale=0.125, out=0x7000, lse=None, stream=None)
    a.update(kw)
    return T.lib.dsel_sparse_attn(*a.values())


@pytest.mark.parametrize("kw,err", [
    (dict(dtype=T.DSEL_F32), "DSEL_ERR_DTYPE"),
    (dict(dtype=T.DSEL_E4M3), "DSEL_ERR_DTYPE"),
    (dict(index_dtype=2), "DSEL_ERR_INDEX_DTYPE"),
    (dict(tokens=-1), "DSEL_ERR_ROWS"),
    (dict(kv_heads=0), "DSEL_ERR_SHAPE"),
    (dict(kv_heads=3), "DSEL_ERR_SHAPE"),
    (dict(dim=96), "DSEL_ERR_SHAPE"),
    (dict(page_size=0), "DSEL_ERR_SHAPE"),
    (dict(seqs=3), "DSEL_ERR_SHAPE"),
    (dict(take=-1), "DSEL_ERR_SHAPE"),
    (dict(block=0), "DSEL_ERR_SHAPE"),
    (dict(take=1 << 20, block=1 << 12), "DSEL_ERR_SHAPE"),
    (dict(q_head_stride=60), "DSEL_ERR_STRIDE"),
    (dict(q_token_stride=516), "DSEL_ERR_STRIDE"),
    (dict(k_row_stride=56), "DSEL_ERR_STRIDE"),
    (dict(k_page_stride=2052), "DSEL_ERR_STRIDE"),
    (dict(v_head_stride=68), "DSEL_ERR_STRIDE"),
    (dict(table_stride=4), "DSEL_ERR_STRIDE"),
    (dict(idx_token_stride=-1), "DSEL_ERR_STRIDE"),
    (dict(q=None), "DSEL_ERR_NULL"),
    (dict(indices=None), "DSEL_ERR_NULL"),
    (dict(out=None), "DSEL_ERR_NULL"),
    (dict(v=0x3008), "DSEL_ERR_ALIGN"),
    (dict(out=0x7008), "DSEL_ERR_ALIGN"),
])
def test_attn_refusals(kw, err):
    assert attn(**kw) == header_define(err)


def test_attn_zero_tokens_is_a_noop():
    assert attn(tokens=0, q=None, out=None, seqs=0) == T.DSEL_OK


def test_packed_calls():
    import struct
    words = struct.pack("=25q", *([0x1000, T.DSEL_F32, -1] + [0] * 22))
    assert T.lib.dsel_call(T.DSEL_CALL_LOGITS, words) == header_define("DSEL_ERR_ROWS")
    words = struct.pack("=25q", *([0x1000, 1 << 40, 4] + [0] * 22))           # a dtype that no int holds
    assert T.lib.dsel_call(T.DSEL_CALL_LOGITS, words) == header_define("DSEL_ERR_SHAPE")
    words = struct.pack("=30qd3q", *([0x1000, T.DSEL_BF16, 0, 8, 3] + [0] * 25), 0.5, 0, 0, 0)
    assert T.lib.dsel_call(T.DSEL_CALL_SPARSE_ATTN, words) == header_define("DSEL_ERR_SHAPE")
    words = struct.pack("=26q", *([0x1000, T.DSEL_F32] + [0] * 24))
    assert T.lib.dsel_call(T.DSEL_CALL_INDEX_SCORE, words) == header_define("DSEL_ERR_DTYPE")
    assert T.lib.dsel_call(T.DSEL_CALL_LOGITS, None) == header_define("DSEL_ERR_NULL")
    assert T.lib.dsel_call(3, words) == header_define("DSEL_ERR_UNAVAILABLE")
    for name in ("DSEL_CALL_LOGITS", "DSEL_CALL_INDEX_SCORE", "DSEL_CALL_SPARSE_ATTN", "DSEL_F16", "DSEL_E4M3"):
        assert getattr(T, name) == header_define(name)


@pytest.mark.parametrize("pages,width", [(1, 5), (10, 1)])
def test_caches_may_be_null_only_where_there_are_no_keys(pages, width):
    null = header_define("DSEL_ERR_NULL")
    for name in ("keys", "table"):
        assert score(**{name: None, "pages": pages, "table_width": width}) == null
    for name in ("k", "v", "table"):
        assert attn(**{name: None, "pages": pages, "table_width": width}) == null
