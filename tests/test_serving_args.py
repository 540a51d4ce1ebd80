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
