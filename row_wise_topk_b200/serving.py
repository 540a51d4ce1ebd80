"""The operators before and after the TopK of a serving step, over torch tensors.

- ``process_logits`` makes the rows that ``topk_sample`` (or ``topk``) takes: penalties
  for repeated tokens, biases, a grammar mask.
- ``index_score`` makes the rows that ``topk`` selects keys from: the Lightning Indexer's
  score of every cached key for each query.
- ``sparse_attention`` reads the blocks that those indices name out of a paged cache.

Each is one call of the C ABI (``include/dsel.h`` states the formulas and the argument
rules); this module checks the tensors and allocates the outputs.  Calls run on the
tensors' device, on the current stream or on the raw handle given as ``stream``
(outputs are then allocated for that stream).  Argument errors raise before any
launch: ``TypeError`` / ``ValueError`` here, ``DselError`` from the library.

Decoding steps call these with microseconds of work each, so the checks are few and
plain, and the arguments go to the library packed into one array (``dsel_call``).
"""
from __future__ import annotations

import contextlib
import struct

import torch

from . import (DSEL_BF16, DSEL_CALL_INDEX_SCORE, DSEL_CALL_LOGITS, DSEL_CALL_SPARSE_ATTN, DSEL_E4M3, DSEL_F16, DSEL_F32,
               DSEL_I32, DSEL_I64, DSEL_OK, DselError, lib)

# the arguments of the entry points, each in 8 bytes, in their order
_LOGITS = struct.Struct("=25q")
_SCORE = struct.Struct("=26q")
_ATTN = struct.Struct("=30qd3q")

_call = lib.dsel_call
_stream_of = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_I32, _I64, _F32, _BF16, _F16, _E4M3 = (torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.float16,
                                        torch.float8_e4m3fn)


@contextlib.contextmanager
def _on(device, stream):
    """CUDA device `device` as the current one and, where a raw stream handle is given, that stream as torch's."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            # (0 is the default stream's handle, but no external stream: torch would take one of its own pool for it)
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream != 0
                                   else torch.cuda.default_stream(device)):
                yield


def _vector(name, t, device, dtype, count):
    """The address of a contiguous 1-D tensor of `count` entries; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != device or t.shape != (count,):
        raise ValueError(f"{name} must be a 1-D {dtype} tensor on the same device with {count} entries")
    if not t.is_contiguous():   # a copy made here would run on another stream than the call
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows_of(name, t, device, rows):
    """Row stride of a 2-D tensor whose rows are contiguous and do not overlap."""
    shape = t.shape
    if len(shape) != 2 or t.get_device() != device or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} must be a 2-D tensor on the same device" + ("" if rows is None else f" with {rows} rows"))
    stride, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if shape[0] <= 1:
        return shape[1]
    if stride < shape[1]:
        raise ValueError(f"{name} must have rows that do not overlap")
    return stride


def _index_dtype(name, t):
    if t.dtype is _I32:
        return DSEL_I32
    if t.dtype is _I64:
        return DSEL_I64
    raise TypeError(f"{name} must be int32 or int64")


def process_logits(logits, *, tokens=None, prompt_len=None, total_len=None, repetition=None, frequency=None,
                   presence=None, bias_offsets=None, bias_ids=None, bias_values=None, mask=None, mask_rows=None,
                   out=None, stream=None):
    """Penalties, biases and a grammar mask on logits (``dsel_logits``).

    ``logits``: [rows, vocab], bfloat16 or float32, any row stride.  ``tokens``: [rows, width]
    int32 / int64, of which the first ``total_len[r]`` are the row's text and the first
    ``prompt_len[r]`` its prompt.  ``repetition`` / ``frequency`` / ``presence``: float32, one
    per row.  ``bias_ids`` (int32) and ``bias_values`` (float32) hold all rows' biases one
    after another, row r's from ``bias_offsets[r]`` (int32 [rows + 1]) on.  ``mask``: int32
    [n, words], bit v % 32 of word v // 32 set where token v is allowed; row r uses mask
    row ``mask_rows[r]`` (int32; -1: not masked), or row r.

    Returns float32 [rows, n], n = vocab rounded up to the TopK row-stride requirement,
    with -inf in the columns behind the vocabulary.  ``out`` may supply that tensor; it
    may be ``logits`` itself when that is float32, contiguous and of such a width, or the
    buffer of such a width whose first ``vocab`` columns ``logits`` is.
    """
    dev = logits.get_device()
    if dev < 0 or logits.dim() != 2:
        raise ValueError("logits must be a 2-D CUDA tensor [rows, vocab] (there is no CPU path)")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return process_logits(logits, tokens=tokens, prompt_len=prompt_len, total_len=total_len, repetition=repetition,
                                  frequency=frequency, presence=presence, bias_offsets=bias_offsets, bias_ids=bias_ids,
                                  bias_values=bias_values, mask=mask, mask_rows=mask_rows, out=out)
    if logits.dtype is _BF16:
        dt = DSEL_BF16
    elif logits.dtype is _F32:
        dt = DSEL_F32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    rows, vocab = logits.shape
    if vocab < 1:
        raise ValueError("logits must have at least one column")
    x_stride = _rows_of("logits", logits, dev, None)
    p_tokens = t_dt = width = t_stride = 0
    if tokens is not None:
        t_dt = _index_dtype("tokens", tokens)
        t_stride = _rows_of("tokens", tokens, dev, rows)
        width = tokens.shape[1]
        p_tokens = tokens.data_ptr()
    elif not (prompt_len is None and total_len is None and repetition is None and frequency is None
              and presence is None):
        raise ValueError("penalties and lengths need tokens=")
    p_prompt = _vector("prompt_len", prompt_len, dev, _I32, rows)
    p_total = _vector("total_len", total_len, dev, _I32, rows)
    p_rep = _vector("repetition", repetition, dev, _F32, rows)
    p_freq = _vector("frequency", frequency, dev, _F32, rows)
    p_pres = _vector("presence", presence, dev, _F32, rows)
    p_boff = p_bids = p_bval = n_bias = 0
    if bias_ids is not None or bias_offsets is not None or bias_values is not None:
        if bias_ids is None or bias_offsets is None or bias_values is None:
            raise ValueError("bias_offsets, bias_ids and bias_values come together")
        n_bias = bias_ids.shape[0] if bias_ids.dim() == 1 else -1
        p_bids = _vector("bias_ids", bias_ids, dev, _I32, n_bias)
        p_bval = _vector("bias_values", bias_values, dev, _F32, n_bias)
        p_boff = _vector("bias_offsets", bias_offsets, dev, _I32, rows + 1)
        if n_bias == 0:
            p_boff = p_bids = p_bval = 0
    p_mask = m_stride = m_count = p_mrows = 0
    if mask is not None:
        if mask.dtype is not _I32:
            raise TypeError("mask must be int32 words")
        m_stride = _rows_of("mask", mask, dev, None)
        m_count, words = mask.shape
        p_mrows = _vector("mask_rows", mask_rows, dev, _I32, rows)
        if words * 32 < vocab:
            raise ValueError("mask rows must hold a bit for every token")
        if mask_rows is None and m_count < rows:
            raise ValueError("mask needs a row for every row of logits, or mask_rows=")
        if m_count > 0:
            p_mask = mask.data_ptr()
    elif mask_rows is not None:
        raise ValueError("mask_rows needs mask=")
    if out is not None and (out.dtype is not _F32 or out.get_device() != dev or out.dim() != 2 or out.shape[0] != rows
                            or out.shape[1] < vocab or out.shape[1] % 16 or not out.is_contiguous()):
        raise ValueError("out must be a contiguous float32 tensor [rows, n], n >= vocab a multiple of 16")

    o = out if out is not None else logits.new_empty(rows, vocab + 15 & ~15, dtype=_F32)
    status = _call(DSEL_CALL_LOGITS, _LOGITS.pack(
        logits.data_ptr(), dt, rows, vocab, x_stride, p_tokens, t_dt, width, t_stride, p_prompt, p_total, p_rep,
        p_freq, p_pres, p_boff, p_bids, p_bval, n_bias, p_mask, m_stride, m_count, p_mrows, o.data_ptr(),
        o.shape[1], _stream_of(dev)))
    if status != DSEL_OK:
        raise DselError(status)
    return o


def _operand_dtype(name, t, byte):
    """The DSEL code of a 16-bit operand (or, where `byte`, of an e4m3 one)."""
    if t.dtype is _BF16:
        return DSEL_BF16
    if t.dtype is _F16:
        return DSEL_F16
    if byte and t.dtype is _E4M3:
        return DSEL_E4M3
    raise TypeError(f"{name} must be bfloat16" + (", float16 or float8_e4m3fn" if byte else " or float16"))


def _queries(q, table, end, seq_ids):
    """Checks what every query of a paged cache comes with.

    Returns the device, q's shape and strides, the table's shape and row stride, the addresses of end and seq_ids."""
    dev, q_shape = q.get_device(), q.shape
    if dev < 0 or len(q_shape) != 3:
        raise ValueError("q must be a 3-D CUDA tensor [tokens, heads, dim] (there is no CPU path)")
    q_stride, tokens = q.stride(), q_shape[0]
    if q_stride[2] != 1:
        raise ValueError("q must be contiguous in its last dimension")
    if table.dtype is not _I32:
        raise TypeError("block_table must be int32")
    t_stride = _rows_of("block_table", table, dev, None)
    t_shape = table.shape
    if end is None:
        raise ValueError("end (the keys each query sees) must be given")
    p_end = _vector("end", end, dev, _I32, tokens)
    p_seq = 0
    if seq_ids is not None:
        p_seq = _vector("seq_ids", seq_ids, dev, _I32, tokens)
    elif t_shape[0] != 1 and t_shape[0] != tokens:
        raise ValueError("block_table needs one row, or one for each query, or seq_ids=")
    return dev, q_shape, q_stride, t_shape, t_stride, p_end, p_seq


def index_score(q, weights, keys, block_table, end, *, seq_ids=None, key_scale=None, row_stride=None, out_dtype=None,
                out=None, stream=None):
    """Scores of every cached key for each query (``dsel_index_score``), the rows of ``topk``.

    ``q``: [tokens, heads, dim], bfloat16, float16 or float8_e4m3fn.  ``weights``: float32
    [tokens, heads].  ``keys``: [pages, page_size, dim] of q's type, ``key_scale`` float32
    [pages, page_size] or None.  ``block_table``: int32 [sequences, width], the pages of each
    sequence in order (best of this call's sequences alone).  ``end``: int32 [tokens], the keys
    each query sees (the ``end`` of ``topk``).  ``seq_ids``: int32 [tokens], each query's sequence; None: query t is of
    sequence t, or all are of the only one.

    Returns [tokens, row_stride] in ``out_dtype`` (bfloat16, or float32), -inf where a query
    sees no key; ``row_stride`` defaults to the keys a table row can name, rounded up to the
    TopK row-stride requirement.  ``out`` may supply that tensor.
    """
    dt = _operand_dtype("q", q, True)
    dev, (tokens, heads, dim), (q_token, q_head, _), (seqs, t_width), t_stride, p_end, p_seq = _queries(
        q, block_table, end, seq_ids)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return index_score(q, weights, keys, block_table, end, seq_ids=seq_ids, key_scale=key_scale,
                               row_stride=row_stride, out_dtype=out_dtype, out=out)
    k_shape = keys.shape
    if keys.dtype is not q.dtype or keys.get_device() != dev or len(k_shape) != 3 or k_shape[2] != dim or keys.stride()[2] != 1:
        raise ValueError("keys must be [pages, page_size, dim] of q's type on its device, contiguous in the last dimension")
    if weights.dtype is not _F32 or weights.shape != (tokens, heads):
        raise ValueError("weights must be float32 [tokens, heads]")
    w_stride = _rows_of("weights", weights, dev, tokens)
    pages, page, _ = k_shape
    k_page, k_row, _ = keys.stride()
    p_scale = s_stride = 0
    if key_scale is not None:
        if key_scale.dtype is not _F32 or key_scale.shape != (pages, page):
            raise ValueError("key_scale must be float32 [pages, page_size]")
        s_stride = _rows_of("key_scale", key_scale, dev, pages)
        p_scale = key_scale.data_ptr()
    if out is not None:
        if out.dim() != 2 or out.get_device() != dev or out.shape[0] != tokens or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor [tokens, row_stride]")
        if (row_stride is not None and out.shape[1] != row_stride) or (out_dtype is not None and out.dtype is not out_dtype):
            raise ValueError("out must have the row_stride and out_dtype that are given")
        row_stride, out_dtype = out.shape[1], out.dtype
    else:
        if row_stride is None:
            row_stride = max(t_width * page + 15 & ~15, 16)   # (a row of the TopK has some columns)
        if out_dtype is None:
            out_dtype = _BF16
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise TypeError("scores are bfloat16 or float32")

    o = out if out is not None else weights.new_empty(tokens, row_stride, dtype=out_dtype)
    status = _call(DSEL_CALL_INDEX_SCORE, _SCORE.pack(
        q.data_ptr(), dt, tokens, heads, dim, q_token, q_head, weights.data_ptr(), w_stride, keys.data_ptr(),
        pages, page, k_page, k_row, p_scale, s_stride, block_table.data_ptr(), seqs, t_width, t_stride, p_seq,
        p_end, o.data_ptr(), DSEL_F32 if out_dtype is _F32 else DSEL_BF16, row_stride, _stream_of(dev)))
    if status != DSEL_OK:
        raise DselError(status)
    return o


def sparse_attention(q, k_cache, v_cache, block_table, indices, end, *, block=1, seq_ids=None, scale=None, out=None,
                     return_lse=False, stream=None):
    """Attention of each query over the cached blocks its indices name (``dsel_sparse_attn``).

    ``q``: [tokens, q_heads, dim], bfloat16 or float16, dim 64 or 128.  ``k_cache`` / ``v_cache``:
    [pages, page_size, kv_heads, dim] of q's type; query head h reads key head
    h // (q_heads // kv_heads).  ``block_table``, ``end`` (positions each query sees) and
    ``seq_ids``: as for ``index_score``.  ``indices``: int32 or int64 [tokens, k], or
    [tokens, kv_heads, k] for a list per key head: what ``topk`` returns; an index i stands for
    the positions i * block .. i * block + block - 1, negative ones are skipped.  ``scale``
    defaults to dim ** -0.5.

    Returns [tokens, q_heads, dim] (``out`` may supply it), and with ``return_lse`` also the
    float32 logarithms of the sums of exponentials [tokens, q_heads].
    """
    dt = _operand_dtype("q", q, False)
    dev, (tokens, heads, dim), (q_token, q_head, _), (seqs, t_width), t_stride, p_end, p_seq = _queries(
        q, block_table, end, seq_ids)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return sparse_attention(q, k_cache, v_cache, block_table, indices, end, block=block, seq_ids=seq_ids,
                                    scale=scale, out=out, return_lse=return_lse)
    shape = k_cache.shape
    if len(shape) != 4 or shape[3] != dim or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [pages, page_size, kv_heads, dim], dim that of q")
    if (k_cache.dtype is not q.dtype or v_cache.dtype is not q.dtype or k_cache.get_device() != dev
            or v_cache.get_device() != dev):
        raise ValueError("k_cache and v_cache must be of q's type on its device")
    pages, page, kv_heads, _ = shape
    k_page, k_row, k_head, k_step = k_cache.stride()
    v_page, v_row, v_head, v_step = v_cache.stride()
    if k_step != 1 or v_step != 1:
        raise ValueError("k_cache and v_cache must be contiguous in their last dimension")
    i_dt = _index_dtype("indices", indices)
    i_shape, i_stride = indices.shape, indices.stride()
    if len(i_shape) not in (2, 3) or i_shape[0] != tokens or indices.get_device() != dev:
        raise ValueError("indices must be [tokens, k] or [tokens, kv_heads, k] on q's device")
    if len(i_shape) == 3 and i_shape[1] != kv_heads:
        raise ValueError("indices must have one list, or one for each key head")
    take = i_shape[-1]
    if take > 1 and i_stride[-1] != 1:
        raise ValueError("indices must be contiguous in the last dimension")
    if scale is None:
        scale = dim ** -0.5
    if out is not None and (out.dtype is not q.dtype or out.get_device() != dev or out.shape != (tokens, heads, dim)
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor of q's shape and type")

    o = out if out is not None else q.new_empty(tokens, heads, dim)
    lse = q.new_empty(tokens, heads, dtype=_F32) if return_lse else None
    status = _call(DSEL_CALL_SPARSE_ATTN, _ATTN.pack(
        q.data_ptr(), dt, tokens, heads, kv_heads, dim, q_token, q_head, k_cache.data_ptr(), v_cache.data_ptr(),
        pages, page, k_page, k_row, k_head, v_page, v_row, v_head, block_table.data_ptr(), seqs, t_width,
        t_stride, p_seq, p_end, indices.data_ptr(), i_dt, take, i_stride[0],
        i_stride[1] if len(i_shape) == 3 else 0, block, scale, o.data_ptr(),
        0 if lse is None else lse.data_ptr(), _stream_of(dev)))
    if status != DSEL_OK:
        raise DselError(status)
    return (o, lse) if return_lse else o
