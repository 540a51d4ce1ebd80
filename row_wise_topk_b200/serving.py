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
"""
from __future__ import annotations

from . import (DSEL_BF16, DSEL_E4M3, DSEL_F16, DSEL_F32, DSEL_I32, DSEL_I64, DSEL_OK, DselError, lib)

def _run(device, stream, call):
    """``call(stream handle)`` with `device` current and, for a given stream, as torch's current one."""
    import torch

    if stream is None and torch.cuda.current_device() == device.index:
        return call(torch.cuda.current_stream(device).cuda_stream)
    with torch.cuda.device(device):
        if stream is None:
            return call(torch.cuda.current_stream(device).cuda_stream)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
            return call(stream)


def _check(status):
    if status != DSEL_OK:
        raise DselError(status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _vector(name, t, device, dtype, count):
    """A contiguous 1-D tensor of `count` entries, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.device != device or t.dim() != 1 or (count is not None and t.shape[0] != count):
        raise ValueError(f"{name} must be a 1-D {dtype} tensor on {device}"
                         + ("" if count is None else f" with {count} entries"))
    if not t.is_contiguous():   # a copy made here would run on another stream than the call
        raise ValueError(f"{name} must be contiguous")
    return t


def _index_dtype(name, t):
    import torch

    if t.dtype == torch.int32:
        return DSEL_I32
    if t.dtype == torch.int64:
        return DSEL_I64
    raise TypeError(f"{name} must be int32 or int64")


def _rows_of(name, t, device, rows):
    """Row stride of a 2-D tensor whose rows are contiguous and do not overlap."""
    if t.dim() != 2 or t.device != device or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must be a 2-D tensor on {device}" + ("" if rows is None else f" with {rows} rows"))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if t.shape[0] <= 1:
        return t.shape[1]
    if t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t.stride(0)


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
    may be ``logits`` itself when that is float32, contiguous and of such a width.
    """
    import torch

    if logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a 2-D CUDA tensor [rows, vocab] (there is no CPU path)")
    if logits.dtype == torch.bfloat16:
        dt = DSEL_BF16
    elif logits.dtype == torch.float32:
        dt = DSEL_F32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    dev = logits.device
    rows, vocab = logits.shape
    if vocab < 1:
        raise ValueError("logits must have at least one column")
    x_stride = _rows_of("logits", logits, dev, None)
    width = t_stride = 0
    t_dt = DSEL_I32
    if tokens is not None:
        t_dt = _index_dtype("tokens", tokens)
        t_stride = _rows_of("tokens", tokens, dev, rows)
        width = tokens.shape[1]
    elif not (prompt_len is None and total_len is None and repetition is None and frequency is None
              and presence is None):
        raise ValueError("penalties and lengths need tokens=")
    prompt_len = _vector("prompt_len", prompt_len, dev, torch.int32, rows)
    total_len = _vector("total_len", total_len, dev, torch.int32, rows)
    repetition = _vector("repetition", repetition, dev, torch.float32, rows)
    frequency = _vector("frequency", frequency, dev, torch.float32, rows)
    presence = _vector("presence", presence, dev, torch.float32, rows)
    if not (bias_offsets is None) == (bias_ids is None) == (bias_values is None):
        raise ValueError("bias_offsets, bias_ids and bias_values come together")
    bias_count = 0
    if bias_ids is not None:
        bias_ids = _vector("bias_ids", bias_ids, dev, torch.int32, None)
        bias_count = bias_ids.shape[0]
        bias_values = _vector("bias_values", bias_values, dev, torch.float32, bias_count)
        bias_offsets = _vector("bias_offsets", bias_offsets, dev, torch.int32, rows + 1)
        if bias_count == 0:
            bias_offsets = bias_ids = bias_values = None
    m_stride = m_count = 0
    if mask is not None:
        if mask.dtype != torch.int32:
            raise TypeError("mask must be int32 words")
        m_stride = _rows_of("mask", mask, dev, None)
        m_count = mask.shape[0]
        mask_rows = _vector("mask_rows", mask_rows, dev, torch.int32, rows)
        if mask.shape[1] * 32 < vocab:
            raise ValueError("mask rows must hold a bit for every token")
        if mask_rows is None and m_count < rows:
            raise ValueError("mask needs a row for every row of logits, or mask_rows=")
        if m_count == 0:
            mask = mask_rows = None
    elif mask_rows is not None:
        raise ValueError("mask_rows needs mask=")
    if out is not None and (out.dtype != torch.float32 or out.device != dev or out.dim() != 2 or out.shape[0] != rows
                            or out.shape[1] < vocab or out.shape[1] % 16 or not out.is_contiguous()):
        raise ValueError("out must be a contiguous float32 tensor [rows, n], n >= vocab a multiple of 16")

    def call(handle):
        o = out if out is not None else torch.empty((rows, (vocab + 15) // 16 * 16), dtype=torch.float32, device=dev)
        _check(lib.dsel_logits(logits.data_ptr(), dt, rows, vocab, x_stride, _ptr(tokens), t_dt, width, t_stride,
                               _ptr(prompt_len), _ptr(total_len), _ptr(repetition), _ptr(frequency), _ptr(presence),
                               _ptr(bias_offsets), _ptr(bias_ids), _ptr(bias_values), bias_count, _ptr(mask),
                               m_stride, m_count, _ptr(mask_rows), o.data_ptr(), o.shape[1], handle))
        return o

    return _run(dev, stream, call)


def _operand_dtype(name, t, byte):
    """The DSEL code of a 16-bit operand (or, where `byte`, of an e4m3 one)."""
    import torch

    if t.dtype == torch.bfloat16:
        return DSEL_BF16
    if t.dtype == torch.float16:
        return DSEL_F16
    if byte and t.dtype == torch.float8_e4m3fn:
        return DSEL_E4M3
    raise TypeError(f"{name} must be bfloat16" + (", float16 or float8_e4m3fn" if byte else " or float16"))


def _queries(q, table, end, seq_ids):
    """Checks what every query of a paged cache comes with; (device, tokens, table stride)."""
    import torch

    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a 3-D CUDA tensor [tokens, heads, dim] (there is no CPU path)")
    dev, tokens = q.device, q.shape[0]
    if q.stride(2) != 1 and q.shape[2] > 1:
        raise ValueError("q must be contiguous in its last dimension")
    if table.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    t_stride = _rows_of("block_table", table, dev, None)
    _vector("end", end, dev, torch.int32, tokens)
    if seq_ids is not None:
        _vector("seq_ids", seq_ids, dev, torch.int32, tokens)
    elif table.shape[0] not in (1, tokens):
        raise ValueError("block_table needs one row, or one for each query, or seq_ids=")
    return dev, tokens, t_stride


def index_score(q, weights, keys, block_table, end, *, seq_ids=None, key_scale=None, row_stride=None, out_dtype=None,
                out=None, stream=None):
    """Scores of every cached key for each query (``dsel_index_score``), the rows of ``topk``.

    ``q``: [tokens, heads, dim], bfloat16, float16 or float8_e4m3fn.  ``weights``: float32
    [tokens, heads].  ``keys``: [pages, page_size, dim] of q's type, ``key_scale`` float32
    [pages, page_size] or None.  ``block_table``: int32 [sequences, width], the pages of each
    sequence in order.  ``end``: int32 [tokens], the keys each query sees (the ``end`` of
    ``topk``).  ``seq_ids``: int32 [tokens], each query's sequence; None: query t is of
    sequence t, or all are of the only one.

    Returns [tokens, row_stride] in ``out_dtype`` (bfloat16, or float32), -inf where a query
    sees no key; ``row_stride`` defaults to the keys a table row can name, rounded up to the
    TopK row-stride requirement.  ``out`` may supply that tensor.
    """
    import torch

    dt = _operand_dtype("q", q, True)
    dev, tokens, t_stride = _queries(q, block_table, end, seq_ids)
    heads, dim = q.shape[1], q.shape[2]
    if keys.dtype != q.dtype or keys.device != dev or keys.dim() != 3 or keys.shape[2] != dim or keys.stride(2) != 1:
        raise ValueError("keys must be [pages, page_size, dim] of q's type on its device, contiguous in the last dimension")
    if weights.dtype != torch.float32 or weights.shape[1:] != (heads,):
        raise ValueError("weights must be float32 [tokens, heads]")
    w_stride = _rows_of("weights", weights, dev, tokens)
    pages, page = keys.shape[0], keys.shape[1]
    s_stride = 0
    if key_scale is not None:
        if key_scale.dtype != torch.float32 or key_scale.shape != (pages, page):
            raise ValueError("key_scale must be float32 [pages, page_size]")
        s_stride = _rows_of("key_scale", key_scale, dev, pages)
    if out is not None:
        if out.dim() != 2 or out.device != dev or out.shape[0] != tokens or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor [tokens, row_stride]")
        if (row_stride is not None and out.shape[1] != row_stride) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out must have the row_stride and out_dtype that are given")
        row_stride, out_dtype = out.shape[1], out.dtype
    else:
        if row_stride is None:
            row_stride = (block_table.shape[1] * page + 15) // 16 * 16
        if out_dtype is None:
            out_dtype = torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("scores are bfloat16 or float32")

    def call(handle):
        o = out if out is not None else torch.empty((tokens, row_stride), dtype=out_dtype, device=dev)
        _check(lib.dsel_index_score(q.data_ptr(), dt, tokens, heads, dim, q.stride(0), q.stride(1), weights.data_ptr(),
                                    w_stride, keys.data_ptr(), pages, page, keys.stride(0), keys.stride(1),
                                    _ptr(key_scale), s_stride, block_table.data_ptr(), block_table.shape[0],
                                    block_table.shape[1], t_stride, _ptr(seq_ids), end.data_ptr(), o.data_ptr(),
                                    DSEL_F32 if out_dtype == torch.float32 else DSEL_BF16, row_stride, handle))
        return o

    return _run(dev, stream, call)


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
    import torch

    dt = _operand_dtype("q", q, False)
    dev, tokens, t_stride = _queries(q, block_table, end, seq_ids)
    heads, dim = q.shape[1], q.shape[2]
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if c.dtype != q.dtype or c.device != dev or c.dim() != 4 or c.shape[3] != dim or c.stride(3) != 1:
            raise ValueError(f"{name} must be [pages, page_size, kv_heads, dim] of q's type on its device, "
                             "contiguous in the last dimension")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    pages, page, kv_heads = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    i_dt = _index_dtype("indices", indices)
    if indices.device != dev or indices.dim() not in (2, 3) or indices.shape[0] != tokens:
        raise ValueError("indices must be [tokens, k] or [tokens, kv_heads, k] on q's device")
    if indices.dim() == 3 and indices.shape[1] != kv_heads:
        raise ValueError("indices must have one list, or one for each key head")
    take = indices.shape[-1]
    if take > 1 and indices.stride(-1) != 1:
        raise ValueError("indices must be contiguous in the last dimension")
    if scale is None:
        scale = dim ** -0.5
    if out is not None and (out.dtype != q.dtype or out.device != dev or out.shape != (tokens, heads, dim)
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor of q's shape and type")

    def call(handle):
        o = out if out is not None else torch.empty((tokens, heads, dim), dtype=q.dtype, device=dev)
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev) if return_lse else None
        _check(lib.dsel_sparse_attn(q.data_ptr(), dt, tokens, heads, kv_heads, dim, q.stride(0), q.stride(1),
                                    k_cache.data_ptr(), v_cache.data_ptr(), pages, page, *k_cache.stride()[:3],
                                    *v_cache.stride()[:3], block_table.data_ptr(), block_table.shape[0],
                                    block_table.shape[1], t_stride, _ptr(seq_ids), end.data_ptr(),
                                    indices.data_ptr(), i_dt, take, indices.stride(0),
                                    indices.stride(1) if indices.dim() == 3 else 0, block, scale, o.data_ptr(),
                                    _ptr(lse), handle))
        return (o, lse) if return_lse else o

    return _run(dev, stream, call)
