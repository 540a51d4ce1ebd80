"""index_score against the float64 oracle: types, head counts, dims, page sizes, mixed
sequences, empty rows, missing pages, strides, special values, streams, graphs, and the
TopK behind it.

Tolerance: the oracle's bound on the float32 sums, and for bfloat16 scores one rounding of
at most 2^-8 of the value (and of that error)."""
import numpy as np
import pytest
import torch

import oracle.serving_oracle as S
import row_wise_topk_b200 as T

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def make(seed, *, seqs=1, tokens=1, heads=4, dim=64, page=16, width=8, dtype="bf16", scale=False, ends=None, ids=None):
    g = torch.Generator().manual_seed(seed)
    pages = seqs * width + 2
    a = dict(q=torch.randn(tokens, heads, dim, generator=g).to(TYPES[dtype]),
             weights=torch.randn(tokens, heads, generator=g),
             keys=torch.randn(pages, page, dim, generator=g).to(TYPES[dtype]),
             block_table=torch.randperm(pages, generator=g)[: seqs * width].view(seqs, width).to(torch.int32))
    top = width * page
    a["end"] = (torch.randint(0, top + 1, (tokens,), generator=g) if ends is None else torch.tensor(ends)).to(torch.int32)
    if ids is not None:
        a["seq_ids"] = torch.tensor(ids, dtype=torch.int32)
    if scale:
        a["key_scale"] = torch.rand(pages, page, generator=g) + 0.5
    return a


def run(a, **kw):
    d = {k: v.cuda() for k, v in a.items()}
    return T.index_score(d.pop("q"), d.pop("weights"), d.pop("keys"), d.pop("block_table"), d.pop("end"), **d, **kw)


def check(got, a):
    n = {k: (v.double() if v.is_floating_point() else v).numpy() for k, v in a.items()}
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    want, err = S.oracle_score(n["q"], n["weights"], n["keys"], n["block_table"], n["end"], got.shape[1],
                               seq_ids=n.get("seq_ids"), key_scale=n.get("key_scale"))
    got = got.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    off = np.abs(got - want, where=fine, out=np.zeros_like(want))
    bound = err + half * (np.abs(np.where(fine, want, 0)) + err)
    assert np.all(off[fine] <= bound[fine]), (off[fine] - bound[fine]).max()
    assert T.dsel_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("heads,dim", [(1, 32), (4, 64), (16, 128), (17, 96), (40, 64), (64, 128), (100, 128), (128, 32)])
def test_types_heads_dims_one_query(dtype, heads, dim):
    a = make(heads + dim, heads=heads, dim=dim, dtype=dtype, scale=dtype == "e4m3", width=25, ends=[25 * 16 - 3])
    check(run(a), a)
    check(run(a, out_dtype=torch.float32), a)


@pytest.mark.parametrize("heads", [3, 16, 32, 64, 128])
@pytest.mark.parametrize("tokens", [2, 5, 9, 33, 70])
def test_chunks_of_queries(heads, tokens):
    ends = [max(0, 300 - tokens + 1 + i) for i in range(tokens)]
    a = make(tokens, tokens=tokens, heads=heads, dim=64, page=20, width=15, ends=ends)
    check(run(a, out_dtype=torch.float32), a)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
@pytest.mark.parametrize("heads,dim", [(5, 128), (16, 32), (64, 128), (90, 64)])
@pytest.mark.parametrize("tokens,page", [(3, 64), (21, 16), (21, 24)])
def test_chunks_of_other_types(dtype, heads, dim, tokens, page):
    width = -(-700 // page)
    ends = [max(0, 700 - 30 * i) for i in range(tokens)]
    a = make(tokens + heads, tokens=tokens, heads=heads, dim=dim, page=page, width=width, dtype=dtype, scale=True, ends=ends)
    check(run(a, out_dtype=torch.float32), a)


def test_one_long_context():
    a = make(30, heads=4, dim=32, page=64, width=5000, ends=[319_950])
    check(run(a), a)


@pytest.mark.parametrize("page", [1, 7, 16, 33, 64, 128, 200, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_page_sizes(page, dtype):
    width = -(-1000 // page)
    a = make(page, seqs=3, tokens=3, heads=8, dim=128, page=page, width=width, dtype=dtype, scale=True, ends=[1000, 129, 640])
    check(run(a), a)


def test_lengths_and_empty_rows():
    ends = [0, 1, 127, 128, 129, 255, 256, 257, -5, 1 << 30, 383, 384]
    n = len(ends)
    a = make(1, seqs=n, tokens=n, heads=16, dim=64, page=16, width=24, ends=ends)
    got = run(a)
    check(got, a)
    assert (got[0] == float("-inf")).all() and (got[8] == float("-inf")).all()
    check(run(a, row_stride=512), a)          # rows longer than the table
    check(run(a, row_stride=208), a)          # and shorter: ends are clamped


@pytest.mark.parametrize("heads", [16, 64])
def test_mixed_sequences(heads):
    # runs of every length, a sequence that comes back, unknown sequences, in one work item and over several
    ids = [0, 0, 0, 1, 2, 2, -1, -1, 3, 0, 0, 4, 4, 4, 4, 4, 4, 4, 4, 4, 9, 1, 1] + [2] * 40 + [3] * 9
    a = make(7, seqs=5, tokens=len(ids), heads=heads, dim=64, page=33, width=12, ids=ids)
    a["end"][4] = 0
    a["end"][12] = 5
    check(run(a, out_dtype=torch.float32), a)


def test_decode_with_few_tokens_each():
    ids = [s for s in range(20) for _ in range(1 + s % 3)]
    a = make(8, seqs=20, tokens=len(ids), heads=64, dim=128, page=64, width=5, ids=ids)
    check(run(a), a)


def test_missing_pages():
    a = make(9, seqs=2, tokens=2, heads=8, dim=64, page=16, width=20, ends=[320, 311])
    a["block_table"][0, 3] = -1
    a["block_table"][0, 8] = 10 ** 6
    a["block_table"][1, 19] = a["keys"].shape[0]
    got = run(a, row_stride=352)
    check(got, a)
    assert (got[0, 48:64] == float("-inf")).all()


def test_long_rows_many_items():
    a = make(10, seqs=3, tokens=3, heads=32, dim=64, page=64, width=300, ends=[19200, 7, 12345])
    check(run(a), a)
    a = make(11, seqs=1, tokens=24, heads=32, dim=64, page=64, width=170, ends=[10880 - 24 + i for i in range(24)])
    check(run(a), a)


@pytest.mark.parametrize("n", [149, 700, 1300])
@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("heads", [8, 64])
def test_many_short_sequences(page, heads, n):
    # several work items for each CTA (equal shares, and from 1,025 queries on ranges), rows of zero to six tiles in
    # no order, a scale for each key
    ends = [(i * 37) % 730 if i % 5 else (i * 64) % 390 for i in range(n)]
    a = make(page + heads, seqs=n, tokens=n, heads=heads, dim=32, page=page, width=-(-736 // page), dtype="e4m3", scale=True,
             ends=ends)
    check(run(a), a)


def test_strides():
    a = make(12, tokens=6, heads=5, dim=64, page=10, width=9, ends=[90, 80, 3, 0, 55, 90], scale=True)
    d = {k: v.cuda() for k, v in a.items()}
    q = torch.zeros(6, 9, 80, dtype=torch.bfloat16, device="cuda")[:, 2:7, 8:72]
    q.copy_(d["q"])
    keys = torch.full((a["keys"].shape[0], 13, 96), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :10, 16:80]
    keys.copy_(d["keys"])
    w = torch.zeros(6, 11, device="cuda")[:, 3:8]
    w.copy_(d["weights"])
    table = torch.full((1, 30), 7, dtype=torch.int32, device="cuda")[:, 4:13]
    table.copy_(d["block_table"])
    scale = torch.zeros(a["keys"].shape[0], 17, device="cuda")[:, 1:11]
    scale.copy_(d["key_scale"])
    check(T.index_score(q, w, keys, table, d["end"], key_scale=scale), a)


@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("tokens", [1, 7])
def test_layouts(page, tokens):
    # heads before tokens, places before pages, a broadcast query
    a = make(page + tokens, tokens=tokens, heads=6, dim=64, page=page, width=12, ends=[12 * page - i for i in range(tokens)])
    d = {k: v.cuda() for k, v in a.items()}
    q = d["q"].permute(1, 0, 2).contiguous().permute(1, 0, 2)
    keys = d["keys"].permute(1, 0, 2).contiguous().permute(1, 0, 2)
    assert tokens == 1 or not q.is_contiguous()
    args = (d["weights"], keys, d["block_table"], d["end"])
    check(T.index_score(q, *args), a)
    if tokens > 1:
        with pytest.raises(T.DselError):          # queries may not overlap
            T.index_score(d["q"][:1].expand(tokens, 6, 64), *args)


def test_default_stream_by_its_handle():
    a = make(3, tokens=2, heads=4, dim=64, ends=[100, 128])
    check(run(a, stream=torch.cuda.default_stream().cuda_stream), a)


def test_special_values():
    a = make(13, tokens=3, heads=5, dim=32, page=16, width=16, ends=[256, 256, 100])
    a["keys"][a["block_table"][0, 2], 3, 7] = float("nan")
    a["keys"][a["block_table"][0, 5], 1, 9] = float("inf")
    a["q"][1, 2, 4] = float("nan")
    a["weights"][2, 0] = float("inf")
    a["keys"][a["block_table"][0, 6], 4] = 0           # behind query 2's end: its inf * 0 does not count
    check(run(a, out_dtype=torch.float32), a)


def test_far_offsets():
    # pages past 2^32 bytes of the cache
    page, dim = 64, 128
    pages = (1 << 32) // (page * dim * 2) + 40
    keys = torch.zeros(pages, page, dim, dtype=torch.bfloat16, device="cuda")
    a = make(14, heads=8, dim=dim, page=page, width=6, ends=[380])
    where = torch.tensor([pages - 1, 5, pages - 30, pages - 2, 0, 17])
    for i, p in enumerate(where):
        keys[p] = a["keys"][a["block_table"][0, i]].cuda()
    got = T.index_score(a["q"].cuda(), a["weights"].cuda(), keys, where.to(torch.int32).view(1, -1).cuda(), a["end"].cuda())
    check(got, a)


def test_same_bits_on_another_stream_and_in_a_graph():
    a = make(15, seqs=4, tokens=40, heads=64, dim=128, page=64, width=40, ids=[i // 10 for i in range(40)])
    d = {k: v.cuda() for k, v in a.items()}
    args = [d[k] for k in ("q", "weights", "keys", "block_table", "end")]
    first = T.index_score(*args, seq_ids=d["seq_ids"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = T.index_score(*args, seq_ids=d["seq_ids"], stream=s.cuda_stream)
    s.synchronize()
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.index_score(*args, seq_ids=d["seq_ids"], out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, out)
    d["end"].sub_(100)
    g.replay()
    assert torch.equal(out, T.index_score(*args, seq_ids=d["seq_ids"]))
    check(out, dict(a, end=d["end"].cpu()))


def test_topk_takes_the_rows():
    a = make(16, seqs=6, tokens=6, heads=16, dim=64, page=64, width=20, ends=[1280, 1000, 3, 0, 513, 700])
    rows = run(a)
    with_end = T.topk(rows, 64, end=a["end"].cuda(), index_dtype=torch.int32)
    values, idx = T.topk(rows, 64)
    for r, n in enumerate(a["end"].tolist()):
        want = rows[r].float().topk(min(64, n)).values
        if n > 64:
            assert torch.equal(idx[r], with_end[1][r]) and int(idx[r].max()) < n
        assert torch.equal(with_end[0][r][: len(want)].float().sort(descending=True).values, want)


def test_most_queries_see_nothing():
    # shares that begin and end anywhere, long stretches without a key, an unknown sequence between
    n = 600
    ends = [0] * n
    for i, e in ((3, 5000), (4, 128), (300, 1), (301, 4999), (599, 257)):
        ends[i] = e
    ids = list(range(n))
    ids[301], ids[5] = -1, n
    a = make(33, seqs=n, tokens=n, heads=16, dim=32, page=64, width=79, ends=ends, ids=ids)
    check(run(a), a)
    a["end"][:] = 0
    got = run(a)
    assert (got == float("-inf")).all()


def test_no_tokens():
    a = make(17)
    d = {k: v.cuda() for k, v in a.items()}
    got = T.index_score(d["q"][:0], d["weights"][:0], d["keys"], d["block_table"], d["end"][:0])
    assert got.shape == (0, 128)


@pytest.mark.parametrize("tokens,rows", [(40, 40), (40, 64), (33, 500)])
def test_a_chunk_against_a_table_with_spare_rows(tokens, rows):
    # the host sees no more queries than table rows and takes the form for decoding; the scores are the same
    a = make(tokens, tokens=tokens, heads=32, dim=64, page=16, width=20, ends=[320 - tokens + 1 + i for i in range(tokens)],
             ids=[0] * tokens)
    check(run(a, out_dtype=torch.float32), a)
    b = dict(a, block_table=torch.full((rows, 20), -1, dtype=torch.int32), seq_ids=torch.full((tokens,), 7, dtype=torch.int32))
    b["block_table"][7] = a["block_table"][0]
    check(run(b, out_dtype=torch.float32), b)
