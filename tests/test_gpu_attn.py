"""sparse_attention against the float64 oracle: types, head groups, blocks, page sizes, lists
that name nothing, repeated and unknown indices, missing pages, garbage in what is not read,
strides, far offsets, streams, graphs; and scores, TopK and attention as one serving step.

Tolerances: the oracle's bounds (float32 sums, one rounding of each probability, one of o)."""
import numpy as np
import pytest
import torch

import oracle.serving_oracle as S
import row_wise_topk_b200 as T

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(seed, *, seqs=1, tokens=1, hq=4, hk=1, dim=64, page=16, width=16, dtype="bf16", block=1, take=40, ends=None,
         ids=None, per_head=False, idt=torch.int32):
    g = torch.Generator().manual_seed(seed)
    pages = seqs * width + 2
    dt = TYPES[dtype]
    a = dict(q=torch.randn(tokens, hq, dim, generator=g).to(dt),
             k_cache=torch.randn(pages, page, hk, dim, generator=g).to(dt),
             v_cache=torch.randn(pages, page, hk, dim, generator=g).to(dt),
             block_table=torch.randperm(pages, generator=g)[: seqs * width].view(seqs, width).to(torch.int32))
    top = width * page
    a["end"] = (torch.randint(0, top + 1, (tokens,), generator=g) if ends is None else torch.tensor(ends)).to(torch.int32)
    lists = (tokens, hk, take) if per_head else (tokens, take)
    a["indices"] = torch.randint(-1, -(-top // block) + 1, lists, generator=g).to(idt)   # repeats, -1, too far
    if ids is not None:
        a["seq_ids"] = torch.tensor(ids, dtype=torch.int32)
    return a, block


def run(a, block, **kw):
    d = {k: v.cuda() for k, v in a.items()}
    return T.sparse_attention(d.pop("q"), d.pop("k_cache"), d.pop("v_cache"), d.pop("block_table"), d.pop("indices"),
                              d.pop("end"), block=block, return_lse=True, **d, **kw)


def check(got, a, block, scale=None):
    n = {k: (v.double() if v.is_floating_point() else v).numpy() for k, v in a.items()}
    want = S.oracle_attention(n["q"], n["k_cache"], n["v_cache"], n["block_table"], n["indices"], n["end"], block=block,
                              seq_ids=n.get("seq_ids"), scale=scale, eps=EPS[a["q"].dtype])
    for x, y, bound in ((got[0], want[0], want[2]), (got[1], want[1], want[3])):
        x = x.cpu().double().numpy()
        assert np.array_equal(np.isnan(x), np.isnan(y))
        fine = np.isfinite(y)
        assert np.array_equal(x[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)])
        assert np.all(np.abs(x - y)[fine] <= bound[fine]), (np.abs(x - y)[fine] - bound[fine]).max()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (16, 1), (17, 1), (32, 1), (40, 1), (64, 1), (100, 1), (6, 6), (28, 4), (32, 2)])
def test_types_and_head_groups(dtype, dim, hq, hk):
    a, b = make(hq + hk, hq=hq, hk=hk, dim=dim, dtype=dtype, tokens=3, ends=[256, 200, 17], take=70)
    check(run(a, b), a, b)


@pytest.mark.parametrize("block", [1, 3, 16, 64, 100])
@pytest.mark.parametrize("page", [1, 7, 16, 64, 200])
def test_blocks_and_pages(block, page):
    width = -(-600 // page)
    a, b = make(block * page, hq=8, hk=2, page=page, width=width, block=block, take=5 + 40 // block, tokens=2,
                ends=[600, 431])
    check(run(a, b), a, b)


@pytest.mark.parametrize("take", [0, 1, 31, 32, 33, 127, 128, 129, 500, 2048])
@pytest.mark.parametrize("hq", [4, 20, 64])
def test_list_lengths(take, hq):
    a, b = make(take, hq=hq, dim=128, take=take, tokens=2, width=64, page=64, ends=[4096, 3000])
    check(run(a, b), a, b)


def test_many_units_and_splits():
    for tokens in (1, 20, 160, 700):       # one CTA to eight for each query
        a, b = make(tokens, hq=8, hk=2, dim=64, take=300, tokens=tokens, width=40, page=16)
        check(run(a, b), a, b)


def test_one_long_list():
    # 131,072 positions of one query: the running sums of every group over many tiles
    a, b = make(31, hq=4, dim=64, page=64, width=2100, block=64, take=2048, ends=[130_001])
    a["indices"][0] = torch.randperm(2100)[:2048].to(torch.int32)
    check(run(a, b), a, b)


def test_rising_scores():
    # every tile's scores lie above the last one's: the reference moves again and again, or not by enough to
    n = 1024
    for dim, factor in ((64, 0.02), (128, 0.4)):
        a, b = make(32, hq=20, dim=dim, take=n, page=64, width=16, ends=[n])
        a["indices"][0] = torch.arange(n)
        row = a["block_table"][0].long()
        ramp = (torch.arange(n) * factor).view(16, 64, 1, 1)
        a["k_cache"][row] = (a["k_cache"][row].float() * 0.1 + ramp / dim ** 0.5).to(torch.bfloat16)
        a["q"][:] = 1.0
        check(run(a, b), a, b)


def test_nothing_to_read():
    a, b = make(1, tokens=6, hq=5, take=33, ends=[0, -3, 256, 256, 256, 1])
    a["indices"][2] = -1
    a["indices"][3] = torch.arange(33) + 256
    a["indices"][4] = -3
    a["indices"][4, 32] = 255
    a["indices"][5] = torch.arange(33)
    o, lse = got = run(a, b)
    check(got, a, b)
    assert (o[:4] == 0).all() and (lse[:4] == float("-inf")).all()


def test_the_same_index_twice_counts_twice():
    a, b = make(2, hq=4, take=8, ends=[256])
    a["indices"][0] = torch.tensor([5, 5, 9, 200, 5, 9, -1, 255])
    check(run(a, b), a, b)


def test_lists_per_key_head_int64_and_far_indices():
    a, b = make(3, hq=12, hk=3, tokens=4, take=50, per_head=True, idt=torch.int64)
    a["indices"][0, 0, 3] = 1 << 40
    a["indices"][1, 2, 7] = -(1 << 40)
    a["indices"][2, 1, 0] = (1 << 32) + 5      # its low half would be a position
    check(run(a, b), a, b)
    a, b = make(4, hq=4, block=64, page=64, width=8, take=9)
    a["indices"][0, 4] = (1 << 31) - 1
    check(run(a, b), a, b)


def test_mixed_sequences_and_missing_pages():
    ids = [0, 2, 1, 1, -1, 7, 0, 2]
    a, b = make(5, seqs=3, tokens=8, hq=8, hk=2, ids=ids, take=100)
    a["block_table"][1, 4] = -1
    a["block_table"][2, 9] = 10 ** 6
    check(run(a, b), a, b)


@pytest.mark.parametrize("hq", [4, 64])
def test_what_is_not_read_has_no_effect(hq):
    a, b = make(6, hq=hq, dim=128, block=16, page=16, width=16, take=9, ends=[200])
    a["indices"][0] = torch.tensor([0, 3, 12, 5, -1, 15, 12, 9, 2])     # block 12 ends at 208: cut at 200
    clean = run(a, b)
    check(clean, a, b)
    for c in ("k_cache", "v_cache"):
        c = a[c]
        row = a["block_table"][0].long()
        c[row[12], 8:] = float("nan")
        c[row[15]] = float("inf")
        c[row[1]] = float("nan")
        c[~torch.isin(torch.arange(c.shape[0]), row)] = float("nan")
    dirty = run(a, b)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_special_scores():
    a, b = make(7, hq=4, dim=64, take=100, ends=[256], tokens=1)
    a["indices"][0] = torch.arange(100)
    row = a["block_table"][0].long()
    for h, x in ((0, 200.0), (1, -200.0), (2, 1.0)):       # scores of thousands apart
        a["q"][0, h] *= x
    check(run(a, b), a, b)
    a["k_cache"][row[2], 5, 0, 0] = float("nan")
    got = run(a, b)
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()
    a, b = make(8, hq=2, dim=64, take=40, ends=[256])
    a["q"][:] = 1
    a["k_cache"][:] = float("-inf")                          # every score is -inf
    o, lse = run(a, b)
    assert (o == 0).all() and (lse == float("-inf")).all()


def test_scales():
    for scale in (0.0, -0.3, 2.0):
        a, b = make(9, hq=6, hk=2, take=80, tokens=2)
        check(run(a, b, scale=scale), a, b, scale)


def test_strides():
    a, b = make(10, tokens=5, hq=6, hk=2, dim=64, page=10, width=20, take=45)
    d = {k: v.cuda() for k, v in a.items()}
    q = torch.zeros(5, 11, 96, dtype=torch.bfloat16, device="cuda")[:, 3:9, 16:80]
    q.copy_(d["q"])
    # heads before places (another layout of the cache), k and v in one buffer
    both = torch.full((a["k_cache"].shape[0], 2, 2, 10, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = (both[:, i].permute(0, 2, 1, 3)[..., :64] for i in (0, 1))
    k.copy_(d["k_cache"])
    v.copy_(d["v_cache"])
    idx = torch.zeros(5, 60, dtype=torch.int32, device="cuda")[:, 7:52]
    idx.copy_(d["indices"])
    check(T.sparse_attention(q, k, v, d["block_table"], idx, d["end"], return_lse=True), a, b)


def test_far_offsets():
    page, hk, dim = 64, 2, 128
    pages = (1 << 32) // (page * hk * dim * 2) + 30
    k = torch.zeros(pages, page, hk, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    a, b = make(11, hq=8, hk=hk, dim=dim, page=page, width=6, take=100, ends=[380])
    where = torch.tensor([pages - 1, 5, pages - 20, pages - 2, 0, 17])
    for i, p in enumerate(where):
        k[p] = a["k_cache"][a["block_table"][0, i]].cuda()
        v[p] = a["v_cache"][a["block_table"][0, i]].cuda()
    got = T.sparse_attention(a["q"].cuda(), k, v, where.to(torch.int32).view(1, -1).cuda(), a["indices"].cuda(),
                             a["end"].cuda(), return_lse=True)
    check(got, a, b)


def test_same_bits_on_another_stream_and_in_a_graph():
    a, b = make(12, seqs=4, tokens=24, hq=32, hk=4, dim=128, block=16, take=30, width=30, page=64, ids=[i // 6 for i in range(24)])
    d = {k: v.cuda() for k, v in a.items()}
    args = [d[k] for k in ("q", "k_cache", "v_cache", "block_table", "indices", "end")]
    kw = dict(block=b, seq_ids=d["seq_ids"])
    first = T.sparse_attention(*args, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = T.sparse_attention(*args, stream=s.cuda_stream, **kw)
    s.synchronize()
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.sparse_attention(*args, out=out, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, out)
    d["q"].mul_(-1)
    g.replay()
    assert torch.equal(out, T.sparse_attention(*args, **kw))


def test_no_tokens():
    a, b = make(13)
    d = {k: v.cuda() for k, v in a.items()}
    o, lse = T.sparse_attention(d["q"][:0], d["k_cache"], d["v_cache"], d["block_table"], d["indices"][:0], d["end"][:0],
                                return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("tokens,k,block", [(1, 64, 1), (3, 5, 16)])
def test_serving_step(tokens, k, block):
    """Scores -> TopK -> attention -> logits -> draw, as a decoding step runs them, against each
    step's oracle on what the step before gave."""
    seqs, page, width, heads, dim, vocab = 4, 16, 20, 16, 64, 3001
    g = torch.Generator().manual_seed(tokens)
    n = seqs * tokens
    lens = torch.tensor([320, 100, 17, 250])
    end = (lens[:, None] - tokens + 1 + torch.arange(tokens)).reshape(-1).to(torch.int32)
    ids = torch.arange(seqs, dtype=torch.int32).repeat_interleave(tokens)
    a, _ = make(20 + tokens, seqs=seqs, tokens=n, hq=8, hk=2, dim=dim, page=page, width=width, ends=end.tolist(),
                ids=ids.tolist(), take=1)
    # one index key per block, in a paged cache of its own
    blocks = -(-width * page // block)
    bpage, bwidth = 8, -(-blocks // 8)
    ikeys = torch.randn(seqs * bwidth, bpage, dim, generator=g).to(torch.bfloat16)
    itable = torch.randperm(seqs * bwidth, generator=g).view(seqs, bwidth).to(torch.int32)
    iq = torch.randn(n, heads, dim, generator=g).to(torch.bfloat16)
    w = torch.randn(n, heads, generator=g)
    bend = -(-end // block).to(torch.int32)

    rows = T.index_score(iq.cuda(), w.cuda(), ikeys.cuda(), itable.cuda(), bend.cuda(), seq_ids=ids.cuda())
    _, idx = T.topk(rows, k, end=bend.cuda(), return_value=False)
    want, err = S.oracle_score(iq.double().numpy(), w.numpy(), ikeys.double().numpy(), itable.numpy(), bend.numpy(),
                               rows.shape[1], seq_ids=ids.numpy())
    for t in range(n):        # what was chosen scores no less than what was not, within the scores' bound
        chosen = idx[t].cpu().numpy()
        chosen = chosen[chosen >= 0]
        assert len(chosen) == min(k, int(bend[t])) and len(set(chosen.tolist())) == len(chosen)
        left = np.setdiff1d(np.arange(int(bend[t])), chosen)
        if len(left):
            slack = 2 * (err[t].max() + 2.0 ** -8 * np.abs(want[t, : int(bend[t])]).max())
            assert want[t, chosen].min() >= want[t, left].max() - slack
    a["indices"] = idx.cpu()
    got = run(a, block)
    check(got, a, block)

    head = torch.randn(8 * dim, vocab, generator=g).to(torch.bfloat16).cuda()
    logits = got[0].view(n, -1) @ head
    text = torch.randint(0, vocab, (n, 30), generator=g).to(torch.int32)
    rep = torch.full((n,), 1.2)
    y = T.process_logits(logits, tokens=text.cuda(), repetition=rep.cuda())
    ref, mag, rounds = S.oracle_logits(logits.double().cpu().numpy(), y.shape[1], tokens=text.numpy(), repetition=rep.numpy())
    fine = np.isfinite(ref)
    off = np.abs(y.double().cpu().numpy()[fine] - ref[fine])
    assert np.all(off <= rounds[fine] * 2.0 ** -24 * mag[fine])
    token, prob = T.topk_sample(y, 1, torch.zeros(n, device="cuda"))
    assert torch.equal(token, y.argmax(1)) and (prob == 1).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,dim", [(4, 64), (20, 128), (64, 64)])
@pytest.mark.parametrize("far", [0, 17_000, 32_767])
def test_one_score_far_above_a_long_flat_list(dtype, hq, dim, far):
    """Terms e^-18 of the largest each, 32,768 of them: they are all of the result where the largest one's value
    is 0.

    Tolerance: the oracle's bound, and where terms are too small for float16's relative rounding (2^-25 at most
    of what a term of the reference is, 2^11 there): 2^-36 of the largest term for each, times its value."""
    n = 32768
    a, b = make(far + hq, hq=hq, dim=dim, dtype=dtype, page=64, width=n // 64, block=64, take=n // 64, ends=[n])
    a["indices"][0] = torch.arange(n // 64)
    row = a["block_table"][0].long()
    a["q"][:] = 1.0
    a["k_cache"][:] = 0.0
    a["v_cache"][:] = a["v_cache"].abs()
    a["k_cache"][row[far // 64], far % 64] = 18 / dim ** 0.5
    a["v_cache"][row[far // 64], far % 64] = 0.0
    o, lse = run(a, b)
    k = {name: t.double().numpy() if t.is_floating_point() else t.numpy() for name, t in a.items()}
    want = S.oracle_attention(k["q"], k["k_cache"], k["v_cache"], k["block_table"], k["indices"], k["end"], block=b,
                              eps=EPS[a["q"].dtype])
    small = np.abs(k["v_cache"][row.numpy()]).sum(axis=(0, 1))[0] * (2.0 ** -36 if dtype == "f16" else 0.0)
    assert np.all(np.abs(o.cpu().double().numpy() - want[0]) <= want[2] + small)
    assert np.all(np.abs(lse.cpu().double().numpy() - want[1]) <= want[3])
