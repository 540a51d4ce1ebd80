"""process_logits against the float64 oracle: penalties, biases, masks, odd sizes and
strides, the special values, in-place calls, streams, graphs, and the sampler behind it.

Tolerance: each of the n roundings that a value goes through in float32 is off by at most
half a step of an intermediate no larger than the sum of the magnitudes m it is made of:
n * 2^-24 * m (the oracle gives n and m for each value); values that go through none are
equal."""
import numpy as np
import pytest
import torch

import oracle.serving_oracle as S
import row_wise_topk_b200 as T

pytestmark = pytest.mark.gpu


def make(seed, rows, vocab, *, dtype=torch.float32, width=0, biases=0, masked=False, ids=torch.int32, spread=None):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((rows, vocab), dtype=np.float32) * 3).to(dtype)
    a = dict(x=x)
    if width:
        top = spread or vocab
        a["tokens"] = torch.from_numpy(rng.integers(-2, top + 2, (rows, width))).to(ids)
        a["total_len"] = torch.from_numpy(rng.integers(0, width + 1, rows)).to(torch.int32)
        a["prompt_len"] = torch.from_numpy(rng.integers(0, width + 1, rows)).to(torch.int32)
        for name, lo, hi in (("repetition", 0.8, 1.4), ("frequency", -0.3, 0.6), ("presence", -0.5, 1.0)):
            a[name] = torch.from_numpy(rng.uniform(lo, hi, rows).astype(np.float32))
    if biases:
        n = rng.integers(0, biases + 1, rows)
        a["bias_offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(torch.int32)
        a["bias_ids"] = torch.from_numpy(rng.integers(-1, vocab + 1, int(n.sum()))).to(torch.int32)
        a["bias_values"] = torch.from_numpy(rng.standard_normal(int(n.sum())).astype(np.float32) * 4)
    if masked:
        count = rows // 2 + 1
        words = rng.integers(0, 1 << 32, (count, -(-vocab // 32) + 1), dtype=np.uint64).astype(np.uint32)
        words[0] = 0                       # a mask that leaves nothing
        a["mask"] = torch.from_numpy(words.view(np.int32))
        a["mask_rows"] = torch.from_numpy(rng.integers(-1, count, rows)).to(torch.int32)
        a["mask_rows"][0] = 0
    return a


def want(a, stride):
    np_ = {k: v.float().numpy() if v.is_floating_point() else v.numpy() for k, v in a.items()}
    biases = None
    if "bias_ids" in a:
        o = np_["bias_offsets"]
        biases = [list(zip(np_["bias_ids"][o[r]:o[r + 1]].tolist(), np_["bias_values"][o[r]:o[r + 1]].tolist()))
                  for r in range(len(o) - 1)]
    keep = {k: np_.get(k) for k in ("tokens", "prompt_len", "total_len", "repetition", "frequency", "presence",
                                    "mask", "mask_rows")}
    return S.oracle_logits(np_["x"], stride, biases=biases, **keep)


def check(got, a):
    got = got.cpu().numpy().astype(np.float64)
    y, mag, rounds = want(a, got.shape[1])
    assert np.array_equal(np.isnan(got), np.isnan(y))
    fine = np.isfinite(y)
    assert np.array_equal(got[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)])
    err = np.abs(got[fine] - y[fine])
    assert np.all(err <= (rounds * 2.0 ** -24 * mag + 2.0 ** -149 * (rounds > 0))[fine]), err.max()


def run(a, **kw):
    d = {k: v.cuda() for k, v in a.items()}
    return T.process_logits(d.pop("x"), **d, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 31), (2, 33), (5, 1000), (2, 8192), (3, 8193), (2, 16399)])
@pytest.mark.parametrize("width,biases,masked", [(0, 0, True), (1, 0, False), (700, 40, True)])
def test_against_oracle(dtype, rows, vocab, width, biases, masked):
    a = make(rows * 31 + vocab, rows, vocab, dtype=dtype, width=width, biases=biases, masked=masked)
    check(run(a), a)


def test_plain_copy_and_padding():
    a = make(1, 4, 100, dtype=torch.bfloat16)
    out = run(a)
    assert out.shape == (4, 112) and torch.isinf(out[:, 100:]).all() and (out[:, 100:] < 0).all()
    assert torch.equal(out[:, :100].cpu(), a["x"].float())


def test_long_history_many_repeats_int64():
    # 20,000 tokens over 50 ids: counts of hundreds, several passes of the scan
    a = make(2, 3, 9000, width=20000, ids=torch.int64, spread=50)
    a["total_len"] = torch.tensor([20000, 19999, 4097], dtype=torch.int32)
    check(run(a), a)


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("rows,vocab,shift", [(40, 70001, 3), (150, 20000, 0), (75, 33000, 1)])
def test_long_texts_of_a_batch(ids, rows, vocab, shift):
    # batches that fill the GPU, texts of thousands of tokens with many repeats, at any alignment
    a = make(rows + shift, rows, vocab, width=2500, ids=ids, masked=True, biases=20, spread=vocab // 3)
    toks = torch.full((rows, 2500 + shift), 5, dtype=ids, device="cuda")[:, shift:]
    toks.copy_(a["tokens"])
    a["repetition"][1], a["frequency"][1], a["presence"][1] = 1.0, 0.0, 0.0       # its tokens are not read
    a["total_len"][2] = 0
    d = {k: v.cuda() for k, v in a.items() if k not in ("x", "tokens")}
    x = a["x"].cuda()
    got = T.process_logits(x, tokens=toks, **d)
    want = torch.stack([T.process_logits(x[r:r + 1], tokens=toks[r:r + 1], **{k: v[r:r + 1] for k, v in d.items()
                                         if k in ("total_len", "prompt_len", "repetition", "frequency", "presence", "mask_rows")},
                                         mask=d["mask"], bias_offsets=d["bias_offsets"][r:r + 2], bias_ids=d["bias_ids"],
                                         bias_values=d["bias_values"])[0] for r in range(rows)])
    assert torch.equal(got, want)              # a row by itself (the other launch shape) gives the same bits
    few = {k: (v[:3] if k in ("x", "tokens", "total_len", "prompt_len", "repetition", "frequency", "presence", "mask_rows") else v)
           for k, v in a.items()}
    few["bias_offsets"] = a["bias_offsets"][:4]
    check(got[:3], few)


def test_lengths_out_of_range_are_clamped():
    a = make(3, 4, 500, width=64)
    a["total_len"] = torch.tensor([-5, 1000, 64, 0], dtype=torch.int32)
    a["prompt_len"] = torch.tensor([3, -7, 1000, 2], dtype=torch.int32)
    check(run(a), a)


def test_default_lengths_and_single_penalties():
    for name in ("repetition", "frequency", "presence"):
        a = make(4, 3, 700, width=90)
        for other in {"repetition", "frequency", "presence", "total_len", "prompt_len"} - {name}:
            del a[other]
        check(run(a), a)


def test_repeated_biases_add_in_list_order():
    # one id many times over more than one warp step, and beside others; the sum depends on its order
    a = make(5, 2, 300)
    ids = [7] * 70 + [9, 7, 9, 299, -3, 300] * 5
    vals = [(-1.0) ** i * 10.0 ** (i % 9 - 4) for i in range(len(ids))]
    a["bias_ids"] = torch.tensor(ids, dtype=torch.int32)
    a["bias_values"] = torch.tensor(vals, dtype=torch.float32)
    a["bias_offsets"] = torch.tensor([0, len(ids) - 20, len(ids)], dtype=torch.int32)
    first = run(a)
    check(first, a)
    total = np.float32(0)
    for i, v in zip(ids[: len(ids) - 20], a["bias_values"].numpy()):
        total = np.float32(total + v) if i == 7 else total
    assert first[0, 7].item() == np.float32(a["x"][0, 7].item() + total)


def test_offsets_outside_the_list_are_clamped():
    a = make(6, 2, 64, biases=5)
    n = a["bias_ids"].numel()
    a["bias_offsets"] = torch.tensor([-4, n, n + 9], dtype=torch.int32)
    got = run(a)
    a["bias_offsets"] = torch.tensor([0, n, n], dtype=torch.int32)
    check(got, a)


def test_special_values_and_masked_nan():
    a = make(7, 2, 64, width=40, masked=True)
    a["x"][:, 0] = float("nan")
    a["x"][:, 1] = float("inf")
    a["x"][:, 2] = float("-inf")
    a["x"][:, 3] = torch.finfo(torch.float32).min / 2
    a["x"][:, 4] = -0.0
    a["mask_rows"] = torch.tensor([0, -1], dtype=torch.int32)      # row 0 keeps nothing
    out = run(a)
    check(out, a)
    assert (out[0] == float("-inf")).all()
    b = dict(a, mask_rows=torch.tensor([5, 7], dtype=torch.int32))   # rows of the mask that do not exist
    check(run(b), b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_and_offsets(dtype):
    a = make(8, 5, 1003, dtype=dtype, width=33, masked=True)
    big = torch.zeros(5, 1500, dtype=dtype).cuda()
    for shift in (0, 1, 2, 3, 4):
        big[:, shift:shift + 1003] = a["x"].cuda()
        toks = torch.full((5, 70), 3, dtype=torch.int32).cuda()
        toks[:, 5:38] = a["tokens"].cuda()
        d = {k: v.cuda() for k, v in a.items() if k not in ("x", "tokens")}
        check(T.process_logits(big[:, shift:shift + 1003], tokens=toks[:, 5:38], **d), a)


def test_in_place_and_out():
    a = make(9, 6, 4096, width=50, biases=9, masked=True)
    d = {k: v.cuda() for k, v in a.items()}
    x = d.pop("x")
    keep = x.clone()
    wide = torch.full((6, 4128), 7.0, device="cuda")
    assert T.process_logits(x, out=wide, **d) is wide
    check(wide, a)
    assert torch.equal(x, keep)
    got = T.process_logits(x, out=x, **d)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, wide[:, :4096])


def test_same_bits_every_time_on_another_stream_and_in_a_graph():
    a = make(10, 64, 20000, width=3000, biases=30, masked=True, spread=400)
    d = {k: v.cuda() for k, v in a.items()}
    x = d.pop("x")
    first = T.process_logits(x, **d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = T.process_logits(x, stream=s.cuda_stream, **d)
    s.synchronize()
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.process_logits(x, out=out, **d)
    assert not out.any()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, out)
    x.mul_(0.5)      # a replay reads the buffers as they are then
    g.replay()
    assert torch.equal(out, T.process_logits(x, **d))


def test_rows_at_far_offsets():
    # the last row starts past 2^32 bytes and 2^31 elements in
    x = torch.zeros(2, 1 << 31, dtype=torch.bfloat16, device="cuda")[:, :1000]
    a = make(11, 2, 1000, dtype=torch.bfloat16, width=20)
    x.copy_(a["x"])
    d = {k: v.cuda() for k, v in a.items() if k != "x"}
    check(T.process_logits(x, **d), a)


def test_sampler_draws_from_processed_rows():
    # a mask that leaves three tokens: every draw is one of them, whatever the penalties
    rows, vocab = 16, 5001
    a = make(12, rows, vocab, dtype=torch.bfloat16, width=100, biases=8)
    words = np.zeros((1, -(-vocab // 32)), dtype=np.uint32)
    allowed = [17, 2500, 5000]
    for v in allowed:
        words[0, v // 32] |= np.uint32(1 << (v % 32))
    a["mask"] = torch.from_numpy(words.view(np.int32))
    a["mask_rows"] = torch.zeros(rows, dtype=torch.int32)
    y = run(a)
    check(y, a)
    u = torch.linspace(0, 0.999, rows, device="cuda")
    token, prob = T.topk_sample(y, 50, u)
    p = torch.softmax(y.double(), -1)
    got = token.cpu().tolist()
    assert set(got) <= set(allowed)
    assert torch.allclose(prob.double(), p.gather(1, token[:, None])[:, 0], rtol=1e-5, atol=0)


def test_no_rows():
    assert T.process_logits(torch.zeros(0, 10, device="cuda")).shape == (0, 16)


@pytest.mark.parametrize("rows", [1, 2, 5])
@pytest.mark.parametrize("vocab", [1000, 1003, 1008])
def test_in_place_in_a_padded_buffer(rows, vocab):
    # logits are the first columns of the buffer that is written: any number of rows, one as well
    a = make(rows + vocab, rows, vocab, width=50, biases=9, masked=True)
    d = {k: v.cuda() for k, v in a.items()}
    buf = torch.full((rows, 1024), 7.0, device="cuda")
    buf[:, :vocab] = d.pop("x")
    assert T.process_logits(buf[:, :vocab], out=buf, **d) is buf
    check(buf, a)
