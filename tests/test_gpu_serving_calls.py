"""The serving operators' Python calls: refusals of tensors that do not fit (nothing is launched),
several streams at once, one graph that holds a whole step, and a package that imports without torch."""
import subprocess
import sys

import pytest
import torch

import row_wise_topk_b200 as T
from conftest import ROOT


def test_package_imports_without_torch():
    code = ("import sys; import row_wise_topk_b200 as T; assert 'torch' not in sys.modules; "
            "assert callable(T.sparse_attention) and 'torch' in sys.modules")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 64)
    end = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 3, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        T.process_logits(x)
    with pytest.raises(ValueError):
        T.index_score(q, torch.zeros(2, 4), torch.zeros(6, 16, 64, dtype=torch.bfloat16), table, end)
    with pytest.raises(ValueError):
        T.sparse_attention(q, torch.zeros(6, 16, 1, 64, dtype=torch.bfloat16),
                           torch.zeros(6, 16, 1, 64, dtype=torch.bfloat16), table, table, end)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
def test_logits_refusals():
    x = torch.zeros(4, 100, device="cuda")
    ok = dict(tokens=i32(4, 5), total_len=i32(4))
    T.process_logits(x, **ok)
    for kw, err in [
            (dict(tokens=torch.zeros(4, 5, device="cuda")), TypeError),
            (dict(tokens=i32(3, 5)), ValueError),
            (dict(tokens=i32(4, 5).cpu()), ValueError),
            (dict(tokens=i32(4, 10)[:, ::2]), ValueError),
            (dict(total_len=i32(4)), ValueError),                                  # without tokens
            (dict(ok, total_len=i32(3)), ValueError),
            (dict(ok, total_len=i32(8)[::2]), ValueError),
            (dict(ok, repetition=i32(4)), ValueError),
            (dict(bias_ids=i32(3)), ValueError),
            (dict(bias_ids=i32(3), bias_offsets=i32(5), bias_values=torch.zeros(4, device="cuda")), ValueError),
            (dict(mask=i32(4, 3)), ValueError),                                    # 96 bits for 100 tokens
            (dict(mask=i32(3, 4)), ValueError),
            (dict(mask_rows=i32(4)), ValueError),
            (dict(mask=torch.zeros(4, 4, device="cuda")), TypeError),
            (dict(out=torch.zeros(4, 100, device="cuda")), ValueError),
            (dict(out=torch.zeros(4, 96, device="cuda")), ValueError),
            (dict(out=torch.zeros(4, 112, device="cuda", dtype=torch.float64)), ValueError)]:
        with pytest.raises(err):
            T.process_logits(x, **kw)
    with pytest.raises(TypeError):
        T.process_logits(x.half())
    with pytest.raises(ValueError):
        T.process_logits(x.T)
    with pytest.raises(ValueError):
        T.process_logits(x[:1].expand(4, 100))
    buf = torch.zeros(4 * 128 + 128, device="cuda")
    with pytest.raises(T.DselError):                                               # overlaps, another start
        T.process_logits(buf[:448].view(4, 112), out=buf[16:464].view(4, 112))


def paged(dtype=torch.bfloat16):
    return dict(q=torch.zeros(3, 4, 64, dtype=dtype, device="cuda"), table=i32(3, 2), end=i32(3))


@pytest.mark.gpu
def test_score_refusals():
    p = paged()
    w = torch.zeros(3, 4, device="cuda")
    keys = torch.zeros(6, 16, 64, dtype=torch.bfloat16, device="cuda")
    T.index_score(p["q"], w, keys, p["table"], p["end"])
    f = lambda q=p["q"], w=w, keys=keys, table=p["table"], end=p["end"], **kw: T.index_score(q, w, keys, table, end, **kw)
    for kw, err in [
            (dict(q=p["q"].float()), TypeError), (dict(q=p["q"][0]), ValueError), (dict(keys=keys.half()), ValueError),
            (dict(keys=keys[..., :32]), ValueError), (dict(w=w.half()), ValueError), (dict(w=w[:2]), ValueError),
            (dict(table=p["table"].long()), TypeError), (dict(table=i32(2, 2)), ValueError), (dict(end=i32(2)), ValueError),
            (dict(end=None), ValueError), (dict(seq_ids=i32(2)), ValueError), (dict(key_scale=w), ValueError),
            (dict(out_dtype=torch.float16), TypeError), (dict(row_stride=24), T.DselError),
            (dict(out=torch.zeros(3, 32, device="cuda"), row_stride=48), ValueError)]:
        with pytest.raises(err):
            f(**kw)


@pytest.mark.gpu
def test_attention_refusals():
    p = paged()
    c = torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    f = lambda q=p["q"], k=c, v=c, table=p["table"], idx=i32(3, 7), end=p["end"], **kw: T.sparse_attention(
        q, k, v, table, idx, end, **kw)
    f()
    for kw, err in [
            (dict(q=p["q"].float()), TypeError), (dict(k=c.half()), ValueError), (dict(v=c[:5]), ValueError),
            (dict(k=c[..., :32], v=c[..., :32]), ValueError), (dict(idx=i32(3, 7).float()), TypeError),
            (dict(idx=i32(2, 7)), ValueError), (dict(idx=i32(3, 3, 7)), ValueError), (dict(idx=i32(3, 14)[:, ::2]), ValueError),
            (dict(k=c[:, :, :1].expand(6, 16, 3, 64), v=c[:, :, :1].expand(6, 16, 3, 64)), T.DselError),   # 4 over 3 heads
            (dict(block=0), T.DselError), (dict(out=p["q"].float()), ValueError)]:
        with pytest.raises(err):
            f(**kw)
    # one key head for all, as a broadcast view, is a cache like any other
    one = torch.randn(6, 16, 1, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    args = dict(q=q, table=i32(3, 2) + 1, idx=torch.arange(7, device="cuda", dtype=torch.int32).repeat(3, 1), end=i32(3) + 20)
    assert torch.equal(f(k=one, v=one, **args), f(k=one.expand(6, 16, 2, 64), v=one.expand(6, 16, 2, 64), **args))


def step(seed, seqs=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    width, page, dim = 40, 32, 64
    t = torch.randperm(seqs * width, device="cuda", generator=g).view(seqs, width).to(torch.int32)
    a = dict(iq=r(seqs, 16, dim).bfloat16(), w=r(seqs, 16), ik=r(seqs * width, page, dim).bfloat16(), table=t,
             end=torch.randint(200, width * page, (seqs,), device="cuda", generator=g).to(torch.int32),
             q=r(seqs, 8, dim).bfloat16(), k=r(seqs * width, page, 2, dim).bfloat16(), v=r(seqs * width, page, 2, dim).bfloat16(),
             head=r(8 * dim, 5000).bfloat16(), text=torch.randint(0, 5000, (seqs, 60), device="cuda", generator=g).to(torch.int32),
             rep=torch.full((seqs,), 1.3, device="cuda"), u=torch.rand(seqs, device="cuda", generator=g))

    def run():
        rows = T.index_score(a["iq"], a["w"], a["ik"], a["table"], a["end"])
        _, idx = T.topk(rows, 64, return_value=False)
        o, lse = T.sparse_attention(a["q"], a["k"], a["v"], a["table"], idx, a["end"], return_lse=True)
        y = T.process_logits(o.view(seqs, -1) @ a["head"], tokens=a["text"], repetition=a["rep"])
        token, prob = T.topk_sample(y, 40, a["u"], top_p=0.9)
        return rows, idx, o, lse, y, token, prob
    return a, run


@pytest.mark.gpu
def test_steps_on_streams_at_once():
    steps = [step(s)[1] for s in range(4)]
    want = [f() for f in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None] * len(steps)
    for _ in range(5):
        for i, (f, s) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(s):
                got[i] = f()
    torch.cuda.synchronize()
    for w, h in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, h))


@pytest.mark.gpu
def test_two_captured_steps_replay_in_any_order():
    runs = [step(s, seqs=5 + 3 * s) for s in range(2)]
    for _, f in runs:
        f()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _, f in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for order in ((0, 1, 0), (1, 1, 0)):
        for a, _ in runs:
            a["q"].mul_(-0.9)
            a["iq"].add_(0.01)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for (_, f), o in zip(runs, outs):
            assert all(torch.equal(x, y) for x, y in zip(f(), o))


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["logits", "attention", "score"])
def test_the_default_streams_handle(op):
    """stream=0 is what current_stream().cuda_stream gives outside every stream context: the default stream
    itself, behind the work that is on it."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    table = torch.arange(20, device="cuda", dtype=torch.int32).view(4, 5)
    end = torch.full((4,), 80, device="cuda", dtype=torch.int32)
    if op == "logits":
        x = r(4, 1000)
        f = lambda **kw: T.process_logits(x, **kw)
    elif op == "attention":
        x, c = r(4, 8, 64).bfloat16(), r(20, 16, 2, 64).bfloat16()
        idx = torch.arange(60, device="cuda", dtype=torch.int32).repeat(4, 1)
        f = lambda **kw: T.sparse_attention(x, c, c, table, idx, end, **kw)
    else:
        x, w, keys = r(4, 16, 64).bfloat16(), r(4, 16), r(20, 16, 64).bfloat16()
        f = lambda **kw: T.index_score(x, w, keys, table, end, **kw)
    want, final = f(), x.clone()
    out = torch.zeros_like(want)    # (an allocation might wait for the device, and so might making streams)
    torch.cuda.Stream()
    handle = torch.cuda.current_stream().cuda_stream
    assert handle == 0
    x.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(1 << 26)      # tens of ms
    x.copy_(final)
    got = f(stream=handle, out=out)
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,seqs", [(1, 1), (4, 4), (4, 0), (40, 1), (300, 300)])
@pytest.mark.parametrize("pages,width,page", [(0, 3, 16), (0, 0, 16), (6, 0, 16), (0, 3, 10), (6, 0, 10)])
def test_caches_without_keys(tokens, seqs, pages, width, page):
    """A cache before its first page, or a table without places: scores of -inf, attention over nothing."""
    table, end = i32(seqs, width), i32(tokens) + 20
    ids = i32(tokens) if seqs == 0 else None
    q = torch.randn(tokens, 8, 64, device="cuda").bfloat16()
    for out_dtype in (torch.bfloat16, torch.float32):
        rows = T.index_score(q, torch.randn(tokens, 8, device="cuda"), q.new_empty(pages, page, 64), table, end, seq_ids=ids,
                             key_scale=torch.empty(pages, page, device="cuda"), out_dtype=out_dtype)
        assert rows.shape == (tokens, max(16, -(-width * page // 16) * 16)) and (rows == float("-inf")).all()
    wide = T.index_score(q, torch.randn(tokens, 8, device="cuda"), q.new_empty(pages, page, 64), table, end, seq_ids=ids,
                         row_stride=20000)
    assert wide.shape == (tokens, 20000) and (wide == float("-inf")).all()
    for idx in (i32(tokens, 9), i32(tokens, 2, 9).long(), i32(tokens, 0)):
        for block in (1, 3, 16):
            c = q.new_empty(pages, page, 2, 64)
            o, lse = T.sparse_attention(q, c, c, table, idx, end, block=block, seq_ids=ids, return_lse=True)
            assert (o == 0).all() and (lse == float("-inf")).all()
    assert T.dsel_device_status() == 0
