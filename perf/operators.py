"""Measured cases of the operators that stand before and after the row-wise TopK in serving.

Three operators, each chained to a TopK call of this package:

- ``logits``: penalties for repeated tokens, biases and grammar masks on the rows that
  ``topk_sample`` draws from (``process_logits``);
- ``score``: the cheap score of every cached key for each query, the rows that ``topk`` selects
  from (``index_score``);
- ``attn``: attention over the cached blocks that those indices name (``sparse_attention``).

``own`` False computes them from elementary torch operations in 32 bits, ``own`` True by the
package's calls.
"""
import math

import torch

own = False

PAD = 16                    # row strides of the TopK input are multiples of this
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}


def _up(n, m):
    return -(-n // m) * m


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def _logits(name, rows, vocab, dtype, history, bias, mask):
    return dict(name=name, op="logits", rows=rows, vocab=vocab, dtype=dtype, history=history, bias=bias, mask=mask)


def _score(name, seqs, each, heads, dim, dtype, ctx, page):
    return dict(name=name, op="score", seqs=seqs, each=each, heads=heads, dim=dim, dtype=dtype, ctx=ctx, page=page)


def _attn(name, seqs, each, q_heads, kv_heads, dim, dtype, ctx, page, block, take):
    return dict(name=name, op="attn", seqs=seqs, each=each, q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                ctx=ctx, page=page, block=block, take=take)


def listed():
    return [
        # one request answering alone: its repetition penalty over a short dialogue (latency)
        _logits("logits 1x129280 f32", 1, 129280, "f32", 512, 0, "none"),
        # an ordinary batch of the sampler: half the rows under a grammar, a few biases
        _logits("logits 64x129280 bf16", 64, 129280, "bf16", 4096, 64, "half"),
        # the sampler's large batch: long dialogues, every row under a grammar
        _logits("logits 256x129280 f32", 256, 129280, "f32", 16384, 16, "all"),
        # a vocabulary of odd size: rows that start at odd addresses
        _logits("logits 37x50001 bf16", 37, 50001, "bf16", 1001, 7, "all"),
        # one token of one short dialogue (latency)
        _score("score 1x8192 bf16", 1, 1, 64, 128, "bf16", 8192, 64),
        # the indexer's batch of decoding requests, contexts of 64 K to 128 K keys
        _score("score 64x131072 bf16", 64, 1, 64, 128, "bf16", 131072, 64),
        # the same batch with the key cache in 8 bits and a scale for each key
        _score("score 64x131072 e4m3", 64, 1, 64, 128, "e4m3", 131072, 64),
        # a chunk of a long prompt: many queries over one request's keys
        _score("score 1024x65536 bf16", 1, 1024, 64, 128, "bf16", 65536, 64),
        # one token reads the 512 keys that its TopK chose out of a long context (latency)
        _attn("attn 1x512 bf16", 1, 1, 64, 1, 128, "bf16", 131072, 64, 1, 512),
        # the indexer's batch of decoding requests: 512 keys of each context, one head of keys
        _attn("attn 64x512 bf16", 64, 1, 64, 1, 128, "bf16", 131072, 64, 1, 512),
        # grouped heads, whole blocks of 64 keys
        _attn("attn 64x32x64 bf16", 64, 1, 32, 4, 128, "bf16", 32768, 64, 64, 32),
        # a chunk of a prompt: each of its tokens chooses 16 blocks
        _attn("attn 1024x16x64 f16", 1, 1024, 32, 4, 128, "f16", 32768, 64, 64, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logits", "score", "attn"])
    if op == "logits":
        vocab = _log(rng, 1000, 160000)
        rows = min(_log(rng, 1, 256), 256 * 129280 // vocab)
        history = _log(rng, 1, 32768)
        history = min(history, 256 * 16384 // rows)
        return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(["f32", "bf16"]), history=history,
                    bias=rng.choice([0, 1, 16, 100, 300]), mask=rng.choice(["none", "half", "all"]))
    if op == "score":
        heads = rng.choice([1, 4, 8, 16, 32, 40, 64])
        dim = rng.choice([64, 128])
        dtype = rng.choice(["bf16", "bf16", "f16", "e4m3"])
        page = rng.choice([16, 33, 64, 128])
        if rng.random() < 0.5:      # decoding: one to four tokens of each of many requests
            seqs, each, ctx = _log(rng, 1, 64), rng.choice([1, 1, 2, 4]), _log(rng, 100, 131072)
            seqs = max(1, seqs // each)
        else:                       # a chunk of a prompt
            seqs, each, ctx = rng.choice([1, 1, 2]), _log(rng, 5, 512), _log(rng, 600, 32768)
        return dict(op=op, seqs=seqs, each=each, heads=heads, dim=dim, dtype=dtype, ctx=max(ctx, each), page=page)
    kv_heads = rng.choice([1, 1, 2, 4])
    group = rng.choice([1, 4, 7, 8, 16, 32, 64] if kv_heads == 1 else [1, 4, 7, 8, 16])
    block = rng.choice([1, 1, 16, 64])
    take = _log(rng, 1, 2048) if block == 1 else _log(rng, 1, 2048 // block)
    if rng.random() < 0.6:
        seqs, each, ctx = _log(rng, 1, 64), 1, _log(rng, 64, 65536)
    else:
        seqs, each, ctx = 1, _log(rng, 5, 512), _log(rng, 600, 32768)
    return dict(op=op, seqs=seqs, each=each, q_heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice([64, 128]),
                dtype=rng.choice(["bf16", "f16"]), ctx=ctx, page=rng.choice([16, 33, 64, 128]), block=block, take=take)


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _lengths(seqs, ctx, each):
    """Keys of each request: spread evenly from half the context to the whole one."""
    lo = max(min(each, ctx), ctx // 2)
    return [lo + (ctx - lo) * (i + 1) // seqs for i in range(seqs)]


def _totals(case):
    """Tokens so far of each row: spread evenly up to the longest."""
    n, rows = case["history"], case["rows"]
    return [max(1, n * (i + 1) // rows) for i in range(rows)]


def _pages(case, g):
    """A table of pages in a shuffled order, and what the queries see of it."""
    seqs, each, page = case["seqs"], case["each"], case["page"]
    lens = _lengths(seqs, case["ctx"], each)
    width = -(-case["ctx"] // page)
    count = seqs * width + 3
    table = torch.randperm(count, device="cuda", generator=g)[: seqs * width].view(seqs, width).to(torch.int32)
    last = torch.tensor(lens, device="cuda", dtype=torch.int32)
    # the tokens of a request are its last ones: each sees the keys up to its own
    end = (last[:, None] - each + 1 + torch.arange(each, device="cuda", dtype=torch.int32)).clamp_min(0).reshape(-1)
    seq = None if each == 1 else torch.arange(seqs, device="cuda", dtype=torch.int32).repeat_interleave(each)
    return table, count, end.contiguous(), seq


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = dict(case)
    if case["op"] == "logits":
        rows, vocab = case["rows"], case["vocab"]
        s["logits"] = (normal(rows, vocab) * 3).to(TYPES[case["dtype"]])
        # tokens come back as in text: a few often, many once
        width = max(case["history"], 1)
        u = torch.rand(rows, width, device="cuda", generator=g)
        s["tokens"] = (u.pow(4) * vocab).long().clamp_max(vocab - 1).to(torch.int32)
        s["total_len"] = torch.tensor(_totals(case), device="cuda", dtype=torch.int32)
        s["prompt_len"] = (s["total_len"] * torch.rand(rows, device="cuda", generator=g)).to(torch.int32)
        s["repetition"] = 1.0 + 0.3 * torch.rand(rows, device="cuda", generator=g)
        s["frequency"] = 0.2 * torch.rand(rows, device="cuda", generator=g)
        s["presence"] = 0.5 * torch.rand(rows, device="cuda", generator=g)
        if case["bias"]:
            nb = min(case["bias"], vocab)
            s["bias_offsets"] = torch.arange(rows + 1, device="cuda", dtype=torch.int32) * nb
            s["bias_ids"] = torch.cat([torch.randperm(vocab, device="cuda", generator=g)[:nb] for _ in range(rows)]).to(torch.int32)
            s["bias_values"] = normal(rows * nb) * 5
        if case["mask"] != "none":
            words = -(-vocab // 32)
            n = rows if case["mask"] == "all" else (rows + 1) // 2
            bits = torch.rand(n, words, 32, device="cuda", generator=g) < 0.2
            s["bitmask"] = (bits.long() << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)
            at = torch.arange(rows, device="cuda", dtype=torch.int32)
            s["mask_rows"] = at if case["mask"] == "all" else torch.where(at % 2 == 0, at // 2, -1).to(torch.int32)
        return s
    table, count, end, seq = _pages(case, g)
    s.update(table=table, end=end, seq=seq)
    tokens, page, dim, dt = end.numel(), case["page"], case["dim"], TYPES[case["dtype"]]
    if case["op"] == "score":
        heads = case["heads"]
        s["q"] = normal(tokens, heads, dim).to(dt)
        s["weights"] = normal(tokens, heads) / math.sqrt(heads * dim)
        s["keys"] = normal(count, page, dim).to(dt)
        if case["dtype"] == "e4m3":
            s["key_scale"] = 0.5 + torch.rand(count, page, device="cuda", generator=g)
        return s
    s["q"] = normal(tokens, case["q_heads"], dim).to(dt)
    s["k_cache"] = normal(count, page, case["kv_heads"], dim).to(dt)
    s["v_cache"] = normal(count, page, case["kv_heads"], dim).to(dt)
    # blocks as a TopK in index order gives them: the query's own among them, -1 behind the last one
    block, take = case["block"], case["take"]
    blocks = -(-case["ctx"] // block)
    pick = torch.rand(tokens, max(blocks, take), device="cuda", generator=g)
    at = torch.arange(pick.shape[1], device="cuda")
    own_block = (end.long() - 1).div(block, rounding_mode="floor")[:, None]
    pick = torch.where(at == own_block, 2.0, pick)
    pick = torch.where(at <= own_block, pick, -1.0)
    top = pick.topk(take, dim=1)
    idx = torch.where(top.values >= 0, top.indices, 1 << 40).sort(dim=1).values
    s["indices"] = torch.where(idx < (1 << 40), idx, -1).to(torch.int32)
    return s


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def run(s):
    if own:
        import row_wise_topk_b200 as T
        if s["op"] == "logits":
            return T.process_logits(s["logits"], tokens=s["tokens"], prompt_len=s["prompt_len"], total_len=s["total_len"],
                                    repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                                    bias_offsets=s.get("bias_offsets"), bias_ids=s.get("bias_ids"),
                                    bias_values=s.get("bias_values"), mask=s.get("bitmask"), mask_rows=s.get("mask_rows"))
        if s["op"] == "score":
            return T.index_score(s["q"], s["weights"], s["keys"], s["table"], s["end"], seq_ids=s["seq"],
                                 key_scale=s.get("key_scale"), row_stride=_up(s["ctx"], PAD))
        return T.sparse_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["indices"], s["end"],
                                  block=s["block"], seq_ids=s["seq"], return_lse=True)
    return {"logits": _plain_logits, "score": _plain_score, "attn": _plain_attn}[s["op"]](s)


def _plain_logits(s):
    rows, vocab = s["rows"], s["vocab"]
    x = s["logits"].float()
    tokens = s["tokens"].long()
    at = torch.arange(tokens.shape[1], device=x.device)
    real = at < s["total_len"][:, None]
    said = real & (at >= s["prompt_len"][:, None])
    count = torch.zeros(rows, vocab, device=x.device).scatter_add_(1, tokens, said.float())
    seen = torch.zeros(rows, vocab, device=x.device).scatter_add_(1, tokens, real.float()) > 0
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if "bias_ids" in s:
        row = torch.arange(rows, device=x.device).repeat_interleave(s["bias_ids"].numel() // rows)
        x.view(-1).index_add_(0, row * vocab + s["bias_ids"], s["bias_values"])
    if "bitmask" in s:
        v = torch.arange(vocab, device=x.device)
        bits = (s["bitmask"][:, v // 32] >> (v % 32)) & 1
        kept = (bits[s["mask_rows"].clamp_min(0).long()] != 0) | (s["mask_rows"] < 0)[:, None]
        x = torch.where(kept, x, float("-inf"))
    out = torch.full((rows, _up(vocab, PAD)), float("-inf"), device=x.device)
    out[:, :vocab] = x
    return out


def _plain_score(s):
    seqs, each, heads, dim, page, ctx = (s[k] for k in ("seqs", "each", "heads", "dim", "page", "ctx"))
    pos = torch.arange(_up(ctx, PAD), device="cuda")
    inside = pos.clamp_max(ctx - 1)
    slot = s["table"].long()[:, inside // page] * page + inside % page
    keys = s["keys"].view(-1, dim)[slot].float()
    z = torch.matmul(s["q"].float().view(seqs, each * heads, dim), keys.transpose(1, 2)).relu_()
    z = torch.einsum("bnhs,bnh->bns", z.view(seqs, each, heads, -1), s["weights"].view(seqs, each, heads))
    if "key_scale" in s:
        z = z * s["key_scale"].view(-1)[slot][:, None]
    z = z.view(seqs * each, -1)
    return torch.where(pos < s["end"][:, None], z, float("-inf")).to(torch.bfloat16)


def _plain_attn(s):
    tokens, hq, dim = s["q"].shape
    hk, page, block = s["kv_heads"], s["page"], s["block"]
    idx = s["indices"].long()
    pos = (idx[:, :, None] * block + torch.arange(block, device="cuda")).view(tokens, -1)
    kept = (pos >= 0) & (pos < s["end"][:, None]) & (idx >= 0).repeat_interleave(block, 1)
    seq = torch.arange(tokens, device="cuda") if s["seq"] is None else s["seq"].long()
    p = torch.where(kept, pos, 0)
    slot = s["table"].long()[seq[:, None], p // page] * page + p % page
    k = s["k_cache"].view(-1, hk, dim)[slot].float()
    v = s["v_cache"].view(-1, hk, dim)[slot].float()
    q = s["q"].float().view(tokens, hk, hq // hk, dim)
    z = torch.einsum("thgd,tnhd->thgn", q, k) / math.sqrt(dim)
    z = torch.where(kept[:, None, None], z, float("-inf"))
    top = z.amax(-1, keepdim=True).clamp_min(-1e30)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("thgn,tnhd->thgd", e / total.clamp_min(1e-37), v)
    lse = (top + torch.log(total)).view(tokens, hq)
    return o.reshape(tokens, hq, dim).to(s["q"].dtype), lse


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    if case["op"] == "logits":
        rows, vocab = case["rows"], case["vocab"]
        masked = {"none": 0, "half": (rows + 1) // 2, "all": rows}[case["mask"]]
        b = rows * vocab * BYTES[case["dtype"]] + rows * _up(vocab, PAD) * 4
        b += sum(_totals(case)) * 4 + masked * _up(vocab, 32) // 8 + rows * min(case["bias"], vocab) * 8 + rows * 24
        return {"bytes": b, "flops": rows * vocab}
    seqs, each, dim, eb = case["seqs"], case["each"], case["dim"], BYTES[case["dtype"]]
    lens = _lengths(seqs, case["ctx"], each)
    ends = [max(0, n - each + 1 + i) for n in lens for i in range(each)]
    tokens = seqs * each
    if case["op"] == "score":
        heads = case["heads"]
        b = sum(lens) * (dim * eb + (4 if case["dtype"] == "e4m3" else 0)) + tokens * heads * (dim * eb + 4)
        b += tokens * _up(case["ctx"], PAD) * 2 + sum(-(-n // case["page"]) for n in lens) * 4 + tokens * 4
        return {"bytes": b, "flops": 2 * sum(ends) * heads * dim}
    block, take = case["block"], case["take"]
    # keys that a query reads: its own block up to itself, and whole blocks
    keys = [min(n, (take - 1) * block + (n - 1) % block + 1) if n else 0 for n in ends]
    # those of one request's tokens overlap: what all of them together reach
    once = 0
    for i, n in enumerate(lens):
        mine = keys[i * each: (i + 1) * each]
        miss = 1.0
        for k in mine:
            miss *= 1 - min(1.0, k / n)
        once += n * (1 - miss) if each > 1 else mine[0]
    b = once * case["kv_heads"] * dim * 2 * eb + tokens * (case["q_heads"] * (dim * 2 * eb + 4) + take * 4 + 4)
    return {"bytes": int(b), "flops": 4 * sum(keys) * case["q_heads"] * dim}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logits":
        return _exact_logits(s)
    if case["op"] == "score":
        return _exact_score(s)
    return _exact_attn(s)


def _exact_logits(s):
    rows, vocab = s["rows"], s["vocab"]
    out = torch.full((rows, _up(vocab, PAD)), float("-inf"), dtype=torch.float64, device="cuda")
    total, prompt = s["total_len"].tolist(), s["prompt_len"].tolist()
    mask_rows = s["mask_rows"].tolist() if "bitmask" in s else [-1] * rows
    for r in range(rows):
        x = s["logits"][r].double()
        text = s["tokens"][r, : total[r]].long()
        count = torch.bincount(text[prompt[r]:], minlength=vocab).double()
        seen = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        seen[text] = True
        rep = s["repetition"][r].double()
        x[seen] = torch.where(x[seen] > 0, x[seen] / rep, x[seen] * rep)
        x -= count * s["frequency"][r].double()
        x[count > 0] -= s["presence"][r].double()
        if "bias_ids" in s:
            a, b = s["bias_offsets"][r], s["bias_offsets"][r + 1]
            x.index_add_(0, s["bias_ids"][a:b].long(), s["bias_values"][a:b].double())
        if mask_rows[r] >= 0:
            words = s["bitmask"][mask_rows[r]].long() & 0xFFFFFFFF
            bits = (words[:, None] >> torch.arange(32, device="cuda")).bitwise_and(1).reshape(-1)[:vocab]
            x[bits == 0] = float("-inf")
        out[r, :vocab] = x
    return out


def _exact_score(s):
    seqs, each, heads, dim, page = (s[k] for k in ("seqs", "each", "heads", "dim", "page"))
    tokens = seqs * each
    out = torch.full((tokens, _up(s["ctx"], PAD)), float("-inf"), dtype=torch.float64, device="cuda")
    end = s["end"].tolist()
    step = max(1, (1 << 31) // (heads * s["ctx"] * 8))
    for b in range(seqs):
        n = max(end[b * each: (b + 1) * each])
        at = s["table"][b].long()
        keys = s["keys"][at].reshape(-1, dim)[:n].double()
        scale = s["key_scale"][at].reshape(-1)[:n].double() if "key_scale" in s else None
        for t in range(b * each, (b + 1) * each, step):
            u = min(t + step, (b + 1) * each)
            z = (s["q"][t:u].double().reshape(-1, dim) @ keys.T).clamp_min_(0).view(u - t, heads, n)
            z = torch.bmm(s["weights"][t:u, None].double(), z)[:, 0]
            if scale is not None:
                z = z * scale
            seen = torch.arange(n, device="cuda") < s["end"][t:u, None]
            out[t:u, :n] = z.masked_fill(~seen, float("-inf"))
    return out


def _exact_attn(s):
    tokens, hq, dim = s["q"].shape
    hk, page, block = s["kv_heads"], s["page"], s["block"]
    out = torch.zeros(tokens, hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((tokens, hq), float("-inf"), dtype=torch.float64, device="cuda")
    chosen, end = s["indices"].tolist(), s["end"].tolist()
    offsets = torch.arange(block)
    for t in range(tokens):
        mine = torch.tensor([i for i in chosen[t] if i >= 0], dtype=torch.long)
        pos = (mine[:, None] * block + offsets).reshape(-1)
        pos = pos[pos < end[t]].cuda()
        if pos.numel() == 0:
            continue
        row = s["table"][t if s["seq"] is None else t // s["each"]].long()
        k = s["k_cache"][row[pos // page], pos % page].double()
        v = s["v_cache"][row[pos // page], pos % page].double()
        q = s["q"][t].double().view(hk, hq // hk, dim)
        z = torch.bmm(q, k.permute(1, 2, 0)) / dim ** 0.5
        out[t] = torch.bmm(torch.softmax(z, -1), v.transpose(0, 1)).view(hq, dim)
        lse[t] = torch.logsumexp(z, -1).view(hq)
    return out, lse
