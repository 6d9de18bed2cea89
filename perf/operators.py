"""Cases of the latent-attention serving operators and of the page copies.

A serving loop of a model that mixes KDA layers with latent-attention layers keeps, for
each latent layer, one row of 576 bf16 values a token (512 of the shared latent, 64 of the
shared positional key) in pages. It appends rows (kda_mla_append), reads them back as dense
rows for the expanded form (kda_mla_gather), attends in the expanded form over whole
sequences (kda_mla_prefill) and in the absorbed form over the pages for one token or a
window of draft tokens (kda_mla_decode), and copies pages when it forks or compacts
(kda_pages_copy).

Each case names its operator in "op"; lengths are ragged and follow from the case's "lens"
seed, so that the work of a case does not depend on the seed of its values.
"""
import random

import torch

own = False

LATENT = 512      # values of the shared latent a token
POS = 64          # values of the shared positional key a token
ROW = LATENT + POS
NOPE = 128        # head size of the expanded keys without position, and of the values
QK = NOPE + POS   # head size of the expanded queries
SCALE = QK ** -0.5
EPS = 1e-6


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # expanded prefill of one fresh sequence, the repository's single-sequence size
        dict(name="prefill 8192 x 12", op="prefill", seqs=1, heads=12, new=8192, prefix=0, lens=-1, causal=True),
        # chunked prefill of a mixed batch: ragged new tokens behind ragged cached prefixes
        dict(name="prefill ragged x 32", op="prefill", seqs=5, heads=32, new=2000, prefix=3900, lens=7, causal=True),
        # the smallest prompt, where the call's latency counts
        dict(name="prefill 256 x 2", op="prefill", seqs=1, heads=2, new=256, prefix=0, lens=-1, causal=True),
        # one token of a million-token context on one rank's 12 heads
        dict(name="decode 1M x 12", op="decode", seqs=1, heads=12, tokens=1, context=1048576, page=64, lens=-1),
        # a full batch of 256 sequences, all 96 heads, ragged contexts
        dict(name="decode 256 x 96", op="decode", seqs=256, heads=96, tokens=1, context=8000, page=64, lens=3),
        # a window of draft tokens of two short contexts: the latency of a verify step
        dict(name="verify 2 x 12 x 8", op="decode", seqs=2, heads=12, tokens=8, context=700, page=32, lens=5),
        # rows of a prefilled batch with the rotation of its 12 query heads
        dict(name="append 65536 x 12", op="append", seqs=8, heads=12, new=8192, context=16384, page=64, lens=-1,
             rope=True),
        # one row each of a full decode batch
        dict(name="append 256 x 96", op="append", seqs=256, heads=96, new=1, context=4000, page=64, lens=9, rope=True),
        # the cached rows of a batch of long contexts, for the expanded form
        dict(name="gather 8 x 30000", op="gather", seqs=8, context=30000, page=64, lens=2),
        # a short prefix read back
        dict(name="gather 3 x 300", op="gather", seqs=3, context=300, page=16, lens=4),
        # compaction: a fifth of the pages of 24 layers move
        dict(name="compact 200 x 24", op="copy", layers=24, pages=1000, pairs=200, page=64),
        # a fork: the last page of one sequence in 24 layers
        dict(name="fork 1 x 24", op="copy", layers=24, pages=200, pairs=1, page=64),
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prefill", "decode", "decode", "append", "gather", "copy"])
    lens = rng.randrange(1 << 20)
    if op == "prefill":
        heads = rng.choice([1, 2, 3, 8, 12, 32, 96])
        seqs = _log(rng, 1, 8)
        most = max(16, int((2.0e8 / heads / seqs) ** 0.5))
        new = _log(rng, 1, min(8192, most))
        prefix = rng.choice([0, rng.randrange(min(8192, most))])
        return dict(op=op, seqs=seqs, heads=heads, new=new, prefix=prefix, lens=lens, causal=rng.random() < 0.75)
    if op == "decode":
        heads = rng.choice([1, 2, 5, 12, 16, 24, 32, 48, 64, 96, 128])
        tokens = rng.choice([1, 1, 1, 2, 4, 7, 16])
        seqs = _log(rng, 1, 256)
        most = int(min((1000000 if seqs < 6 else 1500000) // seqs, 2.0e8 / (heads * tokens * seqs)))
        return dict(op=op, seqs=seqs, heads=heads, tokens=tokens, context=_log(rng, tokens, max(tokens + 1, most)),
                    page=rng.choice([16, 32, 48, 64, 128, 256]), lens=lens)
    if op == "append":
        seqs = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, 65536 // seqs))
        return dict(op=op, seqs=seqs, heads=rng.choice([1, 5, 12, 16]), new=new,
                    context=new + rng.randrange(2000), page=rng.choice([16, 32, 48, 64, 128, 256]), lens=lens,
                    rope=rng.random() < 0.5)
    if op == "gather":
        seqs = _log(rng, 1, 200)
        return dict(op=op, seqs=seqs, context=_log(rng, 1, 240000 // seqs), page=rng.choice([16, 32, 48, 64, 128, 256]),
                    lens=lens)
    page = rng.choice([16, 64, 64, 128])
    pairs = _log(rng, 1, 12000 // page)
    return dict(op=op, layers=rng.choice([1, 3, 12, 24]), pages=2 * pairs + rng.randrange(1, 200), pairs=pairs, page=page)


def _ragged(n, most, seed, least=1):
    """n lengths of least .. most with their mean near the middle; seed -1: all of them most."""
    if seed < 0:
        return [most] * n
    r = random.Random(seed)
    return [r.randrange(min(least, most), most + 1) for _ in range(n)]


def _prefill_lens(case):
    new = _ragged(case["seqs"], case["new"], case["lens"])
    prefix = _ragged(case["seqs"], case["prefix"], case["lens"] + 1 if case["lens"] >= 0 else -1, least=0)
    return new, [a + b for a, b in zip(new, prefix)]


def _append_lens(case):
    new = _ragged(case["seqs"], case["new"], case["lens"])
    r = random.Random(case["lens"] + 1)
    return new, [a + r.randrange(max(1, case["context"] - case["new"] + 1)) for a in new]


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ---------------------------------------------------------------------------- the inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _pages(gen, lens, page):
    """A page table [seqs, most pages] in a shuffled order and the number of pages; -1 where a sequence has no page."""
    need = [(n + page - 1) // page for n in lens]
    total = sum(need)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
    return table, total


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "prefill":
        new, total = _prefill_lens(case)
        tq, tk, h = sum(new), sum(total), case["heads"]
        s.update(q=_normal(gen, tq, h, QK), kv=_normal(gen, tk, h, 2 * NOPE), k_pe=_normal(gen, tk, ROW)[:, LATENT:],
                 cu_q=_ints(_cu(new)), cu_k=_ints(_cu(total)), causal=case["causal"], most_q=max(new),
                 most_k=max(total))
    elif op == "decode":
        lens = _ragged(case["seqs"], case["context"], case["lens"], least=case["tokens"])
        table, pages = _pages(gen, lens, case["page"])
        rows = case["seqs"] * case["tokens"]
        s.update(q_lat=_normal(gen, rows, case["heads"], LATENT), q_pe=_normal(gen, rows, case["heads"], POS),
                 cache=_normal(gen, pages, case["page"], ROW), table=table, lens=_ints(lens), tokens=case["tokens"])
    elif op == "append":
        new, lens = _append_lens(case)
        table, pages = _pages(gen, lens, case["page"])
        t = sum(new)
        down = _normal(gen, t, ROW)  # the down-projection of the tokens: latent, then positional key
        s.update(c=down[:, :LATENT], k_pe=down[:, LATENT:], q_pe=_normal(gen, t, case["heads"], QK)[..., NOPE:],
                 norm_w=1 + 0.1 * torch.randn(LATENT, generator=gen, device="cuda"), cu=_ints(_cu(new)),
                 lens=_ints(lens), table=table, cache=_normal(gen, pages, case["page"], ROW), rope=None)
        if case["rope"]:
            at = torch.arange(max(lens), device="cuda", dtype=torch.float64)
            rate = 10000.0 ** (-torch.arange(POS // 2, device="cuda", dtype=torch.float64) / (POS // 2))
            angle = at[:, None] * rate[None, :]
            s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    elif op == "gather":
        lens = _ragged(case["seqs"], case["context"], case["lens"])
        table, pages = _pages(gen, lens, case["page"])
        s.update(cache=_normal(gen, pages, case["page"], ROW), table=table, cu=_ints(_cu(lens)), rows=sum(lens))
    else:
        order = torch.randperm(case["pages"], generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        s.update(pool=_normal(gen, case["layers"], case["pages"], case["page"], ROW), src=order[:case["pairs"]].clone(),
                 dst=order[case["pairs"]:2 * case["pairs"]].clone())
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if own:
        from linear_attention_serving_02_gb300 import kda

        if op == "prefill":
            return kda.kda_mla_prefill(s["q"], s["kv"], s["k_pe"], s["cu_q"], s["cu_k"], SCALE, causal=s["causal"])
        if op == "decode":
            return kda.kda_mla_decode(s["q_lat"], s["q_pe"], s["cache"], s["table"], s["lens"], SCALE,
                                      num_tokens=s["tokens"])
        if op == "append":
            q_out = kda.kda_mla_append(s["c"], s["k_pe"], s["cache"], s["table"], s["lens"], s["cu"],
                                       norm_w=s["norm_w"], eps=EPS, rope=s["rope"],
                                       q_pe=s["q_pe"] if s["rope"] is not None else None)
            return (s["cache"], q_out) if q_out is not None else (s["cache"],)
        if op == "gather":
            return kda.kda_mla_gather(s["cache"], s["table"], s["cu"], s["rows"])
        kda.kda_pages_copy(s["pool"], s["src"], s["dst"])
        return s["pool"]
    return {"prefill": _prefill, "decode": _decode, "append": _append, "gather": _gather, "copy": _copy}[op](s)


def _at(cu, most):
    """Rows of a packed batch as a padded one: indices [seqs, most] and which of them exist."""
    i = torch.arange(most, device=cu.device)
    there = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None].long() + i[None, :], 0), there


def _softmax(x):
    """exp(x - max) and its sum over the last axis, and the maximum; a row of -inf alone gives zeros."""
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    return x, x.sum(-1, keepdim=True), top


def _prefill(s):
    q_at, q_there = _at(s["cu_q"], s["most_q"])
    k_at, k_there = _at(s["cu_k"], s["most_k"])
    q = s["q"][q_at].float().transpose(1, 2)                      # [seqs, H, Lq, 192]
    kv = s["kv"][k_at].float().transpose(1, 2)                    # [seqs, H, Lk, 256]
    kv = torch.where(k_there[:, None, :, None], kv, 0.0)
    k_pe = s["k_pe"][k_at].float()[:, None]                       # [seqs, 1, Lk, 64]
    x = torch.matmul(q[..., :NOPE], kv[..., :NOPE].transpose(-1, -2))
    x += torch.matmul(q[..., NOPE:], k_pe.transpose(-1, -2))
    x *= SCALE
    seen = k_there[:, None, :].expand(-1, s["most_q"], -1)
    if s["causal"]:
        n_q, n_k = s["cu_q"][1:] - s["cu_q"][:-1], s["cu_k"][1:] - s["cu_k"][:-1]
        last = torch.arange(s["most_q"], device=x.device)[None, :] + (n_k - n_q)[:, None]
        seen = seen & (torch.arange(s["most_k"], device=x.device) <= last[..., None])
    x.masked_fill_(~seen[:, None], float("-inf"))
    p, total, top = _softmax(x)
    o = torch.matmul(p, kv[..., NOPE:]) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0]
    return o.transpose(1, 2)[q_there].to(torch.bfloat16), lse.transpose(1, 2)[q_there]


def _cached(cache, table, most):
    """Rows 0 .. most - 1 of each sequence, [seqs, most, 576], from its pages."""
    i = torch.arange(most, device=cache.device)
    page = table[:, i // cache.shape[1]].long().clamp_(min=0)
    return cache[page, (i % cache.shape[1])[None, :]]


def _decode(s):
    m, n = s["tokens"], s["lens"].shape[0]
    most = s["table"].shape[1] * s["cache"].shape[1]
    there = torch.arange(most, device=s["lens"].device)[None, :] < s["lens"][:, None]
    k = torch.where(there[..., None], _cached(s["cache"], s["table"], most).float(), 0.0)
    q = torch.cat([s["q_lat"], s["q_pe"]], -1).float()
    h = q.shape[1]
    x = torch.matmul(q.view(n, m * h, ROW), k.transpose(-1, -2)).view(n, m, h, most)
    x *= SCALE
    seen = torch.arange(most, device=x.device) < (s["lens"][:, None] - m + 1 + torch.arange(m, device=x.device))[..., None]
    x.masked_fill_(~seen[:, :, None], float("-inf"))
    p, total, top = _softmax(x)
    o = torch.matmul(p.view(n, m * h, most), k[..., :LATENT]).view(n, m, h, LATENT)
    o = o / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0]
    return o.view(n * m, h, LATENT).to(torch.bfloat16), lse.view(n * m, h)


def _rotate(x, cos, sin):
    a, b = x[..., :POS // 2], x[..., POS // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append(s):
    n_new = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(n_new.shape[0], device=n_new.device), n_new, output_size=s["c"].shape[0])
    at = (s["lens"] - s["cu"][1:])[seq] + torch.arange(seq.shape[0], device=seq.device)
    c = s["c"].float()
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["norm_w"]
    k_pe, q = s["k_pe"].float(), None
    if s["rope"] is not None:
        cos, sin = s["rope"][at].split(POS // 2, -1)
        k_pe = _rotate(k_pe, cos, sin)
        q = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None]).to(torch.bfloat16)
    size = s["cache"].shape[1]
    s["cache"][s["table"][seq, at // size].long(), at % size] = torch.cat([c, k_pe], -1).to(torch.bfloat16)
    return (s["cache"], q) if q is not None else (s["cache"],)


def _gather(s):
    i = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["cu"].long()[1:], i, right=True)
    at = i - s["cu"].long()[seq]
    size = s["cache"].shape[1]
    return s["cache"][s["table"][seq, at // size].long(), at % size]


def _copy(s):
    dst, src = s["dst"].to("cuda").long(), s["src"].to("cuda").long()
    s["pool"][:, dst] = s["pool"][:, src]
    return s["pool"]


# ---------------------------------------------------------------------------- what a pass has to do
def work(case):
    op = case["op"]
    if op == "prefill":
        new, total = _prefill_lens(case)
        h, tq, tk = case["heads"], sum(new), sum(total)
        pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(new, total))
        return {"bytes": 2 * (tq * h * (QK + NOPE) + tk * (h * 2 * NOPE + POS)) + 4 * tq * h,
                "flops": 2 * pairs * h * (QK + NOPE)}
    if op == "decode":
        lens = _ragged(case["seqs"], case["context"], case["lens"], least=case["tokens"])
        m, h, n = case["tokens"], case["heads"], case["seqs"]
        pairs = sum(m * x - m * (m - 1) // 2 for x in lens)
        return {"bytes": 2 * sum(lens) * ROW + n * m * h * (2 * (ROW + LATENT) + 4), "flops": 2 * pairs * h * (ROW + LATENT)}
    if op == "append":
        new, _ = _append_lens(case)
        t = sum(new)
        if not case["rope"]:
            return {"bytes": 2 * t * 2 * ROW, "flops": 5 * t * LATENT}
        return {"bytes": 2 * t * 2 * ROW + t * 4 * POS + 2 * t * case["heads"] * 2 * POS,
                "flops": t * (5 * LATENT + 3 * POS * (1 + case["heads"]))}
    if op == "gather":
        return {"bytes": 2 * 2 * ROW * sum(_ragged(case["seqs"], case["context"], case["lens"])), "flops": 0}
    return {"bytes": 2 * 2 * case["layers"] * case["pairs"] * case["page"] * ROW, "flops": 0}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":
        cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
        o = torch.empty(s["q"].shape[0], case["heads"], NOPE, dtype=torch.float64, device="cuda")
        lse = torch.empty(o.shape[:2], dtype=torch.float64, device="cuda")
        for n in range(case["seqs"]):
            a, b, c, d = cu_q[n], cu_q[n + 1], cu_k[n], cu_k[n + 1]
            for h in range(case["heads"]):
                k = torch.cat([s["kv"][c:d, h, :NOPE], s["k_pe"][c:d]], 1).double()
                x = SCALE * (s["q"][a:b, h].double() @ k.T)
                if case["causal"]:
                    x += torch.full_like(x, float("-inf")).triu(d - c - (b - a) + 1)
                lse[a:b, h] = torch.logsumexp(x, 1)
                o[a:b, h] = torch.exp(x - lse[a:b, h, None]) @ s["kv"][c:d, h, NOPE:].double()
        return o, lse
    if op == "decode":
        m, size = case["tokens"], case["page"]
        o = torch.empty(s["q_lat"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(o.shape[:2], dtype=torch.float64, device="cuda")
        for n, length in enumerate(s["lens"].tolist()):
            pages = s["table"][n, :(length + size - 1) // size].long()
            rows = s["cache"][pages].reshape(-1, ROW)[:length].double()
            for t in range(m):
                end, r = length - m + 1 + t, n * m + t
                x = SCALE * (s["q_lat"][r].double() @ rows[:end, :LATENT].T + s["q_pe"][r].double() @ rows[:end, LATENT:].T)
                lse[r] = torch.logsumexp(x, 1)
                o[r] = torch.exp(x - lse[r, :, None]) @ rows[:end, :LATENT]
        return o, lse
    if op == "append":
        cache, cu, size = s["cache"].double(), s["cu"].tolist(), case["page"]
        c = s["c"].double()
        c = s["norm_w"].double() * c / (c.pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt()
        turned = {"k": s["k_pe"].double()[:, None], "q": s["q_pe"].double()}
        q = torch.empty(s["q_pe"].shape, dtype=torch.float64, device="cuda")
        for n, length in enumerate(s["lens"].tolist()):
            a, b = cu[n], cu[n + 1]
            at = torch.arange(length - (b - a), length, device="cuda")
            pe = turned["k"][a:b, 0]
            if case["rope"]:
                turn = torch.complex(s["rope"][at, :POS // 2].double(), s["rope"][at, POS // 2:].double())[:, None]
                got = {}
                for name, x in turned.items():
                    z = torch.complex(x[a:b, :, :POS // 2], x[a:b, :, POS // 2:]) * turn
                    got[name] = torch.cat([z.real, z.imag], -1)
                pe, q[a:b] = got["k"][:, 0], got["q"]
            cache[s["table"][n][at // size].long(), at % size] = torch.cat([c[a:b], pe], 1)
        return (cache, q) if case["rope"] else (cache,)
    if op == "gather":
        rows = []
        for n in range(case["seqs"]):
            length = int(s["cu"][n + 1] - s["cu"][n])
            rows.append(s["cache"][s["table"][n].clamp(min=0).long()].reshape(-1, ROW)[:length])
        return torch.cat(rows).double()
    pool = s["pool"].double()
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        pool[:, b] = pool[:, a]
    return pool
