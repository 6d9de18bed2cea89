"""Cases of latent attention over a paged cache that is held in 8 bits.

The latent layers of a model that mixes them with KDA layers keep one row a token: 512
values of the shared latent and 64 of the shared positional key. In bf16 that is 1152 bytes;
here the latent is held in e4m3 with one scale a row, a power of two, and the positional key
in bf16 in units of that scale: 644 bytes, so that a step over a long context reads a little
more than half as much and a pool holds 1.8 times the tokens.

A page of `size` rows is size * 640 bytes of rows (512 of e4m3, then 64 bf16), then size fp32
scales. A serving loop writes rows as tokens come (kda_mla_append_fp8), reads them back as
dense bf16 rows for the expanded form, whole sequences or windows of them
(kda_mla_gather_fp8), and attends over the pages for one token a sequence or a window of
draft tokens (kda_mla_decode_fp8).

Each case names what it does in "op": "write" (quantise new rows into the pages and read
them back), "read", "decode". Lengths are ragged and follow from the case's "lens" seed, so
that the work of a case does not depend on the seed of its values.
"""
import random

import torch

own = False

LATENT = 512      # values of the shared latent a token
POS = 64          # values of the shared positional key a token
ROW = LATENT + POS
ROW_BYTES = LATENT + 2 * POS
TOKEN_BYTES = ROW_BYTES + 4
NOPE = 128        # head size of the expanded queries without position
SCALE = (NOPE + POS) ** -0.5
EPS = 1e-6
TOP = 448.0       # the largest e4m3 value
EXPONENTS = (-40, 40)  # of a row's scale


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # the rows of a prefilled batch, with the rotation of its 12 query heads
        dict(name="write 65536 x 12", op="write", seqs=8, heads=12, new=8192, context=16384, page=64, lens=-1, rope=True),
        # one row each of a full decode batch, all 96 heads
        dict(name="write 256 x 96", op="write", seqs=256, heads=96, new=1, context=4000, page=64, lens=9, rope=True),
        # ragged chunks of a mixed batch in layers without positions, odd pages
        dict(name="write 5 ragged", op="write", seqs=5, heads=1, new=1900, context=5000, page=48, lens=6, rope=False),
        # the cached rows of a batch of long contexts, for the expanded form
        dict(name="read 8 x 30000", op="read", seqs=8, context=30000, window=0, page=64, lens=2),
        # a window of each of three short prefixes
        dict(name="read 3 x 300", op="read", seqs=3, context=700, window=300, page=16, lens=4),
        # one token of a million-token context on one rank's 12 heads
        dict(name="decode 1M x 12", op="decode", seqs=1, heads=12, tokens=1, context=1048576, page=64, lens=-1),
        # a full batch of 256 sequences, all 96 heads, ragged contexts
        dict(name="decode 256 x 96", op="decode", seqs=256, heads=96, tokens=1, context=8000, page=64, lens=3),
        # a middling batch on one rank's heads
        dict(name="decode 32 x 16", op="decode", seqs=32, heads=16, tokens=1, context=8000, page=32, lens=8),
        # half of the heads on a rank, larger pages
        dict(name="decode 64 x 48", op="decode", seqs=64, heads=48, tokens=1, context=8000, page=128, lens=10),
        # a window of draft tokens of two short contexts: the latency of a verify step
        dict(name="verify 2 x 12 x 8", op="decode", seqs=2, heads=12, tokens=8, context=700, page=32, lens=5),
        # draft tokens of all heads: 384 query rows a sequence
        dict(name="verify 64 x 96 x 4", op="decode", seqs=64, heads=96, tokens=4, context=8000, page=64, lens=12),
        # one token behind one short prompt, where the call's latency counts
        dict(name="decode 1 x 12", op="decode", seqs=1, heads=12, tokens=1, context=500, page=16, lens=-1),
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "decode"])
    lens, page = rng.randrange(1 << 20), rng.choice([16, 32, 48, 64, 80, 128, 256])
    if op == "write":
        seqs = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, 65536 // seqs))
        return dict(op=op, seqs=seqs, heads=rng.choice([1, 5, 12, 16]), new=new, context=new + rng.randrange(2000),
                    page=page, lens=lens, rope=rng.random() < 0.6)
    if op == "read":
        seqs = _log(rng, 1, 200)
        context = _log(rng, 1, 240000 // seqs)
        return dict(op=op, seqs=seqs, context=context, window=rng.choice([0, 1 + rng.randrange(context)]), page=page,
                    lens=lens)
    heads = rng.choice([1, 2, 5, 12, 16, 24, 32, 33, 48, 64, 80, 96, 128])
    tokens = rng.choice([1, 1, 1, 2, 4, 7, 16])
    seqs = _log(rng, 1, 256)
    most = int(min((1000000 if seqs < 6 else 1500000) // seqs, 2.0e8 / (heads * tokens * seqs)))
    return dict(op=op, seqs=seqs, heads=heads, tokens=tokens, context=_log(rng, tokens, max(tokens + 1, most)), page=page,
                lens=lens)


def _ragged(n, most, seed, least=1):
    """n lengths of least .. most with their mean near the middle; seed -1: all of them most."""
    if seed < 0:
        return [most] * n
    r = random.Random(seed)
    return [r.randrange(min(least, most), most + 1) for _ in range(n)]


def _write_lens(case):
    """New tokens of each sequence, and its length with them."""
    new = _ragged(case["seqs"], case["new"], case["lens"])
    r = random.Random(case["lens"] + 1)
    return new, [a + r.randrange(max(1, case["context"] - case["new"] + 1)) for a in new]


def _read_lens(case):
    """First row and number of rows of each sequence: all of them, or a window that ends somewhere behind its middle."""
    lens = _ragged(case["seqs"], case["context"], case["lens"])
    if case["window"] == 0:
        return [0] * len(lens), lens
    r = random.Random(case["lens"] + 1)
    end = [r.randrange(n // 2, n + 1) for n in lens]
    count = [min(case["window"], n) for n in end]
    return [a - b for a, b in zip(end, count)], count


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


def _parts(cache):
    """The rows [pages, size, 640] and the scales [pages, size] of a cache [pages, size, 644]."""
    pages, size, _ = cache.shape
    flat = cache.view(pages, size * TOKEN_BYTES)
    return (flat[:, :size * ROW_BYTES].unflatten(1, (size, ROW_BYTES)),
            flat[:, size * ROW_BYTES:].view(torch.float32))


def _quantise(c, pe):
    """fp32 latents and positional keys as the bytes of their rows and their scales."""
    top = c.abs().amax(-1, keepdim=True)
    mantissa, e = torch.frexp(top / TOP)  # top / 448 = mantissa 2^e with mantissa in [0.5, 1)
    e = torch.where(top == 0, 0, torch.where(mantissa == 0.5, e - 1, e)).clamp_(*EXPONENTS)
    one = torch.ones((), device=c.device)
    low = (c * torch.ldexp(one, -e)).to(torch.float8_e4m3fn).view(torch.uint8)
    at = (pe * torch.ldexp(one, -e)).to(torch.bfloat16).view(torch.uint8)
    return torch.cat([low, at], -1), torch.ldexp(one, e)[..., 0]


def _values(rows, scales):
    """fp32 values of rows [..., 640] with scales [...]."""
    s = scales[..., None]
    c = rows[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float() * s
    return torch.cat([c, rows[..., LATENT:].contiguous().view(torch.bfloat16).float() * s], -1)


def _filled(gen, pages, page):
    """A cache whose rows hold normalised latents and positional keys."""
    cache = torch.empty(pages, page, TOKEN_BYTES, dtype=torch.uint8, device="cuda")
    rows, scales = _parts(cache)
    step = max(1, 262144 // page)
    weight = 1 + 0.1 * torch.randn(LATENT, generator=gen, device="cuda")
    for a in range(0, pages, step):
        x = torch.randn(min(step, pages - a), page, ROW, generator=gen, device="cuda")
        rows[a:a + step], scales[a:a + step] = _quantise(x[..., :LATENT] * weight, x[..., LATENT:])
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "write":
        new, lens = _write_lens(case)
        table, pages = _pages(gen, lens, case["page"])
        t = sum(new)
        down = _normal(gen, t, ROW)  # the down-projection of the tokens: latent, then positional key
        s.update(c=down[:, :LATENT], k_pe=down[:, LATENT:], q_pe=_normal(gen, t, case["heads"], NOPE + POS)[..., NOPE:],
                 norm_w=1 + 0.1 * torch.randn(LATENT, generator=gen, device="cuda"), cu=_ints(_cu(new)), lens=_ints(lens),
                 starts=_ints([b - a for a, b in zip(new, lens)]), table=table,
                 cache=torch.zeros(pages, case["page"], TOKEN_BYTES, dtype=torch.uint8, device="cuda"), rope=None)
        if case["rope"]:
            at = torch.arange(max(lens), device="cuda", dtype=torch.float64)
            rate = 10000.0 ** (-torch.arange(POS // 2, device="cuda", dtype=torch.float64) / (POS // 2))
            angle = at[:, None] * rate[None, :]
            s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    elif op == "read":
        starts, count = _read_lens(case)
        table, pages = _pages(gen, _ragged(case["seqs"], case["context"], case["lens"]), case["page"])
        s.update(cache=_filled(gen, pages, case["page"]), table=table, cu=_ints(_cu(count)), rows=sum(count),
                 starts=_ints(starts) if case["window"] else None)
    else:
        lens = _ragged(case["seqs"], case["context"], case["lens"], least=case["tokens"])
        table, pages = _pages(gen, lens, case["page"])
        rows = case["seqs"] * case["tokens"]
        s.update(q_lat=_normal(gen, rows, case["heads"], LATENT), q_pe=_normal(gen, rows, case["heads"], POS),
                 cache=_filled(gen, pages, case["page"]), table=table, lens=_ints(lens), tokens=case["tokens"])
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if own:
        from linear_attention_serving_02_gb300 import kda

        if op == "write":
            q_out = kda.kda_mla_append_fp8(s["c"], s["k_pe"], s["cache"], s["table"], s["lens"], s["cu"],
                                           norm_w=s["norm_w"], eps=EPS, rope=s["rope"],
                                           q_pe=s["q_pe"] if s["rope"] is not None else None)
            rows = kda.kda_mla_gather_fp8(s["cache"], s["table"], s["cu"], s["c"].shape[0], starts=s["starts"])
            return (rows, q_out) if q_out is not None else (rows,)
        if op == "read":
            return kda.kda_mla_gather_fp8(s["cache"], s["table"], s["cu"], s["rows"], starts=s["starts"])
        return kda.kda_mla_decode_fp8(s["q_lat"], s["q_pe"], s["cache"], s["table"], s["lens"], SCALE,
                                      num_tokens=s["tokens"])
    return {"write": _write, "read": _read, "decode": _decode}[op](s)


def _places(cu, first, total):
    """Sequence and row of each of the `total` rows of a packed batch whose sequences begin at row `first`."""
    i = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu.long()[1:], i, right=True)
    at = i - cu.long()[seq]
    return seq, at if first is None else at + first.long()[seq]


def _rotate(x, cos, sin):
    a, b = x[..., :POS // 2], x[..., POS // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _read_at(cache, table, seq, at):
    rows, scales = _parts(cache)
    size = cache.shape[1]
    page = table[seq, at // size].long()
    return _values(rows[page, at % size], scales[page, at % size])


def _write(s):
    seq, at = _places(s["cu"], s["starts"], s["c"].shape[0])
    c = s["c"].float()
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["norm_w"]
    k_pe, q = s["k_pe"].float(), None
    if s["rope"] is not None:
        cos, sin = s["rope"][at].split(POS // 2, -1)
        k_pe = _rotate(k_pe, cos, sin)
        q = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None]).to(torch.bfloat16)
    rows, scales = _parts(s["cache"])
    size = s["cache"].shape[1]
    page = s["table"][seq, at // size].long()
    rows[page, at % size], scales[page, at % size] = _quantise(c, k_pe)
    back = _read_at(s["cache"], s["table"], seq, at).to(torch.bfloat16)
    return (back, q) if q is not None else (back,)


def _read(s):
    seq, at = _places(s["cu"], s["starts"], s["rows"])
    return _read_at(s["cache"], s["table"], seq, at).to(torch.bfloat16)


def _decode(s):
    m, n = s["tokens"], s["lens"].shape[0]
    size = s["cache"].shape[1]
    most = s["table"].shape[1] * size
    i = torch.arange(most, device=s["lens"].device)
    seq = torch.arange(n, device=i.device)[:, None]
    k = _read_at(s["cache"], s["table"].clamp(min=0), seq, i[None])
    k.masked_fill_((i[None] >= s["lens"][:, None])[..., None], 0.0)
    q = torch.cat([s["q_lat"], s["q_pe"]], -1).float()
    h = q.shape[1]
    x = torch.matmul(q.view(n, m * h, ROW), k.transpose(-1, -2)).view(n, m, h, most)
    x *= SCALE
    seen = i < (s["lens"][:, None] - m + 1 + torch.arange(m, device=i.device))[..., None]
    x.masked_fill_(~seen[:, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(n, m * h, most), k[..., :LATENT]).view(n, m, h, LATENT)
    o = o / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0]
    return o.view(n * m, h, LATENT).to(torch.bfloat16), lse.view(n * m, h)


# ---------------------------------------------------------------------------- what a pass has to do
def work(case):
    op = case["op"]
    if op == "write":
        new, _ = _write_lens(case)
        t, h = sum(new), case["heads"]
        moved = 2 * t * ROW + 2 * t * TOKEN_BYTES + 2 * t * ROW  # read the input, write the rows, read them back, write them
        if case["rope"]:
            moved += 4 * t * POS + 2 * t * h * 2 * POS
        return {"bytes": moved, "flops": t * (7 * LATENT + (3 * POS * (1 + h) if case["rope"] else 0))}
    if op == "read":
        return {"bytes": (TOKEN_BYTES + 2 * ROW) * sum(_read_lens(case)[1]), "flops": 0}
    lens = _ragged(case["seqs"], case["context"], case["lens"], least=case["tokens"])
    m, h, n = case["tokens"], case["heads"], case["seqs"]
    pairs = sum(m * x - m * (m - 1) // 2 for x in lens)
    return {"bytes": sum(lens) * TOKEN_BYTES + n * m * h * (2 * (ROW + LATENT) + 4), "flops": 2 * pairs * h * (ROW + LATENT)}


# ---------------------------------------------------------------------------- the definition in 64 bits
def _e4m3(x):
    """64-bit values at the nearest e4m3 value, ties to the even one (none is past the largest)."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-5) - 4)
    return torch.round(x / step) * step


def _stands_for(byte):
    """The 64-bit values of e4m3 bytes."""
    b = torch.arange(256, dtype=torch.float64, device=byte.device)
    mantissa, e = b % 8, (b // 8) % 16
    value = torch.where(e == 0, mantissa / 8 * 2.0 ** -6, (1 + mantissa / 8) * 2.0 ** (e - 7))
    return torch.where(b >= 128, -value, value)[byte.long()]


def _sequence(cache, pages, length):
    """The 64-bit rows of one sequence."""
    size = cache.shape[1]
    flat = cache[pages.long()].reshape(pages.numel(), size * TOKEN_BYTES)
    rows = flat[:, :size * ROW_BYTES].reshape(-1, ROW_BYTES)[:length]
    scale = flat[:, size * ROW_BYTES:].contiguous().view(torch.float32).reshape(-1, 1)[:length].double()
    at = rows[:, LATENT:].contiguous().view(torch.bfloat16).double()
    return torch.cat([_stands_for(rows[:, :LATENT]), at], 1) * scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    size = case["page"]
    if op == "write":
        cu = s["cu"].tolist()
        c = s["c"].double()
        c = s["norm_w"].double() * c / (c.pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt()
        e = torch.ceil(torch.log2(c.abs().amax(1, keepdim=True) / TOP)).clamp(*EXPONENTS)
        c = _e4m3(c / 2.0 ** e) * 2.0 ** e
        turned = {"k": s["k_pe"].double()[:, None], "q": s["q_pe"].double()}
        if not case["rope"]:
            return (torch.cat([c, turned["k"][:, 0]], 1),)
        q, pe = torch.empty_like(turned["q"]), torch.empty_like(turned["k"][:, 0])
        for n, length in enumerate(s["lens"].tolist()):
            a, b = cu[n], cu[n + 1]
            turn = s["rope"][length - (b - a):length].double()
            turn = torch.complex(turn[:, :POS // 2], turn[:, POS // 2:])[:, None]
            for name, x in turned.items():
                z = torch.complex(x[a:b, :, :POS // 2], x[a:b, :, POS // 2:]) * turn
                z = torch.cat([z.real, z.imag], -1)
                if name == "q":
                    q[a:b] = z
                else:
                    pe[a:b] = z[:, 0]
        return torch.cat([c, pe], 1), q
    if op == "read":
        starts, count = _read_lens(case)
        out = []
        for n, (a, k) in enumerate(zip(starts, count)):
            out.append(_sequence(s["cache"], s["table"][n, :(a + k + size - 1) // size], a + k)[a:])
        return torch.cat(out)
    m = case["tokens"]
    o = torch.empty(s["q_lat"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(o.shape[:2], dtype=torch.float64, device="cuda")
    for n, length in enumerate(s["lens"].tolist()):
        rows = _sequence(s["cache"], s["table"][n, :(length + size - 1) // size], length)
        for t in range(m):
            end, r = length - m + 1 + t, n * m + t
            q = torch.cat([s["q_lat"][r], s["q_pe"][r]], -1).double()
            x = SCALE * (q @ rows[:end].T)
            lse[r] = torch.logsumexp(x, 1)
            o[r] = torch.exp(x - lse[r, :, None]) @ rows[:end, :LATENT]
    return o, lse
