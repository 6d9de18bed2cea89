"""Plain 64-bit forms of the latent-attention operators and the error bounds of the kernels,
used by the GPU tests.

Bounds (u = half a step of a type: bf16 2^-8, fp32 2^-24, relative to the value):
  scores   products of bf16 values are exact in fp32 and d = 192 or 576 of them are summed in
           fp32, each addition off by at most a whole step 2^-23 (tensor cores may truncate):
           |ds| <= ds = (d + 16) 2^-23 scale sum|q k|, the 16 for scaling and exponent
  p        e^{s - M} is off by 2 ds (numerator and maximum) + 2^-20 (the exponential), and by
           bf16's 2^-8 where it multiplies the values
  sums     of n terms in fp32: n 2^-23 at most, for the denominator and each output; the join of
           parts adds the like, so 2 n 2^-23 in all (n counts keys)
  o        |do| <= (2^-8 + 4 ds + 2 n 2^-23 + 2^-18) sum p|v| / sum p, then 2^-8 |o| of its rounding
           (second-order terms are covered by the factor 1.02)
  lse      |d| <= ds + 2 n 2^-23 + 2^-20 + 2^-22 |lse|
"""
import torch

U_BF16, STEP32 = 2.0 ** -8, 2.0 ** -23
LATENT, POS, ROW, NOPE, QK = 512, 64, 576, 128, 192


def attend(q, k, v, scale, seen):
    """One head or a stack of rows: q [R, d], k [n, d], v [n, e] in bf16, seen bool [R, n]. Returns fp64
    (o, lse, bound on |do| with bf16 rounding, bound on |dlse|). A row that sees nothing gives 0, -inf."""
    q, k, v = q.double(), k.double(), v.double()
    R, n = q.shape[0], k.shape[0]
    if n == 0:
        z = torch.zeros(R, v.shape[1], dtype=torch.float64, device=q.device)
        ninf = torch.full((R,), float("-inf"), dtype=torch.float64, device=q.device)
        return z, ninf, torch.zeros_like(z), torch.zeros_like(ninf)
    s = scale * (q @ k.T)
    s = torch.where(seen, s, torch.full_like(s, float("-inf")))
    ds = (q.shape[1] + 16) * STEP32 * scale * torch.where(seen, q.abs() @ k.abs().T, torch.zeros_like(s)).amax(1)
    top = s.amax(1, keepdim=True)
    any_ = torch.isfinite(top)
    p = torch.exp(s - torch.where(any_, top, torch.zeros_like(top)))
    tot = p.sum(1, keepdim=True)
    safe = torch.where(any_, tot, torch.ones_like(tot))
    o, ab = (p @ v) / safe, (p @ v.abs()) / safe
    lse = (top + tot.log())[:, 0]
    cnt = seen.sum(1).double()
    bo = 1.02 * ((U_BF16 + 4 * ds + 2 * cnt * STEP32 + 2.0 ** -18)[:, None] * ab + U_BF16 * o.abs())
    bl = ds + 2 * cnt * STEP32 + 2.0 ** -20 + 2.0 ** -22 * torch.where(any_[:, 0], lse, torch.zeros_like(lse)).abs()
    return o, lse, bo, bl


def check_rows(o, lse, ref):
    """Kernel rows o (bf16), lse (fp32) against attend()'s answer."""
    ro, rl, bo, bl = ref
    d = (o.double() - ro).abs()
    assert bool((d <= bo + 1e-30).all()), "o off by %.3e (allowed there %.3e)" % (
        float((d - bo).max()), float(bo.flatten()[(d - bo).argmax()]))
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none)
    dl = torch.where(none, torch.zeros_like(rl), (lse.double() - rl).abs())
    assert bool((dl <= bl).all()), "lse off by %.3e" % float((dl - bl).max())


def prefill_ref(q, kv, k_pe, cu_q, cu_k, scale, causal, n, h):
    """attend() of head h of sequence n of a packed batch."""
    a, b, c, d = cu_q[n], cu_q[n + 1], cu_k[n], cu_k[n + 1]
    k = torch.cat([kv[c:d, h, :NOPE], k_pe[c:d]], 1)
    i, j = torch.arange(b - a, device=q.device)[:, None], torch.arange(d - c, device=q.device)[None]
    seen = (j <= i + (d - c) - (b - a)) if causal else (j >= 0).expand(b - a, d - c)
    return attend(q[a:b, h], k, kv[c:d, h, NOPE:], scale, seen)


def cached_rows(cache, table, length):
    """Rows 0 .. length - 1 of one sequence."""
    size = cache.shape[1]
    pages = table[:(length + size - 1) // size].long()
    return cache[pages].reshape(-1, ROW)[:length]


def decode_ref(q_lat, q_pe, cache, table, lens, m, scale, n):
    """attend() of all rows (token, head) of sequence n: [m H, 512]."""
    length, H = int(lens[n]), q_lat.shape[1]
    rows = cached_rows(cache, table[n], length)
    q = torch.cat([q_lat[n * m:(n + 1) * m], q_pe[n * m:(n + 1) * m]], -1).reshape(m * H, ROW)
    t = torch.arange(m, device=q.device).repeat_interleave(H)[:, None]
    seen = torch.arange(length, device=q.device)[None] <= t + length - m
    return attend(q, rows, rows[:, :LATENT], scale, seen)


def rotate_ref(x, cos, sin, interleaved):
    """x [..., 64] fp64, cos / sin broadcastable [..., 32]."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y, z = a * cos - b * sin, b * cos + a * sin
    return torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)


def make_pages(gen, lens, size, extra=2, garbage=True):
    """A page table of shuffled distinct pages for lens, its unused entries out of range, and the
    number of pages."""
    need = [(max(0, n) + size - 1) // size for n in lens]
    total = sum(need) + extra
    order = torch.randperm(total, generator=gen).to(torch.int32)
    bad = [-1, -2147483648, total, 2147483647]
    table = torch.empty((len(lens), max(need + [0]) + 1), dtype=torch.int32)
    at = 0
    for n, k in enumerate(need):
        table[n] = bad[n % 4] if garbage else -1
        table[n, :k] = order[at:at + k]
        at += k
    return table, total
