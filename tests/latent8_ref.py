"""Plain 64-bit forms of the latent-attention operators over the cache in 8 bits, and the error bounds of the
kernels, used by their tests.

Bounds (half steps relative to the value: bf16 2^-8, e4m3 2^-4, e5m2 2^-3, fp16 2^-11, fp32 2^-24):
  scores   a query row enters the products as two e4m3 in a unit 2^a for which its largest latent is in
           (224, 448]: together they hold a bf16 value exactly, but for what lies below half their last step,
           2^-10 2^a <= 2^-10 / 224 max|q| < 2^-17.8 max|q|. With the sums (576 + 512 terms, and 16 for scaling
           and exponent, a whole step 2^-23 each, as tensor cores may truncate):
           ds = scale (2^-17.8 max|q_lat| sum|k_lat| + 1104 2^-23 1.07 sum|q k|) + 2^-23 max|e|, k the value with
           its scale 2^e, which is added to the score's exponent
  weights  e^{s - M} is off by 2 ds + 2^-20. For the product with the stored values c = v / s_j the weight
           w = e^{s - M} s_j goes to fp16 and then into an e4m3 and, its remainder, an e5m2: off by at most
           2^-4 2^-3 w + 2^-11 w, and where w is below the e4m3's normal range (2^-6 in the row's unit) by 2^-10 2^-3,
           or half of e5m2's last step, 2^-17: 2^-12.9 of the unit in all. The unit is at most twice the largest
           weight of the current window of 4 tiles of 64 cached rows or of the one before it (a tile after each window
           whose largest is less than half of it, it is set to less than that largest), the windows counting from
           any tile: of the 9 tiles before a tile and the 3 behind it; and at least 2^-43 of the largest weight of all
  sums     2 n 2^-23 in all, n the keys
  o        |do| <= (2^-7 + 2^-11 + 4 ds + 2 n 2^-23 + 2^-18) sum p|v| / sum p
                   + 2^-11.9 sum_tiles (max(p s) of those tiles + 2^-42 of all) sum|c| / sum p + 2^-8 |o|
           (1.02 for second-order terms)
  lse      |d| <= ds + 2 n 2^-23 + 2^-20 + 2^-22 |lse|
"""
import torch

from tests import latent_ref as ref
from tests.latent_ref import LATENT, POS, ROW, STEP32, U_BF16

ROW8, TOKEN8, TOP, TILE = 640, 644, 448.0, 64


def parts(cache):
    """Views of the rows [pages, size, 640] and the scales [pages, size] of a cache [pages, size, 644]."""
    pages, size, token = cache.shape
    assert token == TOKEN8
    rows = cache.as_strided((pages, size, ROW8), (cache.stride(0), ROW8, 1))
    tail = cache.as_strided((pages, 4 * size), (cache.stride(0), 1), cache.storage_offset() + size * ROW8)
    return rows, tail.view(torch.float32)


def exponent(top):
    """Exponent of the scale of rows whose largest |latent| is `top` (fp64)."""
    m, e = torch.frexp(top / TOP)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(top == 0, torch.zeros_like(e), e.clamp(-40, 40))


def quantise(x):
    """fp32 rows [..., 576] as the bytes of rows [..., 640] and their scales."""
    x = x.float()
    e = exponent(x[..., :LATENT].abs().amax(-1).double())
    s = torch.ldexp(torch.ones(e.shape, device=x.device), e)
    y = x / s[..., None]
    return torch.cat([y[..., :LATENT].to(torch.float8_e4m3fn).view(torch.uint8),
                      y[..., LATENT:].contiguous().to(torch.bfloat16).view(torch.uint8)], -1), s


def codes(rows):
    """fp64 stored values of rows [..., 640], without the scale."""
    c = rows[..., :LATENT].contiguous().view(torch.float8_e4m3fn).double()
    return torch.cat([c, rows[..., LATENT:].contiguous().view(torch.bfloat16).double()], -1)


def fill(cache, x):
    """Write fp32 rows [pages, size, 576] into a cache."""
    rows, scales = parts(cache)
    b, s = quantise(x)
    rows.copy_(b)
    scales.copy_(s)
    return cache


def cached(cache, table, length, first=0):
    """Stored values and scales of rows first .. length - 1 of one sequence (fp64)."""
    size = cache.shape[1]
    rows, scales = parts(cache)
    i = torch.arange(first, length, device=cache.device)
    page = table.to(cache.device)[i // size].long()
    return codes(rows[page, i % size]), scales[page, i % size].double()


def attend(q, c, s, scale, seen):
    """A stack of query rows q [R, 576] (bf16) over stored values c [n, 576] with scales s [n], seen bool [R, n].
    Returns fp64 (o, lse, bound on |do| with its rounding, bound on |dlse|)."""
    q = q.double()
    R, n = q.shape[0], c.shape[0]
    if n == 0:
        z = torch.zeros(R, LATENT, dtype=torch.float64, device=q.device)
        ninf = torch.full((R,), float("-inf"), dtype=torch.float64, device=q.device)
        return z, ninf, torch.zeros_like(z), torch.zeros_like(ninf)
    k = c * s[:, None]
    x = torch.where(seen, scale * (q @ k.T), torch.full((), float("-inf"), dtype=torch.float64, device=q.device))
    part = 2.0 ** -17.8 * q[:, :LATENT].abs().amax(1, keepdim=True) * k[:, :LATENT].abs().sum(1)
    ds = scale * torch.where(seen, part + 1104 * 1.07 * STEP32 * (q.abs() @ k.abs().T), torch.zeros_like(x)).amax(1)
    ds = ds + STEP32 * s.log2().abs().amax()
    top = x.amax(1, keepdim=True)
    any_ = torch.isfinite(top)
    p = torch.exp(x - torch.where(any_, top, torch.zeros_like(top)))
    tot = p.sum(1, keepdim=True)
    safe = torch.where(any_, tot, torch.ones_like(tot))
    v = k[:, :LATENT]
    o, ab = (p @ v) / safe, (p @ v.abs()) / safe
    lse = (top + tot.log())[:, 0]
    pad = -n % TILE
    w = torch.nn.functional.pad(p * s, (0, pad)).view(R, -1, TILE).amax(2)
    size = torch.nn.functional.pad(c[:, :LATENT].abs(), (0, 0, 0, pad)).view(-1, TILE, LATENT).sum(1)
    near = torch.nn.functional.max_pool1d(torch.nn.functional.pad(w, (9, 3))[:, None], 13, 1)[:, 0]
    tiles = ((near + 2.0 ** -42 * w.amax(1, keepdim=True)) @ size) / safe
    cnt = seen.sum(1).double()
    bo = 1.02 * ((2.0 ** -7 + 2.0 ** -11 + 4 * ds + 2 * cnt * STEP32 + 2.0 ** -18)[:, None] * ab + 2.0 ** -11.9 * tiles +
                 U_BF16 * o.abs())
    bl = ds + 2 * cnt * STEP32 + 2.0 ** -20 + 2.0 ** -22 * torch.where(any_[:, 0], lse, torch.zeros_like(lse)).abs()
    return o, lse, bo, bl


def decode_ref(q_lat, q_pe, cache, table, lens, m, scale, n):
    """attend() of all rows (token, head) of sequence n: [m H, 512]."""
    length, H = int(lens[n]), q_lat.shape[1]
    c, s = cached(cache, table[n], length)
    q = torch.cat([q_lat[n * m:(n + 1) * m], q_pe[n * m:(n + 1) * m]], -1).reshape(m * H, ROW)
    t = torch.arange(m, device=q.device).repeat_interleave(H)[:, None]
    seen = torch.arange(length, device=q.device)[None] <= t + length - m
    return attend(q, c, s, scale, seen)


check_rows, make_pages, rotate_ref = ref.check_rows, ref.make_pages, ref.rotate_ref
