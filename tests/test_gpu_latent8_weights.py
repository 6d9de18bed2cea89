"""Latent attention over the 8-bit cache where a few keys outweigh all others: what the others carry keeps its bits.

The bound. A weight w = p s (s the row's scale) is held in a unit u of its query row as fp16, e4m3 and, its remainder,
e5m2. From 2^-6 u on the e4m3 is off by at most half of its last step, 2^-4 of w's power of two, and the e5m2 by half
of its own, so by 2^-8 w in all; below, the e4m3 is a multiple of 2^-9 u, the remainder at most 2^-10 u, and its e5m2 off by at
most 2^-14 u. fp16 adds 2^-11 w, or 2^-25 u. The unit is set anew by a tile whose largest weight is above it (to 2^-6 of
that), by a stretch's first tile (2^-2.5), behind low weights (2^-2.5 of the tile's largest or 2^-7 of four tiles' sum), and else
stays for the next tiles only where four tiles' weights sum to 8 u. Each of these happened in the 9 tiles up to a weight's own,
so there u <= max(2^-2.5 w, sum of w over 4 tiles / 8). The first 8 rows of a sequence count 2^-6.2 of theirs in its first tile. The
unit stays above 2^-40 of the largest weight of all (2^-46.2 of those rows'), which adds 2^-53 of it.
Scores, sums and roundings are as in tests/latent8_ref.py, whose own term for low weights (2^-11.9 of the largest one near,
counted for all 64 rows of a tile) follows from a unit held by the largest weight of four tiles: the outputs that it is used
for stay within it, but what the kernel promises is the bound here."""
import math

import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent8_ref as ref
from tests.test_gpu_latent import LATENT, NAN, POS, ROW, SCALE, _gen, _ints, _status
from tests.test_gpu_latent8 import _cache

pytestmark = pytest.mark.gpu

TILE, EARLY = 64, 8


def _bounds(q, c, s, scale):
    """ref.attend() of query rows that see all n rows, with the bound on |do| from above."""
    n = c.shape[0]
    seen = torch.ones(q.shape[0], n, dtype=torch.bool, device=q.device)
    o, lse, _, bl = ref.attend(q, c, s, scale, seen)
    q, k, v = q.double(), c * s[:, None], (c * s[:, None])[:, :LATENT]
    p = torch.softmax(scale * (q @ k.T), 1)
    part = 2.0 ** -17.8 * q[:, :LATENT].abs().amax(1, keepdim=True) * k[:, :LATENT].abs().sum(1)
    ds = scale * (part + 1104 * 1.07 * ref.STEP32 * (q.abs() @ k.abs().T)).amax(1) + ref.STEP32 * s.log2().abs().amax()
    w = p * s
    counted = w.clone()
    counted[:, :EARLY] *= 2.0 ** -6.2
    counted = torch.nn.functional.pad(counted, (0, -n % TILE)).view(q.shape[0], -1, TILE)

    def last(x, tiles, of):  # over `tiles` tiles up to each one
        return of(torch.nn.functional.pad(x, (tiles - 1, 0)).unfold(1, tiles, 1))

    four = last(counted.sum(2), 4, lambda x: x.sum(2))
    u = torch.maximum(last(four, 9, lambda x: x.amax(2)) / 8, 2.0 ** -2.5 * last(counted.amax(2), 9, lambda x: x.amax(2)))
    u = u.repeat_interleave(TILE, 1)[:, :n]
    dw = torch.maximum(2.0 ** -8 * w, (2.0 ** -14 + 2.0 ** -25) * u) + 2.0 ** -11 * w + 2.0 ** -53 * w.amax(1, keepdim=True)
    # (the probabilities themselves, times the values, carry the scores' errors)
    bo = 1.02 * ((4 * ds + 2 * n * ref.STEP32 + 2.0 ** -18)[:, None] * (p @ v.abs()) + dw @ c[:, :LATENT].abs() +
                 ref.U_BF16 * o.abs())
    return o, lse, bo, bl


def _mixed(n):
    return torch.rand(n, generator=_gen(9)) * 3 - 3


# scores by row, and the rows that outweigh the others
def _sinks(share, count=1, at=0):
    def of(n):
        x = _mixed(n)
        strong = torch.arange(at, at + count)
        x[strong] = -100
        x[strong] = math.log(share / (1 - share) / count) + torch.logsumexp(x, 0)
        return x, strong
    return of


def _windows(low):
    """One key far above the others in four tiles, and a first key above these."""
    def of(n):
        x = torch.full((n,), -low * math.log(2.0))
        strong = torch.arange(5, n, 4 * TILE)
        x[strong] = 0
        x[0] = 3.49 * math.log(2.0)
        return x, torch.cat([torch.tensor([0]), strong])
    return of


def _falls(by, after):
    def of(n):
        x = _mixed(n)
        x[after:] -= by
        return x, torch.arange(after)
    return of


PATTERNS = {
    "a first key of 0.8": _sinks(0.8), "a first key of 0.95": _sinks(0.95), "a first key of 0.99": _sinks(0.99),
    "four first keys of 0.97": _sinks(0.97, 4), "a key of 0.9 in the middle": _sinks(0.9, 1, 200),
    "a key of 0.99 in the middle": _sinks(0.99, 1, 200),
    "one key in four tiles": _windows(9.84), "one key in four tiles, far above": _windows(12.0),
    "a fall of 2^10": _falls(10 * math.log(2.0), 40), "a fall of 2^30": _falls(30 * math.log(2.0), 100),
    "a fall of 2^41": _falls(41 * math.log(2.0), 70),
}


@pytest.mark.parametrize("name", PATTERNS)
@pytest.mark.parametrize("H", [3, 48, 96])
def test_what_the_low_weights_carry(name, H):
    """Several sequences a thread block over the same rows, of which the strong ones share a latent and two or three of the
    others each of the remaining: the output shows every key's weight."""
    g, n, size, N = _gen(71), 1100, 64, 300
    scores, strong = PATTERNS[name](n)
    table, pages = ref.make_pages(g, [n], size)
    x = torch.zeros(pages, size, ROW)
    i = torch.arange(n)
    values = torch.nn.functional.one_hot(i % (LATENT - 1), LATENT).float()
    values[strong] = 0
    values[strong, LATENT - 1] = 1.0
    x[table[0, i // size].long(), i % size, :LATENT] = values
    x[table[0, i // size].long(), i % size, LATENT] = scores.to(torch.bfloat16).float()
    cache, table = ref.fill(_cache(pages, size), x.cuda()), table.cuda()
    q_lat = torch.zeros(1, H, LATENT)
    q_pe = torch.zeros(1, H, POS)
    q_pe[..., 0] = 1
    q_lat, q_pe = q_lat.bfloat16().cuda(), q_pe.bfloat16().cuda()
    st = _status()
    o, lse = kda.kda_mla_decode_fp8(q_lat.expand(N, H, LATENT).contiguous(), q_pe.expand(N, H, POS).contiguous(), cache,
                                    table.expand(N, -1).contiguous(), _ints([n] * N), 1.0, status=st)
    assert st.item() == 0
    c, s = ref.cached(cache, table[0].cpu(), n)
    want = _bounds(torch.cat([q_lat, q_pe], -1)[0, :1], c, s, 1.0)  # (every head's query is the same)
    ref.check_rows(o.view(N * H, LATENT), lse.view(N * H), [x.expand(N * H, *x.shape[1:]) for x in want])

@pytest.mark.parametrize("H", [12, 48, 96])
def test_a_row_of_nan_does_not_slow_the_others(H):
    """A padded row whose queries are NaN goes through its tiles as fast as the others. (1.4 to 1.5 times the time
    where such a row looks for a unit in every tile.)"""
    g, n, size, N = _gen(72), 4096, 64, 64
    table, pages = ref.make_pages(g, [n], size)  # (of all sequences)
    cache = ref.fill(_cache(pages, size), torch.randn(pages, size, ROW, generator=g).cuda())
    q = torch.randn(N, H, ROW, generator=g).to(torch.bfloat16).cuda()
    table, lens = table.cuda().expand(N, -1).contiguous(), _ints([n] * N)
    ws = torch.empty(kda.kda_mla_decode_fp8_workspace_size(N, H, 1), dtype=torch.uint8, device="cuda")

    def best(q_lat, q_pe):
        out = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, lens, SCALE, workspace=ws)
            b.record()
            b.synchronize()
            out.append(a.elapsed_time(b))
        return min(out)

    q_lat, q_pe = q[..., :LATENT].contiguous(), q[..., LATENT:].contiguous()
    want = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, lens, SCALE)
    with_nan = q_lat.clone()
    with_nan[:, 1, 7] = NAN
    o, lse = kda.kda_mla_decode_fp8(with_nan, q_pe, cache, table, lens, SCALE)
    assert bool(o[:, 1].isnan().all()) and bool(lse[:, 1].isnan().all())
    keep = [h for h in range(H) if h != 1]
    assert torch.equal(o[:, keep], want[0][:, keep]) and torch.equal(lse[:, keep], want[1][:, keep])
    plain = best(q_lat, q_pe)
    assert best(with_nan, q_pe) <= 1.14 * plain
