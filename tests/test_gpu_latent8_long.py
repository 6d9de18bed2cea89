"""Latent attention over the 8-bit cache where a thread block goes through many tiles and several sequences, and over
millions of rows: inputs in which every tile has a value column of its own, so that one left out or taken twice shows
however long the sequence is, and keys of a few kinds, for which the answer has a closed form.

Errors, relative to positive values: a weight in fp16, e4m3 and e5m2 2^-7 + 2^-11 (tests/latent8_ref.py) and 2^-19 for its
score and exponential; the products' sums 2^-11 (at most 4096 additions a part in the tensor core, each low by less than a
step 2^-23) and 2^-13 (at most 1024 parts added to nearest, 2^-24 each, and some for the join); the denominator 2^-13 (at
most 1024 tiles a part, 1024 parts and 32 of a tile, 2^-24 each); the output's rounding 2^-8."""
import math

import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent8_ref as ref
from tests.test_gpu_latent import LATENT, POS, ROW, SCALE, _gen, _ints, _status
from tests.test_gpu_latent8 import _cache, _check, _inputs

pytestmark = pytest.mark.gpu

TILE = 64
LN2 = math.log(2.0)
TOL_O = 2.0 ** -7 + 2.0 ** -11 + 2.0 ** -19 + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -8
TOL_LSE = 2.0 ** -13 + 2.0 ** -19


@pytest.mark.parametrize("H,m,size", [(12, 1, 64), (40, 1, 16), (96, 1, 64), (65, 2, 64), (96, 2, 16), (128, 2, 48),
                                      (64, 5, 32), (96, 4, 64), (64, 16, 128)])
def test_decode_of_many_short_sequences_a_block(H, m, size):
    """Several sequences a thread block, empty ones and ones of less than a tile among them, cut at any place."""
    g = _gen(H * m)
    lens = [(n * 389) % 1201 if n % 9 else (0, 1, m, 64, 65)[n // 9 % 5] for n in range(360 if H * m <= 96 else 90)]
    q_lat, q_pe, cache, table = _inputs(g, lens, size, H, m)
    st, lens_d = _status(), _ints(lens)
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, lens_d, SCALE, num_tokens=m, status=st)
    assert st.item() == 0
    _check(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE, seqs=range(0, len(lens), 1 if len(lens) < 100 else 3))
    o2, lse2 = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, lens_d, SCALE, num_tokens=m)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


COUNTED = [[(1 << 20) + 5], [LATENT * TILE, 0, 300011], [900 + 1061 * n for n in range(20)],
           [LATENT * TILE, 0, 20016, 1, 64, 30011, 4500, 127] + [900 + 61 * n for n in range(40)]]


@pytest.mark.parametrize("lens", COUNTED, ids=lambda lens: "%d sequences" % len(lens))
@pytest.mark.parametrize("H,m", [(12, 1), (64, 1), (96, 1), (65, 2), (40, 5), (96, 4), (64, 16)])
def test_decode_counts_every_tile_once(lens, H, m):
    """All scores are 0 and row i holds 1 in latent i // 64 % 512, so o[d] is the share of the visible rows in the
    tiles d, d + 512, ..: of 32 tiles a latent at most, one too few or too many moves it by 3%."""
    g, size = _gen(60), 64
    table, pages = ref.make_pages(g, lens, size)
    cache = _cache(pages, size, 0xFF)
    rows, scales = ref.parts(cache)
    one, s = ref.quantise(torch.eye(LATENT, ROW, device="cuda"))
    for n, k in enumerate(lens):
        i = torch.arange(k)
        page, at, kind = table[n, i // size].long().cuda(), (i % size).cuda(), (i // TILE % LATENT).cuda()
        rows[page, at], scales[page, at] = one[kind], s[kind]
    N = len(lens)
    q_lat = torch.zeros(N * m, H, LATENT, dtype=torch.bfloat16, device="cuda")
    q_pe = torch.randn(N * m, H, POS, generator=g).to(torch.bfloat16).cuda()
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table.cuda(), _ints(lens), SCALE, num_tokens=m)
    for n, k in enumerate(lens):
        for t in range(m):
            seen = max(0, k - (m - 1 - t))
            tiles = LATENT * (1 + k // (TILE * LATENT))
            tiles = TILE * torch.arange(tiles, dtype=torch.float64, device="cuda")
            want = (seen - tiles).clamp(0, TILE).view(-1, LATENT).sum(0) / max(1, seen)
            got = o[n * m + t].double()
            assert bool(((got - want).abs() <= TOL_O * want).all()), (n, t)
            l = torch.tensor(float(seen), dtype=torch.float64).log()
            if seen == 0:
                assert bool((lse[n * m + t] == -float("inf")).all())
            else:
                assert bool(((lse[n * m + t].double().cpu() - l).abs() <= TOL_LSE + 2.0 ** -22 * l).all())


def _values(kind):
    """Positive values of every last bit of e4m3."""
    return 1 + (torch.arange(LATENT) * (3 + 2 * kind) + kind) % 8 / 8.0


FAR = {
    # lengths, kinds' scores in powers of two, pages of each kind in turn, H, m
    "alike, several row tiles": ([1 << 26, 100], [0.0], [(0, 1)], 64, 16),
    "alike, 96 rows": ([200 << 20], [0.0], [(0, 1)], 96, 1),
    "alike, 48 rows": ([100 << 20, 1], [0.0], [(0, 1)], 48, 1),
    "a new maximum behind many rows": ([(1 << 25) + 33], [0.0, 9.0, 18.0],
                                       [(0, 1200), (1, 3), (0, 2100), (2, 1), (1, 900)], 64, 16),
    "a new maximum behind many rows, 12 heads": ([(1 << 27) + 1], [0.0, 9.0, 18.0],
                                                 [(0, 1200), (1, 3), (0, 2100), (2, 1), (1, 900)], 12, 1),
    "whole sequences of many tiles": ([80000 + 31 * n for n in range(170)], [0.0, 9.0],
                                      [(0, 1100), (1, 1), (0, 3)], 12, 1),
    "weights that are no power of two": ([1 << 26], [0.0, -3.296875], [(0, 1), (1, 3000)], 40, 2),
}


@pytest.mark.parametrize("what", list(FAR))
def test_decode_over_millions_of_rows(what):
    """A page of each kind, which the page tables name again and again. Beside a page that weighs 2^9 and more
    of its neighbours, up to 12 of these are off by 2^-11.9 of its weight (tests/latent8_ref.py)."""
    lens, scores, turns, H, m = FAR[what]
    size, kinds, N = 64, len(scores), len(lens)
    cycle = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in turns])
    most = max(-(-n // size) for n in lens)
    row = cycle.repeat(-(-most // cycle.numel()))[:most]
    values = torch.stack([_values(a) for a in range(kinds)])
    x = torch.zeros(kinds, size, ROW)
    x[..., :LATENT] = values[:, None]
    x[..., LATENT] = torch.tensor(scores)[:, None]
    cache = ref.fill(_cache(kinds, size), x.cuda())
    q_lat = torch.zeros(N * m, H, LATENT, dtype=torch.bfloat16, device="cuda")
    q_pe = torch.zeros(N * m, H, POS, dtype=torch.bfloat16, device="cuda")
    q_pe[..., 0] = 1
    st = _status()
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, row.cuda().repeat(N, 1), _ints(lens), LN2, num_tokens=m, status=st)
    assert st.item() == 0
    w = torch.exp2(torch.tensor(scores, dtype=torch.float64))
    near = 0.0 if max(scores) == 0 else 24 * 2.0 ** -11.9  # (values up to twice one another)
    for n, length in enumerate(lens):
        for t in range(m):
            full, rest = divmod(length - (m - 1 - t), size)
            counts = size * torch.bincount(row[:full], minlength=kinds)
            if rest:
                counts[row[full]] += rest
            share = counts.double() * w
            wo, wl = (share @ values.double()) / share.sum(), share.sum().log()
            assert bool(((lse[n * m + t].double().cpu() - wl).abs() <= TOL_LSE + 2.0 ** -22 * wl).all()), (n, t)
            assert bool(((o[n * m + t].double().cpu() - wo).abs() <= (TOL_O + near) * wo).all()), (n, t)


@pytest.mark.parametrize("H", [2, 40, 96])
def test_decode_of_positional_scores_alone(H):
    """Queries without latents over rows whose latents are next to nothing: the positional key, in units of the row's
    scale, is then huge, and the queries' unit is small."""
    g, n, size = _gen(61), 300, 32
    table, pages = ref.make_pages(g, [n], size)
    x = torch.randn(pages, size, ROW, generator=g)
    x[..., :LATENT] *= 2.0 ** -30
    cache = ref.fill(_cache(pages, size), x.cuda())
    q_lat = torch.zeros(1, H, LATENT, dtype=torch.bfloat16, device="cuda")
    q_lat[0, 0] = 2.0 ** -80
    q_pe = torch.randn(1, H, POS, generator=g).to(torch.bfloat16).cuda()
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table.cuda(), _ints([n]), SCALE)
    _check(o, lse, q_lat, q_pe, cache, table.cuda(), [n], 1, SCALE)


@pytest.mark.parametrize("H,m", [(2, 1), (33, 3)])
def test_the_longest_sequence_and_the_largest_pages(H, m):
    """Pages of 65,536 rows and the 2,147,418,112 that 32,767 of them hold: rows written and read back at the end, and all of
    them attended. Half of the pages' rows hold 1 in latent 0, the others' in latent 1, but the last three, the new ones, in 2."""
    size, pages = 65536, 32767
    n = size * pages
    cache = _cache(3, size)
    rows, scales = ref.parts(cache)
    one, s = ref.quantise(torch.eye(3, ROW, device="cuda"))
    for page, kind in ((0, 0), (1, 1), (2, 1)):
        rows[page], scales[page] = one[kind], s[kind]
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None] % 2
    table[0, -1] = 2
    down = torch.zeros(3, ROW, dtype=torch.bfloat16, device="cuda")
    down[:, 2] = 1
    st, lens = _status(), _ints([n])
    kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table, lens, status=st)
    end = kda.kda_mla_gather_fp8(cache, table, _ints([0, 9]), 9, starts=_ints([n - 9]), status=st)
    want = torch.zeros(9, ROW, device="cuda")
    want[:6, 1] = want[6:, 2] = 1
    assert torch.equal(end.float(), want)
    q_lat = torch.zeros(m, H, LATENT, dtype=torch.bfloat16, device="cuda")
    q_pe = torch.zeros(m, H, POS, dtype=torch.bfloat16, device="cuda")
    q_lat[..., 2] = 16 * LN2  # the new rows score 2^16
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, lens, 1.0, num_tokens=m, status=st)
    assert st.item() == 0
    score = float(torch.tensor(16 * LN2).bfloat16())
    for t in range(m):
        new = (3 - (m - 1 - t)) * math.exp(score)
        share = torch.tensor([size * (pages // 2), size * (pages // 2 + 1) - 3, new], dtype=torch.float64)
        total = share.sum()
        want = torch.zeros(LATENT, dtype=torch.float64)
        want[:3] = share / total
        # (beside the new rows the last nine tiles' weights are off by 2^-13.9 of a unit of 2^-2.5 of theirs: 576 2^-16.4 2^16 in all)
        more = 576 * 2.0 ** -16.4 * math.exp(score) / total
        assert bool(((o[t].double().cpu() - want).abs() <= TOL_O * want + more * (want > 0)).all()), t
        assert bool(((lse[t].double().cpu() - total.log()).abs() <= TOL_LSE + 2.0 ** -22 * total.log()).all()), t
    far = kda.kda_mla_gather_fp8(cache, table, _ints([0, 2]), 2, starts=_ints([n - 1]), status=st)
    assert st.item() == -4 and bool(far[1].isnan().all()) and torch.equal(far[0].float(), end[8].float())
