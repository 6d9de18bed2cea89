"""Latent attention over millions of keys: sums that stay near the exact ones however long they are.

All keys of a kind are alike, so the answer has a closed form: with n_a keys of weight 2^{s_a} and value v_a,
o = sum n_a 2^{s_a} v_a / sum n_a 2^{s_a} and lse = ln sum n_a 2^{s_a}. The scale is ln 2 in fp32 and the kernel's
exponent s scale log2(e) rounds twice, so a weight is off by at most 2 ln 2 |s| 2^-24 < 2^-19 of itself for |s| <= 25.
Where the weights are powers of two (and all values are positive) rounding P changes nothing, and a sum is off by
  2^-11   at most 4096 additions a part in the tensor core, each low by less than a step 2^-23
  2^-13   at most 512 parts (2^25 keys of a row, or of a thread block's stretch) added to nearest, 2^-24 each, and
          2^-17 of the denominator's additions (a tile's for themselves, then at most 2^18 tiles: where tiles are alike
          their sums are whole numbers below 2^24 times a power of two, exact)
and o then is rounded to bf16. With other weights P's rounding is a bf16 rounding more, and the denominator's
additions, of tiles alike, all round one way: at most 1024 a part and 512 parts, 2^-24 each, and 32 in a tile, in all
less than 2^-13."""
import math

import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent_ref as ref
from tests.test_gpu_latent import LATENT, NOPE, POS, QK, ROW, _ints

pytestmark = pytest.mark.gpu

LN2 = math.log(2.0)
TOL_O = ref.U_BF16 + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -17
TOL_LSE = 2.0 ** -16


def _values(n, kind):
    """Values of a kind of key: positive, of every last bit of bf16."""
    return (1 + (torch.arange(n) * (37 + 10 * kind) % 128 + kind) / 128.0 % 1).to(torch.bfloat16)


def _want(counts, scores, values):
    """(o, lse) in 64 bits of counts [.., kinds]."""
    w = counts.double() * torch.exp2(torch.tensor(scores, dtype=torch.float64))
    return (w @ values.double()) / w.sum(-1, keepdim=True), w.sum(-1).log()


def _close(o, lse, want, scores):
    o, lse = o.double().cpu(), lse.double().cpu()
    exact = all(float(s).is_integer() for s in scores)
    to, tl = (TOL_O, TOL_LSE) if exact else (TOL_O + ref.U_BF16 + 2.0 ** -13, 2.0 ** -13)
    assert bool(((lse - want[1]).abs() <= tl + 2.0 ** -22 * want[1]).all()), float((lse - want[1]).abs().max())
    assert bool(((o - want[0]).abs() <= to * want[0]).all()), float((o / want[0] - 1).abs().max())


# runs of keys: (kind, length). Scores of the kinds in powers of two.
MILLION = 1 << 20
PREFILL = {
    "alike": ([0.0], [(0, 4 * MILLION + 77)]),
    "one key of weight 1 before many of 2^-25": ([0.0, -25.0], [(0, 1), (1, 4 * MILLION)]),
    "a new maximum behind many keys, and small ones again": (
        [0.0, 9.0, 20.0], [(0, 70000), (1, 3), (0, 131072 + 5), (2, 1), (1, 200000), (0, MILLION)]),
    "weights that are no power of two": ([0.0, -3.296875], [(0, 1), (1, 8 * MILLION)]),
    "the same, and a new maximum": ([0.0, -3.296875, 9.0], [(0, 1), (1, 2 * MILLION), (2, 1), (1, 100), (0, 3 * MILLION)]),
}


@pytest.mark.parametrize("what", list(PREFILL))
@pytest.mark.parametrize("new", [3, 300])
def test_prefill_over_millions_of_keys(what, new):
    """Causal: the last rows see up to 299 keys more than the first; `new` gives one or two query tiles."""
    scores, runs = PREFILL[what]
    kind = torch.cat([torch.full((n,), a) for a, n in runs]).cuda()
    n, H = kind.numel(), 2
    kv = torch.empty(n, H, 2 * NOPE, dtype=torch.bfloat16, device="cuda")
    kv[..., :NOPE] = 0
    for a in range(len(scores)):
        for h in range(H):
            kv[kind == a, h, NOPE:] = _values(NOPE, a + 3 * h).cuda()
    pe = torch.zeros(n, POS, dtype=torch.bfloat16, device="cuda")
    pe[:, 0] = torch.tensor(scores, device="cuda").to(torch.bfloat16)[kind]
    q = torch.zeros(new, H, QK, dtype=torch.bfloat16, device="cuda")
    q[..., NOPE] = 1
    o, lse = kda.kda_mla_prefill(q, kv, pe, _ints([0, new]), _ints([0, n]), LN2)
    total = torch.bincount(kind.cpu(), minlength=len(scores))
    # what a row does not see
    tail = torch.nn.functional.one_hot(kind[n - new + 1:].cpu(), len(scores)).flip(0).cumsum(0).flip(0)
    counts = total - torch.cat([tail, torch.zeros(1, len(scores), dtype=torch.long)])
    for h in range(H):
        values = torch.stack([_values(NOPE, a + 3 * h) for a in range(len(scores))])
        _close(o[:, h], lse[:, h], _want(counts, scores, values), scores)


def test_prefill_of_one_query_tile_that_takes_longer_than_a_wait():
    """The warps of the second query tile, which has no rows, wait for the item's end: 1.5 us a key tile, 2.4 s, where
    a wait gives up after 2. Needs 135 GB for its 2.1e8 keys."""
    n = 210_000_000
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < n * 2 * (2 * NOPE + POS) + (4 << 30):
        pytest.skip("not enough free device memory")
    kv = torch.empty(n, 1, 2 * NOPE, dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros(n, POS, dtype=torch.bfloat16, device="cuda")
    kv[:] = torch.cat([torch.zeros(NOPE), _values(NOPE, 2)]).to(torch.bfloat16).cuda()
    q = torch.randn(5, 1, QK, device="cuda").to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kda.kda_mla_prefill(q, kv, pe, _ints([0, 5]), _ints([0, n]), LN2, causal=False, status=st)
    assert st.item() == 0
    # 3205 parts instead of 512, and a denominator of 128 a tile, whole numbers of fewer than 24 bits
    want = _want(torch.tensor([[n]]), [0.0], _values(NOPE, 2)[None])
    assert bool(((o[:, 0].double().cpu() - want[0]).abs() <= (TOL_O + 2.0 ** -12) * want[0]).all())
    assert bool(((lse[:, 0].double().cpu() - want[1]).abs() <= TOL_LSE + 2.0 ** -22 * want[1]).all())
    del kv, pe
    torch.cuda.empty_cache()


DECODE = {
    # lengths, kinds' scores, pages of each kind in turn, H, m
    "alike, 13 blocks a list": ([1 << 26, 100], [0.0], [(0, 1)], 64, 16),
    "alike, 96 rows": ([200 << 20], [0.0], [(0, 1)], 96, 1),
    "a new maximum behind many rows": ([(1 << 25) + 33], [0.0, 9.0, 18.0],
                                       [(0, 1200), (1, 3), (0, 2100), (2, 1), (1, 900)], 64, 16),
    "whole sequences of many tiles": ([80000 + 31 * n for n in range(170)], [0.0, 9.0],
                                      [(0, 1100), (1, 1), (0, 3)], 12, 1),
    "weights that are no power of two": ([1 << 26], [0.0, -3.296875], [(0, 1), (1, 3000)], 64, 16),
}


@pytest.mark.parametrize("what", list(DECODE))
def test_decode_over_millions_of_rows(what):
    """A page of each kind, which the page tables name again and again."""
    lens, scores, turns, H, m = DECODE[what]
    size, kinds, N = 64, len(scores), len(lens)
    cycle = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in turns])
    most = max(-(-n // size) for n in lens)
    row = cycle.repeat(-(-most // cycle.numel()))[:most]
    values = torch.stack([_values(LATENT, a) for a in range(kinds)])
    cache = torch.zeros(kinds, size, ROW, dtype=torch.bfloat16, device="cuda")
    cache[..., :LATENT] = values.cuda()[:, None]
    cache[..., LATENT] = torch.tensor(scores, device="cuda").to(torch.bfloat16)[:, None]
    q_lat = torch.zeros(N * m, H, LATENT, dtype=torch.bfloat16, device="cuda")
    q_pe = torch.zeros(N * m, H, POS, dtype=torch.bfloat16, device="cuda")
    q_pe[..., 0] = 1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, row.cuda().repeat(N, 1), _ints(lens), LN2, num_tokens=m, status=st)
    assert st.item() == 0
    for n, length in enumerate(lens):
        for t in range(m):
            seen = length - (m - 1 - t)
            full, rest = divmod(seen, size)
            counts = size * torch.bincount(row[:full], minlength=kinds)
            if rest:
                counts[row[full]] += rest
            wo, wl = _want(counts, scores, values)
            _close(o[n * m + t], lse[n * m + t], (wo.expand(H, -1), wl.expand(H)), scores)
