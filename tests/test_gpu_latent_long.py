"""Latent attention where a thread block goes through many tiles and several sequences or items: rings that
wrap, slots refilled, queries of the next piece of work loaded under the last one's end. Beside the 64-bit forms
there are inputs in which every tile has a value column of its own, so that one left out or taken twice
shows however long the sequence is."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent_ref as ref
from tests.test_gpu_latent import (LATENT, NOPE, POS, QK, ROW, SCALE, _check_decode, _cu, _decode_inputs, _gen, _ints,
                                   _prefill_inputs, _status)

pytestmark = pytest.mark.gpu

TILE_K, TILE_ROWS = 128, 64  # keys of a tile in the prefill, cached rows of a tile in the decode


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("H,m,size", [(65, 2, 64), (96, 2, 16), (128, 2, 48), (64, 5, 32), (96, 4, 64), (64, 16, 128)])
def test_decode_of_many_tiles_with_several_row_tiles(H, m, size):
    """More than 96 query rows a sequence: at least ten tiles a thread block, of one to four sequences."""
    g = _gen(H * m)
    lens = [(n * 389) % 1201 if n % 9 else (0, 1, m, 64, 65)[n // 9 % 5] for n in range(90)]
    # two row tiles at least, so half the SMs' blocks share the list at most
    assert sum(max(1, -(-n // TILE_ROWS)) for n in lens) >= 10 * (_sms() // 2)
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, size, H, m)
    st, lens_d = _status(), _ints(lens)
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, lens_d, SCALE, num_tokens=m, status=st)
    assert st.item() == 0
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE)
    o2, lse2 = kda.kda_mla_decode(q_lat, q_pe, cache, table, lens_d, SCALE, num_tokens=m)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# one long sequence (all blocks' parts joined by 16 warps a row), some (by four), many (by one)
COUNTED = [[(1 << 20) + 5], [LATENT * TILE_ROWS, 0, 300011], [900 + 1061 * n for n in range(20)],
           [LATENT * TILE_ROWS, 0, 20016, 1, 64, 30011, 4500, 127] + [900 + 61 * n for n in range(40)]]


@pytest.mark.parametrize("lens", COUNTED, ids=lambda lens: "%d sequences" % len(lens))
@pytest.mark.parametrize("H,m", [(12, 1), (64, 1), (96, 1), (65, 2), (96, 4), (64, 16)])
def test_decode_counts_every_tile_once(lens, H, m):
    """All scores are 0 and row i holds 1 in latent i // 64 % 512, so o[d] is the share of the visible rows in the
    tiles d, d + 512, ..: weights of 1 and counts are exact, what is left is the quotient and its rounding. Of 32 tiles
    a latent at most, one too few or too many moves it by 3%."""
    g, size = _gen(60), 64
    table, pages = ref.make_pages(g, lens, size)
    cache = torch.full((pages, size, ROW), float("nan"), dtype=torch.bfloat16, device="cuda")
    for n, k in enumerate(lens):
        i = torch.arange(k)
        at = (table[n, i // size].long() * size + i % size).cuda()
        one = torch.eye(LATENT, ROW, dtype=torch.bfloat16, device="cuda")
        cache.view(-1, ROW)[at] = one[(i // TILE_ROWS % LATENT).cuda()]
    N = len(lens)
    q_lat = torch.zeros(N * m, H, LATENT, dtype=torch.bfloat16, device="cuda")
    q_pe = torch.randn(N * m, H, POS, generator=g).to(torch.bfloat16).cuda()
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table.cuda(), _ints(lens), SCALE, num_tokens=m)
    for n, k in enumerate(lens):
        for t in range(m):
            seen = max(0, k - (m - 1 - t))
            tiles = LATENT * (1 + k // (TILE_ROWS * LATENT))
            tiles = TILE_ROWS * torch.arange(tiles, dtype=torch.float64, device="cuda")
            want = (seen - tiles).clamp(0, TILE_ROWS).view(-1, LATENT).sum(0) / max(1, seen)
            got = o[n * m + t].double()
            assert bool(((got - want).abs() <= (ref.U_BF16 + 2.0 ** -21) * want).all()), (n, t)
            l = torch.tensor(float(seen), dtype=torch.float64).log()
            if seen == 0:
                assert bool((lse[n * m + t] == -float("inf")).all())
            else:
                assert bool(((lse[n * m + t].double().cpu() - l).abs() <= 2.0 ** -20 + 2.0 ** -22 * l).all())


# ------------------------------------------------------------------ prefill
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_of_several_items_a_block(causal):
    """Several hundred items of up to eleven key tiles and one or two query tiles, some without keys, so that every
    block takes others over and carries its rings from item to item."""
    g, H = _gen(61), 32
    new = [300, 700, 1, 411, 128, 0, 640, 257, 129, 550, 90, 513, 256, 385, 40]
    prefix = [0, 900, 650, 333, 0, 40, 128, 71, 500, 1, 0, 899, 256, 64, 0]
    total = [a + b for a, b in zip(new, prefix)]
    total[10], total[14] = 0, 17  # queries without keys, and more queries than keys
    assert H * sum(-(-n // 256) for n in new) >= 4 * _sms()
    q, kv, pe = _prefill_inputs(g, new, total, H)
    cu_q, cu_k, st = _cu(new), _cu(total), _status()
    args = (q, kv, pe, _ints(cu_q), _ints(cu_k), SCALE)
    o, lse = kda.kda_mla_prefill(*args, causal=causal, status=st)
    assert st.item() == 0
    for n in range(len(new)):
        a, b = cu_q[n], cu_q[n + 1]
        for h in (0, 1, 7, 14, 22, 31):
            ref.check_rows(o[a:b, h], lse[a:b, h], ref.prefill_ref(q, kv, pe, cu_q, cu_k, SCALE, causal, n, h))
    for _ in range(3):
        o2, lse2 = kda.kda_mla_prefill(*args, causal=causal)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new,total,H", [([16384], [16384], 4), ([700, 3000, 257, 5000], [9000, 3000, 16200, 5300], 9),
                                         ([300, 5], [1 << 19, 70001], 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_counts_every_key_tile_once(new, total, H, causal):
    """All scores are 0 and key j holds 1 in value j // 128 % 128: o[d] is the share of the visible keys in the tiles
    d, d + 128, .., of 32 at most, so that one moves it by 3%."""
    g, cu_q, cu_k = _gen(62), _cu(new), _cu(total)
    q = torch.zeros(sum(new), H, QK, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(sum(total), H, 2 * NOPE, dtype=torch.bfloat16, device="cuda")
    kv[..., :NOPE] = torch.randn(H, NOPE, generator=g).to(torch.bfloat16).cuda()
    j = torch.cat([torch.arange(n) for n in total]).cuda() // TILE_K % NOPE
    kv[..., NOPE:] = torch.eye(NOPE, dtype=torch.bfloat16, device="cuda")[j][:, None]
    pe = torch.randn(sum(total), POS, generator=g).to(torch.bfloat16).cuda()
    o, lse = kda.kda_mla_prefill(q, kv, pe, _ints(cu_q), _ints(cu_k), SCALE, causal=causal)
    for n, (k, a) in enumerate(zip(total, new)):
        tiles = TILE_K * torch.arange(NOPE * (1 + k // (TILE_K * NOPE)), dtype=torch.float64, device="cuda")
        seen = torch.arange(k - a + 1, k + 1, device="cuda", dtype=torch.float64)
        seen = seen if causal else torch.full_like(seen, k)
        want = ((seen[:, None] - tiles).clamp(0, TILE_K).view(a, -1, NOPE).sum(1) / seen[:, None])[:, None]
        got = o[cu_q[n]:cu_q[n + 1]].double()
        assert bool(((got - want).abs() <= (ref.U_BF16 + 2.0 ** -21) * want).all()), n
        l = seen.log()[:, None]
        assert bool(((lse[cu_q[n]:cu_q[n + 1]].double() - l).abs() <= 2.0 ** -20 + 2.0 ** -22 * l).all()), n
