"""Latent attention over the cache in 8 bits on the GPU, against plain 64-bit forms (tests/latent8_ref.py, which
derives the bounds)."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from linear_attention_serving_02_gb300.paging import PagePool
from tests import latent8_ref as ref
from tests.test_gpu_latent import (DECODE, LATENT, NAN, NOPE, POS, QK, ROW, SCALE, _capture, _cu, _gen, _ints, _rand,
                                   _rope, _status)

pytestmark = pytest.mark.gpu

ROW8, TOKEN8 = ref.ROW8, ref.TOKEN8


def _cache(pages, size, fill=0):
    return torch.full((pages, size, TOKEN8), fill, dtype=torch.uint8, device="cuda")


def _random_cache(g, pages, size, spread=0.0):
    """Rows of normal values; spread: of the rows' magnitudes, in powers of two."""
    x = torch.randn(pages, size, ROW, generator=g)
    if spread:
        x *= torch.exp2(spread * torch.randn(pages, size, 1, generator=g)).clamp(2.0 ** -20, 2.0 ** 20)
    return ref.fill(_cache(pages, size), x.cuda())


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("new,before,size,H,rope,norm,cu", [
    ([1], [0], 16, 1, False, True, True),
    ([5, 0, 17], [11, 3, 0], 16, 3, True, True, True),
    ([1] * 40, list(range(40)), 32, 12, True, True, False),
    ([64, 65, 130], [63, 0, 500], 64, 17, True, False, True),
    ([3] * 33, [7] * 33, 48, 96, True, True, True),
    ([2000], [1], 128, 5, False, False, True),
])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(new, before, size, H, rope, norm, cu, interleaved):
    g = _gen(len(new) + size)
    lens = [a + b for a, b in zip(new, before)]
    table, pages = ref.make_pages(g, lens, size)
    table_d, T = table.cuda(), sum(new)
    down, q = _rand(g, T, ROW), _rand(g, T, H, QK)
    down[:, :LATENT] *= torch.exp2(torch.randint(-9, 9, (T, 1), generator=g).float()).to(torch.bfloat16).cuda()
    cache = torch.randint(0, 256, (pages, size, TOKEN8), generator=g, dtype=torch.uint8).cuda()
    was, w = cache.clone(), (1 + 0.1 * torch.randn(LATENT, generator=g)).cuda() if norm else None
    tab, st = _rope(max(lens)) if rope else None, _status()
    args = (table_d, _ints(lens), _ints(_cu(new)) if cu else None)
    more = dict(norm_w=w, eps=1e-5, rope=tab, rope_interleaved=interleaved, q_pe=q[..., NOPE:] if rope else None, status=st)
    q_out = kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, *args, **more)
    assert st.item() == 0
    seq = [n for n, k in enumerate(new) for _ in range(k)]
    pos = [before[n] + i for n, k in enumerate(new) for i in range(k)]
    page = torch.tensor([int(table[n, p // size]) for n, p in zip(seq, pos)], device="cuda")
    at = torch.tensor([p % size for p in pos], device="cuda")
    c, pe = down[:, :LATENT].double(), down[:, LATENT:].double()
    if norm:
        c = c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    rows, scales = ref.parts(cache)
    got, s = ref.codes(rows[page, at]), scales[page, at].double()
    # the scale is a power of two that puts the largest value into (224, 448]; fp32 may be off by 300 steps
    top, off = c.abs().amax(1) / s, 300 * 2.0 ** -23
    assert torch.equal(torch.frexp(s)[0], torch.full_like(s, 0.5))
    assert bool((top <= ref.TOP * (1 + off)).all()) and bool((top > ref.TOP / 2 * (1 - off)).all())
    val = got[:, :LATENT] * s[:, None]
    half = torch.maximum(2.0 ** -4 * c.abs(), 2.0 ** -10 * s[:, None])
    assert bool(((val - c).abs() <= half * (1 + 2.0 ** -10) + off * c.abs()).all())
    if not norm:  # bf16 values: the scale and every rounding are exact
        b, se = ref.quantise(torch.cat([c, pe], 1))
        assert torch.equal(rows[page, at][:, :LATENT], b[:, :LATENT]) and torch.equal(s, se.double())
    p_val = got[:, LATENT:] * s[:, None]
    if rope:
        # the positional key and the queries are those of the bf16 cache, bit for bit
        plain = torch.zeros(pages, size, ROW, dtype=torch.bfloat16, device="cuda")
        q_plain = kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], plain, *args, **more)
        assert torch.equal(q_out, q_plain) and torch.equal(p_val, plain[page, at][:, LATENT:].double())
    else:
        assert q_out is None and torch.equal(p_val, pe)
    left = torch.ones(pages, size, dtype=torch.bool, device="cuda")
    left[page, at] = False
    was_rows, was_scales = ref.parts(was)
    assert torch.equal(rows[left], was_rows[left])
    assert torch.equal(scales.contiguous().view(torch.int32)[left], was_scales.contiguous().view(torch.int32)[left])


def test_append_of_extreme_rows():
    """Rows of zeros, at and next to the largest e4m3 value, subnormal, past the largest scale, with infinities and NaN."""
    inf = float("inf")
    tops = [0.0, 448.0, 450.0, 224.0, 225.0, 1.0, 2.0 ** -31, 2.0 ** -32, 2.0 ** -60, 1e-40, 448 * 2.0 ** 40, 452 * 2.0 ** 40,
            3e38, inf, -448.0, -450.0, -inf]
    T = len(tops) + 2
    down = torch.zeros(T, ROW, dtype=torch.bfloat16, device="cuda")
    down[:, LATENT:] = _rand(_gen(1), T, POS)
    for i, t in enumerate(tops):
        down[i, 7 + i] = t
        down[i, 300:340] = t / 3 if abs(t) < inf else 5.0
    down[-2, 100], down[-2, 200] = NAN, 3.0
    down[-1, :LATENT] = NAN
    cache, table = _cache(2, 32), _ints([[1, 0]])
    kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table, _ints([T]))
    c, s = ref.cached(cache, table[0].cpu(), T)
    x = down[:, :LATENT].double()
    for i, t in enumerate(tops):
        e = int(ref.exponent(torch.tensor(min(abs(t), 3.4e38), dtype=torch.float64)))
        assert s[i].item() == 2.0 ** e, t
        y = (x[i] / 2.0 ** e).clamp(-448, 448)
        assert bool(((c[i, :LATENT] - y).abs() <= torch.maximum(2.0 ** -4 * y.abs(), torch.full_like(y, 2.0 ** -10))).all()), t
        if 2.0 ** -40 < abs(t) < 1e6:
            assert torch.equal(c[i, LATENT:] * s[i], down[i, LATENT:].double()), t
    assert c[-2, 200] * s[-2] == 3 and c[-2, 100].isnan() and int(c[-2].isnan().sum()) == 1
    assert bool(c[-1, :LATENT].isnan().all()) and s[-1].item() == 1


def test_append_leaves_padding_alone_and_rotates_queries_in_place():
    g = _gen(3)
    new, lens, size = [3, 2], [20, 40], 16
    table, pages = ref.make_pages(g, lens, size)
    down, q, cache = _rand(g, 9, ROW), _rand(g, 9, 4, QK), _cache(pages, size, 7)
    was = q.clone()
    out = kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table.cuda(), _ints(lens), _ints(_cu(new)),
                                 rope=_rope(40), q_pe=q[..., NOPE:], q_out=q[..., NOPE:])
    assert out.data_ptr() == q[..., NOPE:].data_ptr()
    assert torch.equal(q[..., :NOPE], was[..., :NOPE]) and torch.equal(q[5:], was[5:]) and not torch.equal(q[:5], was[:5])
    rows, _ = ref.parts(cache)
    assert int((rows != 7).any(-1).sum()) == 5


@pytest.mark.parametrize("what,code", [("page", -9), ("short", -4), ("long", -4), ("rope", -4)])
def test_append_bad_tables(what, code):
    g = _gen(5)
    size, lens = 16, [20, 30, 25]
    table, pages = ref.make_pages(g, lens, size)
    down, q, cache = _rand(g, 6, ROW), _rand(g, 6, 2, POS), _cache(pages, size, 9)
    tab = _rope(30 if what != "rope" else 29)
    if what == "page":
        table[1, 1] = pages
    elif what == "short":
        lens[1] = 0
    elif what == "long":
        lens[1] = table.shape[1] * size + 2
        tab = _rope(200)
    st = _status()
    q_out = kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table.cuda(), _ints(lens), None, rope=tab,
                                   q_pe=q, status=st)
    assert st.item() == code and kda.kda_workspace_status(st) == code
    bad = {"rope": [3]}.get(what, [2, 3])
    bad = torch.tensor([i in bad for i in range(6)], device="cuda")
    assert torch.equal(torch.isnan(q_out).all(-1).all(-1), bad) and not torch.isnan(q_out[~bad]).any()
    rows, _ = ref.parts(cache)
    assert int((rows != 9).any(-1).sum()) == 6 - int(bad.sum())


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("lens,size", [([1], 16), ([0, 5, 0, 0, 33, 16, 0], 16), ([700, 1, 64], 64), ([3] * 70, 48)])
@pytest.mark.parametrize("window", [False, True])
def test_gather(lens, size, window):
    g = _gen(sum(lens))
    table, pages = ref.make_pages(g, lens, size)
    pool = torch.randint(0, 256, (pages, 2, size, TOKEN8), generator=g, dtype=torch.uint8).cuda()
    cache, st = pool[:, 1], _status()  # two layers in turn: a page stride of two pages
    ref.fill(cache, torch.randn(pages, size, ROW, generator=g).cuda() * torch.exp2(torch.randn(pages, size, 1, generator=g)).cuda())
    starts = [(3 * n + k // 2) % (k + 1) for n, k in enumerate(lens)] if window else [0] * len(lens)
    count = [k - a for k, a in zip(lens, starts)]
    T = sum(count)
    out = torch.full((T + 7, ROW), 5.0, dtype=torch.bfloat16, device="cuda")
    got = kda.kda_mla_gather_fp8(cache, table.cuda(), _ints(_cu(count)), T + 7, starts=_ints(starts) if window else None,
                                 out=out, status=st)
    assert got is out and st.item() == 0
    want = []
    for n, k in enumerate(lens):
        c, s = ref.cached(cache, table[n], k, starts[n])
        want.append(c * s[:, None])
    assert torch.equal(out[:T].double(), torch.cat(want)) and bool((out[T:] == 5).all())


def test_gather_bad_page_start_and_length():
    g = _gen(9)
    lens, size = [20, 40, 5], 16
    table, pages = ref.make_pages(g, lens, size)
    cache = _random_cache(g, pages, size)
    table[1, 1] = -3
    st = _status()
    out = kda.kda_mla_gather_fp8(cache, table.cuda(), _ints(_cu(lens)), 65, status=st)
    bad = torch.zeros(65, dtype=torch.bool, device="cuda")
    bad[36:52] = True
    assert st.item() == -9 and torch.equal(torch.isnan(out).all(1), bad) and not torch.isnan(out[~bad]).any()
    table[1, 1], table[2] = 0, 1
    most = table.shape[1] * size
    for n, first, k, nan in ((2, most - 3, 5, 2), (0, -2, 20, 2), (0, -2147483648, 20, 20), (2, 2147483647, 5, 5)):
        st, starts, count = _status(), [0, 0, 0], list(lens)
        starts[n], count[n] = first, k
        table_d = table.clone()
        table_d[n] = 1
        out = kda.kda_mla_gather_fp8(cache, table_d.cuda(), _ints(_cu(count)), sum(count), starts=_ints(starts), status=st)
        assert st.item() == -4 and int(torch.isnan(out).all(1).sum()) == nan == int(torch.isnan(out).any(1).sum())


# ------------------------------------------------------------------ decode
def _inputs(g, lens, size, H, m, scale=1.0, tails=True, spread=0.0):
    table, pages = ref.make_pages(g, lens, size)
    cache = _random_cache(g, pages, size, spread)
    if tails:  # NaN and infinities in every row and scale that no sequence has
        used = torch.zeros(pages, size, dtype=torch.bool)
        for n, k in enumerate(lens):
            i = torch.arange(max(0, k))
            used[table[n, i // size].long(), i % size] = True
        used = used.cuda()
        rows, scales = ref.parts(cache)
        b = rows.clone()
        b[~used] = 0x7F
        b[~used, LATENT + 1:] = 0xFF
        rows.copy_(b)
        s = scales.clone()
        s[~used] = NAN
        s[~used & (torch.arange(size, device="cuda") % 2 == 0)] = float("inf")
        scales.copy_(s)
    N = len(lens)
    return _rand(g, N * m, H, LATENT, scale=scale), _rand(g, N * m, H, POS, scale=scale), cache, table.cuda()


def _check(o, lse, q_lat, q_pe, cache, table, lens, m, scale, seqs=None):
    H = q_lat.shape[1]
    for n in range(len(lens)) if seqs is None else seqs:
        r = slice(n * m, (n + 1) * m)
        ref.check_rows(o[r].reshape(m * H, LATENT), lse[r].reshape(-1),
                       ref.decode_ref(q_lat, q_pe, cache, table, lens, m, scale, n))


# 1 to 32, 33 to 64 and 65 to 96 query rows, and several row tiles, at the borders of each
MORE = [([70, 200], 16, 32, 1), ([129, 64], 64, 33, 1), ([300, 1], 48, 31, 1), ([63], 32, 63, 1), ([200, 0, 65], 64, 64, 1),
        ([640, 2], 64, 97, 1), ([100, 700], 16, 7, 16), ([500], 80, 8, 4), ([2, 1000], 64, 11, 3), ([333, 90], 256, 95, 2),
        ([64 * 9], 64, 128, 1), ([5000, 3], 64, 33, 1), ([4100], 32, 96, 2)]


@pytest.mark.parametrize("lens,size,H,m", DECODE + MORE)
def test_decode(lens, size, H, m):
    g = _gen(sum(lens) + H)
    q_lat, q_pe, cache, table = _inputs(g, lens, size, H, m)
    st = _status()
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=m, status=st)
    assert st.item() == 0
    _check(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE)


@pytest.mark.parametrize("H", [12, 48, 96])
@pytest.mark.parametrize("scale", [0.01, 30.0])
def test_decode_flat_and_sharp_scores(scale, H):
    g, lens = _gen(31), [3000, 130]
    q_lat, q_pe, cache, table = _inputs(g, lens, 64, H, 2 if H < 96 else 1, scale=scale)
    m = q_lat.shape[0] // 2
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=m)
    _check(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE)


@pytest.mark.parametrize("H", [3, 40, 96])
def test_decode_of_rows_of_different_magnitudes(H):
    """Every token's scale is another one."""
    g, lens = _gen(36), [900, 70]
    q_lat, q_pe, cache, table = _inputs(g, lens, 64, H, 1, spread=3.0)
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), 0.01)
    _check(o, lse, q_lat, q_pe, cache, table, lens, 1, 0.01)


def _scored(H, n, scores, size=64, seed=32):
    """A cache whose row j scores scores[j] for every head (scale 1), by its first positional value, and is
    otherwise random, and queries."""
    g = _gen(seed)
    table, pages = ref.make_pages(g, [n], size)
    x = torch.randn(pages, size, ROW, generator=g)
    i = torch.arange(n)
    x[..., LATENT:] = 0
    x[table[0, i // size].long(), i % size, LATENT] = scores.float()
    q_lat, q_pe = torch.zeros(1, H, LATENT), torch.zeros(1, H, POS)
    q_pe[..., 0] = 1
    q_lat[..., 1] = 0.01
    return q_lat.bfloat16().cuda(), q_pe.bfloat16().cuda(), ref.fill(_cache(pages, size), x.cuda()), table.cuda()


SCORES = {
    "rising": lambda n: torch.arange(n) * 0.5,
    "falling": lambda n: -torch.arange(n) * 0.5,
    "a first key far above": lambda n: torch.where(torch.arange(n) == 0, 24.0, 0.0),
    "a first tile far above": lambda n: torch.where(torch.arange(n) < 64, 12.0, 0.0),
    "a key far above in the middle": lambda n: torch.where(torch.arange(n) == n // 2, 30.0, 0.0),
    "every 64th key above": lambda n: torch.where(torch.arange(n) % 64 == 5, 7.0, 0.0),
    "every 64th key far above": lambda n: torch.where(torch.arange(n) % 64 == 40, 13.0, 0.0),
    "tiles in turn": lambda n: torch.where((torch.arange(n) // 64) % 2 == 0, 9.0, 0.0),
    "halves in turn": lambda n: torch.where((torch.arange(n) // 32) % 3 == 0, 11.0, 0.0),
    "steps down": lambda n: -(torch.arange(n) // 64) * 2.0,
    "a fall past every exponent": lambda n: torch.where(torch.arange(n) < 64, 0.0, -300.0),
    "a rise past every exponent": lambda n: torch.where(torch.arange(n) < n - 64, -300.0, 0.0),
}


@pytest.mark.parametrize("name", SCORES)
@pytest.mark.parametrize("H", [2, 40, 96])
def test_decode_of_scores_that_move(name, H):
    n = 1500
    scores = SCORES[name](n).to(torch.bfloat16)
    q_lat, q_pe, cache, table = _scored(H, n, scores)
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints([n]), 1.0)
    _check(o, lse, q_lat, q_pe, cache, table, [n], 1, 1.0)


@pytest.mark.parametrize("H", [2, 48, 70])
def test_decode_of_uneven_queries(H):
    """Query rows of zeros, of one value far above the others, tiny and huge ones; one of NaN and one with an
    infinity make their own row NaN alone."""
    g, lens = _gen(37), [400]
    q_lat, q_pe, cache, table = _inputs(g, lens, 64, H, 4)
    q_lat[0, 0], q_pe[0, 0] = 0, 0
    q_lat[0, 1, 5] = 300.0
    q_lat[1, 0] *= 2.0 ** -60
    q_lat[1, 1] *= 2.0 ** 60
    q_pe[1, 1] *= 0
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=4)
    keep = torch.ones(4, H, dtype=torch.bool, device="cuda")
    keep[1, 1] = False
    want = [x[keep.flatten()] for x in ref.decode_ref(q_lat, q_pe, cache, table, lens, 4, SCALE, 0)]
    ref.check_rows(o[keep], lse[keep], want)
    assert torch.isfinite(o[1, 1]).all()
    q_lat[2, 1, 9], q_lat[3, 0, 100] = NAN, float("inf")
    q_lat[1, 1] = 1
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=4)
    bad = torch.zeros(4, H, dtype=torch.bool, device="cuda")
    bad[2, 1] = bad[3, 0] = True
    assert bool(o[bad].isnan().all()) and bool(lse[bad].isnan().all())
    want = [x[~bad.flatten()] for x in ref.decode_ref(q_lat.nan_to_num(1.0, 1.0), q_pe, cache, table, lens, 4, SCALE, 0)]
    ref.check_rows(o[~bad], lse[~bad], want)


def test_decode_agrees_with_the_bf16_cache_of_the_same_values():
    """The rows read back, put into a bf16 cache: both decodes are within their bounds of the same answer."""
    from tests import latent_ref as bf

    g, lens, size = _gen(38), [700, 64, 0, 333], 64
    q_lat, q_pe, cache, table = _inputs(g, lens, size, 12, 2, tails=False)
    pages = cache.shape[0]
    rows = kda.kda_mla_gather_fp8(cache, torch.arange(pages, dtype=torch.int32, device="cuda")[:, None],
                                  _ints(_cu([size] * pages)), pages * size)
    a = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=2)
    plain = rows.view(pages, size, ROW)
    b = kda.kda_mla_decode(q_lat, q_pe, plain, table, _ints(lens), SCALE, num_tokens=2)
    _check(*a, q_lat, q_pe, cache, table, lens, 2, SCALE)
    for n in range(4):
        r = slice(2 * n, 2 * n + 2)
        x = ref.decode_ref(q_lat, q_pe, cache, table, lens, 2, SCALE, n)
        y = bf.decode_ref(q_lat, q_pe, plain, table, lens, 2, SCALE, n)
        assert bool(((a[0][r].reshape(-1, LATENT).double() - b[0][r].reshape(-1, LATENT).double()).abs() <= x[2] + y[2] + 1e-30).all())


def test_decode_pages_of_interleaved_layers():
    g, lens, size = _gen(33), [200, 90], 32
    q_lat, q_pe, cache, table = _inputs(g, lens, size, 12, 1)
    pool = torch.full((cache.shape[0], 3, size, TOKEN8), 0x7F, dtype=torch.uint8, device="cuda")
    pool[:, 1] = cache
    a = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE)
    b = kda.kda_mla_decode_fp8(q_lat, q_pe, pool[:, 1], table, _ints(lens), SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("H", [12, 40, 96])
@pytest.mark.parametrize("what,code", [("page", -9), ("negative page", -9), ("negative", -4), ("long", -4)])
def test_decode_bad_tables(what, code, H):
    """The bad sequence's rows are NaN and the others exact."""
    g, lens, size, m = _gen(34), [500, 400, 90], 16, 1 if H == 96 else 2
    q_lat, q_pe, cache, table = _inputs(g, lens, size, H, m)
    if what == "page":
        table[1, 11] = cache.shape[0]
    elif what == "negative page":
        table[1, 24] = -1
    lens_bad = list(lens)
    if what == "negative":
        lens_bad[1] = -7
    elif what == "long":
        lens_bad[1] = table.shape[1] * size + 1
    st = _status()
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens_bad), SCALE, num_tokens=m, status=st)
    assert st.item() == code
    assert bool(torch.isnan(o[m:2 * m]).all()) and bool(torch.isnan(lse[m:2 * m]).all())
    _check(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE, seqs=(0, 2))


def test_decode_of_a_cache_without_pages():
    g, lens = _gen(35), [40, 0]
    q_lat, q_pe, cache, table = _inputs(g, lens, 16, 2, 1, tails=False)
    o, lse, st = torch.zeros(2, 2, LATENT, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, device="cuda"), _status()
    ws = torch.empty(kda.kda_mla_decode_fp8_workspace_size(2, 2, 1), dtype=torch.uint8, device="cuda")
    rc = kda.library().kda_mla_decode_fp8(q_lat.data_ptr(), q_pe.data_ptr(), cache.data_ptr(), 16 * TOKEN8, 0, 16,
                                          table.data_ptr(), table.shape[1], _ints(lens).data_ptr(), 2, 2, 1, SCALE,
                                          o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), st.data_ptr(),
                                          torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and st.item() == -9
    assert o[0].isnan().all() and lse[0].isnan().all()
    assert (o[1] == 0).all() and (lse[1] == -float("inf")).all()


@pytest.mark.parametrize("H", [12, 48, 96])
def test_decode_gives_the_same_bits_again_and_on_another_stream(H):
    """A used workspace, another stream and a second call change nothing."""
    g, lens = _gen(35), [5000, 64, 700]
    q_lat, q_pe, cache, table = _inputs(g, lens, 64, H, 1)
    ws = torch.full((kda.kda_mla_decode_fp8_workspace_size(3, H, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    a = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, workspace=ws)
    b = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, workspace=ws)
    side, lens_d = torch.cuda.Stream(), _ints(lens)
    torch.cuda.synchronize()
    c = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, lens_d, SCALE, stream=side)
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


# ------------------------------------------------------------------ graphs, and all of them together
def test_a_captured_serving_step_follows_its_tables():
    """append, decode and gather captured once; lengths, page table and rows change between replays."""
    g, size, N, H = _gen(41), 16, 3, 12
    lens = [5, 100, 33]
    table, pages = ref.make_pages(g, [n + 40 for n in lens], size)
    cache, table = _random_cache(g, pages, size), table.cuda()
    lens_d, down, q = _ints(lens), _rand(g, N, ROW), _rand(g, N, H, ROW)
    tab = _rope(300)
    cu, starts = _ints(_cu([3, 3, 3])), _ints([2, 90, 30])

    def step():
        q_pe = kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table, lens_d, rope=tab,
                                      q_pe=q[..., LATENT:])
        o, lse = kda.kda_mla_decode_fp8(q[..., :LATENT].contiguous(), q_pe, cache, table, lens_d, SCALE)
        return o, lse, kda.kda_mla_gather_fp8(cache, table, cu, 9, starts=starts)

    keep = cache.clone()
    graph, out = _capture(step)
    for k in range(3):
        cache.copy_(keep)
        lens_d.copy_(_ints([n + 11 * k for n in lens]))
        starts.copy_(_ints([n - 3 + 11 * k for n in lens]))
        down.copy_(_rand(g, N, ROW))
        graph.replay()
        torch.cuda.synchronize()
        got, after = [x.clone() for x in out], cache.clone()
        cache.copy_(keep)
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(after, cache)


def test_two_graphs_share_a_workspace_in_order():
    g, lens = _gen(42), [3000, 900]
    args = [_inputs(g, lens, 64, 12, 1) for _ in range(2)]
    ws = torch.empty(kda.kda_mla_decode_fp8_workspace_size(2, 12, 1), dtype=torch.uint8, device="cuda")
    lens_d = _ints(lens)
    runs = [_capture(lambda a=a: kda.kda_mla_decode_fp8(*a, lens_d, SCALE, workspace=ws)) for a in args]
    for _ in range(2):
        for graph, _o in runs:
            graph.replay()
    torch.cuda.synchronize()
    for a, (_g, out) in zip(args, runs):
        _check(out[0], out[1], *a, lens, 1, SCALE)


def test_serving_run_across_a_fork():
    """A prompt is appended in two chunks, its prefix read back window by window and attended in the expanded form
    beside the absorbed one; the sequence is forked, both go on with tokens of their own, and a compaction moves
    the pages: the decode's bits stay."""
    g, H, size, P = _gen(43), 4, 16, 37
    pool = PagePool(24, size)
    cache = torch.full((1, 24, size, TOKEN8), 0x7F, dtype=torch.uint8, device="cuda")
    norm_w, tab, st = (1 + 0.1 * torch.randn(LATENT, generator=g)).cuda(), _rope(128), _status()
    w_k = (0.05 * torch.randn(H, NOPE, LATENT, generator=g)).cuda()
    w_v = (0.05 * torch.randn(H, NOPE, LATENT, generator=g)).cuda()
    pool.add("x")
    pool.grow("x", 50)
    pool.add("a")

    def append(names, new, q_pe):
        table, lens = pool.table(names)
        down = _rand(g, sum(new), ROW)
        q = kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache[0], table.cuda(), lens.cuda(), _ints(_cu(new)),
                                   norm_w=norm_w, rope=tab, q_pe=q_pe, status=st)
        return table.cuda(), lens.cuda(), q

    pool.grow("a", 20)
    append(["a"], [20], None)
    pool.grow("a", P - 20)
    q = _rand(g, P - 20, H, QK)
    table, lens, q_pe = append(["a"], [P - 20], q[..., NOPE:])
    rows = kda.kda_mla_gather_fp8(cache[0], table, _ints([0, P]), P, status=st)
    windows = [kda.kda_mla_gather_fp8(cache[0], table, _ints([0, b - a]), b - a, starts=_ints([a]), status=st)
               for a, b in ((0, 7), (7, 33), (33, P))]
    assert torch.equal(torch.cat(windows), rows)
    c = rows[:, :LATENT].float()
    kv = torch.cat([torch.einsum("hdl,tl->thd", w_k, c), torch.einsum("hdl,tl->thd", w_v, c)], -1).to(torch.bfloat16)
    o, lse = kda.kda_mla_prefill(torch.cat([q[..., :NOPE], q_pe], -1), kv, rows[:, LATENT:], _ints([0, P - 20]),
                                 _ints([0, P]), SCALE, status=st)
    q_lat = torch.einsum("hdl,thd->thl", w_k, q[-1:, :, :NOPE].float()).to(torch.bfloat16)
    ol, lse_l = kda.kda_mla_decode_fp8(q_lat, q_pe[-1:].contiguous(), cache[0], table, lens, SCALE, status=st)
    _check(ol, lse_l, q_lat, q_pe[-1:], cache[0], table, [P], 1, SCALE)
    # the expanded form of the last token: k_nope and v are rounded to bf16 there, q_lat here, which moves a score by
    # at most ds each and a weight by twice that; weights (2^-7 and 2^-11.9 a tile of 64 here, 2^-8 there), v and the
    # outputs are rounded besides, the latent output before W_V spreads it over 512 values
    u = 1.1 * 2.0 ** -8
    ds = u * SCALE * float((q_lat[0].float().abs() @ c.abs().T).amax() + torch.einsum(
        "hd,thd->ht", q[-1, :, :NOPE].float().abs(), kv[..., :NOPE].float().abs()).amax())
    assert float((lse_l - lse[-1:]).abs().max()) <= ds + 1e-3
    spread = float(torch.einsum("hdl,hl->hd", w_v.abs(), c.abs().amax(0).expand(H, -1)).amax())
    o_abs = torch.einsum("hdl,thl->thd", w_v, ol.float())
    assert float((o_abs - o[-1:].float()).abs().max()) <= (3 * u + 2 * ds) * float(kv[..., NOPE:].float().abs().max()) + \
        (2 + 2 + 64 * 2.0 ** -3.9) * u * spread + 1e-3

    pool.fork("a", "b")
    for s in ("a", "b"):
        kda.kda_pages_copy(cache, *pool.grow(s, 3))
    shared = kda.kda_mla_gather_fp8(cache[0], pool.table(["a", "b"])[0].cuda(), _ints([0, P, 2 * P]), 2 * P)
    assert torch.equal(shared[:P], rows) and torch.equal(shared[P:], rows)
    qd = _rand(g, 6, H, ROW)
    table, lens, q_pe = append(["a", "b"], [3, 3], qd[..., LATENT:])
    q_lat = qd[..., :LATENT].contiguous()
    before = kda.kda_mla_decode_fp8(q_lat, q_pe, cache[0], table, lens, SCALE, num_tokens=3, status=st)
    _check(*before, q_lat, q_pe, cache[0], table, [P + 3, P + 3], 3, SCALE)
    pool.free("x")
    src, dst = pool.compact()
    assert src
    kda.kda_pages_copy(cache, src, dst)
    cache[0, pool.num_pages - pool.free_pages:] = 0x7F
    table, lens = [t.cuda() for t in pool.table(["a", "b"])]
    after = kda.kda_mla_decode_fp8(q_lat, q_pe, cache[0], table, lens, SCALE, num_tokens=3, status=st)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1]) and st.item() == 0
