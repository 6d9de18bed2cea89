"""The latent-attention operators and the page copies on the GPU against plain 64-bit forms
(tests/latent_ref.py, which derives the bounds)."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from linear_attention_serving_02_gb300.paging import PagePool
from tests import latent_ref as ref

pytestmark = pytest.mark.gpu

LATENT, POS, ROW, NOPE, QK = 512, 64, 576, 128, 192
SCALE = QK ** -0.5
NAN = float("nan")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16).cuda()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _rope(n):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([ang.cos(), ang.sin()], 1).float().cuda()


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
    cache = _rand(g, pages, size, ROW)
    was, w = cache.clone(), (1 + 0.1 * torch.randn(LATENT, generator=g)).cuda() if norm else None
    tab, st = _rope(max(lens)) if rope else None, _status()
    q_out = kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table_d, _ints(lens),
                               _ints(_cu(new)) if cu else None, norm_w=w, eps=1e-5, rope=tab,
                               rope_interleaved=interleaved, q_pe=q[..., NOPE:] if rope else None, status=st)
    assert st.item() == 0
    seq = [n for n, k in enumerate(new) for _ in range(k)]
    pos = [before[n] + i for n, k in enumerate(new) for i in range(k)]
    at = [int(table[n, p // size]) * size + p % size for n, p in zip(seq, pos)]
    c, pe = down[:, :LATENT].double(), down[:, LATENT:].double()
    if norm:
        c = c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    got = cache.view(-1, ROW)[torch.tensor(at, device="cuda")]
    # the sum of 512 squares, its root and two products in fp32, then one rounding
    tol_c = (ref.U_BF16 + 300 * 2.0 ** -23) * c.abs()
    if not norm:
        assert torch.equal(got[:, :LATENT], down[:, :LATENT])
    assert bool(((got[:, :LATENT].double() - c).abs() <= tol_c).all())
    if rope:
        cos, sin = tab[torch.tensor(pos)].double().split(32, 1)
        # two products and a sum in fp32 of terms up to |a| + |b| <= 2 max
        def close(x, r, raw):
            return bool(((x.double() - r).abs() <= ref.U_BF16 * 1.001 * r.abs() + 2.0 ** -21 * raw.abs().amax()).all())
        assert close(got[:, LATENT:], ref.rotate_ref(pe, cos, sin, interleaved), pe)
        qr = q[..., NOPE:].double()
        assert close(q_out, ref.rotate_ref(qr, cos[:, None], sin[:, None], interleaved), qr)
    else:
        assert q_out is None and torch.equal(got[:, LATENT:], down[:, LATENT:])
    left = torch.ones(pages * size, dtype=torch.bool, device="cuda")
    left[torch.tensor(at)] = False
    assert torch.equal(cache.view(-1, ROW)[left], was.view(-1, ROW)[left])


def test_append_rotates_queries_in_place_and_leaves_padding_alone():
    g = _gen(3)
    new, lens, size = [3, 2], [20, 40], 16
    table, pages = ref.make_pages(g, lens, size)
    T = 9  # four rows behind the last sequence
    down, q, cache = _rand(g, T, ROW), _rand(g, T, 4, QK), _rand(g, pages, size, ROW)
    tab, was = _rope(40), q.clone()
    out = kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table.cuda(), _ints(lens), _ints(_cu(new)),
                             rope=tab, q_pe=q[..., NOPE:], q_out=q[..., NOPE:])
    sep = kda.kda_mla_append(down[:5, :LATENT], down[:5, LATENT:], cache, table.cuda(), _ints(lens), _ints(_cu(new)),
                             rope=tab, q_pe=was[:5, :, NOPE:])
    assert out.data_ptr() == q[..., NOPE:].data_ptr() and torch.equal(q[:5, :, NOPE:], sep)
    assert torch.equal(q[..., :NOPE], was[..., :NOPE]) and torch.equal(q[5:], was[5:])


def test_append_of_one_token_and_head_with_odd_strides():
    """A dimension of one has no step: whatever its stride says, the call is taken."""
    g, rope = _gen(7), _rope(8)
    down, q = _rand(g, 1, ROW), _rand(g, 1, 1, POS)
    table, lens = _ints([[0]]), _ints([5])
    outs = []
    for odd in (False, True):
        cache, q_out = torch.zeros(1, 16, ROW, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(q)
        views = [x.as_strided((1, 1, POS), (1001, 77, 1)) if odd else x for x in (q, q_out)]
        c, k_pe = down[:, :LATENT], down[:, LATENT:]
        if odd:
            c, k_pe = c.as_strided((1, LATENT), (7, 1)), k_pe.as_strided((1, POS), (3, 1), LATENT)
        kda.kda_mla_append(c, k_pe, cache, table, lens, _ints([0, 1]), rope=rope, q_pe=views[0], q_out=views[1])
        outs.append((cache, q_out))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert (outs[0][1] != 0).any()


@pytest.mark.parametrize("what,code", [("page", -9), ("short", -4), ("long", -4), ("rope", -4)])
def test_append_bad_tables(what, code):
    g = _gen(5)
    size, lens = 16, [20, 30, 25]
    table, pages = ref.make_pages(g, lens, size)
    down, q, cache = _rand(g, 6, ROW), _rand(g, 6, 2, POS), _rand(g, pages, size, ROW)
    tab = _rope(30 if what != "rope" else 29)
    if what == "page":
        table[1, 1] = pages
    elif what == "short":
        lens[1] = 0
    elif what == "long":
        lens[1] = table.shape[1] * size + 2
        tab = _rope(200)
    was, st = cache.clone(), _status()
    q_out = kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table.cuda(), _ints(lens), None, rope=tab,
                               q_pe=q, status=st)
    assert st.item() == code and kda.kda_workspace_status(st) == code
    bad = {"rope": [3]}.get(what, [2, 3])
    bad = torch.tensor([i in bad for i in range(6)], device="cuda")
    assert torch.equal(torch.isnan(q_out).all(-1).all(-1), bad) and not torch.isnan(q_out[~bad]).any()
    changed = (cache != was).any(-1)
    assert int(changed.sum()) == 6 - int(bad.sum())


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("lens,size", [([1], 16), ([0, 5, 0, 0, 33, 16, 0], 16), ([700, 1, 64], 64), ([3] * 70, 48)])
def test_gather(lens, size):
    g = _gen(sum(lens))
    table, pages = ref.make_pages(g, lens, size)
    big = _rand(g, pages, 2, size, ROW)  # two layers in turn: a page stride of two pages
    cache, st = big[:, 1], _status()
    T = sum(lens)
    out = torch.full((T + 7, ROW), 5.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_mla_gather(cache, table.cuda(), _ints(_cu(lens)), T + 7, out=out, status=st)
    want = torch.cat([ref.cached_rows(cache, table[n].cuda(), k) for n, k in enumerate(lens)])
    assert st.item() == 0 and torch.equal(out[:T], want) and bool((out[T:] == 5).all())


def test_gather_bad_page_and_length():
    g = _gen(9)
    lens, size = [20, 40, 5], 16
    table, pages = ref.make_pages(g, lens, size)
    cache = _rand(g, pages, size, ROW)
    table[1, 1] = -3
    st = _status()
    out = kda.kda_mla_gather(cache, table.cuda(), _ints(_cu(lens)), 65, status=st)
    bad = torch.zeros(65, dtype=torch.bool, device="cuda")
    bad[36:52] = True
    assert st.item() == -9 and torch.equal(torch.isnan(out).all(1), bad)
    lens[2] = table.shape[1] * size + 1
    st = _status()
    table[1, 1], table[2] = 0, 1
    out = kda.kda_mla_gather(cache, table.cuda(), _ints(_cu(lens)), sum(lens), status=st)
    assert st.item() == -4 and bool(torch.isnan(out[-1]).all()) and not torch.isnan(out[:-1]).any()


# ------------------------------------------------------------------ prefill
PREFILL = [
    # new, prefix, H, causal
    ([1], [0], 1, True),
    ([1], [0], 2, False),
    ([1, 1, 1], [5, 127, 128], 3, True),
    ([127], [0], 2, True),
    ([128], [0], 2, True),
    ([129], [0], 2, True),
    ([256], [0], 2, True),
    ([257, 0, 300], [0, 9, 77], 3, True),
    ([300], [1000], 1, True),
    ([300, 20], [1000, 5], 1, False),
    ([1000], [0], 2, True),
    ([70] * 9, [0, 1, 2, 63, 64, 65, 127, 128, 129], 2, True),
    ([640, 513], [128, 255], 5, True),
]


def _prefill_inputs(g, new, total, H, pad_q=0, pad_k=0, scale=1.0):
    tq, tk = sum(new) + pad_q, sum(total) + pad_k
    return _rand(g, tq, H, QK, scale=scale), _rand(g, tk, H, 2 * NOPE), _rand(g, tk, ROW)[:, LATENT:]


@pytest.mark.parametrize("new,prefix,H,causal", PREFILL)
def test_prefill(new, prefix, H, causal):
    g = _gen(sum(new) + sum(prefix))
    total = [a + b for a, b in zip(new, prefix)]
    q, kv, pe = _prefill_inputs(g, new, total, H)
    cu_q, cu_k, st = _cu(new), _cu(total), _status()
    o, lse = kda.kda_mla_prefill(q, kv, pe, _ints(cu_q), _ints(cu_k), SCALE, causal=causal, status=st)
    assert st.item() == 0
    for n in range(len(new)):
        for h in range(H):
            a, b = cu_q[n], cu_q[n + 1]
            ref.check_rows(o[a:b, h], lse[a:b, h], ref.prefill_ref(q, kv, pe, cu_q, cu_k, SCALE, causal, n, h))


@pytest.mark.parametrize("scale", [0.01, 30.0])
def test_prefill_flat_and_sharp_scores(scale):
    """Nearly uniform weights, and scores of hundreds whose maximum moves from tile to tile."""
    g = _gen(21)
    q, kv, pe = _prefill_inputs(g, [500], [900], 2, scale=scale)
    o, lse = kda.kda_mla_prefill(q, kv, pe, _ints([0, 500]), _ints([0, 900]), SCALE)
    for h in range(2):
        ref.check_rows(o[:, h], lse[:, h], ref.prefill_ref(q, kv, pe, [0, 500], [0, 900], SCALE, True, 0, h))


def test_prefill_rising_scores():
    """Every key scores higher than the one before, over a range far past a float's exponent."""
    g = _gen(22)
    q, kv, pe = _prefill_inputs(g, [300], [700], 1)
    q[:] = 0
    q[..., 0] = 8
    kv[:, 0, 0] = torch.arange(700, device="cuda").to(torch.bfloat16)
    for sign in (1, -1):
        kv[:, 0, 0] *= sign
        o, lse = kda.kda_mla_prefill(q, kv, pe, _ints([0, 300]), _ints([0, 700]), 1.0)
        ref.check_rows(o[:, 0], lse[:, 0], ref.prefill_ref(q, kv, pe, [0, 300], [0, 700], 1.0, True, 0, 0))


def test_prefill_rows_that_see_nothing_and_rows_of_no_sequence():
    """More queries than keys under the causal mask, sequences without keys, NaN and infinities in every row
    that belongs to no sequence or to another one, and output rows of no sequence left alone."""
    g = _gen(23)
    new, total, H = [200, 40, 0, 3], [150, 0, 30, 70], 2
    cu_q, cu_k = [x + 5 for x in _cu(new)], [x + 9 for x in _cu(total)]
    q, kv, pe = _prefill_inputs(g, new, total, H, pad_q=12, pad_k=20)
    good_q, good_kv = q.clone(), kv.clone()
    q[:5], q[cu_q[-1]:], kv[:9], pe[:9] = NAN, NAN, float("inf"), NAN
    kv[cu_k[-1]:], pe[cu_k[-1]:] = NAN, float("-inf")
    kv[cu_k[2]:cu_k[3]], pe[cu_k[2]:cu_k[3]] = NAN, NAN  # keys of the sequence without queries
    for causal in (True, False):
        st = _status()
        o = torch.full((q.shape[0], H, NOPE), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((q.shape[0], H), 7.0, device="cuda")
        kda.kda_mla_prefill(q, kv, pe, _ints(cu_q), _ints(cu_k), SCALE, causal=causal, o=o, lse=lse, status=st)
        assert st.item() == 0
        for n in (0, 1, 3):
            for h in range(H):
                a, b = cu_q[n], cu_q[n + 1]
                ref.check_rows(o[a:b, h], lse[a:b, h],
                               ref.prefill_ref(good_q, good_kv, pe, cu_q, cu_k, SCALE, causal, n, h))
        for x in (o, lse):
            assert bool((x[:5] == 7).all()) and bool((x[cu_q[-1]:] == 7).all())


def test_prefill_bad_offsets_leave_the_sequence_alone():
    g = _gen(24)
    q, kv, pe = _prefill_inputs(g, [100, 60], [100, 60], 1)
    for cu_q, cu_k in (([0, 100, 400], [0, 100, 160]), ([0, 100, 160], [0, 100, 400]), ([0, 100, 160], [0, 100, 90]),
                       ([0, 100, 160], [0, 100, -5])):
        st = _status()
        o = torch.full((160, 1, NOPE), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((160, 1), 7.0, device="cuda")
        kda.kda_mla_prefill(q, kv, pe, _ints(cu_q), _ints(cu_k), SCALE, o=o, lse=lse, status=st)
        assert st.item() == -4 and bool((o[100:] == 7).all()) and bool((lse[100:] == 7).all())
        ref.check_rows(o[:100, 0], lse[:100, 0], ref.prefill_ref(q, kv, pe, [0, 100], [0, 100], SCALE, True, 0, 0))


# ------------------------------------------------------------------ decode
DECODE = [
    # lens, page size, H, m
    ([1], 16, 1, 1),
    ([0, 1, 2, 15, 16, 17], 16, 2, 1),
    ([63, 64, 65, 127, 128, 129], 64, 12, 1),
    ([300, 5], 32, 12, 4),
    ([3, 0, 16, 15, 200], 48, 5, 16),       # windows longer than their sequences: rows that see nothing
    ([1000, 77], 128, 64, 1),
    ([500, 64], 64, 65, 1),
    ([700, 333, 64], 64, 96, 1),
    ([257], 256, 128, 2),
    ([190, 300], 80, 24, 3),
    ([20000], 64, 12, 1),
    ([9000, 1, 0, 4000], 64, 16, 2),
    ([100 + 7 * i for i in range(170)], 16, 3, 1),
    # several row tiles: 384, 130 and 2000 query rows
    ([300, 0, 71], 64, 96, 4),
    ([513, 2], 32, 130, 1),
    ([100, 40], 16, 125, 16),
    ([40 + 5 * i for i in range(160)], 64, 72, 1),
    ([6000, 1], 64, 96, 1),
    # one and two row tiles of more than 64 rows
    ([500, 31, 0], 16, 80, 1),
    ([200, 1, 65], 48, 12, 8),
    ([300, 40, 0], 64, 96, 2),
    ([129, 4000], 32, 65, 2),
    # eight row tiles of 56 rows, the last one without any (385 and 388 query rows)
    ([70, 200, 0], 16, 77, 5),
    ([64], 64, 97, 4),
]


def _decode_inputs(g, lens, size, H, m, scale=1.0, tails=True):
    table, pages = ref.make_pages(g, lens, size)
    N = len(lens)
    cache = _rand(g, pages, size, ROW)
    if tails:  # NaN and infinities in every row that no sequence has
        used = torch.zeros(pages * size, dtype=torch.bool)
        for n, k in enumerate(lens):
            i = torch.arange(max(0, k))
            used[table[n, i // size].long() * size + i % size] = True
        cache.view(-1, ROW)[~used.cuda()] = NAN
        cache.view(-1, ROW)[~used.cuda(), ::3] = float("inf")
    return _rand(g, N * m, H, LATENT, scale=scale), _rand(g, N * m, H, POS, scale=scale), cache, table.cuda()


def _check_decode(o, lse, q_lat, q_pe, cache, table, lens, m, scale, seqs=None):
    H = q_lat.shape[1]
    for n in range(len(lens)) if seqs is None else seqs:
        r = slice(n * m, (n + 1) * m)
        ref.check_rows(o[r].reshape(m * H, LATENT), lse[r].reshape(-1),
                       ref.decode_ref(q_lat, q_pe, cache, table, lens, m, scale, n))


@pytest.mark.parametrize("lens,size,H,m", DECODE)
def test_decode(lens, size, H, m):
    g = _gen(sum(lens) + H)
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, size, H, m)
    st = _status()
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=m, status=st)
    assert st.item() == 0
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE)


@pytest.mark.parametrize("scale", [0.01, 30.0])
def test_decode_flat_and_sharp_scores(scale):
    g, lens = _gen(31), [3000, 130]
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, 64, 12, 2, scale=scale)
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=2)
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, 2, SCALE)


def test_decode_rising_scores():
    g, lens = _gen(32), [700, 1]
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, 64, 3, 1, tails=False)
    q_lat[:], q_pe[:] = 0, 0
    q_lat[..., 0] = torch.tensor([8.0, -8.0, 1.0]).cuda().to(torch.bfloat16)
    i = torch.arange(700)
    cache[table[0, (i // 64).cuda()].long(), (i % 64).cuda(), 0] = i.cuda().to(torch.bfloat16)
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), 1.0)
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, 1, 1.0)


def test_decode_pages_of_interleaved_layers():
    g, lens, size = _gen(33), [200, 90], 32
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, size, 12, 1)
    pool = torch.full((cache.shape[0], 3, size, ROW), NAN, dtype=torch.bfloat16, device="cuda")
    pool[:, 1] = cache
    a = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE)
    b = kda.kda_mla_decode(q_lat, q_pe, pool[:, 1], table, _ints(lens), SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("what,code", [("page", -9), ("negative page", -9), ("negative", -4), ("long", -4)])
def test_decode_bad_tables(what, code):
    """The bad sequence's rows are NaN and the others exact."""
    g, lens, size, H, m = _gen(34), [500, 400, 90], 16, 12, 2
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, size, H, m)
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
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens_bad), SCALE, num_tokens=m, status=st)
    assert st.item() == code
    assert bool(torch.isnan(o[m:2 * m]).all()) and bool(torch.isnan(lse[m:2 * m]).all())
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE, seqs=(0, 2))


def test_decode_of_a_cache_without_pages():
    g, lens = _gen(35), [40, 0]
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, 16, 2, 1, tails=False)
    o, lse, st = torch.zeros(2, 2, LATENT, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, device="cuda"), _status()
    ws = torch.empty(kda.kda_mla_decode_workspace_size(2, 2, 1), dtype=torch.uint8, device="cuda")
    rc = kda.library().kda_mla_decode(q_lat.data_ptr(), q_pe.data_ptr(), cache.data_ptr(), 16 * ROW, 0, 16,
                                      table.data_ptr(), table.shape[1], _ints(lens).data_ptr(), 2, 2, 1, SCALE, o.data_ptr(),
                                      lse.data_ptr(), ws.data_ptr(), ws.numel(), st.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and st.item() == -9
    assert o[0].isnan().all() and lse[0].isnan().all()
    assert (o[1] == 0).all() and (lse[1] == -float("inf")).all()


def test_decode_gives_the_same_bits_again_and_on_another_stream():
    """A used workspace, another stream and a second call change nothing."""
    g, lens = _gen(35), [5000, 64, 700]
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, 64, 12, 1)
    ws = torch.full((kda.kda_mla_decode_workspace_size(3, 12, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    a = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE, workspace=ws)
    b = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE, workspace=ws)
    side, lens_d = torch.cuda.Stream(), _ints(lens)
    torch.cuda.synchronize()
    c = kda.kda_mla_decode(q_lat, q_pe, cache, table, lens_d, SCALE, stream=side)
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


# ------------------------------------------------------------------ page copies
@pytest.mark.parametrize("shape,dtype,swap", [
    ((1, 9, 16), torch.uint8, False), ((3, 9, 16, ROW), torch.bfloat16, False),
    ((9, 3, 16, ROW), torch.bfloat16, True), ((2, 9, 5, 128, 128), torch.float32, False),
    ((2, 9, 4097, 16), torch.uint8, False)])
def test_pages_copy_in_list_order(shape, dtype, swap):
    """Chains, pages written twice, pages copied onto themselves."""
    pool = torch.randint(0, 100, shape, device="cuda").to(dtype)
    if swap:
        pool = pool.transpose(0, 1)
    src, dst = [0, 1, 2, 4, 3, 8, 0, 5, 5], [1, 2, 3, 4, 0, 7, 8, 6, 1]
    want = pool.clone()
    for a, b in zip(src, dst):
        want[:, b] = want[:, a].clone()
    assert kda.kda_pages_copy(pool, src, dst) is pool
    assert torch.equal(pool, want)
    kda.kda_pages_copy(pool, [], [])
    assert torch.equal(pool, want)


@pytest.mark.parametrize("n", [31, 33, 481, 2001, 4500])
def test_pages_copy_of_long_lists(n):
    pool = torch.randint(0, 1 << 30, (2, 2 * n, 64), dtype=torch.int32, device="cuda")
    order = torch.randperm(2 * n, generator=_gen(n))
    src, dst = order[:n], order[n:]
    want = pool.clone()
    want[:, dst.cuda()] = pool[:, src.cuda()]
    kda.kda_pages_copy(pool, src, dst)
    assert torch.equal(pool, want)


# ------------------------------------------------------------------ graphs, and all of them together
def _capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    return g, out


def test_a_captured_serving_step_follows_its_tables():
    """append, decode and gather captured once; lengths, page table and rows change between replays."""
    g, size, N, H = _gen(41), 16, 3, 12
    lens = [5, 100, 33]
    table, pages = ref.make_pages(g, [n + 40 for n in lens], size)
    cache, table = _rand(g, pages, size, ROW), table.cuda()
    lens_d, down, q = _ints(lens), _rand(g, N, ROW), _rand(g, N, H, ROW)
    tab = _rope(300)
    cu = _ints(_cu([20, 20, 20]))

    def step():
        q_pe = kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table, lens_d, rope=tab,
                                  q_pe=q[..., LATENT:])
        o, lse = kda.kda_mla_decode(q[..., :LATENT].contiguous(), q_pe, cache, table, lens_d, SCALE)
        return o, lse, kda.kda_mla_gather(cache, table, cu, 60)

    keep = cache.clone()
    graph, out = _capture(step)
    for k in range(3):
        cache.copy_(keep)
        lens_d.copy_(_ints([n + 11 * k for n in lens]))
        down.copy_(_rand(g, N, ROW))
        graph.replay()
        torch.cuda.synchronize()
        got, after = [x.clone() for x in out], cache.clone()
        cache.copy_(keep)
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())
        assert torch.equal(after, cache)


def test_two_graphs_share_a_workspace_in_order():
    g, lens = _gen(42), [3000, 900]
    args = [_decode_inputs(g, lens, 64, 12, 1) for _ in range(2)]
    ws = torch.empty(kda.kda_mla_decode_workspace_size(2, 12, 1), dtype=torch.uint8, device="cuda")
    lens_d = _ints(lens)
    runs = [_capture(lambda a=a: kda.kda_mla_decode(*a, lens_d, SCALE, workspace=ws)) for a in args]
    for _ in range(2):
        for graph, _o in runs:
            graph.replay()
    torch.cuda.synchronize()
    for a, (_g, out) in zip(args, runs):
        _check_decode(out[0], out[1], *a, lens, 1, SCALE)


def test_serving_run_expanded_and_absorbed_forms_agree_across_a_fork():
    """A prompt is appended, gathered and attended in the expanded form, with W_K and W_V applied by
    torch; the sequence is forked and both go on with other tokens through decode; a compaction
    moves the pages. The last token's outputs of both forms agree with the 64-bit form, and
    the KDA state slots are copied along by the same call."""
    g, H, size, P = _gen(43), 4, 16, 37
    pool = PagePool(24, size)
    cache = torch.full((1, 24, size, ROW), NAN, dtype=torch.bfloat16, device="cuda")
    states = torch.randn((2, 4, H, 128, 128), device="cuda")
    w_k, w_v = (0.05 * torch.randn(H, NOPE, LATENT, generator=g)).cuda(), (0.05 * torch.randn(H, NOPE, LATENT, generator=g)).cuda()
    norm_w, tab, st = (1 + 0.1 * torch.randn(LATENT, generator=g)).cuda(), _rope(128), _status()
    # another sequence first, freed later, so that compaction has holes to fill
    pool.add("x")
    pool.grow("x", 50)
    pool.add("a")

    def append(seq_names, new, q_pe):
        table, lens = pool.table(seq_names)
        down = _rand(g, sum(new), ROW)
        q = kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache[0], table.cuda(), lens.cuda(), _ints(_cu(new)),
                               norm_w=norm_w, rope=tab, q_pe=q_pe, status=st)
        return table.cuda(), lens.cuda(), q

    pool.grow("a", P)
    q = _rand(g, P, H, QK)
    table, lens, q_pe = append(["a"], [P], q[..., NOPE:])
    rows = kda.kda_mla_gather(cache[0], table, _ints([0, P]), P, status=st)
    c = rows[:, :LATENT].float()
    kv = torch.cat([torch.einsum("hdl,tl->thd", w_k, c), torch.einsum("hdl,tl->thd", w_v, c)], -1).to(torch.bfloat16)
    o, lse = kda.kda_mla_prefill(torch.cat([q[..., :NOPE], q_pe], -1), kv, rows[:, LATENT:], _ints([0, P]), _ints([0, P]),
                                 SCALE, status=st)
    # the absorbed form of the prompt's last token
    q_lat = torch.einsum("hdl,thd->thl", w_k, q[-1:, :, :NOPE].float()).to(torch.bfloat16)
    ol, lse_l = kda.kda_mla_decode(q_lat, q_pe[-1:].contiguous(), cache[0], table, lens, SCALE, status=st)
    _check_decode(ol, lse_l, q_lat, q_pe[-1:], cache[0], table, [P], 1, SCALE)
    o_abs = torch.einsum("hdl,thl->thd", w_v, ol.float())
    # each form rounds its up-projected operand to bf16 (k_nope and v here, q_lat there), which moves a
    # score by at most ds; weights move by 2 ds, and p, v and o are rounded once each, ol once more
    # before W_V spreads its rounding over 512 values
    u = 1.1 * ref.U_BF16
    ds = u * SCALE * float((q_lat[0].float().abs() @ c.abs().T).amax() + torch.einsum(
        "hd,thd->ht", q[-1, :, :NOPE].float().abs(), kv[..., :NOPE].float().abs()).amax())
    assert float((lse_l - lse[-1:]).abs().max()) <= ds + 1e-3
    spread = float(torch.einsum("hdl,hl->hd", w_v.abs(), c.abs().amax(0).expand(H, -1)).amax())
    assert float((o_abs - o[-1:].float()).abs().max()) <= (3 * u + 2 * ds) * float(kv[..., NOPE:].float().abs().max()) + \
        2 * u * spread + 1e-3

    pool.fork("a", "b")
    kda.kda_pages_copy(states, [0], [1])
    assert torch.equal(states[:, 0], states[:, 1])
    for s in ("a", "b"):
        kda.kda_pages_copy(cache, *pool.grow(s, 3))
    shared = kda.kda_mla_gather(cache[0], pool.table(["a", "b"])[0].cuda(), _ints([0, P, 2 * P]), 2 * P)
    assert torch.equal(shared[:P], rows) and torch.equal(shared[P:], rows)
    qd = _rand(g, 6, H, ROW)
    table, lens, q_pe = append(["a", "b"], [3, 3], qd[..., LATENT:])
    q_lat = qd[..., :LATENT].contiguous()
    before = kda.kda_mla_decode(q_lat, q_pe, cache[0], table, lens, SCALE, num_tokens=3, status=st)
    _check_decode(*before, q_lat, q_pe, cache[0], table, [P + 3, P + 3], 3, SCALE)
    pool.free("x")
    src, dst = pool.compact()
    assert src
    kda.kda_pages_copy(cache, src, dst)
    cache[0, pool.num_pages - pool.free_pages:] = NAN
    table, lens = [t.cuda() for t in pool.table(["a", "b"])]
    after = kda.kda_mla_decode(q_lat, q_pe, cache[0], table, lens, SCALE, num_tokens=3, status=st)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1]) and st.item() == 0
