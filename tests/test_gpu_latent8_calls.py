"""Calls of the 8-bit cache's operators as a serving program makes them: other streams, several at once, captured
and replayed, far offsets, many short sequences, pages used twice, calls of nothing."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent8_ref as ref
from tests.test_gpu_latent import (LATENT, NOPE, POS, QK, ROW, SCALE, _capture, _cu, _gen, _ints, _rand, _rope, _status)
from tests.test_gpu_latent8 import TOKEN8, _cache, _check, _inputs, _random_cache

pytestmark = pytest.mark.gpu


def _calls(seed, H=12):
    """The three calls on inputs of their own; each returns the tensors it wrote."""
    g, size, lens, new = _gen(seed), 32, [300, 41], [70, 5]
    q_lat, q_pe, cache, table = _inputs(g, lens, size, H, 1, tails=False)
    q, down, rope = _rand(g, sum(new), 3, QK), _rand(g, sum(new), ROW), _rope(300)
    lens_d, cu_q, cu_k, starts = _ints(lens), _ints(_cu(new)), _ints([0, 90, 121]), _ints([210, 10])
    ws = torch.empty(kda.kda_mla_decode_fp8_workspace_size(2, H, 1), dtype=torch.uint8, device="cuda")
    work = torch.empty_like(cache)

    def append(stream=None):
        with torch.cuda.stream(stream):
            work.copy_(cache)
        out = kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], work, table, lens_d, cu_q, rope=rope,
                                     q_pe=q[..., NOPE:], stream=stream)
        return work, out

    return [append,
            lambda stream=None: (kda.kda_mla_gather_fp8(cache, table, cu_k, 121, starts=starts, stream=stream),),
            lambda stream=None: kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, lens_d, SCALE, workspace=ws, stream=stream)]


@pytest.mark.parametrize("which", range(3))
def test_another_stream_and_a_captured_call_give_the_same_bits(which):
    call = _calls(50)[which]
    want = [x.clone() for x in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, out = _capture(call)
    for _ in range(2):
        for x in out:
            x.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("H", [12, 48, 96])
def test_two_streams_at_once(H):
    runs, side = [_calls(51, H), _calls(52, H)], [torch.cuda.Stream(), torch.cuda.Stream()]
    want = [[[x.clone() for x in call()] for call in calls] for calls in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[call(s) for call in calls] for calls, s in zip(runs, side)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for u, v in zip(a, b) for x, y in zip(u, v))


def test_graphs_of_two_streams_with_workspaces_of_their_own():
    calls, side = [_calls(53)[2], _calls(54, 96)[2]], [torch.cuda.Stream(), torch.cuda.Stream()]
    want = [[x.clone() for x in call()] for call in calls]
    runs = [_capture(call) for call in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for (graph, _), s in zip(runs, side):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), w in zip(runs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_cache_past_two_to_the_32():
    """Pages behind byte 2^32 of the cache, appended, read back and attended."""
    g, size, H, pages = _gen(55), 64, 2, 110000
    cache = torch.empty(pages, size, TOKEN8, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 32
    lens = [150, 64]
    table = _ints([[109999, 3, 109000], [108990, -1, -1]])
    down = _rand(g, sum(lens), ROW)
    kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table, _ints(lens), _ints(_cu(lens)))
    rows = kda.kda_mla_gather_fp8(cache, table, _ints(_cu(lens)), sum(lens))
    b, s = ref.quantise(down)
    assert torch.equal(rows, (ref.codes(b) * s.double()[:, None]).to(torch.bfloat16))
    q_lat, q_pe = _rand(g, 2, H, LATENT), _rand(g, 2, H, POS)
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE)
    _check(o, lse, q_lat, q_pe, cache, table, lens, 1, SCALE)


@pytest.mark.parametrize("count", [33, 1500])
@pytest.mark.parametrize("size", [16, 80])
def test_many_short_sequences(count, size):
    """More sequences than a warp looks at in one round and than there are SMs, empty ones among them."""
    g = _gen(count)
    new = [(7 * n) % 4 for n in range(count)]
    lens = [a + (5 * n) % 23 for n, a in enumerate(new)]
    cu_q, cu_k, st = _cu(new), _cu(lens), _status()
    table, pages = ref.make_pages(g, lens, size)
    cache, table = _random_cache(g, pages, size), table.cuda()
    down = _rand(g, sum(new), ROW)
    kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table, _ints(lens), _ints(cu_q), status=st)
    rows = kda.kda_mla_gather_fp8(cache, table, _ints(cu_k), sum(lens), status=st)
    values = [ref.cached(cache, table[n], k) for n, k in enumerate(lens)]
    assert torch.equal(rows, torch.cat([c * s[:, None] for c, s in values]).to(torch.bfloat16))
    b, s = ref.quantise(down)
    down8 = (ref.codes(b) * s.double()[:, None]).to(torch.bfloat16)
    for n in range(count):
        k, a = cu_k[n + 1], new[n]
        assert a == 0 or torch.equal(rows[k - a:k], down8[cu_q[n]:cu_q[n + 1]])
    for H in (12, 50, 96):
        q_lat, q_pe = _rand(g, count, H, LATENT), _rand(g, count, H, POS)
        o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, status=st)
        _check(o, lse, q_lat, q_pe, cache, table, lens, 1, SCALE, seqs=range(0, count, 1 if count < 100 else 13))
    assert st.item() == 0


def test_a_page_twice_in_one_sequence_and_in_two():
    g, size, H = _gen(56), 32, 12
    cache = _random_cache(g, 4, size)
    table, lens = _ints([[2, 0, 2, 2, 1], [2, 0, 3, -1, -1]]), [150, 70]
    q_lat, q_pe = _rand(g, 4, H, LATENT), _rand(g, 4, H, POS)
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=2)
    _check(o, lse, q_lat, q_pe, cache, table, lens, 2, SCALE)
    rows = kda.kda_mla_gather_fp8(cache, table, _ints(_cu(lens)), sum(lens))
    values = [ref.cached(cache, table[n], k) for n, k in enumerate(lens)]
    assert torch.equal(rows, torch.cat([c * s[:, None] for c, s in values]).to(torch.bfloat16))


def test_calls_of_nothing_write_nothing():
    g = _gen(57)
    cache = _random_cache(g, 2, 16)
    was, none, one, st = cache.clone(), _ints([]), _ints([0]), _status()
    no_table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    kda.kda_mla_append_fp8(_rand(g, 0, LATENT), _rand(g, 0, POS), cache, no_table, none, one, status=st)
    kda.kda_mla_append_fp8(_rand(g, 5, LATENT), _rand(g, 5, POS), cache, no_table, none, one, status=st)
    out = torch.full((4, ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_mla_gather_fp8(cache, no_table, one, 4, out=out, status=st)
    kda.kda_mla_gather_fp8(cache, _ints([[0, 1, 0]]), _ints([0, 0]), 4, out=out, starts=_ints([20]), status=st)
    assert bool((out == 7).all())
    o, lse = kda.kda_mla_decode_fp8(_rand(g, 0, 2, LATENT), _rand(g, 0, 2, POS), cache, no_table, none, SCALE, status=st)
    assert o.shape == (0, 2, LATENT) and lse.shape == (0, 2)
    # sequences without rows: zeros and -inf
    o, lse = kda.kda_mla_decode_fp8(_rand(g, 6, 40, LATENT), _rand(g, 6, 40, POS), cache, _ints([[5]] * 3), _ints([0, 0, 0]),
                                    SCALE, num_tokens=2, status=st)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
    torch.cuda.synchronize()
    assert st.item() == 0 and torch.equal(cache, was)


def test_the_status_word_is_never_cleared():
    g, lens = _gen(58), [40]
    q_lat, q_pe, cache, table = _inputs(g, lens, 16, 2, 1)
    st = torch.full((1,), -4, dtype=torch.int32, device="cuda")
    kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, status=st)
    kda.kda_mla_gather_fp8(cache, table, _ints(_cu(lens)), 40, status=st)
    assert st.item() == -4


@pytest.mark.parametrize("H,m", [(2, 1), (48, 1), (96, 1), (96, 4)])
def test_calls_that_follow_one_another_wait_for_one_another(H, m):
    """Each call reads what the one before it wrote, and writes what it read: without any pause between
    them, and as one graph, they give the bits of calls with a synchronisation behind each."""
    g, size, lens = _gen(59 + H), 32, [700, 90, 33]
    N = len(lens)
    q0, p0, cache0, table = _inputs(g, lens, size, H, m, tails=False)
    down0, rope, lens_d, cu = _rand(g, N * m, ROW), _rope(800), _ints(lens), _ints(_cu(lens))
    cu_q = _ints(_cu([m] * N))
    ws = torch.empty(kda.kda_mla_decode_fp8_workspace_size(N, H, m), dtype=torch.uint8, device="cuda")
    q, cache, down = q0.clone(), cache0.clone(), down0.clone()
    q_pe, o, lse = p0.clone(), torch.empty_like(q0), torch.empty(N * m, H, device="cuda")
    rows = torch.empty(sum(lens), ROW, dtype=torch.bfloat16, device="cuda")
    src, dst = [int(table[1, 0])], [int(table[0, 3])]

    def chain(pause):
        q.copy_(q0), cache.copy_(cache0), down.copy_(down0), q_pe.copy_(p0)
        for _ in range(4):
            steps = [
                lambda: kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table, lens_d, cu_q, rope=rope,
                                               q_pe=q_pe, q_out=q_pe),
                lambda: kda.kda_mla_decode_fp8(q, q_pe, cache, table, lens_d, SCALE, m, o, lse, ws),
                lambda: kda.kda_pages_copy(cache[None], src, dst),
                lambda: kda.kda_mla_decode_fp8(o, q_pe, cache, table, lens_d, SCALE, m, q, lse, ws),
                lambda: kda.kda_mla_gather_fp8(cache, table, cu, sum(lens), out=rows),
                lambda: down.copy_(rows[100:100 + N * m]),
            ]
            for step in steps:
                step()
                if pause:
                    torch.cuda.synchronize()

    def state():
        return [x.clone() for x in (q, cache, down, q_pe, o, lse, rows)]

    chain(True)
    want = state()
    assert all(torch.isfinite(x.float()).all() for x in want)
    for _ in range(5):
        chain(False)
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
    graph, _ = _capture(lambda: chain(False))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(state(), want))


@pytest.mark.parametrize("H,m,spare", [(12, 1, 0), (33, 1, 0), (40, 1, 5000), (96, 1, 0), (96, 1, 5000), (64, 3, 0), (100, 2, 5000),
                                       (128, 16, 0)])
def test_decode_stays_within_its_workspace(H, m, spare):
    """Every part of the list's cuts is written (one long sequence and short ones): the bytes on both sides of a
    workspace of just the size that is asked for stay."""
    g, lens = _gen(60 + H), [12000, 3, 900]
    q_lat, q_pe, cache, table = _inputs(g, lens, 64, H, m, tails=False)
    table = torch.cat([table, torch.full((3, spare), -1, dtype=torch.int32, device="cuda")], 1)
    size, edge = kda.kda_mla_decode_fp8_workspace_size(3, H, m), 1 << 20
    room = torch.full((size + 2 * edge,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=m,
                                    workspace=room[edge:edge + size])
    assert bool((room[:edge] == 0x5A).all()) and bool((room[edge + size:] == 0x5A).all())
    _check(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE, seqs=(1, 2))


@pytest.mark.parametrize("H,m,spare", [(12, 1, 0), (33, 1, 0), (40, 1, 5000), (96, 1, 0), (96, 1, 5000), (64, 3, 0), (100, 2, 5000),
                                       (128, 16, 0)])
def test_decode_of_a_long_sequence_from_a_workspace_of_its_size(H, m, spare):
    """The sequence that is cut into many parts, joined from just the workspace that is asked for: parts that overlapped in
    it would show."""
    g, lens = _gen(80 + H), [12000, 3, 900]
    q_lat, q_pe, cache, table = _inputs(g, lens, 64, H, m)
    table = torch.cat([table, torch.full((3, spare), -1, dtype=torch.int32, device="cuda")], 1)
    ws = torch.full((kda.kda_mla_decode_fp8_workspace_size(3, H, m),), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=m, workspace=ws)
    _check(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE)


@pytest.mark.parametrize("H,m,lens", [(2048, 5, [700, 90, 33]), (65535, 1, [70]), (4000, 16, [100, 0]), (300, 8, [2000, 17, 300])])
def test_decode_of_very_many_rows(H, m, lens):
    """More row tiles than SMs: one list for all blocks and no join; and about as many."""
    g = _gen(H)
    q_lat, q_pe, cache, table = _inputs(g, lens, 32, H, m)
    st = _status()
    o, lse = kda.kda_mla_decode_fp8(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=m, status=st)
    assert st.item() == 0
    _check(o, lse, q_lat, q_pe, cache, table, lens, m, SCALE)


@pytest.mark.parametrize("H,m", [(12, 1), (96, 4), (2048, 5)])
def test_streams_that_fork_and_join(H, m):
    """main: append, decode, | side: gather of what append wrote; joined: a page copy over both, a decode of the copy.
    Eagerly without pauses and as a graph they give the bits of calls with a synchronisation behind each."""
    g, size, lens = _gen(70 + H), 32, [700, 90, 33]
    N = len(lens)
    q0, p0, cache0, table = _inputs(g, lens, size, H, m, tails=False)
    down, rope, lens_d, cu = _rand(g, N * m, ROW), _rope(800), _ints(lens), _ints(_cu(lens))
    cu_q = _ints(_cu([m] * N))
    ws = [torch.empty(kda.kda_mla_decode_fp8_workspace_size(N, H, m), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache, q_pe = cache0.clone(), p0.clone()
    o, lse = torch.empty_like(q0), torch.empty(N * m, H, device="cuda")
    o2, lse2 = torch.empty_like(q0), torch.empty_like(lse)
    rows = torch.empty(sum(lens), ROW, dtype=torch.bfloat16, device="cuda")
    side, src, dst = torch.cuda.Stream(), int(table[1, 0]), int(table[0, 3])

    def step(pause=lambda: None):
        main = torch.cuda.current_stream()
        cache.copy_(cache0), q_pe.copy_(p0)
        kda.kda_mla_append_fp8(down[:, :LATENT], down[:, LATENT:], cache, table, lens_d, cu_q, rope=rope, q_pe=q_pe, q_out=q_pe)
        pause()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kda.kda_mla_gather_fp8(cache, table, cu, sum(lens), out=rows)
            pause()
        kda.kda_mla_decode_fp8(q0, q_pe, cache, table, lens_d, SCALE, m, o, lse, ws[0])
        pause()
        main.wait_stream(side)
        kda.kda_pages_copy(cache[None], [src], [dst])
        pause()
        kda.kda_mla_decode_fp8(o, q_pe, cache, table, lens_d, SCALE, m, o2, lse2, ws[1])
        pause()

    def state():
        torch.cuda.synchronize()
        return [x.clone() for x in (cache, q_pe, o, lse, rows, o2, lse2)]

    step(torch.cuda.synchronize)
    want = state()
    assert all(bool(torch.isfinite(x.float()).all()) for x in want)
    for _ in range(5):
        step()
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=warm):
        step()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
