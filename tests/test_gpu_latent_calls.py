"""Calls of the latent-attention operators and the page copies as a serving program makes them: other
streams, captured and replayed, far offsets, many short sequences, pages used twice, calls of nothing."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent_ref as ref
from tests.test_gpu_latent import (LATENT, NOPE, QK, ROW, SCALE, _capture, _check_decode, _cu, _decode_inputs, _gen,
                                   _ints, _prefill_inputs, _rand, _rope, _status)

pytestmark = pytest.mark.gpu


def _calls(seed):
    """The five calls on inputs of their own; each returns the tensors it wrote."""
    g, size, lens, new = _gen(seed), 32, [300, 41], [70, 5]
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, size, 12, 1, tails=False)
    q, kv, pe = _prefill_inputs(g, new, lens, 3)
    down, rope, lens_d, cu_q, cu_k = _rand(g, sum(new), ROW), _rope(300), _ints(lens), _ints(_cu(new)), _ints(_cu(lens))
    ws = torch.empty(kda.kda_mla_decode_workspace_size(2, 12, 1), dtype=torch.uint8, device="cuda")
    pool = _rand(g, 3, 8, 64, 128)
    work, copy = torch.empty_like(cache), torch.empty_like(pool)

    def append(stream=None):
        with torch.cuda.stream(stream):
            work.copy_(cache)
        out = kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], work, table, lens_d, cu_q, rope=rope,
                                 q_pe=q[..., NOPE:], stream=stream)
        return work, out

    def pages(stream=None):
        with torch.cuda.stream(stream):
            copy.copy_(pool)
        return (kda.kda_pages_copy(copy, [0, 1, 5, 0], [1, 2, 5, 7], stream=stream),)

    return [append, pages,
            lambda stream=None: (kda.kda_mla_gather(cache, table, cu_k, sum(lens), stream=stream),),
            lambda stream=None: kda.kda_mla_prefill(q, kv, pe, cu_q, cu_k, SCALE, stream=stream),
            lambda stream=None: kda.kda_mla_decode(q_lat, q_pe, cache, table, lens_d, SCALE, workspace=ws, stream=stream)]


@pytest.mark.parametrize("which", range(5))
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
            x.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    runs, side = [_calls(51), _calls(52)], [torch.cuda.Stream(), torch.cuda.Stream()]
    want = [[[x.clone() for x in call()] for call in calls] for calls in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[call(s) for call in calls] for calls, s in zip(runs, side)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for u, v in zip(a, b) for x, y in zip(u, v))


def test_cache_and_rows_past_two_to_the_31():
    """Pages behind element 2^31 (and byte 2^32) of the cache, and a batch that starts there in its tensors."""
    g, size, H, pages = _gen(53), 64, 2, 60000
    cache = torch.empty(pages, size, ROW, dtype=torch.bfloat16, device="cuda")
    assert cache.numel() > 2 ** 31
    lens = [150, 64]
    table = _ints([[59999, 3, 59000], [58990, -1, -1]])
    down = _rand(g, sum(lens), ROW)
    kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table, _ints(lens), _ints(_cu(lens)))
    assert torch.equal(kda.kda_mla_gather(cache, table, _ints(_cu(lens)), sum(lens)), down)
    q_lat, q_pe = _rand(g, 2, H, LATENT), _rand(g, 2, H, ROW - LATENT)
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE)
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, 1, SCALE)
    kda.kda_pages_copy(cache[None], [59999], [59998])
    assert torch.equal(cache[59998], cache[59999])
    del cache
    T, H = 180000, 64
    q = torch.empty(T, H, QK, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(T, H, 2 * NOPE, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 2 ** 31 and kv.numel() > 2 ** 31
    at, n = T - 140, 140
    q[at:], kv[at:], pe[at:] = _rand(g, n, H, QK), _rand(g, n, H, 2 * NOPE), _rand(g, n, 64)
    o, lse = kda.kda_mla_prefill(q, kv, pe, _ints([at, T]), _ints([at, T]), SCALE)
    for h in (0, 63):
        ref.check_rows(o[at:, h], lse[at:, h], ref.prefill_ref(q, kv, pe, [at, T], [at, T], SCALE, True, 0, h))


@pytest.mark.parametrize("count", [33, 1500])
def test_many_short_sequences(count):
    """More sequences than a warp looks at in one round and than there are SMs, empty ones among them."""
    g, size, H = _gen(count), 16, 2
    new = [(7 * n) % 4 for n in range(count)]
    lens = [a + (5 * n) % 23 for n, a in enumerate(new)]
    q, kv, pe = _prefill_inputs(g, new, lens, H)
    cu_q, cu_k, st = _cu(new), _cu(lens), _status()
    o, lse = kda.kda_mla_prefill(q, kv, pe, _ints(cu_q), _ints(cu_k), SCALE, status=st)
    for n in range(0, count, 1 if count < 100 else 13):
        a, b = cu_q[n], cu_q[n + 1]
        for h in range(H):
            ref.check_rows(o[a:b, h], lse[a:b, h], ref.prefill_ref(q, kv, pe, cu_q, cu_k, SCALE, True, n, h))
    table, pages = ref.make_pages(g, lens, size)
    cache, table = _rand(g, pages, size, ROW), table.cuda()
    down = _rand(g, sum(new), ROW)
    kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table, _ints(lens), _ints(cu_q), status=st)
    rows = kda.kda_mla_gather(cache, table, _ints(cu_k), sum(lens), status=st)
    for n in range(count):
        k, a = cu_k[n + 1], new[n]
        assert a == 0 or torch.equal(rows[k - a:k], down[cu_q[n]:cu_q[n + 1]])
    assert torch.equal(rows, torch.cat([ref.cached_rows(cache, table[n], k) for n, k in enumerate(lens)]))
    q_lat, q_pe = _rand(g, count, 12, LATENT), _rand(g, count, 12, ROW - LATENT)
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE, status=st)
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, 1, SCALE, seqs=range(0, count, 1 if count < 100 else 13))
    assert st.item() == 0


def test_prefill_output_aligned_to_16_bytes_only():
    g, n, H = _gen(54), 150, 3
    q, kv, pe = _prefill_inputs(g, [n], [n], H)
    room = torch.full((n * H * NOPE + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = room[8:8 + n * H * NOPE].view(n, H, NOPE)
    assert o.data_ptr() % 32 == 16
    kda.kda_mla_prefill(q, kv, pe, _ints([0, n]), _ints([0, n]), SCALE, o=o)
    want, _ = kda.kda_mla_prefill(q, kv, pe, _ints([0, n]), _ints([0, n]), SCALE)
    assert torch.equal(o, want) and bool((room[:8] == 7).all()) and bool((room[-8:] == 7).all())


def test_a_page_twice_in_one_sequence_and_in_two():
    g, size, H = _gen(55), 32, 12
    cache = _rand(g, 4, size, ROW)
    table, lens = _ints([[2, 0, 2, 2, 1], [2, 0, 3, -1, -1]]), [150, 70]
    q_lat, q_pe = _rand(g, 4, H, LATENT), _rand(g, 4, H, ROW - LATENT)
    o, lse = kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE, num_tokens=2)
    _check_decode(o, lse, q_lat, q_pe, cache, table, lens, 2, SCALE)
    rows = kda.kda_mla_gather(cache, table, _ints(_cu(lens)), sum(lens))
    assert torch.equal(rows, torch.cat([ref.cached_rows(cache, table[n], k) for n, k in enumerate(lens)]))


def test_calls_of_nothing_write_nothing():
    g = _gen(56)
    cache = _rand(g, 2, 16, ROW)
    was, none, one, st = cache.clone(), _ints([]), _ints([0]), _status()
    no_table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    kda.kda_mla_append(_rand(g, 0, LATENT), _rand(g, 0, 64), cache, no_table, none, one, status=st)
    kda.kda_mla_append(_rand(g, 5, LATENT), _rand(g, 5, 64), cache, no_table, none, one, status=st)
    out = torch.full((4, ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_mla_gather(cache, no_table, one, 4, out=out, status=st)
    assert bool((out == 7).all())
    o = torch.full((5, 2, NOPE), 7.0, dtype=torch.bfloat16, device="cuda")
    q, kv, pe = _prefill_inputs(g, [5], [5], 2)
    kda.kda_mla_prefill(q, kv, pe, one, one, SCALE, o=o, status=st)
    assert bool((o == 7).all())
    # queries without any key at all
    o, lse = kda.kda_mla_prefill(q, kv[:0], pe[:0], _ints([0, 5]), _ints([0, 0]), SCALE, status=st)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())
    o, lse = kda.kda_mla_decode(_rand(g, 0, 2, LATENT), _rand(g, 0, 2, 64), cache, no_table, none, SCALE, status=st)
    assert o.shape == (0, 2, LATENT) and lse.shape == (0, 2)
    kda.kda_pages_copy(cache[None], [], [])
    torch.cuda.synchronize()
    assert st.item() == 0 and torch.equal(cache, was)


def test_the_status_word_is_never_cleared():
    g, lens = _gen(57), [40]
    q_lat, q_pe, cache, table = _decode_inputs(g, lens, 16, 2, 1)
    st = torch.full((1,), -4, dtype=torch.int32, device="cuda")
    kda.kda_mla_decode(q_lat, q_pe, cache, table, _ints(lens), SCALE, status=st)
    kda.kda_mla_gather(cache, table, _ints(_cu(lens)), 40, status=st)
    assert st.item() == -4


def test_page_ids_of_every_kind():
    g = _gen(58)
    pool = _rand(g, 2, 9, 16)
    want = pool.clone()
    want[:, 5], want[:, 7] = pool[:, 1], pool[:, 2]

    class Id:
        def __init__(self, v):
            self.v = v

        def __index__(self):
            return self.v

    for src, dst in (([1, 2], [5, 7]), ((1, 2), (5, 7)), (range(1, 3), iter([5, 7])), ([Id(1), Id(2)], [5, True + 6]),
                     (torch.tensor([1, 2]), torch.tensor([5, 7], dtype=torch.uint8)),
                     (torch.tensor([1, 0, 2, 0], dtype=torch.int32)[::2], torch.tensor([5, 7], dtype=torch.int32))):
        got = pool.clone()
        kda.kda_pages_copy(got, src, dst)
        assert torch.equal(got, want)
    for bad, error in (([1.0, 2], TypeError), (["1", 2], TypeError), ([1], ValueError), ([1, 2 ** 40], kda.KdaError),
                       ([1, -2 ** 70], kda.KdaError), ([1, 9], kda.KdaError), (torch.tensor([1.0, 2.0]), TypeError),
                       (torch.tensor([[1, 2]]), ValueError), (torch.tensor([1, -1]), kda.KdaError)):
        got = pool.clone()
        with pytest.raises(error):
            kda.kda_pages_copy(got, bad, [5, 7])
        assert torch.equal(got, pool)


@pytest.mark.parametrize("H,m", [(2, 1), (12, 1), (96, 1), (96, 4)])
def test_calls_that_follow_one_another_wait_for_one_another(H, m):
    """Each call reads what the one before it wrote, and writes what it read: without any pause between
    them, and as one graph, they give the bits of calls with a synchronisation behind each."""
    g, size, lens = _gen(59 + H), 32, [700, 90, 33]
    N = len(lens)
    q0, p0, cache0, table = _decode_inputs(g, lens, size, H, m, tails=False)
    down0, rope, lens_d, cu = _rand(g, N * m, ROW), _rope(800), _ints(lens), _ints(_cu(lens))
    cu_q = _ints(_cu([m] * N))
    ws = torch.empty(kda.kda_mla_decode_workspace_size(N, H, m), dtype=torch.uint8, device="cuda")
    q, cache, down = q0.clone(), cache0.clone(), down0.clone()
    q_pe, o, lse = p0.clone(), torch.empty_like(q0), torch.empty(N * m, H, device="cuda")
    rows = torch.empty(sum(lens), ROW, dtype=torch.bfloat16, device="cuda")
    qx, kv = torch.empty(N * m, 2, QK, dtype=torch.bfloat16, device="cuda"), _rand(g, sum(lens), 2, 2 * NOPE)
    ox, lx = torch.empty(N * m, 2, NOPE, dtype=torch.bfloat16, device="cuda"), torch.empty(N * m, 2, device="cuda")

    def chain(pause):
        q.copy_(q0), cache.copy_(cache0), down.copy_(down0), q_pe.copy_(p0)
        for _ in range(4):
            steps = [
                lambda: kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table, lens_d, cu_q, rope=rope,
                                           q_pe=q_pe, q_out=q_pe),
                lambda: kda.kda_mla_decode(q, q_pe, cache, table, lens_d, SCALE, m, o, lse, ws),
                lambda: kda.kda_pages_copy(o.view(1, N, -1), [0], [2]),
                lambda: kda.kda_mla_decode(o, q_pe, cache, table, lens_d, SCALE, m, q, lse, ws),
                lambda: kda.kda_mla_gather(cache, table, cu, sum(lens), rows),
                lambda: qx.view(N * m, -1).copy_(q.view(N * m, -1)[:, :2 * QK]),
                lambda: kda.kda_mla_prefill(qx, kv, rows[:, LATENT:], cu_q, cu, SCALE, o=ox, lse=lx),
                lambda: down[:, :2 * NOPE].copy_(ox.view(N * m, -1)),
            ]
            for step in steps:
                step()
                if pause:
                    torch.cuda.synchronize()

    def state():
        return [x.clone() for x in (q, cache, down, q_pe, o, lse, rows, ox, lx)]

    chain(True)
    want = state()
    assert all(torch.isfinite(x).all() for x in want)
    for _ in range(5):
        chain(False)
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
    graph, _ = _capture(lambda: chain(False))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
