"""Latent attention and page copies on two streams that fork and join by events, eagerly and captured: a call that is
launched while its predecessor ends still waits for the work that an event brings in from the other stream."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests.test_gpu_latent import (LATENT, NOPE, QK, ROW, SCALE, _cu, _decode_inputs, _gen, _ints, _rand, _rope)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,m", [(12, 1), (96, 4), (2048, 5)])
def test_streams_that_fork_and_join(H, m):
    """main: append, decode, | side: gather, prefill on what append wrote; joined: a page copy over both, a decode of
    the copy. (2048, 5): one list for all blocks, so no join kernel stands between the decode and what follows."""
    g, size, lens = _gen(70 + H), 32, [700, 90, 33]
    N = len(lens)
    q0, p0, cache0, table = _decode_inputs(g, lens, size, H, m, tails=False)
    down, rope, lens_d, cu = _rand(g, N * m, ROW), _rope(800), _ints(lens), _ints(_cu(lens))
    cu_q = _ints(_cu([m] * N))
    ws = [torch.empty(kda.kda_mla_decode_workspace_size(N, H, m), dtype=torch.uint8, device="cuda") for _ in range(2)]
    qx, kv = _rand(g, N * m, 2, QK), _rand(g, sum(lens), 2, 2 * NOPE)
    cache, q_pe = cache0.clone(), p0.clone()
    o, lse = torch.empty_like(q0), torch.empty(N * m, H, device="cuda")
    o2, lse2 = torch.empty_like(q0), torch.empty_like(lse)
    rows = torch.empty(sum(lens), ROW, dtype=torch.bfloat16, device="cuda")
    ox, lx = torch.empty(N * m, 2, NOPE, dtype=torch.bfloat16, device="cuda"), torch.empty(N * m, 2, device="cuda")
    side, src, dst = torch.cuda.Stream(), int(table[1, 0]), int(table[0, 3])

    def step(pause=lambda: None):
        main = torch.cuda.current_stream()
        cache.copy_(cache0), q_pe.copy_(p0)
        kda.kda_mla_append(down[:, :LATENT], down[:, LATENT:], cache, table, lens_d, cu_q, rope=rope, q_pe=q_pe, q_out=q_pe)
        pause()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kda.kda_mla_gather(cache, table, cu, sum(lens), rows)
            pause()
            kda.kda_mla_prefill(qx, kv, rows[:, LATENT:], cu_q, cu, SCALE, o=ox, lse=lx)
            pause()
        kda.kda_mla_decode(q0, q_pe, cache, table, lens_d, SCALE, m, o, lse, ws[0])
        pause()
        main.wait_stream(side)
        kda.kda_pages_copy(o.view(1, N, -1), [0], [1])
        kda.kda_pages_copy(cache[None], [src], [dst])
        pause()
        kda.kda_mla_decode(o, q_pe, cache, table, lens_d, SCALE, m, o2, lse2, ws[1])
        pause()

    def state():
        torch.cuda.synchronize()
        return [x.clone() for x in (cache, q_pe, o, lse, rows, ox, lx, o2, lse2)]

    step(torch.cuda.synchronize)
    want = state()
    assert all(bool(torch.isfinite(x).all()) for x in want)
    for _ in range(5):
        step()
    assert all(torch.equal(a, b) for a, b in zip(state(), want))
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=warm):
        step()
    for x in (o, lse, rows, ox, lx, o2, lse2):
        x.fill_(3.0)
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
