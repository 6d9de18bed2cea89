"""The 8-bit decode's tests once more with page tables that are wide: what the tables could hold decides how many query
rows a block takes, and without the spare entries these small batches would all be given 32."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import test_gpu_latent8 as narrow
from tests.test_gpu_latent8 import (test_decode, test_decode_agrees_with_the_bf16_cache_of_the_same_values,  # noqa: F401
                                    test_decode_flat_and_sharp_scores,
                                    test_decode_gives_the_same_bits_again_and_on_another_stream,
                                    test_decode_of_rows_of_different_magnitudes,
                                    test_decode_of_scores_that_move, test_decode_of_uneven_queries,
                                    test_two_graphs_share_a_workspace_in_order)
from tests.test_gpu_latent8_calls import (test_a_page_twice_in_one_sequence_and_in_two,  # noqa: F401
                                          test_calls_that_follow_one_another_wait_for_one_another,
                                          test_graphs_of_two_streams_with_workspaces_of_their_own, test_two_streams_at_once)
from tests.test_gpu_latent8_long import test_decode_of_positional_scores_alone  # noqa: F401

pytestmark = pytest.mark.gpu

TILES = 4096  # of a sequence: more than 24 for each SM


@pytest.fixture(autouse=True)
def wide_tables(monkeypatch):
    real = kda.kda_mla_decode_fp8

    def padded(q_lat, q_pe, cache, table, *args, **more):
        most = -(-TILES * 64 // cache.shape[1])
        spare = torch.full((table.shape[0], max(0, most - table.shape[1])), -1, dtype=torch.int32, device="cuda")
        return real(q_lat, q_pe, cache, torch.cat([table, spare], 1), *args, **more)

    monkeypatch.setattr(kda, "kda_mla_decode_fp8", padded)


@pytest.mark.parametrize("H", [12, 40, 96, 150])
@pytest.mark.parametrize("what,code", [("page", -9), ("negative page", -9), ("negative", -4)])
def test_decode_bad_wide_tables(what, code, H):
    narrow.test_decode_bad_tables(what, code, H)


@pytest.mark.parametrize("H,m", [(33, 1), (96, 1), (64, 3), (64, 16)])
def test_decode_agrees_with_narrow_tables(H, m, monkeypatch):
    """Both cuts of the same work are within the bounds of the same answer."""
    g, lens = narrow._gen(H), [700, 64, 0, 2000, 65]
    inputs = narrow._inputs(g, lens, 64, H, m)
    o, lse = kda.kda_mla_decode_fp8(*inputs, narrow._ints(lens), narrow.SCALE, num_tokens=m)
    monkeypatch.undo()
    o2, lse2 = kda.kda_mla_decode_fp8(*inputs, narrow._ints(lens), narrow.SCALE, num_tokens=m)
    for a, b in ((o, lse), (o2, lse2)):
        narrow._check(a, b, *inputs, lens, m, narrow.SCALE)
