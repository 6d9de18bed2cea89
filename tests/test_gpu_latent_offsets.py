"""Offsets that fall in kda_mla_prefill: what is sound is computed, what is not is left alone, wherever it stands."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent_ref as ref
from tests.test_gpu_latent import NOPE, SCALE, _cu, _gen, _ints, _prefill_inputs, _status

pytestmark = pytest.mark.gpu


def _run(cu_q, cu_k, Tq, Tk, H, good, causal=True):
    """The sequences in `good` are computed and set nothing; every other row keeps its 7; the status says so."""
    q, kv, pe = _prefill_inputs(_gen(Tq + Tk), [Tq], [Tk], H)
    st = _status()
    o = torch.full((Tq, H, NOPE), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Tq, H), 7.0, device="cuda")
    kda.kda_mla_prefill(q, kv, pe, _ints(cu_q), _ints(cu_k), SCALE, causal=causal, o=o, lse=lse, status=st)
    assert st.item() == -4
    left = torch.ones(Tq, dtype=torch.bool, device="cuda")
    for n in good:
        a, b = cu_q[n], cu_q[n + 1]
        left[a:b] = False
        for h in range(H):
            ref.check_rows(o[a:b, h], lse[a:b, h], ref.prefill_ref(q, kv, pe, cu_q, cu_k, SCALE, causal, n, h))
    assert bool((o[left] == 7).all()) and bool((lse[left] == 7).all())


@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("cu_q,cu_k,good", [
    # the same rows twice: more tiles than total_q and the number of sequences allow for
    ([0, 1000, 0, 1000], [0, 500, 500, 1000], [0]),
    ([0, 1000, 0, 1000, 0, 1000], [0, 300, 300, 600, 600, 1000], [0]),
    # a part of the rows twice, and a sound sequence behind
    ([0, 300, 100, 700, 1000], [0, 300, 300, 900, 1000], [0, 3]),
    ([0, 300, 200, 300, 1000], [0, 300, 300, 400, 1000], [0, 3]),
    # offsets that leave the tensor and come back behind the rows taken
    ([0, 300, 1200, 300, 1000], [0, 300, 400, 400, 1000], [0, 3]),
    ([0, 300, -4, 300, 1000], [0, 300, 400, 400, 1000], [0, 3]),
    # the keys' offsets alone
    ([0, 300, 600, 1000], [0, 500, 200, 1000], [0, 2]),
])
def test_offsets_that_fall(cu_q, cu_k, good, H):
    _run(cu_q, cu_k, 1000, 1000, H, good)


@pytest.mark.parametrize("at", [31, 32, 33, 70])
def test_offsets_that_fall_among_many_sequences(at):
    """The warp that looks for a block's work sees 32 sequences at a time: a fall in an earlier round still counts."""
    new = [5 + n % 7 for n in range(100)]
    cu_q = _cu(new)
    cu_k, Tq = list(cu_q), cu_q[-1]
    cu_q[at] = 3  # sequence at - 1 falls, sequence `at` begins inside earlier ones
    _run(cu_q, cu_k, Tq, Tq, 2, [n for n in range(100) if n not in (at - 1, at)])
