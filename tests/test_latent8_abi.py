"""Refusals of the 8-bit latent-cache entry points, on the CPU: the C entries with fake (never dereferenced)
addresses, and the binding's own checks; the 64-bit helpers of the GPU tests. Nothing is launched."""
import pytest
import torch

from linear_attention_serving_02_gb300 import kda
from tests import latent8_ref as ref
from tests.test_latent_abi import ALIGN, F, NULL, SHAPE, UNSUPPORTED, WORKSPACE, _call
from tests.test_latent_abi import APPEND as APPEND_BF16, DECODE as DECODE_BF16

PS = 64 * 644
APPEND = dict(APPEND_BF16, page_stride=PS)
DECODE = dict(DECODE_BF16, page_stride=PS)
GATHER = dict(cache=F, page_stride=PS, pages=8, size=64, cu=F, starts=None, table=F, max_pages=4, out=F, T=4, N=2,
              status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(size=0), UNSUPPORTED), (dict(size=24), UNSUPPORTED), (dict(size=1 << 17, page_stride=644 << 17), UNSUPPORTED),
    (dict(page_stride=PS - 16), SHAPE), (dict(page_stride=PS + 8), SHAPE), (dict(pages=-1), SHAPE),
    (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 26), SHAPE), (dict(page_stride=1 << 60, pages=1 << 20), SHAPE),
    (dict(eps=-1.0), UNSUPPORTED), (dict(eps=float("nan")), UNSUPPORTED), (dict(il=2), UNSUPPORTED),
    (dict(q_out=None), UNSUPPORTED), (dict(q_pe=None), UNSUPPORTED), (dict(rope=None), UNSUPPORTED),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(N=-1), SHAPE), (dict(cu=None, T=5), SHAPE),
    (dict(N=0, cu=None), SHAPE), (dict(c_stride=511), SHAPE), (dict(k_pe_stride=56), SHAPE), (dict(H=0), SHAPE),
    (dict(qo_ts=64, qo_hs=128), SHAPE), (dict(rope_len=-1), SHAPE), (dict(c=None), NULL), (dict(cache=None), NULL),
    (dict(lens=None), NULL), (dict(c=F + 8), ALIGN), (dict(cache=F + 8), ALIGN), (dict(cu=F + 2), ALIGN),
    (dict(T=0), 0), (dict(N=0, T=0), 0)])
def test_append_refusals(over, code):
    assert _call("kda_mla_append_fp8", APPEND, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(size=-16), UNSUPPORTED), (dict(page_stride=0), SHAPE), (dict(page_stride=PS + 4), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=1 << 31), SHAPE), (dict(N=-1), SHAPE), (dict(cache=None), NULL), (dict(cu=None), NULL), (dict(table=None), NULL),
    (dict(out=None), NULL), (dict(out=F + 8), ALIGN), (dict(starts=F + 2), ALIGN), (dict(status=F + 1), ALIGN),
    (dict(T=0), 0), (dict(N=0), 0)])
def test_gather_refusals(over, code):
    assert _call("kda_mla_gather_fp8", GATHER, over) == code


@pytest.mark.parametrize("over,code", [
    (dict(size=8), UNSUPPORTED), (dict(page_stride=PS - 16), SHAPE), (dict(page_stride=PS + 8), SHAPE),
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=float("nan")), UNSUPPORTED), (dict(scale=float("inf")), UNSUPPORTED),
    (dict(m=17), UNSUPPORTED), (dict(m=-1), SHAPE), (dict(N=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=65536), SHAPE),
    (dict(N=1 << 28, H=16), SHAPE), (dict(page_stride=1 << 39), SHAPE), (dict(q_lat=None), NULL), (dict(q_pe=None), NULL),
    (dict(cache=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(o=None), NULL), (dict(ws=None), NULL),
    (dict(q_lat=F + 8), ALIGN), (dict(cache=F + 8), ALIGN), (dict(ws=F + 64), ALIGN), (dict(ws_bytes=8), WORKSPACE),
    (dict(N=0), 0), (dict(m=0), 0)])
def test_decode_refusals(over, code):
    assert _call("kda_mla_decode_fp8", DECODE, over) == code


def test_decode_workspace_size():
    size = kda.kda_mla_decode_fp8_workspace_size
    assert size(-1, 1, 1) == 0 and size(1, -1, 1) == 0 and size(1, 1, -1) == 0
    assert size(1, 12, 1) > 0 and size(256, 96, 16) > 0


def test_binding_refuses_cpu_tensors_and_bad_types():
    bf, i32 = torch.bfloat16, torch.int32
    cache, table, lens = torch.zeros(2, 16, 644, dtype=torch.uint8), torch.zeros(1, 2, dtype=i32), torch.ones(1, dtype=i32)
    c, pe = torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf)
    with pytest.raises(ValueError):
        kda.kda_mla_append_fp8(c, pe, cache, table, lens)
    with pytest.raises(TypeError):
        kda.kda_mla_append_fp8(c.float(), pe, cache, table, lens)
    with pytest.raises(ValueError):
        kda.kda_mla_gather_fp8(cache, table, torch.zeros(2, dtype=i32), 1)
    with pytest.raises(TypeError):
        kda.kda_mla_gather_fp8(cache.to(bf), table, torch.zeros(2, dtype=i32), 1)
    with pytest.raises(ValueError):
        kda.kda_mla_decode_fp8(torch.zeros(1, 2, 512, dtype=bf), torch.zeros(1, 2, 64, dtype=bf), cache, table, lens, 0.1)


def test_reference_quantiser_rounds_to_the_nearest_value_and_keeps_rows_it_made():
    """The tests' own quantiser: powers of two as scales, the largest value in (224, 448], half a step at most,
    and a row that is read back is held as the same values (the scale may halve: 230 becomes 224, which is 448 / 2)."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(50, 576, generator=g) * torch.exp2(torch.randint(-30, 30, (50, 1), generator=g).float())
    x[0, :512], x[1, 3] = 0, 448 * 2.0 ** 7
    b, s = ref.quantise(x)
    c = ref.codes(b)
    assert s[0] == 1 and torch.equal(torch.frexp(s)[0], torch.full_like(s, 0.5))
    top = x[1:, :512].abs().amax(1) / s[1:]
    assert bool((top <= 448).all()) and bool((top > 224).all())
    y = x.double() / s[:, None].double()
    lat = (c[:, :512] - y[:, :512]).abs()
    assert bool((lat <= torch.maximum(2.0 ** -4 * y[:, :512].abs(), torch.full_like(lat, 2.0 ** -10))).all())
    back = (c * s[:, None].double()).float()
    b2, s2 = ref.quantise(back)
    assert torch.equal(ref.codes(b2) * s2[:, None].double(), back.double())


def test_decode_workspace_size_grows_with_the_rows():
    """More heads or tokens never need less, so a workspace for the most serves the others; and it counts no sequences."""
    size = kda.kda_mla_decode_fp8_workspace_size
    for m in (1, 2, 16):
        sizes = [size(4, H, m) for H in range(1, 200)]
        assert sizes == sorted(sizes)
    assert all(size(4, H, 1) <= size(4, H, 2) <= size(4, H, 16) for H in range(1, 200))
    assert size(1, 96, 4) == size(5000, 96, 4)
