"""Refusals of the latent-attention and page entry points, on the CPU: the C entries with fake
(never dereferenced) addresses, and the binding's own checks. Nothing is launched."""
import ctypes

import pytest
import torch

from linear_attention_serving_02_gb300 import kda

F = 1 << 20
NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE, PAGES = -1, -2, -3, -5, -6, -9
PS = 64 * 576


def _call(fn, args, over):
    a = dict(args)
    a.update(over)
    return getattr(kda.library(), fn)(*a.values())


APPEND = dict(c=F, c_stride=576, k_pe=F, k_pe_stride=576, norm_w=None, eps=1e-6, rope=F, rope_len=100, il=0, q_pe=F,
              q_ts=768, q_hs=192, q_out=F, qo_ts=256, qo_hs=64, H=4, cu=F, lens=F, table=F, max_pages=4, cache=F,
              page_stride=PS, pages=8, size=64, T=4, N=2, status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(size=0), UNSUPPORTED), (dict(size=24), UNSUPPORTED), (dict(size=1 << 17, page_stride=576 << 17), UNSUPPORTED),
    (dict(page_stride=PS - 8), SHAPE), (dict(page_stride=PS + 4), SHAPE), (dict(pages=-1), SHAPE),
    (dict(max_pages=-1), SHAPE), (dict(max_pages=1 << 26), SHAPE), (dict(page_stride=1 << 60, pages=1 << 20), SHAPE),
    (dict(eps=-1.0), UNSUPPORTED), (dict(eps=float("nan")), UNSUPPORTED), (dict(il=2), UNSUPPORTED),
    (dict(q_out=None), UNSUPPORTED), (dict(q_pe=None), UNSUPPORTED), (dict(rope=None), UNSUPPORTED),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(N=-1), SHAPE), (dict(cu=None, T=5), SHAPE),
    (dict(N=0, cu=None), SHAPE), (dict(c_stride=511), SHAPE), (dict(c_stride=516), SHAPE), (dict(k_pe_stride=56), SHAPE),
    (dict(H=0), SHAPE), (dict(H=65536), SHAPE), (dict(q_ts=-768), SHAPE), (dict(q_hs=4), SHAPE),
    (dict(qo_hs=56), SHAPE), (dict(qo_ts=192), SHAPE), (dict(qo_ts=64, qo_hs=128), SHAPE),
    (dict(rope_len=-1), SHAPE),
    (dict(c=None), NULL), (dict(k_pe=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL),
    (dict(cache=None), NULL), (dict(c=F + 8), ALIGN), (dict(rope=F + 4), ALIGN), (dict(q_out=F + 2), ALIGN),
    (dict(cu=F + 2), ALIGN), (dict(T=0), 0), (dict(N=0, T=0), 0), (dict(T=0, qo_ts=0, H=2), 0)])
def test_append_refusals(over, code):
    assert _call("kda_mla_append", APPEND, over) == code


GATHER = dict(cache=F, page_stride=PS, pages=8, size=64, cu=F, table=F, max_pages=4, out=F, T=4, N=2, status=None,
              stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(size=-16), UNSUPPORTED), (dict(page_stride=0), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(N=-1), SHAPE), (dict(cache=None), NULL), (dict(cu=None), NULL), (dict(table=None), NULL), (dict(out=None), NULL),
    (dict(out=F + 8), ALIGN), (dict(status=F + 1), ALIGN), (dict(T=0), 0), (dict(N=0), 0)])
def test_gather_refusals(over, code):
    assert _call("kda_mla_gather", GATHER, over) == code


PREFILL = dict(q=F, kv=F, k_pe=F, k_pe_stride=64, cu_q=F, cu_k=F, Tq=4, Tk=4, N=1, H=2, causal=1, scale=0.1, o=F,
               lse=None, status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=-1.0), UNSUPPORTED), (dict(scale=float("nan")), UNSUPPORTED),
    (dict(scale=float("inf")), UNSUPPORTED), (dict(causal=2), UNSUPPORTED), (dict(Tq=-1), SHAPE), (dict(Tk=-1), SHAPE),
    (dict(Tq=1 << 31), SHAPE), (dict(Tk=1 << 31), SHAPE), (dict(N=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=65536), SHAPE),
    (dict(k_pe_stride=63), SHAPE), (dict(k_pe_stride=68), SHAPE), (dict(q=None), NULL), (dict(kv=None), NULL),
    (dict(k_pe=None), NULL), (dict(cu_q=None), NULL), (dict(cu_k=None), NULL), (dict(o=None), NULL),
    (dict(q=F + 8), ALIGN), (dict(kv=F + 2), ALIGN), (dict(k_pe=F + 8), ALIGN), (dict(o=F + 8), ALIGN),
    (dict(lse=F + 2), ALIGN), (dict(N=0), 0), (dict(Tq=0), 0)])
def test_prefill_refusals(over, code):
    assert _call("kda_mla_prefill", PREFILL, over) == code


DECODE = dict(q_lat=F, q_pe=F, cache=F, page_stride=PS, pages=8, size=64, table=F, max_pages=4, lens=F, N=2, H=12, m=1,
              scale=0.1, o=F, lse=None, ws=F, ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(size=8), UNSUPPORTED), (dict(page_stride=PS - 8), SHAPE), (dict(scale=0.0), UNSUPPORTED),
    (dict(scale=float("nan")), UNSUPPORTED), (dict(m=17), UNSUPPORTED), (dict(m=-1), SHAPE), (dict(N=-1), SHAPE),
    (dict(H=0), SHAPE), (dict(H=65536), SHAPE), (dict(N=1 << 28, H=16), SHAPE), (dict(q_lat=None), NULL),
    (dict(q_pe=None), NULL), (dict(cache=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(o=None), NULL), (dict(ws=None), NULL), (dict(q_lat=F + 8), ALIGN), (dict(cache=F + 8), ALIGN),
    (dict(ws=F + 64), ALIGN), (dict(ws_bytes=8), WORKSPACE), (dict(N=0), 0), (dict(m=0), 0)])
def test_decode_refusals(over, code):
    assert _call("kda_mla_decode", DECODE, over) == code


def test_decode_workspace_size():
    size = kda.kda_mla_decode_workspace_size
    assert size(-1, 1, 1) == 0 and size(1, -1, 1) == 0 and size(1, 1, -1) == 0
    assert 0 < size(1, 12, 1) <= size(256, 96, 1) <= size(256, 96, 16)


def _copy(src, dst, **over):
    a = dict(pool=F, page_stride=4096, page_bytes=4096, pages=8, layer_stride=8 * 4096, layers=2)
    a.update(over)
    s, d = (ctypes.c_int32 * max(1, len(src)))(*src), (ctypes.c_int32 * max(1, len(dst)))(*dst)
    return kda.library().kda_pages_copy(*a.values(), ctypes.addressof(s), ctypes.addressof(d), len(src), None)


@pytest.mark.parametrize("over,code", [
    (dict(page_bytes=8), SHAPE), (dict(page_stride=4104), SHAPE), (dict(layer_stride=8), SHAPE), (dict(pages=-1), SHAPE),
    (dict(layers=-1), SHAPE), (dict(layers=65536), SHAPE), (dict(page_bytes=-16), SHAPE), (dict(page_stride=-4096), SHAPE),
    (dict(page_bytes=4112), SHAPE),                               # pages overlap
    (dict(layer_stride=7 * 4096), SHAPE),                         # layers overlap
    (dict(page_stride=4096, layer_stride=4096), SHAPE), (dict(page_bytes=1 << 41, page_stride=1 << 41), SHAPE),
    (dict(page_stride=1 << 61), SHAPE), (dict(pool=None), NULL), (dict(pool=F + 8), ALIGN), (dict(layers=0), 0),
    (dict(page_bytes=0), 0)])
def test_pages_copy_refusals(over, code):
    assert _copy([0], [1], **over) == code


@pytest.mark.parametrize("src,dst", [([8], [0]), ([0], [8]), ([-1], [0]), ([0], [-1]), ([0, 1, 2], [3, 4, 1 << 30])])
def test_pages_copy_refuses_ids_before_any_launch(src, dst):
    assert _copy(src, dst) == PAGES


def test_pages_copy_of_nothing():
    assert _copy([], []) == 0 and _copy([3], [3]) == 0


def test_status_text():
    assert "page" in kda.kda_status_string(-9)


def test_binding_refuses_cpu_tensors_and_bad_types():
    bf, i32 = torch.bfloat16, torch.int32
    cache, table, lens = torch.zeros(2, 16, 576, dtype=bf), torch.zeros(1, 2, dtype=i32), torch.ones(1, dtype=i32)
    with pytest.raises(ValueError):
        kda.kda_mla_append(torch.zeros(1, 512, dtype=bf), torch.zeros(1, 64, dtype=bf), cache, table, lens)
    with pytest.raises(TypeError):
        kda.kda_mla_append(torch.zeros(1, 512), torch.zeros(1, 64, dtype=bf), cache, table, lens)
    with pytest.raises(ValueError):
        kda.kda_mla_gather(cache, table, torch.zeros(2, dtype=i32), 1)
    with pytest.raises(ValueError):
        kda.kda_mla_prefill(torch.zeros(1, 2, 192, dtype=bf), torch.zeros(1, 2, 256, dtype=bf), torch.zeros(1, 64, dtype=bf),
                            torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), 0.1)
    with pytest.raises(ValueError):
        kda.kda_mla_decode(torch.zeros(1, 2, 512, dtype=bf), torch.zeros(1, 2, 64, dtype=bf), cache, table, lens, 0.1)
    with pytest.raises(ValueError):
        kda.kda_pages_copy(torch.zeros(1, 2, 16, dtype=torch.uint8), [0], [1])
    with pytest.raises(ValueError):
        kda.kda_pages_copy(torch.zeros(4), [0], [1])
