"""Refusals of the operators over a ragged cache, on the host before any launch (no GPU needed)."""

import ctypes
import os

import pytest
import torch

from precision_attention_fmha_b200 import build as build_mod
from precision_attention_fmha_b200 import fmha

P = 0x10000  # an aligned address that no refused call ever reaches


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fmha.LIB_PATH):
        build_mod.build()
    return fmha.load_library()


def cache(paged=True, D=128, Hq=8, Hkv=2, T=4, B=2):
    a = fmha._CacheArgs()
    for t in (a.q, a.k, a.v, a.o):
        t.ptr, t.dtype = P, fmha.BF16
    for t, H, S in ((a.q, Hq, T), (a.o, Hq, T), (a.k, Hkv, 64), (a.v, Hkv, 64)):
        t.stride_h, t.stride_s, t.stride_b = D, H * D, S * H * D
    a.B, a.T, a.Hq, a.Hkv, a.D = B, T, Hq, Hkv, D
    a.lens = P
    if paged:
        a.page_table, a.num_pages, a.page_size, a.max_pages_per_seq = P, 10, 64, 5
    else:
        a.capacity = 64
    return a


def set_(obj, **kw):
    for k, v in kw.items():
        setattr(obj, k, v)


COMMON = [
    (lambda a: set_(a, D=96), 2), (lambda a: set_(a, D=192), 2), (lambda a: set_(a, Hkv=3), 1), (lambda a: set_(a, B=-1), 1),
    (lambda a: set_(a, lens=None), 1), (lambda a: set_(a, lens=P + 2), 1), (lambda a: set_(a, q_lens=P + 1), 1),
    (lambda a: set_(a.q, dtype=fmha.E4M3), 2), (lambda a: set_(a.q, dtype=fmha.FP16), 2), (lambda a: set_(a.q, ptr=P + 8), 1),
    (lambda a: set_(a.q, ptr=None), 1), (lambda a: set_(a.k, ptr=None), 1), (lambda a: set_(a.k, dtype=fmha.INT8), 2),
    (lambda a: set_(a.k, stride_s=2 * 128 + 4), 1), (lambda a: set_(a.k, stride_h=64), 1), (lambda a: set_(a.k, reserved=1), 1),
    (lambda a: set_(a, page_size=48), 2), (lambda a: set_(a, num_pages=0), 1), (lambda a: set_(a, page_table=P + 2), 1),
    (lambda a: set_(a, capacity=321), 1), (lambda a: set_(a, capacity=-1), 1), (lambda a: set_(a, max_pages_per_seq=1 << 28), 2),
    (lambda a: set_(a, lse=P + 2), 1), (lambda a: set_(a.sf_k, kind=1, ptr=P), 2),  # a scale on BF16 keys
]
ATTEND = COMMON + [
    (lambda a: set_(a.v, dtype=fmha.FP16), 2), (lambda a: set_(a.k, dtype=fmha.E4M3), 2),  # E4M3 keys, BF16 values
    (lambda a: set_(a.o, dtype=fmha.E4M3), 2), (lambda a: set_(a.o, ptr=None), 1), (lambda a: set_(a.sf_v, kind=1, ptr=P), 2),
    (lambda a: (set_(a.v, dtype=fmha.E4M3), set_(a.sf_v, kind=4, ptr=P)), 2),  # per-channel V scales
    (lambda a: (set_(a.v, dtype=fmha.E4M3), set_(a.sf_v, kind=1)), 1),
]


BIG = 1 << 40


@pytest.mark.parametrize("mutate,status", ATTEND)
def test_tree_refuses(lib, mutate, status):
    a = cache()
    mutate(a)
    assert lib.fmha_fwd_tree(ctypes.byref(a), None, 0, P, BIG, None) == status
    assert lib.fmha_last_error_message() != b""


def test_tree_refuses_workspace_and_mask(lib):
    a = cache()
    need = lib.fmha_fwd_tree_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert lib.fmha_fwd_tree(ctypes.byref(a), None, 0, None, need, None) == 1
    assert lib.fmha_fwd_tree(ctypes.byref(a), None, 0, P + 4, need, None) == 1
    assert lib.fmha_fwd_tree(ctypes.byref(a), None, 0, P, need - 1, None) == 1
    assert lib.fmha_fwd_tree(ctypes.byref(a), P, -1, P, need, None) == 1
    assert lib.fmha_fwd_tree(None, None, 0, P, need, None) == 1


@pytest.mark.parametrize("mutate,status", ATTEND)
def test_selected_refuses(lib, mutate, status):
    a = cache()
    mutate(a)
    assert lib.fmha_fwd_selected(ctypes.byref(a), P, 4, 64, P, BIG, None) == status


@pytest.mark.parametrize("blocks,top,block,status", [(None, 4, 64, 1), (P + 2, 4, 64, 1), (P, 0, 64, 1), (P, 4, 48, 2),
                                                     (P, 4, 256, 2), (P, 1 << 26, 64, 1)])
def test_selected_refuses_lists(lib, blocks, top, block, status):
    assert lib.fmha_fwd_selected(ctypes.byref(cache()), blocks, top, block, P, BIG, None) == status


@pytest.mark.parametrize("mutate,status", [
    (lambda a: set_(a, D=96), 2), (lambda a: set_(a.k, ptr=None), 1), (lambda a: set_(a.k, dtype=fmha.INT8), 2),
    (lambda a: set_(a, page_size=8), 2), (lambda a: set_(a, lens=None), 1)])
def test_bounds_refuse(lib, mutate, status):
    a = cache()
    mutate(a)
    assert lib.fmha_key_bounds(ctypes.byref(a), P, 5, 64, None, None) == status


def test_bounds_refuse_arguments(lib):
    a = cache()
    r = ctypes.byref(a)
    assert lib.fmha_key_bounds(r, None, 5, 64, None, None) == 1
    assert lib.fmha_key_bounds(r, P + 8, 5, 64, None, None) == 1
    assert lib.fmha_key_bounds(r, P, -1, 64, None, None) == 1
    assert lib.fmha_key_bounds(r, P, 5, 24, None, None) == 2
    assert lib.fmha_key_bounds(r, P, 5, 64, P + 1, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(n=20000), 2), (dict(n=-1), 1), (dict(block=8), 2), (dict(top=0), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1),
    (dict(tile=64), 2), (dict(tile=128, block=64), 2), (dict(bounds=None), 1), (dict(bounds=P + 4), 1), (dict(out=None), 1),
    (dict(out=P + 2), 1)])
def test_select_refuses(lib, kw, status):
    d = dict(bounds=P, n=5, block=64, top=2, sinks=0, recent=1, tile=1, out=P)
    d.update(kw)
    assert lib.fmha_select_blocks(ctypes.byref(cache()), d["bounds"], d["n"], d["block"], d["top"], d["sinks"], d["recent"],
                                  d["tile"], d["out"], None) == status


@pytest.mark.parametrize("mutate,status", COMMON)
@pytest.mark.parametrize("T", [4, 100])
def test_weights_refuse(lib, mutate, status, T):
    a = cache(T=T)
    a.lse = P
    mutate(a)
    assert lib.fmha_key_weights(ctypes.byref(a), P, 320, 1, 1, P, BIG, None) == status


def test_weights_refuse_arguments(lib):
    a = cache(T=100)
    r = ctypes.byref(a)
    assert lib.fmha_key_weights(r, P, 320, 1, 1, P, BIG, None) == 1  # no lse
    a.lse = P
    assert lib.fmha_key_weights(r, None, 320, 1, 1, P, BIG, None) == 1
    assert lib.fmha_key_weights(r, P, -1, 1, 1, P, BIG, None) == 1
    need = lib.fmha_key_weights_workspace_bytes(r, 320, 1)
    assert need > 0
    assert lib.fmha_key_weights(r, P, 320, 1, 1, P, need - 1, None) == 1
    assert lib.fmha_key_weights(r, P, 320, 1, 1, None, need, None) == 1


@pytest.mark.parametrize("budget,sinks,recent,status", [(0, 0, 0, 1), (4, 3, 2, 1), (4, -1, 0, 1), (4, 0, -1, 1)])
def test_evict_refuses(lib, budget, sinks, recent, status):
    assert lib.fmha_evict_select(ctypes.byref(cache()), P, 100, budget, sinks, recent, P, P, None) == status


def test_evict_and_compact_refuse_arguments(lib):
    a, o = cache(), cache()
    r = ctypes.byref(a)
    assert lib.fmha_evict_select(r, None, 100, 4, 0, 0, P, P, None) == 1
    assert lib.fmha_evict_select(r, P, 100, 4, 0, 0, None, P, None) == 1
    assert lib.fmha_evict_select(r, P, 100, 4, 0, 0, P, P + 1, None) == 1

    def compact(out=None, keep=P, kb=4, kh=0, n=4, counts=P, start=None, w=None, nw=0, wo=None, nwo=0):
        return lib.fmha_cache_compact(r, out, keep, kb, kh, n, counts, start, w, nw, wo, nwo, None)

    assert compact(keep=None) == 1 and compact(counts=None) == 1 and compact(n=-1) == 1 and compact(kb=-1) == 1
    assert compact(w=P, nw=10) == 1                                  # weights without a place
    assert compact(w=P, nw=10, wo=P + 64, nwo=10) == 1               # inside one cache: the same weights
    assert compact(w=P, nw=10, wo=P, nwo=9) == 1
    assert compact(out=ctypes.byref(o), w=P, nw=10, wo=P, nwo=10) == 1
    o.D = 64
    assert compact(out=ctypes.byref(o)) == 1
    o = cache()
    o.k.dtype = o.v.dtype = fmha.E4M3
    assert compact(out=ctypes.byref(o)) == 1


def test_nothing_to_do_is_fine(lib):
    a = cache()
    a.B = 0
    r = ctypes.byref(a)
    assert lib.fmha_fwd_tree(r, None, 0, None, 0, None) == 0
    assert lib.fmha_fwd_selected(r, P, 4, 64, None, 0, None) == 0
    assert lib.fmha_key_bounds(r, P, 5, 64, None, None) == 0
    assert lib.fmha_key_weights(r, P, 320, 1, 1, None, 0, None) == 0
    assert lib.fmha_fwd_tree_workspace_bytes(r) == 0


def test_binding_checks_shapes():
    """The binding's own checks, with CPU tensors (the device check comes last)."""
    bf = torch.bfloat16
    q, k = torch.zeros(2, 3, 8, 64, dtype=bf), torch.zeros(2, 32, 4, 64, dtype=bf)
    lens = torch.zeros(2, dtype=torch.int32)
    i32 = torch.int32

    def refused(f, *a, **kw):
        with pytest.raises(ValueError):
            f(*a, **kw)

    refused(fmha.fmha_fwd_tree, q, k, k, lens)                               # not on a GPU
    refused(fmha.fmha_fwd_tree, q, k, k, lens.long())
    refused(fmha.fmha_fwd_tree, q, k, k[:, :16], lens)
    refused(fmha.fmha_fwd_tree, q[:1], k, k, lens)
    refused(fmha.fmha_fwd_tree, q, k, k, lens, tree_mask=torch.zeros(2, 3, 3))
    refused(fmha.fmha_fwd_tree, q, k, k, lens, tree_mask=torch.zeros(2, 3, 4, dtype=torch.uint8))
    refused(fmha.fmha_fwd_tree, q, k, k, lens, tree_mask=torch.zeros(2, 3, 6, dtype=torch.uint8)[:, :, ::2])
    refused(fmha.fmha_fwd_selected, q, k, k, torch.zeros(2, 3, 4, dtype=i32), lens, 16)
    refused(fmha.fmha_fwd_selected, q, k, k, torch.zeros(2, 3, 8, 2, dtype=i32), lens, 16)
    refused(fmha.key_bounds, k, lens, 16, bounds=torch.zeros(2, 4, 2, 64, dtype=bf))
    refused(fmha.select_blocks, q, torch.zeros(2, 4, 2, 2, 64), lens, 16, 1)
    refused(fmha.select_blocks, q, torch.zeros(2, 4, 2, 2, 64, dtype=bf), lens, 16, 1, out=torch.zeros(2, 3, 4, 2, dtype=i32))
    refused(fmha.key_weights, q, k, torch.zeros(2, 8, 3), torch.zeros(2, 4, 9, dtype=torch.float64), lens)
    refused(fmha.key_weights, q, k, torch.zeros(2, 3, 8), torch.zeros(2, 4, 9), lens)
    refused(fmha.evict_select, torch.zeros(2, 4), lens, 3)
    refused(fmha.cache_compact, k, k, torch.zeros(2, 3, 2, dtype=i32), lens)
    refused(fmha.cache_compact, k, k, torch.zeros(2, 4, 2, dtype=i32), lens, k_out=k)
    refused(fmha.cache_compact, k, k, torch.zeros(2, 4, 2, dtype=i32), lens, weights_out=torch.zeros(2, 4, 9))
    refused(fmha.fmha_fwd_tree, q, k, k, lens, sf_k=fmha.Scale(torch.zeros(3, 3), "per_head"))


def test_numbers_that_32_bits_do_not_hold():
    """Sizes past a 32-bit argument are refused, not cut to their low bits."""
    big = (1 << 32) + 4
    lens = torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(1, 1, 8)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 128, 1, 64, dtype=torch.bfloat16)
    bounds = torch.zeros(1, 1, 8, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: fmha.evict_select(w, lens, big), lambda: fmha.evict_select(w, lens, 4, sinks=big),
              lambda: fmha.evict_select(w, lens, 4, recent=big), lambda: fmha.key_bounds(k, lens, big),
              lambda: fmha.select_blocks(q, bounds, lens, big, 4), lambda: fmha.select_blocks(q, bounds, lens, 16, big),
              lambda: fmha.select_blocks(q, bounds, lens, 16, 4, sink_blocks=big),
              lambda: fmha.select_blocks(q, bounds, lens, 16, 4, recent_blocks=big),
              lambda: fmha.select_blocks(q, bounds, lens, 16, 4, q_tile=big),
              lambda: fmha.fmha_fwd_selected(q, k, k, torch.zeros(1, 1, 1, 2, dtype=torch.int32), lens, big),
              lambda: fmha.key_bounds(k, lens, 16, page_table=torch.empty(1, 1 << 25, dtype=torch.int32))):
        with pytest.raises(ValueError, match="out of range"):
            f()


@pytest.mark.parametrize("empty", ["T", "Hq"])
def test_weights_without_query_rows_refuse(lib, empty):
    """Sums over no query row are written where they overwrite: what is written to and the cache are checked all the same."""
    def call(w=P, accumulate=0, **kw):
        a = cache()
        set_(a, **{empty: 0, **kw})
        a.q.ptr = None
        return lib.fmha_key_weights(ctypes.byref(a), w, 320, 1, accumulate, None, 0, None)

    assert call(accumulate=1) == 0 and call(B=0) == 0 and call(**{"Hq": 0, "Hkv": 0}) == 0
    assert call(w=None) == 1 and call(w=P + 2) == 1 and call(lens=None) == 1 and call(D=96) == 2 and call(page_size=48) == 2


def test_scattered_workspaces_are_refused():
    """A workspace's bytes are counted from its elements: one whose elements repeat or lie apart is none of that size."""
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    whole = torch.empty(256, dtype=torch.float32)
    assert fmha._scratch(whole, 1024, q)[1:] == (whole.data_ptr(), 1024)
    for w in (torch.empty(1, dtype=torch.uint8).expand(1024), whole[::2], whole.view(16, 16).t()):
        with pytest.raises(ValueError, match="contiguous"):
            fmha._scratch(w, 16, q)
