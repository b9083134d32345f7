"""Block bounds and picks, gathered key weights, eviction and compaction over a ragged cache, against plain forms."""

import pytest
import torch

import cache_ref as ref
from test_cache_attn_gpu import DEV, i32, make, poison, to_pages

pytestmark = pytest.mark.gpu


def nan_like(x):
    return torch.full((1,), float("nan"), device=DEV).to(x.dtype)


# ------------------------------------------------------------------ bounds --
@pytest.mark.parametrize("B,Hkv,D,lens,block,page,kv", [
    (1, 1, 64, [1], 16, 0, "bf16"), (2, 3, 128, [17, 200], 16, 16, "bf16"), (2, 2, 64, [0, 333], 32, 64, "bf16"),
    (3, 8, 128, [1000, 64, 65], 64, 16, "bf16"), (1, 2, 128, [513], 128, 32, "bf16"),
    (2, 2, 64, [129, 31], 64, 128, "e4m3"), (2, 4, 128, [300, 255], 128, 64, "e4m3"), (1, 1, 128, [40], 32, 0, "e4m3"),
])
def test_bounds(B, Hkv, D, lens, block, page, kv):
    from precision_attention_fmha_b200 import fmha

    q, k, v, _, g = make(B + D, B, 1, Hkv, Hkv, D, max(lens) + 20, page, kv)
    poison(k, lens)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    nb = -(-max(lens) // block) + 1
    before = torch.randn(B, Hkv, nb, 2, D, generator=g, device=DEV).bfloat16()
    got = fmha.key_bounds(k, i32(lens), block, table, bounds=before.clone())
    fmha.get_device_error()
    assert torch.equal(got.double(), ref.bounds(k, lens, block, before, table))
    # from a start on: earlier blocks keep what they held
    start = [max(0, n - 20) for n in lens]
    got = fmha.key_bounds(k, i32(lens), block, table, bounds=before.clone(), start=i32(start))
    want = ref.bounds(k, lens, block, before, table)
    for b in range(B):
        want[b, :, : start[b] // block] = before[b, :, : start[b] // block].double()
    assert torch.equal(got.double(), want)


# ------------------------------------------------------------------- picks --
@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,block,top,sinks,recent", [
    (1, 1, 1, 1, 64, [1], 16, 1, 0, 1), (1, 1, 8, 2, 128, [1000], 16, 5, 1, 2), (2, 3, 12, 4, 64, [700, 90], 32, 4, 0, 0),
    (1, 2, 4, 1, 128, [40000], 16, 64, 2, 3), (1, 1, 2, 2, 64, [120000], 16, 700, 1, 1), (3, 2, 8, 8, 128, [64, 65, 63], 64, 1, 0, 1),
    (2, 1, 4, 2, 128, [5000, 1], 128, 40, 1, 1), (1, 1, 4, 2, 128, [3000], 16, 2, 3, 4),
    (1, 1, 2, 1, 64, [16384 * 16], 16, 2000, 1, 1),  # the most blocks
])
def test_pick_lists(B, T, Hq, Hkv, D, lens, block, top, sinks, recent):
    from precision_attention_fmha_b200 import fmha

    g = torch.Generator(device=DEV)
    g.manual_seed(top)
    nb = -(-max(lens) // block)
    q = torch.randn(B, T, Hq, D, generator=g, device=DEV).bfloat16()
    x = torch.randn(B, Hkv, nb, 2, D, generator=g, device=DEV)
    bnd = torch.stack([x.amin(3), x.amax(3)], 3).bfloat16()
    q_lens = i32([max(0, min(T, n) - b % 2) for b, n in enumerate(lens)])
    for b in range(B):
        q[b, int(q_lens[b]):] = float("nan")
    got = fmha.select_blocks(q, bnd, i32(lens), block, top, sinks, recent, q_lens)
    fmha.get_device_error()
    want = torch.full_like(got, -1)
    for b, rows in enumerate(ref.pick(q, bnd, lens, block, top, sinks, recent, q_lens)):
        for t, heads in enumerate(rows):
            for h, ids in enumerate(heads):
                want[b, t, h, : len(ids)] = torch.tensor(ids, dtype=torch.int32)
    assert torch.equal(got, want)


def test_pick_ties_go_to_the_lowest_block():
    from precision_attention_fmha_b200 import fmha

    q = torch.ones(1, 1, 2, 64, device=DEV).bfloat16()
    bnd = torch.zeros(1, 1, 40, 2, 64, device=DEV).bfloat16()
    bnd[0, 0, 1::2] = -0.0  # equal to zero all the same
    bnd[0, 0, 20:23, 1] = 1.0
    got = fmha.select_blocks(q, bnd, i32([640]), 16, 9, 0, 1)
    assert got.flatten().tolist() == [0, 1, 2, 3, 4, 20, 21, 22, 39]
    bnd[:] = -1.0
    got = fmha.select_blocks(q, bnd, i32([640]), 16, 4, 0, 0)
    assert got.flatten().tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("D", [64, 128])
def test_pick_over_the_whole_range_of_values(D):
    """Queries and bounds of every BF16 magnitude, subnormals and the largest among them, in every channel."""
    from precision_attention_fmha_b200 import fmha

    g = torch.Generator(device=DEV)
    g.manual_seed(D + 1)

    def any_bf16(*shape):
        bits = torch.randint(0, 0x7f80, shape, generator=g, device=DEV) | torch.randint(0, 2, shape, generator=g, device=DEV) << 15
        return torch.where(bits >= 0x8000, bits - 0x10000, bits).to(torch.int16).view(torch.bfloat16)

    q = any_bf16(2, 2, 6, D)
    q[1] *= 2.0 ** -100  # one sequence's scores are all tiny
    x = any_bf16(2, 3, 200, 2, D)
    x[1] *= 2.0 ** -30
    bnd = torch.stack([x.amin(3), x.amax(3)], 3)
    lens = [200 * 16, 150 * 16 + 3]
    got = fmha.select_blocks(q, bnd, i32(lens), 16, 30, 1, 2)
    for b, rows in enumerate(ref.pick(q, bnd, lens, 16, 30, 1, 2)):
        for t, heads in enumerate(rows):
            for h, ids in enumerate(heads):
                assert got[b, t, h].tolist() == ids
    tiny = torch.full((1, 1, 1, D), 2.0 ** -133, device=DEV).bfloat16()  # the smallest of all
    low = torch.zeros(1, 1, 9, 2, D, device=DEV).bfloat16()
    low[0, 0, 4, 1, D - 1] = low[0, 0, 6, 1, 2] = 2.0 ** -133
    assert fmha.select_blocks(tiny, low, i32([9 * 16]), 16, 2, 0, 0).flatten().tolist() == [4, 6]


@pytest.mark.parametrize("D", [64, 128])
def test_pick_near_ties(D):
    """Scores that differ by less than 32 bits can tell (many blocks within 2^-24 of each other): the exact ones decide."""
    from precision_attention_fmha_b200 import fmha

    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    n = 1000
    q = torch.randn(2, 2, 6, D, generator=g, device=DEV).bfloat16()
    one = torch.randn(2, 3, 1, 2, D, generator=g, device=DEV)
    one = torch.stack([one.amin(3), one.amax(3)], 3).bfloat16().expand(2, 3, n, 2, D).contiguous()
    # one channel moves by a tiny amount: products of 2^-20 and less next to a score of order 10
    one[..., 0, 3] = -(torch.randint(1, 100, (2, 3, n), generator=g, device=DEV) * 2.0 ** -27).bfloat16()
    one[..., 1, 3] = (torch.randint(1, 100, (2, 3, n), generator=g, device=DEV) * 2.0 ** -27).bfloat16()
    lens = [n * 16, n * 16 - 40]
    got = fmha.select_blocks(q, one, i32(lens), 16, 300, 1, 2)
    for b, rows in enumerate(ref.pick(q, one, lens, 16, 300, 1, 2)):
        for t, heads in enumerate(rows):
            for h, ids in enumerate(heads):
                assert got[b, t, h].tolist() == ids


@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,top,sinks,recent", [
    (1, 128, 2, 1, 64, [128], 1, 0, 1), (1, 700, 8, 2, 128, [700], 3, 1, 1), (2, 300, 4, 4, 128, [300, 900], 2, 0, 1),
    (2, 513, 4, 1, 64, [513, 200], 4, 1, 2),
])
def test_pick_masks(B, T, Hq, Hkv, D, lens, top, sinks, recent):
    from precision_attention_fmha_b200 import fmha

    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    nb = -(-max(lens) // 128)
    q = torch.randn(B, T, Hq, D, generator=g, device=DEV).bfloat16()
    x = torch.randn(B, Hkv, nb, 2, D, generator=g, device=DEV)
    bnd = torch.stack([x.amin(3), x.amax(3)], 3).bfloat16()
    q_lens = i32([min(T, n) for n in lens])
    for b in range(B):
        q[b, int(q_lens[b]):] = float("nan")
    got = fmha.select_blocks(q, bnd, i32(lens), 128, top, sinks, recent, q_lens, q_tile=128)
    fmha.get_device_error()
    want = torch.zeros_like(got)
    for b, rows in enumerate(ref.pick(q, bnd, lens, 128, top, sinks, recent, q_lens, 128)):
        for i, heads in enumerate(rows):
            for h, ids in enumerate(heads):
                want[b, h, i, ids] = 1
    assert torch.equal(got, want)


# ----------------------------------------------------------------- weights --
# A weight is a sum of R exponentials. Each is off by at most 2^-13 relative (the score bound of cache_ref), the
# 32-bit sums inside a tile of at most 4096 terms by 2^-24 * 4096 / 2 relative at the very worst, 2^-13 again.
WEIGHT_RTOL = 2.0 ** -12


@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,page,kv", [
    (1, 1, 1, 1, 64, [1], 0, "bf16"), (2, 1, 8, 2, 128, [700, 65], 16, "bf16"), (3, 2, 12, 4, 128, [64, 63, 1000], 64, "bf16"),
    (2, 5, 14, 2, 64, [300, 40], 32, "bf16"), (2, 33, 8, 4, 128, [150, 33], 128, "bf16"), (2, 3, 8, 2, 128, [130, 500], 16, "e4m3"),
    (1, 2, 4, 4, 64, [257], 0, "e4m3"), (1, 64, 2, 1, 64, [64], 0, "bf16"), (1, 300, 6, 2, 128, [300], 64, "bf16"),
    (2, 130, 4, 1, 128, [1000, 77], 16, "bf16"), (2, 200, 4, 2, 64, [200, 513], 0, "bf16"), (2, 100, 4, 2, 128, [140, 99], 32, "e4m3"),
    (1, 257, 2, 2, 64, [300], 0, "e4m3"),
])
@pytest.mark.parametrize("causal", [True, False])
def test_weights(B, T, Hq, Hkv, D, lens, page, kv, causal):
    from precision_attention_fmha_b200 import fmha

    q, k, v, sf, g = make(T + B, B, T, Hq, Hkv, D, max(lens) + 9, page, kv)
    poison(k, lens)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    q_lens = i32([max(0, min(T, n) - b) for b, n in enumerate(lens)])
    for b in range(B):
        q[b, int(q_lens[b]):] = float("nan")
    lse = torch.randn(B, Hq, T, generator=g, device=DEV) + 4
    lse[0, 0, 0] = float("-inf")  # a row that saw nothing
    n = max(lens) + 5
    w0 = torch.rand(B, Hkv, n, generator=g, device=DEV)
    add = ref.weights(q, k, torch.where(torch.isinf(lse), torch.full_like(lse, float("inf")), lse), lens, n, q_lens, table, causal, sf[0])
    for accumulate in (True, False):
        w = fmha.key_weights(q, k, lse, w0.clone(), i32(lens), q_lens, table, causal, accumulate, sf_k=sf[0])
        fmha.get_device_error()
        for b, s in enumerate(lens):
            want = add[b, :, :s] + (w0[b, :, :s].double() if accumulate else 0)
            err = (w[b, :, :s].double() - want).abs()
            assert bool((err <= want.abs() * WEIGHT_RTOL + 1e-30).all()), float((err / want.abs().clamp(min=1e-30)).max())
            assert torch.equal(w[b, :, s:], w0[b, :, s:])
        again = fmha.key_weights(q, k, lse, w0.clone(), i32(lens), q_lens, table, causal, accumulate, sf_k=sf[0])
        assert torch.equal(w, again)


# ------------------------------------------------------- evict and compact --
@pytest.mark.parametrize("B,Hkv,lens,budget,sinks,recent", [
    (1, 1, [1], 1, 0, 0), (2, 2, [100, 5], 10, 2, 3), (1, 3, [5000], 1000, 4, 64), (3, 1, [33, 32, 31], 32, 0, 32),
    (1, 2, [40000], 7, 0, 0), (2, 1, [3000, 0], 2999, 1, 1), (1, 1, [70], 8, 4, 4),
    (1, 1, [120000], 30001, 16, 100), (3, 8, [9000, 20000, 8193], 8192, 1, 0), (40, 4, [600 + i for i in range(40)], 601, 0, 1),
    (160, 1, [60000] * 160, 100, 1, 1),  # too many keys for shared memory
    (3, 1, [49149, 31745, 31744], 20000, 3, 5), (2, 1, [32768, 993], 992, 0, 0), (2, 2, [65000, 49153], 48000, 7, 9),
])
def test_evict_select(B, Hkv, lens, budget, sinks, recent):
    from precision_attention_fmha_b200 import fmha

    g = torch.Generator(device=DEV)
    g.manual_seed(budget)
    w = torch.rand(B, Hkv, max(lens) + 3, generator=g, device=DEV)
    w = (w * 50).round() / 50 if budget != 1000 else w ** 8  # many ties
    w[0, 0, ::7] = 0.0
    w[0, 0, ::14] = -0.0
    if lens[0] > 60:
        w[0, 0, 20:24] = float("nan")
    keep, counts = fmha.evict_select(w, i32(lens), budget, sinks, recent)
    fmha.get_device_error()
    assert counts.tolist() == [min(n, budget) for n in lens]
    want = torch.full_like(keep, -1)
    for b, heads in enumerate(ref.kept(w, lens, budget, sinks, recent)):
        for h, at in enumerate(heads):
            want[b, h, : len(at)] = torch.tensor(at, dtype=torch.int32)
    assert torch.equal(keep, want)


def rows(x, table, b):
    n = x.shape[1] if table is None else table.shape[1] * x.shape[1]
    return ref.gather(x, table, b, n)


@pytest.mark.parametrize("B,Hkv,D,lens,budget,page,kv", [
    (1, 1, 64, [40], 9, 0, "bf16"), (2, 2, 128, [300, 700], 120, 16, "bf16"), (1, 4, 128, [2500], 1300, 64, "bf16"),
    (2, 2, 64, [500, 20], 300, 32, "e4m3"), (1, 2, 128, [700], 650, 128, "e4m3"), (1, 2, 128, [400], 100, 16, "bf16_e4m3"),
])
@pytest.mark.parametrize("inside", [False, True])
def test_compact(B, Hkv, D, lens, budget, page, kv, inside):
    from precision_attention_fmha_b200 import fmha

    q, k, v, _, g = make(D + B, B, 1, Hkv, Hkv, D, max(lens), page, kv)
    table = out_table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    n = max(lens) + 2
    w = torch.rand(B, Hkv, n, generator=g, device=DEV)
    keep, counts = fmha.evict_select(w, i32(lens), budget, 2, 5)
    kw = {}
    if not inside:
        per = -(-budget // page) if page else 0
        shape = (B, budget) if not page else (B * per + 1, page)
        ko = torch.ones(shape + (Hkv, D), device=DEV).to(k.dtype)
        vo = torch.ones(shape + (Hkv, D), device=DEV).to(v.dtype)
        if page:
            out_table = torch.randperm(B * per + 1, generator=g, device=DEV)[: B * per].to(torch.int32).view(B, per)
        wo = torch.full((B, Hkv, budget + 3), 9.0, device=DEV)
        kw = dict(k_out=ko, v_out=vo, out_page_table=out_table, weights_out=wo)
    bits = lambda x: x.view(torch.uint8)  # noqa: E731
    want = []
    for x, y in ((k, k if inside else ko), (v, v if inside else vo)):
        res = y.clone()
        for b in range(B):
            m = int(counts[b])
            for h in range(Hkv):
                at = keep[b, h, :m].long()
                src = rows(x, table, b)[at, h]
                to = torch.arange(m, device=DEV)
                t2 = table if inside else out_table
                if t2 is None:
                    res[b, to, h] = src
                else:
                    res[t2[b].long()[to // page], to % page, h] = src
        want.append(res)
    ww = torch.zeros_like(w if inside else wo)
    for b in range(B):
        for h in range(Hkv):
            m = int(counts[b])
            ww[b, h, :m] = w[b, h, keep[b, h, :m].long()]
    gk, gv = fmha.cache_compact(k, v, keep, counts, page_table=table, weights=w, **kw)
    fmha.get_device_error()
    assert torch.equal(bits(gk), bits(want[0])) and torch.equal(bits(gv), bits(want[1]))
    assert torch.equal(w if inside else wo, ww)


def test_compact_commits_a_tree_path():
    """An accepted path of a drafted tree moves to the end of the context, in every head."""
    from precision_attention_fmha_b200 import fmha

    ctx, path = [37, 60], [[0, 2, 5], [0, 1]]
    q, k, v, _, g = make(3, 2, 1, 2, 2, 64, 80, 16)
    k, v, table = to_pages(k, v, 16, g)
    keep = torch.full((2, 1, 3), -1, dtype=torch.int32, device=DEV)
    for b in range(2):
        keep[b, 0, : len(path[b])] = torch.tensor([ctx[b] + i for i in path[b]], dtype=torch.int32)
    before = [rows(k, table, b).clone() for b in range(2)]
    fmha.cache_compact(k, v, keep, i32([3, 2]), dst_start=i32(ctx), page_table=table)
    fmha.get_device_error()
    for b in range(2):
        want = before[b].clone()
        for i, n in enumerate(path[b]):
            want[ctx[b] + i] = before[b][ctx[b] + n]
        assert torch.equal(rows(k, table, b), want)
