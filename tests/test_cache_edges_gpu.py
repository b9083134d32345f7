"""The operators over a ragged cache at their edges: many-row trees (contexts on the packed tensor-memory tiles) with
non-finite keys, bad lengths and pages, strides and many sequences; long flat tails; empty groups of queries."""

import math

import pytest
import torch

import cache_ref as ref
from test_cache_attn_gpu import DEV, i32, make, poison, random_tree, to_pages

pytestmark = pytest.mark.gpu

PACKED = [
    # B, T, Hq, Hkv, room, page
    (1, 16, 16, 2, 1300, 0),    # 128 rows (two tiles of the same rows take alternate keys), one split
    (1, 16, 16, 2, 3300, 64),   # several splits
    (1, 40, 16, 2, 1300, 16),   # 320 rows
    (1, 40, 16, 2, 3300, 0),
    (10, 5, 64, 8, 1300, 0),    # 40 rows on many heads
    (10, 5, 64, 8, 2500, 128),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,room,page", PACKED)
@pytest.mark.parametrize("bad", ["k nan", "k inf", "v nan"])
@pytest.mark.parametrize("where", ["middle", "last"])
def test_packed_non_finite_context(B, T, Hq, Hkv, room, page, bad, where):
    """A key of the context whose score is NaN makes every row of its KV head NaN, as in the few-row kernel, whatever tile
    or split it is in; a NaN value its column. All other rows keep their bits."""
    from precision_attention_fmha_b200 import fmha

    D, G = 128, Hq // Hkv
    ctx = [room - T - 20 - 7 * b for b in range(B)]
    q, k, v, _, g = make(41, B, T, Hq, Hkv, D, room, page)
    at = 3 * 128 + 5 if where == "middle" else ctx[-1] // 128 * 128 - 1
    x, y = k.clone(), v.clone()
    if bad == "v nan":
        y[-1, at, -1, 7] = float("nan")
    else:
        x[-1, at, -1, 3] = float("nan" if bad == "k nan" else "inf")

    def run(k, v):
        table = None
        if page:
            k, v, table = to_pages(k, v, page, torch.Generator(device=DEV).manual_seed(1))
        lse = torch.empty(B, Hq, T, device=DEV)
        return fmha.fmha_fwd_tree(q, k, v, i32(ctx), None, None, table, lse=lse), lse

    want, want_lse = run(k, v)
    o, lse = run(x, y)
    fmha.get_device_error()
    assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
    heads = slice(Hq - G, Hq)  # of the last KV head
    if bad == "v nan":
        assert torch.isnan(o[-1, :, heads, 7]).all()
        o[-1, :, heads, 7] = want[-1, :, heads, 7]
    else:
        hit = (q[-1, :, heads, 3] >= 0) if bad == "k inf" else torch.ones(T, G, dtype=torch.bool, device=DEV)
        assert torch.equal(torch.isnan(o[-1, :, heads]).all(-1), hit)
        assert torch.equal(~torch.isfinite(lse[-1, heads]).t(), hit)
        assert torch.equal(torch.isfinite(o[-1, :, heads]).all(-1), ~hit)
        o[-1, :, heads], lse[-1, heads] = want[-1, :, heads], want_lse[-1, heads]
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("kv", ["bf16", "bf16_e4m3", "e4m3"])
@pytest.mark.parametrize("Hq", [8, 16, 32, 64])  # rows a KV head: every arrangement of the few-row kernel
def test_long_flat_tail(Hq, kv):
    """One dominant key, then 65536 keys of 2^-27 of its weight each: what they add up to (2^-11) is neither lost nor
    skewed by the 16-bit weights. All sequences read the same pages, and there are enough for a CTA to walk a sequence
    whole. Lifted as
    they are, all 16-bit weights are normal numbers, so the tolerance is that of cache_ref.check (A = O: no value is negative);
    the tail's weights are equal, and the 32-bit sums of 2^14 of them per warp and column are off by 2^-24 * 2^14 / 16
    relative at the worst (one addition per 16 keys), 2^-14, which 2^-12 A holds beside the rest."""
    from precision_attention_fmha_b200 import fmha

    B, D, page, N = 444, 64, 128, 65536
    wide = N // page + 1
    kt = torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16
    vt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    k, v = torch.zeros(wide, page, 1, D, device=DEV), torch.zeros(wide, page, 1, D, device=DEV)
    k[0, 0, 0, 0] = 12.0
    v[..., :32] = 1.0  # the tail's columns
    v[0, 0, 0, :32], v[0, 0, 0, 32:] = 0.0, 1.0
    q = torch.zeros(B, 1, Hq, D, device=DEV, dtype=torch.bfloat16)
    q[..., 0] = 12.5
    table = torch.arange(wide, device=DEV, dtype=torch.int32).expand(B, wide).contiguous()
    lse = torch.empty(B, Hq, 1, device=DEV)
    o = fmha.fmha_fwd_tree(q, k.to(kt), v.to(vt), i32([N] * B), page_table=table, lse=lse)
    fmha.get_device_error()
    z = 12.5 * 12.0 / 8.0
    tail = N * math.exp(-z)  # the node is the last of the N keys behind the first
    want = torch.full((D,), tail / (1 + tail), dtype=torch.float64, device=DEV)
    want[32:] = 1 / (1 + tail)
    ref.check(o, lse, (want.expand(B, 1, Hq, D), torch.full((B, Hq, 1), z + math.log1p(tail), dtype=torch.float64, device=DEV),
                       want.expand(B, 1, Hq, D)), v8=kv != "bf16")


@pytest.mark.parametrize("T,Hq", [(0, 4), (3, 0), (0, 0)])
@pytest.mark.parametrize("page", [0, 16])
def test_weights_without_query_rows(T, Hq, page):
    """An empty sum is zero: written over what the weights held up to each length, or added to it."""
    from precision_attention_fmha_b200 import fmha

    B, Hkv, D, lens = 3, 2, 64, [1500, 0, 33]
    _, k, v, _, g = make(51, B, 1, 2, Hkv, D, 1504, page)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    q = torch.empty(B, T, Hq, D, device=DEV, dtype=torch.bfloat16)
    w0 = torch.rand(B, Hkv, 1501, generator=g, device=DEV)
    want = w0.clone()
    for b, n in enumerate(lens):
        want[b, :, :n] = 0
    lse = torch.empty(B, Hq, T, device=DEV)
    assert torch.equal(fmha.key_weights(q, k, lse, w0.clone(), i32(lens), page_table=table, accumulate=False), want)
    assert torch.equal(fmha.key_weights(q, k, lse, w0.clone(), i32(lens), page_table=table, accumulate=True), w0)
    fmha.get_device_error()
    far = [1505, -1, 33]
    want[0, :, 1500] = 0
    assert torch.equal(fmha.key_weights(q, k, lse, w0.clone(), i32(far), page_table=table, accumulate=False), want)
    with pytest.raises(fmha.FmhaError) as e:
        fmha.get_device_error()
    assert e.value.status == fmha.FMHA_ERR_DEVICE_INDEX


@pytest.mark.parametrize("q_tile", [1, 128])
def test_picks_without_query_heads(q_tile):
    """No query head: every score is an empty sum, so the ties' rule picks, and the whole of `picked` is written."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hkv, D, lens, block, top, sinks, recent = 2, 130, 2, 64, [1100, 140], 128, 4, 1, 1
    q = torch.empty(B, T, 0, D, device=DEV, dtype=torch.bfloat16)
    nb = 9
    bnd = torch.randn(B, Hkv, nb, 2, D, device=DEV).bfloat16()
    shape, dtype = ((B, T, Hkv, top), torch.int32) if q_tile == 1 else ((B, Hkv, 2, nb), torch.uint8)
    got = fmha.select_blocks(q, bnd, i32(lens), block, top, sinks, recent, q_tile=q_tile, out=torch.full(shape, 99, device=DEV).to(dtype))
    fmha.get_device_error()
    want = torch.full(shape, -1 if q_tile == 1 else 0, device=DEV).to(dtype)
    for b, rows in enumerate(ref.pick(q, bnd, lens, block, top, sinks, recent, None, q_tile)):
        for i, heads in enumerate(rows):
            for h, ids in enumerate(heads):
                if q_tile == 1:
                    want[b, i, h, : len(ids)] = i32(ids)
                else:
                    want[b, h, i, ids] = 1
    assert torch.equal(got, want)


@pytest.mark.parametrize("inside", [True, False])
@pytest.mark.parametrize("page", [0, 16])
def test_compact_leaves_out_a_row_with_its_weight(inside, page):
    """A position past the cache, out of order or on a bad page is reported, and its row and its weight stay as they were."""
    from precision_attention_fmha_b200 import fmha

    Hkv, D, n, room = 2, 64, 96, 64
    _, k, v, _, g = make(61, 1, 1, 2, Hkv, D, room, page)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
        bad = table.clone()
        bad[0, 2] = 1 << 20  # positions 32..47
    keep = i32([[[0, 2, 9, 8, 20, 35, 40, 50, 63, 70, 80]]])  # 8: out of order (inside one cache); 70, 80: past the cache
    count, start = 10, 0
    w = torch.rand(1, Hkv, n, generator=g, device=DEV)
    ko, vo = (k, v) if inside else (torch.ones(1, 16, Hkv, D, device=DEV).bfloat16(), torch.ones(1, 16, Hkv, D, device=DEV).bfloat16())
    wo = w if inside else torch.full((1, Hkv, 14), 5.0, device=DEV)
    left_out = {9} | ({3} if inside else set()) | ({5, 6} if page else set())
    want_w, rows_k = wo.clone(), (ref.gather(ko, table, 0, room) if inside else ko[0]).clone()
    src = ref.gather(k, table, 0, room)
    for i in range(count):
        if i not in left_out:
            want_w[0, :, start + i] = w[0, :, int(keep[0, 0, i])]
            rows_k[start + i] = src[int(keep[0, 0, i])]
    want_w[0, :, start + count:] = 0
    fmha.cache_compact(k, v, keep, i32([count]), page_table=bad if page else None, weights=w,
                       **({} if inside else dict(k_out=ko, v_out=vo, weights_out=wo)))
    with pytest.raises(fmha.FmhaError) as e:
        fmha.get_device_error()
    assert e.value.status == fmha.FMHA_ERR_DEVICE_INDEX
    assert torch.equal(ref.gather(ko, table, 0, room) if inside else ko[0], rows_k)
    assert torch.equal(wo, want_w)


@pytest.mark.parametrize("start", [2 ** 31 - 1, 2 ** 31 - 3, -2 ** 31, 2 ** 30, 64])
@pytest.mark.parametrize("inside", [True, False])
def test_compact_to_a_start_outside_the_cache(start, inside):
    """Sums of a start and a row number stay in range: nothing moves, no weight changes but those past a negative start."""
    from precision_attention_fmha_b200 import fmha

    k, v, n = torch.randn(1, 64, 2, 64, device=DEV).bfloat16(), torch.randn(1, 64, 2, 64, device=DEV).bfloat16(), 70
    w = torch.rand(1, 2, n, device=DEV)
    out = dict(k_out=torch.zeros_like(k), v_out=torch.zeros_like(v), weights_out=torch.full_like(w, 3.0))
    to = (k, v, w) if inside else tuple(out.values())
    before = [x.clone() for x in to]
    if start == 64:  # past the cache, not past the weights
        before[2][:, :, 64 + 5:] = 0
    if start < 0 and inside:
        before[2][:] = 0
    fmha.cache_compact(k, v, i32([[[40, 41, 42, 50, 63]]]), i32([5]), dst_start=i32([start]), weights=w, **({} if inside else out))
    with pytest.raises(fmha.FmhaError) as e:
        fmha.get_device_error()
    assert e.value.status == fmha.FMHA_ERR_DEVICE_INDEX
    assert all(torch.equal(a, b) for a, b in zip(to, before))


@pytest.mark.parametrize("page", [0, 16])
def test_packed_lengths_past_the_cache(page):
    """Lengths outside a cache whose room is no whole number of key tiles are cut to it and reported, as with few rows."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, room = 5, 17, 16, 2, 128, 1040
    q, k, v, _, g = make(71, B, T, Hq, Hkv, D, room, page)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    given, nodes = [1500, 1040, 1030, -3, 600], [17, 17, 17, 17, 40]
    cut, left = [1040, 1040, 1030, 0, 600], [0, 0, 10, 17, 17]

    def run(ctx, nodes):
        lse = torch.empty(B, Hq, T, device=DEV)
        return fmha.fmha_fwd_tree(q, k, v, i32(ctx), None, i32(nodes), table, lse=lse), lse

    o, lse = run(given, nodes)
    with pytest.raises(fmha.FmhaError) as e:
        fmha.get_device_error()
    assert e.value.status == fmha.FMHA_ERR_DEVICE_INDEX
    want = run(cut, left)
    fmha.get_device_error()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    ref.check(o, lse, ref.tree(q, k, v, cut, None, i32(left), table))


@pytest.mark.parametrize("T", [1, 17])  # the few-row kernel alone, and with the packed one before it
def test_bad_pages_read_zeros(T):
    from precision_attention_fmha_b200 import fmha

    B, Hq, Hkv, D, room, page = 2, 16, 2, 128, 1280, 64
    q, k, v, _, g = make(72, B, T, Hq, Hkv, D, room, page)
    k, v, table = to_pages(k, v, page, g)
    k, v, zero = k.nan_to_num(0), v.nan_to_num(0), k.shape[0] - 1
    k[-1], v[-1] = 0, 0
    table = torch.where(table == zero, zero - 1, table).to(torch.int32)  # no sequence reads the page of zeros
    ctx = i32([1200, 1263 - T])
    for at, bad in ((3, 1 << 20), (18, -1), (0, k.shape[0])):
        wrong, right = table.clone(), table.clone()
        wrong[1, at], right[1, at] = bad, zero
        lse, want_lse = torch.empty(B, Hq, T, device=DEV), torch.empty(B, Hq, T, device=DEV)
        o = fmha.fmha_fwd_tree(q, k, v, ctx, page_table=wrong, lse=lse)
        with pytest.raises(fmha.FmhaError) as e:
            fmha.get_device_error()
        assert e.value.status == fmha.FMHA_ERR_DEVICE_INDEX
        want = fmha.fmha_fwd_tree(q, k, v, ctx, page_table=right, lse=want_lse)
        fmha.get_device_error()
        assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("page", [0, 32])
def test_packed_many_sequences(page):
    """More sequences than the packed kernel orders by length; strided q, out, K and V; masks with empty rows; padding."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, room = 37, 17, 8, 1, 128, 1280
    q, k, v, _, g = make(73, B, T + 2, Hq + 3, Hkv + 1, D, room, page)
    q = q[:, 1:T + 1, 2:Hq + 2]
    ctx = [(397 * b + 11 * b * b) % (room - T + 1) for b in range(B)]
    ctx[5], ctx[6], ctx[7] = 0, 1024, room - T
    nodes = [(T - 3 * b) % (T + 1) for b in range(B)]
    ends = [c + n for c, n in zip(ctx, nodes)]
    poison(k, ends), poison(v, ends)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    k, v = k[:, :, 1:], v[:, :, :1]
    for b in range(B):
        q[b, nodes[b]:] = float("nan")
    mask = random_tree(B, T, g)
    wide = torch.full((B, T + 1, Hq * 2, D), 5.0, device=DEV).bfloat16()
    lse = torch.empty(B, Hq, T, device=DEV)
    o = fmha.fmha_fwd_tree(q, k, v, i32(ctx), mask, i32(nodes), table, out=wide[:, :T, ::2], lse=lse)
    fmha.get_device_error()
    ref.check(o, lse, ref.tree(q, k, v, ctx, mask, i32(nodes), table))
    assert bool((wide[:, T:] == 5).all()) and bool((wide[:, :, 1::2] == 5).all())


def test_packed_hidden_nodes_may_hold_anything():
    """A drafted node that a row does not see holds NaN and infinities, behind a context on the packed tiles."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, ctx = 2, 20, 16, 2, 128, [1100, 1279]
    q, k, v, _, g = make(74, B, T, Hq, Hkv, D, 1320)
    mask = torch.eye(T, device=DEV, dtype=torch.uint8).expand(B, T, T).contiguous()
    mask[:, :, 0] = 1
    for i, n in enumerate([3, 9, 16]):
        mask[:, :, n] = 0
        for b in range(B):
            k[b, ctx[b] + n] = float("nan")
            v[b, ctx[b] + n, :, i::5] = float("nan")
            v[b, ctx[b] + n, :, i + 1::7] = float("inf")
    lse = torch.empty(B, Hq, T, device=DEV)
    o = fmha.fmha_fwd_tree(q, k, v, i32(ctx), mask, lse=lse)
    fmha.get_device_error()
    ref.check(o, lse, ref.tree(q, k, v, ctx, mask, None, None))


def test_many_rows_in_a_replayed_graph():
    """One capture of a wide tree, a prompt's weights, a choice and a compaction in place; between replays the lengths, the
    drafted nodes and the queries change. Each replay gives what the calls give, and the calls what the formulas say."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, room, page = 3, 70, 16, 2, 128, 1600, 64
    q, k, v, _, g = make(81, B, T, Hq, Hkv, D, room, page)
    k0, v0, table = to_pages(k, v, page, g)
    k, v = k0.clone(), v0.clone()
    ctx, nodes, lens = i32([10, 1400, 900]), i32([T] * B), i32([10 + T, 1400 + T, 900 + T])
    lse = torch.empty(B, Hq, T, device=DEV)
    weights = torch.zeros(B, Hkv, room, device=DEV)

    def step():
        o = fmha.fmha_fwd_tree(q, k, v, ctx, None, nodes, table, lse=lse)
        fmha.key_weights(q, k, lse, weights, lens, nodes, table, accumulate=False)
        keep, counts = fmha.evict_select(weights, lens, 200, 4, 32)
        fmha.cache_compact(k, v, keep, counts, page_table=table, weights=weights)
        return o, keep, counts

    def fresh():
        k.copy_(k0), v.copy_(v0), weights.fill_(9.0), lse.fill_(9.0)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for c, m in (([0, 1530, 128], [70, 70, 70]), ([1279, 1280, 1281], [64, 0, 1]), ([640, 3, 1529], [33, 70, 69])):
        ctx.copy_(i32(c)), nodes.copy_(i32(m)), lens.copy_(i32([a + b for a, b in zip(c, m)]))
        q.copy_(torch.randn(q.shape, generator=g, device=DEV))
        fresh()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*out, lse, k, v, weights)]
        fresh()
        want = [*step(), lse, k, v, weights]
        assert all(torch.equal(a.nan_to_num(7), b.nan_to_num(7)) for a, b in zip(got, want))
        ref.check(got[0], got[3], ref.tree(q, k0, v0, c, None, i32(m), table))
    fmha.get_device_error()
    del graph
