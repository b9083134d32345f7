"""The operators over a ragged cache as a server calls them: strided tensors, streams, graphs, concurrent calls, far
positions, reported errors, and a run of them together."""

import math

import pytest
import torch

import cache_ref as ref
from test_cache_attn_gpu import DEV, i32, make, random_tree, to_pages

pytestmark = pytest.mark.gpu


def test_strided_tensors():
    """K and V as halves of one pool, heads before tokens in memory, q and out as slices of wider tensors."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, page = 2, 5, 6, 2, 128, 32
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    pool = torch.randn(9, 2, Hkv, page, D, generator=g, device=DEV).bfloat16()
    k, v = pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2)
    table = torch.randperm(9, generator=g, device=DEV)[:8].view(2, 4).to(torch.int32)
    wide = torch.randn(B, T + 2, Hq + 3, D + 64, generator=g, device=DEV).bfloat16()
    q = wide[:, 1:T + 1, 2:Hq + 2, 64:]
    ctx = [100, 37]
    mask = random_tree(B, T, g)
    out = torch.full((B, T + 1, Hq * 2, D), 5.0, device=DEV).bfloat16()
    o = out[:, :T, ::2]
    lse = torch.empty(B, Hq, T, device=DEV)
    fmha.fmha_fwd_tree(q, k, v, i32(ctx), mask, None, table, out=o, lse=lse)
    want = ref.tree(q, k, v, ctx, mask, None, table)
    ref.check(o, lse, want)
    assert bool((out[:, T:] == 5).all()) and bool((out[:, :, 1::2] == 5).all())
    lens = [105, 42]
    bounds = fmha.key_bounds(k, i32(lens), 16, table)
    assert torch.equal(bounds.double(), ref.bounds(k, lens, 16, torch.zeros_like(bounds), table))
    blocks = fmha.select_blocks(q, bounds, i32(lens), 16, 3, 1, 1)
    got = fmha.fmha_fwd_selected(q, k, v, blocks, i32(lens), 16, None, table, lse=lse)
    ref.check(got, lse, ref.selected(q, k, v, blocks, lens, 16, None, table))
    w = fmha.key_weights(q, k, lse, torch.zeros(B, Hkv, 128, device=DEV), i32(lens), page_table=table)
    assert bool((w.double() - ref.weights(q, k, lse, lens, 128, None, table)).abs().max() < 1e-3)


def test_streams_and_threads():
    """Calls on side streams, two at once, give what one call gives."""
    import threading

    from precision_attention_fmha_b200 import fmha

    q, k, v, _, g = make(2, 4, 8, 32, 8, 128, 2100)
    ctx = i32([2000, 1, 700, 1333])
    mask = random_tree(4, 8, g)
    lens = i32([2000, 9, 708, 1341])
    bounds = fmha.key_bounds(k, lens, 64)
    torch.cuda.synchronize()

    def work(stream=None):
        lse = torch.empty(4, 32, 8, device=DEV)
        torch.cuda.synchronize()
        o = fmha.fmha_fwd_tree(q, k, v, ctx, mask, lse=lse, stream=stream)
        blocks = fmha.select_blocks(q, bounds, lens, 64, 9, 1, 2, stream=stream)
        s = fmha.fmha_fwd_selected(q, k, v, blocks, lens, 64, stream=stream)
        w = fmha.key_weights(q, k, lse, torch.zeros(4, 8, 2100, device=DEV), lens, stream=stream, accumulate=False)
        return o, lse, blocks, s

    want = work()
    got = [None] * 4

    def run(i):
        stream = torch.cuda.Stream()
        for _ in range(10):
            got[i] = work(stream)
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_threads_with_calls_of_different_sizes():
    """The kernels whose shared memory follows the call's size: large and small calls under way at once."""
    import threading

    from precision_attention_fmha_b200 import fmha

    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    sizes = [40, 45000, 3000, 20000]
    cases = []
    for n in sizes:
        w = torch.rand(1, 2, n, generator=g, device=DEV)
        n_blocks = max(4, n // 4)
        q = torch.randn(1, 1, 4, 64, generator=g, device=DEV).bfloat16()
        bounds = torch.randn(1, 2, n_blocks, 2, 64, generator=g, device=DEV).bfloat16()
        cases.append((w, i32([n]), q, bounds, i32([n_blocks * 16])))

    def work(c, stream=None):
        w, lens, q, bounds, tokens = c
        return fmha.evict_select(w, lens, 17, stream=stream)[0], fmha.select_blocks(q, bounds, tokens, 16, 3, stream=stream)

    want = [work(c) for c in cases]
    torch.cuda.synchronize()
    errors, got = [], [None] * len(cases)

    def run(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(200):
                got[i] = work(cases[i], stream)
            stream.synchronize()
        except Exception as e:  # an assertion of the main thread reports it
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(cases))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for r, x in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(r, x))


def test_graph_replay_with_grown_sequences():
    """One capture; between replays the lengths, keys and queries change in place."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, S = 3, 2, 8, 2, 64, 600
    q, k, v, _, g = make(3, B, T, Hq, Hkv, D, S)
    lens = i32([10, 500, 64])
    lse = torch.empty(B, Hq, T, device=DEV)
    weights = torch.zeros(B, Hkv, S, device=DEV)
    bounds = torch.zeros(B, Hkv, -(-S // 16), 2, D, device=DEV).bfloat16()

    def step():
        fmha.key_bounds(k, lens, 16, bounds=bounds)
        blocks = fmha.select_blocks(q, bounds, lens, 16, 6, 1, 2)
        o = fmha.fmha_fwd_selected(q, k, v, blocks, lens, 16, lse=lse)
        t = fmha.fmha_fwd_tree(q, k, v, lens, lse=None)
        fmha.key_weights(q, k, lse, weights, lens)
        keep, counts = fmha.evict_select(weights, lens, 100, 4, 8)
        return blocks, o, t, keep, counts

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in ([11, 501, 65], [300, 598, 2], [598, 17, 333]):
        lens.copy_(i32(n))
        q.copy_(torch.randn(q.shape, generator=g, device=DEV))
        k[:, :, :, 1].mul_(-1)
        weights.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out] + [lse.clone(), weights.clone()]
        weights.zero_()
        want = list(step()) + [lse, weights]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        ref.check(got[1], got[5], ref.selected(q, k, v, got[0], n, 16))
    fmha.get_device_error()
    del graph


def test_far_positions():
    """A cache of more than 2^31 elements: offsets are 64 bits wide."""
    from precision_attention_fmha_b200 import fmha

    B, Hq, Hkv, D, S = 2, 16, 16, 128, 560000  # 2.3e9 elements each of K and V
    k = torch.zeros(B, S, Hkv, D, device=DEV, dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    n = S - 70
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    tail = slice(n - 200, n + 64)
    k[:, tail] = torch.randn(B, 264, Hkv, D, generator=g, device=DEV).bfloat16() * 3
    v[:, tail] = torch.randn(B, 264, Hkv, D, generator=g, device=DEV).bfloat16()
    q = torch.randn(B, 1, Hq, D, generator=g, device=DEV).bfloat16()
    lens = i32([n, n - 3])
    top = torch.full((B, 1, Hkv, 2), -1, dtype=torch.int32, device=DEV)
    top[..., 0] = (n - 4) // 64
    top[..., 1] = (n - 4) // 64 - 1
    lse = torch.empty(B, Hq, 1, device=DEV)
    o = fmha.fmha_fwd_selected(q, k, v, top, lens, 64, lse=lse)
    ref.check(o, lse, ref.selected(q, k, v, top, [n, n - 3], 64))
    o = fmha.fmha_fwd_tree(q, k, v, lens, lse=lse)
    # every other key scores 0 and has value 0
    for b in range(B):
        end = n - 3 * b + 1
        for h in (0, Hq - 1):
            x, y = k[b, end - 200:end, h].double(), v[b, end - 200:end, h].double()
            z = (x @ q[b, 0, h].double()) / math.sqrt(D)
            total = math.log(float(z.exp().sum()) + end - 200)
            assert abs(float(lse[b, h, 0]) - total) < 1e-4
            want = (z - total).exp() @ y
            assert bool(((o[b, 0, h].double() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -8 * ((z - total).exp() @ y.abs())).all())
    w = fmha.key_weights(q, k, lse, torch.zeros(B, Hkv, S, device=DEV), i32([n + 1, n - 2]))
    assert abs(float(w[1, Hkv - 1, :n - 2].double().sum()) - 1) < 1e-3 and float(w[1, :, n - 2:].abs().max()) == 0
    bounds = fmha.key_bounds(k, lens, 128)
    j = (n - 4) // 128
    part = k[1, 128 * j:n - 3].double()
    assert torch.equal(bounds[1, :, j, 0].double(), part.amin(0)) and torch.equal(bounds[1, :, j, 1].double(), part.amax(0))
    keep = i32(list(range(n - 40, n))).view(1, 1, 40).expand(B, 1, 40).contiguous()
    before = k[1, n - 40:n].clone()
    fmha.cache_compact(k, v, keep, i32([40, 40]), dst_start=i32([5, n - 100]))
    assert torch.equal(k[1, n - 100:n - 60], before)
    fmha.get_device_error()


def test_bounds_with_far_more_blocks_than_keys():
    """Room for more blocks than 32-bit positions reach: what lies past the cache is left as it was."""
    from precision_attention_fmha_b200 import fmha

    n = (1 << 24) + 3
    k = torch.randn(1, 300, 1, 64, device=DEV).bfloat16()
    bounds = torch.empty(1, 1, n, 2, 64, dtype=torch.bfloat16, device=DEV)
    bounds[0, 0, 3:] = 7
    fmha.key_bounds(k, i32([300]), 128, bounds=bounds)
    first = fmha.key_bounds(k, i32([300]), 128)
    assert torch.equal(bounds[:, :, :3], first)
    assert bool((bounds[0, 0, 3:] == 7).all())
    fmha.get_device_error()


def test_reported_errors():
    """Bad pages, ids and lengths are reported, and what they name is left out or cut."""
    from precision_attention_fmha_b200 import fmha

    q, k, v, _, g = make(5, 2, 1, 4, 2, 64, 128, 32)
    k, v, table = to_pages(k.nan_to_num(0), v.nan_to_num(0), 32, g, extra=0)
    lens = i32([100, 127])
    fmha.get_device_error()

    def reported(f):
        f()
        with pytest.raises(fmha.FmhaError) as e:
            fmha.get_device_error()
        assert e.value.status == fmha.FMHA_ERR_DEVICE_INDEX
        fmha.get_device_error()  # cleared

    bad = table.clone()
    bad[1, 2] = 1 << 20
    for n in (bad, torch.where(bad == 1 << 20, -1, bad).to(torch.int32)):
        reported(lambda: fmha.fmha_fwd_tree(q, k, v, lens, page_table=n))
        reported(lambda: fmha.key_bounds(k, lens, 16, n))
        reported(lambda: fmha.key_weights(q, k, torch.zeros(2, 4, 1, device=DEV), torch.zeros(2, 2, 128, device=DEV), lens, page_table=n))
    ids = torch.zeros(2, 1, 2, 2, dtype=torch.int32, device=DEV)
    ids[1, 0, 1, 1] = 1 << 24
    reported(lambda: fmha.fmha_fwd_selected(q, k, v, ids, lens, 32, page_table=table))
    one = torch.where(ids == 1 << 24, -1, ids).to(torch.int32)
    o = fmha.fmha_fwd_selected(q, k, v, ids, lens, 32, page_table=table)
    assert torch.equal(o, fmha.fmha_fwd_selected(q, k, v, one, lens, 32, page_table=table))
    with pytest.raises(fmha.FmhaError):
        fmha.get_device_error()
    for n in (i32([100, 129]), i32([-1, 5])):
        reported(lambda: fmha.fmha_fwd_tree(q, k, v, n, page_table=table))
        reported(lambda: fmha.key_bounds(k, n, 16, table))
        reported(lambda: fmha.evict_select(torch.zeros(2, 2, 128, device=DEV), n, 7))
        reported(lambda: fmha.fmha_fwd_selected(q, k, v, one, n, 32, page_table=table))
    w = torch.rand(2, 2, 128, device=DEV)
    order = i32([[[5, 4], [7, 9]], [[1, 2], [3, 4]]])
    reported(lambda: fmha.cache_compact(k, v, order, i32([2, 2]), page_table=table, weights=w))      # out of order
    reported(lambda: fmha.cache_compact(k, v, order, i32([3, 2]), page_table=table))                 # more than listed
    reported(lambda: fmha.cache_compact(k, v, order, i32([2, 2]), dst_start=i32([6, 0]), page_table=table))  # moving up
    out = torch.zeros(2, 4, 2, 64, device=DEV).bfloat16()
    far = i32([[[5, 999], [7, 9]], [[1, 2], [3, 4]]])
    reported(lambda: fmha.cache_compact(k, v, far, i32([2, 2]), page_table=table, k_out=out, v_out=out.clone()))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_request_from_prompt_to_evicted_cache(kv):
    """A prompt's weights shrink its cache; blocks are picked from what is left; a draft is verified, its accepted path
    committed, and the next draft attends to it. Each step against its 64-bit form on the same state."""
    from precision_attention_fmha_b200 import fmha

    B, S, Hq, Hkv, D, page = 2, 900, 8, 2, 128, 16
    q, k, v, sf, g = make(6, B, S, Hq, Hkv, D, S, 0, kv)
    lens = [900, 777]
    # the prompt: its own tokens gather the weights (one padded sequence)
    lse = torch.empty(B, Hq, S, device=DEV)
    fmha.fmha_fwd_tree(q, k, v, i32([0, 0]), None, i32(lens), sf_k=sf[0], sf_v=sf[1], lse=lse)
    w = torch.zeros(B, Hkv, S, device=DEV)
    fmha.key_weights(q, k, lse, w, i32(lens), i32(lens), sf_k=sf[0])
    total = torch.tensor(lens, device=DEV).double()[:, None] * (Hq // Hkv)
    assert bool(((w.double().sum(-1) - total).abs() < 1e-3 * total).all())  # every row's weights sum to 1
    # shrink to 256 keys a head, into a paged cache with room for 320
    keep, counts = fmha.evict_select(w, i32(lens), 256, 4, 32)
    per = 320 // page
    kp = torch.zeros(B * per, page, Hkv, D, device=DEV).to(k.dtype)
    vp = torch.zeros(B * per, page, Hkv, D, device=DEV).to(v.dtype)
    table = torch.randperm(B * per, generator=g, device=DEV).to(torch.int32).view(B, per)
    w2 = torch.empty(B, Hkv, 320, device=DEV)
    fmha.cache_compact(k, v, keep, counts, k_out=kp, v_out=vp, out_page_table=table, weights=w, weights_out=w2)
    for b in range(B):
        for h in range(Hkv):
            at = keep[b, h].long()
            assert torch.equal(ref.gather(kp, table, b, 256)[:, h].float(), k[b, at, h].float())
            assert torch.equal(w2[b, h, :256], w[b, h, at]) and float(w2[b, h, 256:].abs().max()) == 0
    ctx = counts  # the new lengths
    # a drafted tree of 9 nodes behind the kept keys
    T = 9
    qt = torch.randn(B, T, Hq, D, generator=g, device=DEV).bfloat16()
    new_k, new_v = torch.randn(B, T, Hkv, D, generator=g, device=DEV), torch.randn(B, T, Hkv, D, generator=g, device=DEV)
    for b in range(B):
        for i in range(T):
            s = 256 + i
            kp[table[b, s // page].long(), s % page] = (new_k[b, i] * (32 if kv == "e4m3" else 1)).to(k.dtype)
            vp[table[b, s // page].long(), s % page] = (new_v[b, i] * (32 if kv != "bf16" else 1)).to(v.dtype)
    mask = random_tree(B, T, g)
    tl = torch.empty(B, Hq, T, device=DEV)
    o = fmha.fmha_fwd_tree(qt, kp, vp, ctx, mask, page_table=table, sf_k=sf[0], sf_v=sf[1], lse=tl)
    ref.check(o, tl, ref.tree(qt, kp, vp, [256, 256], mask, None, table, *sf), v8=kv != "bf16")
    # accept nodes 0, 3, 7 of one sequence and 0, 1 of the other
    path = i32([[[256, 259, 263]], [[256, 257, -1]]])
    fmha.cache_compact(kp, vp, path, i32([3, 2]), dst_start=ctx, page_table=table)
    lens2 = [259, 258]
    # the next token picks blocks out of the cache and attends to them; its weights are added
    q1 = torch.randn(B, 1, Hq, D, generator=g, device=DEV).bfloat16()
    bounds = fmha.key_bounds(kp, i32(lens2), 16, table)
    blocks = fmha.select_blocks(q1, bounds, i32(lens2), 16, 6, 1, 2)
    want = ref.pick(q1, bounds, lens2, 16, 6, 1, 2)
    assert [[[x for x in h if x >= 0] for h in t] for t in blocks[0].tolist()] == want[0]
    l1 = torch.empty(B, Hq, 1, device=DEV)
    o = fmha.fmha_fwd_selected(q1, kp, vp, blocks, i32(lens2), 16, page_table=table, sf_k=sf[0], sf_v=sf[1], lse=l1)
    ref.check(o, l1, ref.selected(q1, kp, vp, blocks, lens2, 16, None, table, *sf), v8=kv != "bf16")
    o = fmha.fmha_fwd_tree(q1, kp, vp, i32([n - 1 for n in lens2]), page_table=table, sf_k=sf[0], sf_v=sf[1], lse=l1)
    add = ref.weights(q1, kp, l1, lens2, 320, None, table, True, sf[0])
    w3 = fmha.key_weights(q1, kp, l1, w2.clone(), i32(lens2), page_table=table, sf_k=sf[0])
    assert bool(((w3.double() - w2.double() - add).abs() <= 2.0 ** -12 * (w2.double() + add)).all())
    # and the cache shrinks again, in place
    keep, counts = fmha.evict_select(w3, i32(lens2), 200, 4, 16)
    before = [ref.gather(kp, table, b, 320).clone() for b in range(B)]
    fmha.cache_compact(kp, vp, keep, counts, page_table=table, weights=w3)
    for b in range(B):
        for h in range(Hkv):
            assert torch.equal(ref.gather(kp, table, b, 200)[:, h].float(), before[b][keep[b, h].long(), h].float())
    fmha.get_device_error()


def test_prompt_by_picked_masks():
    """128-token query tiles pick the block mask that the prefill kernel takes."""
    from precision_attention_fmha_b200 import fmha

    B, S, Hq, Hkv, D = 1, 1000, 4, 2, 128
    q, k, v, _, g = make(7, B, S, Hq, Hkv, D, S)
    lens = i32([S])
    bounds = fmha.key_bounds(k, lens, 128)
    mask = fmha.select_blocks(q, bounds, lens, 128, 3, 1, 1, q_tile=128)
    lse = torch.empty(B, Hq, S, device=DEV)
    o = fmha.fmha_fwd_block_sparse(q, k, v, mask, causal=True, lse=lse)
    fmha.get_device_error()
    sees = mask.bool().repeat_interleave(128, 2)[:, :, :S].repeat_interleave(128, 3)[..., :S] & torch.ones(S, S, device=DEV).tril().bool()
    for h in (0, 3):
        rows = torch.arange(0, S, 37, device=DEV)
        want = ref.attend(q[0, rows, h].double(), k[0, :, h // 2].double(), v[0, :, h // 2].double(), sees[0, h // 2][rows], 1 / math.sqrt(D))
        assert bool(((o[0, rows, h].double() - want[0]).abs() < 1e-2).all())  # the prefill kernel's stated tolerance
    assert int(mask[0, 0].sum(-1).max()) == 3


def test_other_device_is_made_current():
    from precision_attention_fmha_b200 import fmha

    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    q, k, v, _, g = make(9, 1, 2, 4, 2, 64, 50)
    want = fmha.fmha_fwd_tree(q, k, v, i32([30]))
    at = [x.to("cuda:1") for x in (q, k, v, i32([30]))]
    assert torch.equal(fmha.fmha_fwd_tree(*at).cpu(), want.cpu())


def test_wait_that_runs_out_is_reported():
    """With a limit of one cycle device waits give up: the call returns, reports it, and later calls are whole. The cache
    is long enough that every CTA's ring fills, so some wait has to run out."""
    from precision_attention_fmha_b200 import fmha

    n = 60000
    q, k, v, _, g = make(10, 2, 4, 8, 2, 128, n)
    lens, lse = i32([n - 4, n - 9]), torch.zeros(2, 8, 4, device=DEV)
    wide = torch.randn(2, 200, 8, 128, generator=g, device=DEV).bfloat16()
    want = fmha.fmha_fwd_tree(q, k, v, lens)
    fmha.get_device_error()
    for f in (lambda: fmha.fmha_fwd_tree(q, k, v, lens),
              lambda: fmha.fmha_fwd_tree(wide, k, v, i32([n - 300, n - 500])),
              lambda: fmha.key_weights(q, k, lse, torch.zeros(2, 2, n, device=DEV), lens),
              lambda: fmha.key_weights(wide, k, torch.zeros(2, 8, 200, device=DEV), torch.zeros(2, 2, n, device=DEV), lens)):
        fmha.set_wait_timeout_cycles(1)
        try:
            f()
            with pytest.raises(fmha.FmhaError) as e:
                fmha.get_device_error()
        finally:
            fmha.set_wait_timeout_cycles(0)
        assert e.value.status == fmha.FMHA_ERR_TIMEOUT
    assert torch.equal(fmha.fmha_fwd_tree(q, k, v, lens), want)
    fmha.get_device_error()


@pytest.mark.parametrize("cycles", [1, 300, 1000, 3000, 10000, 100000])
def test_weights_whose_waits_run_out_in_any_turn(cycles):
    """A prompt's weights take each CTA through many turns: whichever turn's wait runs out, first or later, all warps leave
    after the same one; the call returns, says so if a wait ran out, and the next call is whole."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, n = 2, 1500, 8, 2, 64, 4000
    q, k, v, _, g = make(12, B, T, Hq, Hkv, D, n)
    lens, lse = i32([n, n - 9]), torch.full((B, Hq, T), 8.0, device=DEV)
    want = fmha.key_weights(q, k, lse, torch.zeros(B, Hkv, n, device=DEV), lens)
    fmha.get_device_error()
    for _ in range(5):
        fmha.set_wait_timeout_cycles(cycles)
        try:
            fmha.key_weights(q, k, lse, torch.zeros(B, Hkv, n, device=DEV), lens)
            torch.cuda.synchronize()
        finally:
            fmha.set_wait_timeout_cycles(0)
        try:
            fmha.get_device_error()
        except fmha.FmhaError as e:
            assert e.status == fmha.FMHA_ERR_TIMEOUT
        assert torch.equal(fmha.key_weights(q, k, lse, torch.zeros(B, Hkv, n, device=DEV), lens), want)
    fmha.get_device_error()
