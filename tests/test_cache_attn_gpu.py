"""Attention over a ragged cache (tree of drafted tokens, picked blocks) against its 64-bit form."""

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make(seed, B, T, Hq, Hkv, D, S, page=0, kv="bf16"):
    """q, k, v, table and scales: caches with room for S tokens; slots past a sequence's end hold NaN."""
    from precision_attention_fmha_b200 import fmha

    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q = torch.randn(B, T, Hq, D, generator=g, device=DEV).bfloat16()
    rows = S if page == 0 else -(-S // page) * page
    shape = (B, rows, Hkv, D)
    k, v = torch.randn(shape, generator=g, device=DEV), torch.randn(shape, generator=g, device=DEV)
    sf = None
    kt = vt = torch.bfloat16
    if kv != "bf16":
        vt = torch.float8_e4m3fn
        kt = vt if kv == "e4m3" else kt
        sf = (fmha.Scale(torch.full((1,), 1 / 32, device=DEV), "per_tensor") if kv == "e4m3" else None,
              fmha.Scale(torch.rand(B, Hkv, generator=g, device=DEV) * 0.05 + 0.01, "per_head"))
        k, v = k * (32 if kv == "e4m3" else 1), v * 32
    k, v = k.to(kt), v.to(vt)
    return q, k, v, sf or (None, None), g


def poison(x, lens):
    """NaN in the rows of [B, S, H, D] past each sequence's length."""
    nan = torch.full((1,), float("nan"), device=DEV).to(x.dtype)
    for b, n in enumerate(lens):
        x[b, n:] = nan
    return x


def to_pages(k, v, page, g, extra=3):
    """Contiguous rows -> pools in shuffled pages (the extra pages hold NaN) and the page table."""
    B, S, H, D = k.shape
    per = S // page
    perm = torch.randperm(B * per + extra, generator=g, device=DEV)[: B * per].view(B, per)
    out = []
    for x in (k, v):
        pool = torch.full((B * per + extra, page, H, D), float("nan"), device=DEV).to(x.dtype)
        pool[perm.reshape(-1)] = x.reshape(B * per, page, H, D)
        out.append(pool)
    return out[0], out[1], perm.to(torch.int32)


def random_tree(B, T, g):
    """Every node sees itself and its ancestors; one row of each tree sees nothing of the tree."""
    m = torch.zeros(B, T, T, dtype=torch.uint8, device=DEV)
    r = torch.rand(B, T, generator=g, device=DEV).tolist()
    for b in range(B):
        for i in range(T):
            m[b, i, i] = 1
            if i:
                p = int(r[b][i] * i)
                m[b, i] |= m[b, p]
    m[:, T - 1] = 0
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


TREES = [
    # B, T, Hq, Hkv, D, ctx, page, kv
    (1, 1, 1, 1, 64, [0], 0, "bf16"),
    (1, 1, 8, 8, 128, [1], 16, "bf16"),
    (2, 3, 4, 2, 64, [63, 64], 0, "bf16"),
    (3, 8, 8, 2, 128, [65, 0, 700], 64, "bf16"),
    (2, 5, 12, 4, 128, [127, 300], 32, "bf16"),    # 3 heads a group
    (2, 17, 14, 2, 64, [129, 1000], 16, "bf16"),   # 7 heads a group, 119 rows
    (1, 33, 64, 8, 128, [515], 128, "bf16"),
    (4, 1, 32, 8, 128, [1, 4095, 33, 1024], 64, "bf16"),
    (3, 8, 8, 2, 128, [65, 0, 700], 64, "e4m3"),
    (2, 17, 8, 2, 64, [129, 1000], 16, "e4m3"),
    (2, 1, 16, 1, 128, [2047, 90], 0, "e4m3"),
    (2, 6, 8, 4, 128, [100, 200], 32, "bf16_e4m3"),
    (2, 40, 4, 2, 64, [31, 257], 0, "bf16_e4m3"),
    (24, 5, 64, 8, 128, [900 + 7 * i for i in range(24)], 64, "bf16"),  # 40 rows on many heads
    # many rows and room: contexts on the packed tensor-memory tiles, the rest joined
    (2, 16, 64, 8, 128, [1500, 100], 64, "bf16"),
    (3, 17, 64, 8, 128, [1023, 1024, 0], 16, "bf16"),  # 136 rows
    (1, 40, 32, 4, 128, [2049], 0, "bf16"),            # 320 rows: three 128-row tiles
    (2, 140, 4, 4, 128, [1279, 1408], 128, "bf16"),    # one head a group
    (1, 3, 128, 2, 128, [3000], 32, "bf16"),           # 64 heads a group
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,ctx,page,kv", TREES)
@pytest.mark.parametrize("masked", [False, True])
def test_tree(B, T, Hq, Hkv, D, ctx, page, kv, masked):
    from precision_attention_fmha_b200 import fmha

    S = max(ctx) + T + 5
    q, k, v, sf, g = make(T * 1000 + B, B, T, Hq, Hkv, D, S, page, kv)
    nodes = i32([max(0, T - b) for b in range(B)]) if masked else None
    ends = [c + (T if nodes is None else int(nodes[b])) for b, c in enumerate(ctx)]
    poison(k, ends), poison(v, ends)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    mask = random_tree(B, T, g) if masked else None
    if nodes is not None:  # the padding rows of q hold NaN
        for b in range(B):
            q[b, int(nodes[b]):] = float("nan")
    lse = torch.full((B, Hq, T), 7.0, device=DEV)
    o = fmha.fmha_fwd_tree(q, k, v, i32(ctx), mask, nodes, table, sf_k=sf[0], sf_v=sf[1], lse=lse)
    fmha.get_device_error()
    ref.check(o, lse, ref.tree(q, k, v, ctx, mask, nodes, table, *sf), v8=kv != "bf16")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_tree_hidden_nodes_may_hold_anything(kv):
    """A node that a row does not see holds NaN and infinities in K and V: the row's result is that of finite ones."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hq, Hkv, D, ctx = 1, 20, 4, 2, 128, [77]
    q, k, v, sf, g = make(5, B, T, Hq, Hkv, D, 128, 0, kv)
    mask = torch.eye(T, device=DEV, dtype=torch.uint8)[None].contiguous()
    mask[0, :, 0] = 1
    bad = [3, 9, 16]
    nan = torch.full((1,), float("nan"), device=DEV).to(k.dtype)
    for i, n in enumerate(bad):
        mask[0, :, n] = 0
        k[0, ctx[0] + n] = nan
        v[0, ctx[0] + n, :, i::5] = nan
        if kv == "bf16":
            v[0, ctx[0] + n, :, i + 1::7] = float("inf")
    lse = torch.empty(B, Hq, T, device=DEV)
    o = fmha.fmha_fwd_tree(q, k, v, i32(ctx), mask, lse=lse, sf_k=sf[0], sf_v=sf[1])
    fmha.get_device_error()
    ref.check(o, lse, ref.tree(q, k, v, ctx, mask, None, None, *sf), v8=kv != "bf16")


def test_tree_visible_nan_reaches_its_row_only():
    from precision_attention_fmha_b200 import fmha

    q, k, v, _, g = make(6, 1, 4, 2, 1, 128, 64)
    k[0, 30] = float("nan")  # node 0
    mask = torch.eye(4, device=DEV, dtype=torch.uint8)[None].contiguous()
    lse = torch.empty(1, 2, 4, device=DEV)
    o = fmha.fmha_fwd_tree(q, k, v, i32([30]), mask, lse=lse)
    assert torch.isnan(o[0, 0]).all() and torch.isnan(lse[0, :, 0]).all()
    assert torch.isfinite(o[0, 1:]).all() and torch.isfinite(lse[0, :, 1:]).all()


SELECTS = [
    # B, T, Hq, Hkv, D, lens, block, top, page, kv
    (1, 1, 1, 1, 64, [1], 16, 1, 0, "bf16"),
    (1, 1, 8, 2, 128, [700], 64, 4, 64, "bf16"),
    (2, 3, 4, 2, 64, [130, 301], 16, 7, 32, "bf16"),
    (2, 2, 24, 2, 128, [1000, 70], 32, 5, 16, "bf16"),  # 12 heads a group
    (1, 2, 40, 2, 128, [555], 128, 3, 64, "bf16"),      # 20 heads a group
    (1, 1, 80, 1, 64, [300], 64, 3, 128, "bf16"),       # 80 heads a group: two row tiles
    (3, 1, 32, 8, 128, [4000, 64, 65], 64, 16, 64, "bf16"),
    (2, 3, 8, 2, 128, [1000, 70], 32, 6, 64, "e4m3"),
    (2, 1, 8, 2, 64, [1000, 70], 16, 9, 0, "e4m3"),
    (2, 1, 8, 2, 128, [900, 10], 64, 4, 32, "bf16_e4m3"),
    (40, 4, 8, 8, 64, [100 + 7 * i for i in range(40)], 16, 3, 0, "bf16"),  # more items than CTAs
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,block,top,page,kv", SELECTS)
def test_selected(B, T, Hq, Hkv, D, lens, block, top, page, kv):
    from precision_attention_fmha_b200 import fmha

    q, k, v, sf, g = make(B * 100 + top, B, T, Hq, Hkv, D, max(lens) + 3, page, kv)
    poison(k, lens), poison(v, lens)
    table = None
    if page:
        k, v, table = to_pages(k, v, page, g)
    q_lens = i32([max(0, min(T, n) - b % 2) for b, n in enumerate(lens)])
    blocks = torch.full((B, T, Hkv, top), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        nb = -(-lens[b] // block)
        for t in range(T):
            for h in range(Hkv):
                some = torch.randperm(nb, generator=g, device=DEV)[: top - (t + h) % 2].to(torch.int32)
                blocks[b, t, h, : some.numel()] = some
    if top > 2:
        blocks[0, 0, 0, 1] = -1  # a gap
    lse = torch.full((B, Hq, T), 7.0, device=DEV)
    o = fmha.fmha_fwd_selected(q, k, v, blocks, i32(lens), block, q_lens, table, sf_k=sf[0], sf_v=sf[1], lse=lse)
    fmha.get_device_error()
    ref.check(o, lse, ref.selected(q, k, v, blocks, lens, block, q_lens, table, *sf), v8=kv != "bf16")


def test_tree_e4m3_visible_nan_codes_reach_their_rows():
    """NaN codes of K and V that a row sees make it NaN (V: that column); rows that do not see them are untouched."""
    from precision_attention_fmha_b200 import fmha

    q, k, v, sf, g = make(8, 1, 4, 4, 2, 128, 64, 0, "e4m3")
    nan = torch.full((1,), float("nan"), device=DEV).to(k.dtype)
    k[0, 30, 0] = nan       # node 0, KV head 0
    v[0, 31, 1, 5] = nan    # node 1, KV head 1, one column
    mask = torch.eye(4, device=DEV, dtype=torch.uint8)[None].contiguous()
    lse = torch.empty(1, 4, 4, device=DEV)
    o = fmha.fmha_fwd_tree(q, k, v, i32([30]), mask, lse=lse, sf_k=sf[0], sf_v=sf[1])
    assert torch.isnan(o[0, 0, :2]).all() and torch.isnan(lse[0, :2, 0]).all()
    assert torch.isnan(o[0, 1, 2:, 5]).all()
    o[0, 0, :2], o[0, 1, 2:, 5] = 0, 0
    lse[0, :2, 0] = 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("T", [1, 9])  # 2 and 18 rows: both arrangements of the few-row kernel
def test_zero_scale(T):
    """A KV head whose key scale is zero: every key in sight weighs the same, also beside keys that are not."""
    from precision_attention_fmha_b200 import fmha

    q, k, v, (_, sv), g = make(21, 2, T, 4, 2, 64, 200, 0, "e4m3")
    sk = fmha.Scale(torch.tensor([[0.0, 0.03], [0.02, 0.0]], device=DEV), "per_head")
    ctx = [70, 130]
    lse = torch.empty(2, 4, T, device=DEV)
    o = fmha.fmha_fwd_tree(q, k, v, i32(ctx), sf_k=sk, sf_v=sv, lse=lse)
    ref.check(o, lse, ref.tree(q, k, v, ctx, None, None, None, sk, sv), v8=True)
    lens = [c + T for c in ctx]
    ids = torch.tensor([0, 3, 2, 7], dtype=torch.int32, device=DEV).expand(2, T, 2, 4).contiguous()
    o = fmha.fmha_fwd_selected(q, k, v, ids, i32(lens), 16, sf_k=sk, sf_v=sv, lse=lse)
    ref.check(o, lse, ref.selected(q, k, v, ids, lens, 16, None, None, sk, sv), v8=True)


@pytest.mark.parametrize("Hq,kv", [(4, "bf16"), (40, "bf16"), (4, "e4m3")])
def test_selected_with_tiles_that_hold_no_block(Hq, kv):
    """Lists with gaps of whole 64-key tiles between their blocks: an empty tile is full at once, and must hide its slot."""
    from precision_attention_fmha_b200 import fmha

    B, T, Hkv, D, lens, block, top = 3, 4, 2, 64, [3000, 64, 1501], 64, 40
    q, k, v, sf, g = make(31, B, T, Hq, Hkv, D, max(lens) + 3, 0, kv)
    poison(k, lens), poison(v, lens)
    blocks = torch.full((B, T, Hkv, top), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        nb = -(-lens[b] // block)
        for t in range(T):
            for h in range(Hkv):
                n = min(nb, (5 * t + 3 * h + b) % 18)
                at = torch.randperm(top, generator=g, device=DEV)[:n]
                blocks[b, t, h, at] = torch.randperm(nb, generator=g, device=DEV)[:n].to(torch.int32)
    lse = torch.empty(B, Hq, T, device=DEV)
    o = fmha.fmha_fwd_selected(q, k, v, blocks, i32(lens), block, sf_k=sf[0], sf_v=sf[1], lse=lse)
    fmha.get_device_error()
    ref.check(o, lse, ref.selected(q, k, v, blocks, lens, block, None, None, *sf), v8=kv != "bf16")
    for _ in range(50):
        assert torch.equal(fmha.fmha_fwd_selected(q, k, v, blocks, i32(lens), block, sf_k=sf[0], sf_v=sf[1]), o)
