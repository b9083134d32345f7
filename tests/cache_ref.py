"""Plain 64-bit forms of the operators over a ragged cache, one (sequence, head) at a time, and their tolerances.

Tolerances, derived before any run. O is rounded once to BF16 (half a step: 2^-9 of a value's binade, at most
2^-8 / 2 = 2^-9 relative to the binade's top, 2^-8 of the value at its foot) after a sum whose weights were rounded
to the value type's 16 bits. With V of unit scale and weights p_j / l that sum to 1, each weight off by at most
eps/2 relative (BF16: 2^-8, F16: 2^-11) moves O by at most eps/2 * sum_j p_j |v_j| / l, so

    |O - O_ref| <= 2^-8 |O_ref| + eps_p/2 * A + 2^-16 A,   A = softmax(|v|) = sum_j p_j |v_j| / l,

where the last term covers the 32-bit arithmetic: scores are sums of D <= 128 exact products, off by at most
D * 2^-24 * sum_d |q_d k_d| * scale, which for the inputs here (|q.k| sums under 2^8, scale >= 2^-4) is under 2^-13
in the exponent per key and far less on average, and ex2 is off by 2^-22; a worst-case bound of 2^-13 would be
looser than needed, and 2^-12 * A is allowed to stay safe. The log-sum-exp is a 32-bit number of size under 2^6
whose score errors are as above: 2^-13 + 2^-18 * |lse|.
"""

import math

import torch

LSE_ATOL = 2.0 ** -13


def gather(x, table, b, n):
    """Rows 0..n-1 of sequence b: [n, H, D]."""
    if table is None:
        return x[b, :n]
    page = x.shape[1]
    s = torch.arange(n, device=x.device)
    return x[table[b].long()[s // page], s % page]


def scale_of(sf, b, h):
    if sf is None:
        return 1.0
    return float(sf.tensor.reshape(-1)[0]) if sf.kind == "per_tensor" else float(sf.tensor[b, h])


def attend(q, k, v, sees, scale):
    """q [R, D], k / v [N, D], sees bool [R, N], all 64 bits. O, lse and A (see above); hidden keys never enter."""
    R, D = q.shape
    o, a = torch.zeros(R, v.shape[1], dtype=torch.float64, device=q.device), torch.zeros(R, v.shape[1], dtype=torch.float64, device=q.device)
    lse = torch.full((R,), -math.inf, dtype=torch.float64, device=q.device)
    for r in range(R):
        at = sees[r].nonzero()[:, 0]
        if at.numel() == 0:
            continue
        z = (k[at] @ q[r]) * scale
        lse[r] = torch.logsumexp(z, 0)
        w = torch.exp(z - lse[r])
        o[r] = w @ v[at]
        a[r] = w @ v[at].abs()
    return o, lse, a


def tree(q, k, v, ctx, mask, nodes, table=None, sf_k=None, sf_v=None, scale=None):
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale = scale or 1 / math.sqrt(D)
    o = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        c = int(ctx[b])
        m = T if nodes is None else int(nodes[b])
        kk, vv = gather(k, table, b, c + m).double(), gather(v, table, b, c + m).double()
        tm = torch.ones(T, T, device=q.device).tril() if mask is None else mask[b if mask.shape[0] > 1 else 0]
        sees = torch.ones(m, c + m, dtype=torch.bool, device=q.device)
        sees[:, c:] = tm[:m, :m] != 0
        for h in range(Hq):
            g = h // G
            o[b, :m, h], lse[b, h, :m], a[b, :m, h] = attend(
                q[b, :m, h].double(), kk[:, g] * scale_of(sf_k, b, g), vv[:, g] * scale_of(sf_v, b, g), sees, scale)
    return o, lse, a


def selected(q, k, v, blocks, lens, block, q_lens=None, table=None, sf_k=None, sf_v=None, scale=None):
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale = scale or 1 / math.sqrt(D)
    o = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(lens[b])
        m = T if q_lens is None else int(q_lens[b])
        kk, vv = gather(k, table, b, n).double(), gather(v, table, b, n).double()
        for t in range(m):
            at = n - m + t
            for g in range(Hkv):
                keys = [s for i in blocks[b, t, g].tolist() if i >= 0 for s in range(i * block, min((i + 1) * block, at + 1))]
                if not keys:
                    continue
                hs = slice(g * G, g * G + G)
                x = kk[keys, g] * scale_of(sf_k, b, g)
                y = vv[keys, g] * scale_of(sf_v, b, g)
                o[b, t, hs], lse[b, hs, t], a[b, t, hs] = attend(
                    q[b, t, hs].double(), x, y, torch.ones(G, len(keys), dtype=torch.bool, device=q.device), scale)
    return o, lse, a


def check(o, lse, ref, v8=False):
    ro, rl, ra = ref
    tol = ro.abs() * 2.0 ** -8 + ra * (2.0 ** -11 if v8 else 2.0 ** -8) + ra * 2.0 ** -12 + 1e-30
    err = (o.double() - ro).abs()
    assert torch.isfinite(o).all(), "non-finite output"
    assert bool((err <= tol).all()), f"O off by {float((err - tol).max()):.3g} more than allowed (max error {float(err.max()):.3g})"
    if lse is not None:
        dead = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse) & (lse < 0), dead), "lse: -inf in other rows"
        off = (lse.double() - rl).abs()[~dead]
        lim = (LSE_ATOL + rl.abs() * 2.0 ** -18)[~dead]
        assert bool((off <= lim).all()), f"lse off by {float(off.max()):.3g}"


def bounds(k, lens, block, before, table=None):
    """The bounds buffer after the call; `before` is what it held."""
    out = before.double().clone()
    for b in range(out.shape[0]):
        kk = gather(k, table, b, int(lens[b])).double()
        for j in range(-(-int(lens[b]) // block)):
            part = kk[j * block: (j + 1) * block]
            out[b, :, j, 0], out[b, :, j, 1] = part.amin(0), part.amax(0)
    return out


def pick(q, bnd, lens, block, top, sinks, recent, q_lens=None, q_tile=1):
    """Picked ids of each (sequence, tile, KV head), as nested lists."""
    B, T, Hq, D = q.shape
    Hkv = bnd.shape[1]
    G = Hq // Hkv
    out = []
    for b in range(B):
        m = T if q_lens is None else int(q_lens[b])
        rows = []
        for t0 in range(0, T, q_tile):
            t1 = min(t0 + q_tile, m)
            last = int(lens[b]) - m + t1 - 1
            seen = last // block + 1 if t1 > t0 and last >= 0 else 0
            heads = []
            for h in range(Hkv):
                x = q[b, t0:t1, h * G:(h + 1) * G].double().reshape(-1, D)
                lo, hi = bnd[b, h, :seen, 0].double(), bnd[b, h, :seen, 1].double()
                score = torch.maximum(x[:, None] * lo, x[:, None] * hi).sum((0, 2)).tolist() if seen else []
                order = sorted(range(seen), key=lambda j: (not (j < sinks or j >= seen - recent), 0.0 if
                                                           (j < sinks or j >= seen - recent) else -score[j], j))
                heads.append(sorted(order[:top]))
            rows.append(heads)
        out.append(rows)
    return out


def weights(q, k, lse, lens, n, q_lens=None, table=None, causal=True, sf_k=None, scale=None):
    """Gathered weights [B, Hkv, n] in 64 bits."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale = scale or 1 / math.sqrt(D)
    out = torch.zeros(B, Hkv, n, dtype=torch.float64, device=q.device)
    for b in range(B):
        m = T if q_lens is None else int(q_lens[b])
        s = int(lens[b])
        kk = gather(k, table, b, s).double()
        at = s - m + torch.arange(m, device=q.device)
        sees = (torch.arange(s, device=q.device) <= at[:, None]) if causal else torch.ones(m, s, dtype=torch.bool, device=q.device)
        for h in range(Hq):
            z = (q[b, :m, h].double() @ (kk[:, h // G] * scale_of(sf_k, b, h // G)).t()) * scale - lse[b, h, :m].double()[:, None]
            out[b, h // G, :s] += torch.where(sees, z.exp(), torch.zeros_like(z)).sum(0)
    return out


def kept(w, lens, budget, sinks, recent):
    """Kept positions of each (sequence, KV head), as nested lists."""
    out = []
    for b in range(w.shape[0]):
        n = int(lens[b])
        heads = []
        for h in range(w.shape[1]):
            if n <= budget:
                heads.append(list(range(n)))
                continue
            x = w[b, h, :n].tolist()
            rest = sorted(range(sinks, n - recent), key=lambda s: (x[s] != x[s], -x[s] if x[s] == x[s] else 0.0, s))
            heads.append(sorted(list(range(sinks)) + list(range(n - recent, n)) + rest[: budget - sinks - recent]))
        out.append(heads)
    return out
