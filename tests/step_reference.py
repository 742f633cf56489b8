"""Plain 64-bit forms of the packed-step operators (plan, rotary positions, cache write, tree
attention), for the tests; written from the definitions in include/mla_step.h."""
import math

import torch

PAGE = 64


def ancestors(parents):
    """[n, n] truth values: token j is token i or an ancestor of it (parents of one request)."""
    n = len(parents)
    seen = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = parents[j]
    return seen


def pack(seen, max_nodes):
    """Truth values [n, m] as int32 words [n, ceil(max_nodes / 32)]."""
    words = (max_nodes + 31) // 32
    out = torch.zeros(seen.shape[0], words, dtype=torch.int32)
    for i, j in seen.nonzero().tolist():
        v = int(out[i, j // 32]) | (1 << (j % 32))
        out[i, j // 32] = v - (1 << 32) if v >= 1 << 31 else v
    return out


def plan(cached, new, free_pages, head, table, num_tokens, parents=None, max_nodes=0):
    """The plan by loops, for lengths that fit; table is changed in place."""
    seq_lens, cu, ids, pos, slots = [], [0], [], [], []
    words = (max_nodes + 31) // 32
    masks = torch.zeros(num_tokens, words, dtype=torch.int32)
    for b, (c, n) in enumerate(zip(cached, new)):
        seq_lens.append(c + n)
        for p in range((c + PAGE - 1) // PAGE, (c + n + PAGE - 1) // PAGE):
            table[b, p] = free_pages[head]
            head += 1
        par = None if parents is None else parents[cu[-1]:cu[-1] + n]
        if par is not None and n:
            seen = ancestors(par)
            masks[cu[-1]:cu[-1] + n] = pack(seen, max_nodes)
        for i in range(n):
            ids.append(b)
            pos.append(c + (i if par is None else int(seen[i].sum()) - 1))
            slots.append(int(table[b, (c + i) // PAGE]) * PAGE + (c + i) % PAGE)
        cu.append(cu[-1] + n)
    pad = [-1] * (num_tokens - len(ids))
    return dict(seq_lens=seq_lens, cu_tokens=cu, seq_ids=ids + pad, positions=pos + pad, slots=slots + pad,
                free_head=[head], masks=masks)


def rotary(x, positions, inv_freq, mscale, layout, offset, inverse=False):
    """(value, bound): x [T, heads, width] turned in fp64, and what an fp32 rotation with cosines
    and sines within 2^-22 may be off before the last rounding."""
    y = x.double().clone()
    rot = 2 * inv_freq.numel()
    a = positions.double()[:, None, None] * inv_freq
    c, s = a.cos() * mscale, a.sin() * mscale * (-1.0 if inverse else 1.0)
    r = y[..., offset:offset + rot]
    x0, x1 = (r[..., :rot // 2], r[..., rot // 2:]) if layout == "half" else (r[..., 0::2], r[..., 1::2])
    x0, x1 = x0.clone(), x1.clone()
    y0, y1 = x0 * c - x1 * s, x0 * s + x1 * c
    size = x0.abs() + x1.abs()
    bound = torch.zeros_like(y)
    for dst, u, v in ((y, y0, y1), (bound, size, size)):
        d = dst[..., offset:offset + rot]
        if layout == "half":
            d[..., :rot // 2], d[..., rot // 2:] = u, v
        else:
            d[..., 0::2], d[..., 1::2] = u, v
    # 2^-22 for each cosine and sine (a series in fp32 of an argument rounded to fp32: a few
    # units of 2^-24), 2^-24 for each of two products, the sum and the factor mscale
    return y, bound * abs(mscale) * 2.0 ** -21


def tree_attention(q, c, k, scale, seen):
    """One sequence in fp64: q [n, H, dc + dr], cache rows c [L, dc], k [L, dr], seen [n, L] truth
    values. Returns (o [n, H, dc], lse [n, H], weight-magnitude A = sum p |c|, score size).
    What a row does not see takes no part, whatever it holds."""
    n, H, D = q.shape
    dc = c.shape[1]
    o = torch.zeros(n, H, dc, dtype=torch.float64, device=q.device)
    A = torch.zeros_like(o)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(lse)
    for i in range(n):
        idx = seen[i].nonzero()[:, 0].to(q.device)
        if idx.numel() == 0:
            continue
        kv = torch.cat([c[idx], k[idx]], -1).double()
        s = q[i].double() @ kv.T * scale
        size[i] = (q[i].double().abs() @ kv.abs().T * scale).amax(-1)
        lse[i] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[i][:, None])
        o[i] = p @ c[idx].double()
        A[i] = p @ c[idx].double().abs()
    return o, lse, A, size


def check_tree(o, lse, ref, tokens):
    """Bounds of the kernels' arithmetic, per element. A score is an fp32 sum of exact products,
    at most D 2^-22 of the sum of their magnitudes off (D = 576 at most; twice the unit of each
    of D truncating additions), so a weight is off by twice that relatively (numerator and sum);
    a weight is rounded to bf16 (2^-8) and the result once more (2^-8 of the value); the
    exponentials, the sum of the weights and the merge are fp32 (2^-16 covers 2^8 units)."""
    ro, rl, A, size = ref
    ds = 576 * 2.0 ** -22 * size
    bound = (2.0 ** -8 + 2.0 ** -16 + 2 * ds[..., None]) * A + 2.0 ** -8 * ro.abs() + 1e-30
    o, lse = o.double(), lse.double()
    assert torch.isfinite(o).all()
    worst = ((o - ro).abs() / bound).max()
    assert worst <= 1, f"o: {worst:.3f} of the bound"
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (o[empty] == 0).all()
    # the logarithm of an fp32 sum of up to `tokens` terms (2^-24 each), a product and a sum in fp32
    lb = ds + tokens * 2.0 ** -24 + 2.0 ** -20 * (1 + rl.abs())
    off = ((lse - rl).abs() / lb)[~empty]
    assert off.numel() == 0 or off.max() <= 1, f"lse: {off.max():.3f} of the bound"
