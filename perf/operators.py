"""The operators of a speculative-decoding step over the paged latent cache, as workloads.

A step plans its pages and slots from the request lengths (``plan``), rotates the new
queries (``rotary``), writes the new tokens into the cache (``append``) and attends from
every drafted node to the cache through the draft tree (``tree``). ``run`` is one pass
through one of them: in elementary torch operations, or through the package's calls.
"""
import math

import torch

own = False

PAGE = 64


def listed():
    return [
        # One request, one small draft, a 16-head shard: latency is all that counts.
        dict(name="tree one request", op="tree", cache="bf16", dc=512, heads=16, batch=1, nodes=8, length=320,
             ragged=False, chain=False),
        # The 128-head decode configuration (16 sequences of 4096 tokens) with a draft of 8 nodes each.
        dict(name="tree 16x4096", op="tree", cache="bf16", dc=512, heads=128, batch=16, nodes=8, length=4096,
             ragged=False, chain=False),
        # Long contexts, 32 nodes each: tensor-core bound.
        dict(name="tree 4x65536", op="tree", cache="bf16", dc=512, heads=128, batch=4, nodes=32, length=65536,
             ragged=False, chain=False),
        # A mixed batch: lengths from 1/32 of the longest up, 1 to 12 nodes per request.
        dict(name="tree ragged", op="tree", cache="bf16", dc=512, heads=128, batch=32, nodes=12, length=32768,
             ragged=True, chain=False),
        # The retrofitted model (32 heads, d_c 64), a chain of 5 drafted tokens, 32 x 8192.
        dict(name="tree retrofit chain", op="tree", cache="bf16", dc=64, heads=32, batch=32, nodes=5, length=8192,
             ragged=False, chain=True),
        # The E4M3 cache: 16 sequences of about 4096 tokens, up to 4 nodes.
        dict(name="tree e4m3 ragged", op="tree", cache="e4m3", dc=512, heads=128, batch=16, nodes=4, length=4096,
             ragged=True, chain=False),
        # The plan of a drafted step of 64 requests, with the tree masks.
        dict(name="plan draft", op="plan", batch=64, new=8, cached=8192, tree=True),
        # The plan of a step that mixes 1024 requests' prompt pieces.
        dict(name="plan prompts", op="plan", batch=1024, new=512, cached=16384, tree=False),
        # The rotary part of a drafted step's queries: 128 tokens, 128 heads.
        dict(name="rotary step", op="rotary", tokens=128, heads=128, width=64, offset=0, rot=64, layout="interleaved",
             scaling="yarn", dtype="bfloat16"),
        # A prompt's queries, rotated in the last third of 192-wide heads, half layout.
        dict(name="rotary prompt", op="rotary", tokens=16384, heads=128, width=192, offset=128, rot=64, layout="half",
             scaling="yarn", dtype="bfloat16"),
        # A drafted step's cache write.
        dict(name="append step", op="append", cache="bf16", dc=512, tokens=128, layout="interleaved"),
        # Eight prompts of 4096 tokens written to the E4M3 cache.
        dict(name="append prompts e4m3", op="append", cache="e4m3", dc=512, tokens=32768, layout="interleaved"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "plan", "rotary", "append"])
    if op == "tree":
        cache, dc = rng.choice([("bf16", 512), ("bf16", 512), ("bf16", 64), ("e4m3", 512)])
        heads = rng.choice([32, 32, 8, 128] if dc == 64 else [128, 128, 64, 16, 24])
        nodes = _log(rng, 1, 64)
        length = max(_log(rng, 64, 65536), 2 * nodes)
        batch = _log(rng, 1, 64)
        # no more rows x tokens than the largest listed case
        while batch > 1 and batch * nodes * heads * length > 4 * 32 * 128 * 65536:
            batch //= 2
        while nodes > 1 and batch * nodes * heads * length > 4 * 32 * 128 * 65536:
            nodes //= 2
        return dict(op=op, cache=cache, dc=dc, heads=heads, batch=batch, nodes=nodes, length=length,
                    ragged=rng.random() < 0.6, chain=rng.random() < 0.3)
    if op == "plan":
        tree = rng.random() < 0.5
        return dict(op=op, batch=_log(rng, 1, 1024), new=_log(rng, 1, 64 if tree else 512), cached=_log(rng, 1, 16384),
                    tree=tree)
    if op == "rotary":
        rot = rng.choice([64, 64, 8, 32, 128, 18])
        width = rot + rng.choice([0, 0, 128, 5])
        heads = rng.choice([1, 16, 24, 128])
        return dict(op=op, tokens=max(1, _log(rng, 1, 16384) * 64 // width), heads=heads, width=width,
                    offset=rng.choice([0, width - rot]), rot=rot, layout=rng.choice(["interleaved", "half"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]))
    cache, dc = rng.choice([("bf16", 512), ("bf16", 64), ("e4m3", 512)])
    return dict(op=op, cache=cache, dc=dc, tokens=_log(rng, 1, 32768), layout=rng.choice(["interleaved", "half"]))


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * std).to(dtype)


def _tables(g, lens, max_pages):
    """A permuted block table for `lens` (host list) and its number of pages."""
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    total = max(1, sum(pages))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(pages, device="cuda")
    col = torch.arange(max_pages, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = (first[:, None] + col[None]).clamp_(max=total - 1)
    return torch.where(col[None] < n[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous(), total


def _parents(g, counts, chain):
    """Parents (index within the request, -1 for a child of the context) of every drafted token."""
    n = torch.tensor(counts, device="cuda")
    i = torch.arange(int(n.sum()), device="cuda") - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    if chain:
        return (i - 1).to(torch.int32)
    u = torch.rand(i.shape, generator=g, device="cuda")
    return ((u * (i + 1)).floor().clamp_(max=i) - 1).to(torch.int32)   # uniform on -1 .. i - 1


def _ancestors(parents, counts, nodes):
    """[T, nodes] truth values: node j is node i or one of its ancestors."""
    n = torch.tensor(counts, device="cuda")
    start = torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    i = torch.arange(parents.numel(), device="cuda") - start
    seen = torch.zeros(parents.numel(), nodes, dtype=torch.bool, device="cuda")
    seen[torch.arange(parents.numel(), device="cuda"), i] = True
    jump = parents.long()
    while True:   # one doubling of the reach per turn
        live = jump >= 0
        at = (start + jump.clamp(min=0))
        seen = seen | (seen[at] & live[:, None])
        jump = torch.where(live, jump[at], jump)
        if not bool((jump >= 0).any()):
            return seen


def _pack(seen):
    """Truth values [T, n] as bits of int32 words [T, ceil(n / 32)]."""
    T, n = seen.shape
    w = (n + 31) // 32
    bits = torch.zeros(T, w * 32, dtype=torch.int64, device=seen.device)
    bits[:, :n] = seen
    words = (bits.view(T, w, 32) << torch.arange(32, device=seen.device)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def _frequencies(rot, scaling):
    """Plain rotary frequencies in 64 bits, and the amplitude, of a context 32 times the trained 4096."""
    theta, s, trained = 10000.0, 32.0, 4096
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        theta *= s ** (rot / max(1, rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / s
    if scaling != "yarn":
        return f, 1.0
    turns = lambda r: rot * math.log(trained / (r * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=host).tolist()  # noqa: E731
    def split(lo, hi, n):   # counts of lo .. hi whose total goes by the case alone, in the seed's order
        same = torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(n))
        return same[torch.randperm(n, generator=host)].tolist()
    s = dict(case)
    if case["op"] == "tree":
        B, H, n, L, dc = (case[k] for k in ("batch", "heads", "nodes", "length", "dc"))
        dr, dn = (64, 128) if dc == 512 else (8, 120)
        counts = split(1, n, B) if case["ragged"] else [n] * B
        lens = pick(max(n, L // 32), L, B) if case["ragged"] else [L] * B
        max_pages = (L + PAGE - 1) // PAGE
        s["block_table"], pages = _tables(g, lens, max_pages)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["cu_tokens"] = torch.cumsum(torch.tensor([0] + counts), 0).to("cuda", torch.int32)
        T = sum(counts)
        # an absorbed query: its latent part has the spread that q_c W_UK gives
        s["q"] = torch.cat([_randn(g, T, H, dc, std=math.sqrt(dn / dc)), _randn(g, T, H, dr)], -1).contiguous()
        s["masks"] = _pack(_ancestors(_parents(g, counts, case["chain"]), counts, n))
        s["kr_pool"] = _randn(g, pages, PAGE, dr)
        s["scale"] = 1.0 / math.sqrt(dn + dr)
        if case["cache"] == "e4m3":
            x = _randn(g, pages, PAGE, dc, dtype=torch.float32)
            s["scales"] = (x.abs().amax(-1) / 448.0).contiguous()
            s["ckv_pool"] = (x / s["scales"][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            s["ckv_pool"] = _randn(g, pages, PAGE, dc)
        if own:
            from mla_latent_kv_18_b200 import api
            s["dims"] = api.make_dims(H, 1, dn, dc, dr, 128, PAGE, s["scale"])
            s["workspace"] = api.alloc_tree_workspace(s["dims"], "cuda")
    elif case["op"] == "plan":
        B, new, cached = case["batch"], case["new"], case["cached"]
        counts = split(0 if B > 4 else 1, new, B)
        before = pick(0, cached, B)
        max_pages = (cached + new + PAGE - 1) // PAGE + 1
        table, pages = _tables(g, before, max_pages)
        s["block_table"] = table
        T = sum(counts)
        s["num_tokens"] = max(64, -(-T // 64) * 64)   # a captured step's fixed number of token rows
        s["cached_lens"] = torch.tensor(before, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        room = T // PAGE + B + 3
        s["free_pages"] = (pages + torch.randperm(room, generator=g, device="cuda")).to(torch.int32)
        s["free_head"] = torch.tensor([3], dtype=torch.int32, device="cuda")
        s["parents"] = None
        if case["tree"]:
            s["parents"] = torch.full((s["num_tokens"],), -1, dtype=torch.int32, device="cuda")
            s["parents"][:T] = _parents(g, counts, False)
    elif case["op"] == "rotary":
        T, H = case["tokens"], case["heads"]
        s["x"] = _randn(g, T, H, case["width"], dtype=getattr(torch, case["dtype"]))
        s["k"] = _randn(g, T, 1, case["width"], dtype=getattr(torch, case["dtype"]))
        s["positions"] = torch.randint(0, 131072, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"], s["mscale"] = _frequencies(case["rot"], case["scaling"])
        s["inv_freq"] = s["inv_freq"].cuda()
        s["out"], s["k_out"] = torch.empty_like(s["x"]), torch.empty_like(s["k"])
    else:
        T, dc = case["tokens"], case["dc"]
        dr = 64 if dc == 512 else 8
        both = _randn(g, T, dc + dr)   # the new tokens' [c_KV | k_R], one projection's output
        s["ckv_new"], s["kr_new"] = both[:, :dc], both[:, dc:]
        pages = T // PAGE + 2
        s["slots"] = torch.randperm(pages * PAGE, generator=g, device="cuda")[:T].contiguous()
        s["slots"][torch.rand(T, generator=g, device="cuda") < 0.01] = -1   # rows of a padded batch
        s["positions"] = torch.randint(0, 131072, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"], s["mscale"] = _frequencies(dr, "yarn")
        s["inv_freq"] = s["inv_freq"].cuda()
        s["kr_pool"] = torch.zeros(pages, PAGE, dr, dtype=torch.bfloat16, device="cuda")
        if case["cache"] == "e4m3":
            s["ckv_pool"] = torch.zeros(pages, PAGE, dc, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.zeros(pages, PAGE, device="cuda")
        else:
            s["ckv_pool"] = torch.zeros(pages, PAGE, dc, dtype=torch.bfloat16, device="cuda")
        if own:
            from mla_latent_kv_18_b200 import api
            s["dims"] = api.make_dims(1, 1, 128 if dc == 512 else 120, dc, dr, 128, PAGE)
    return s


# ------------------------------------------------------------------ the package's calls

def _run_own(s):
    from mla_latent_kv_18_b200 import api
    if s["op"] == "tree":
        if s["cache"] == "e4m3":
            return api.decode_tree_fp8(s["q"], s["ckv_pool"], s["scales"], s["kr_pool"], s["block_table"],
                                       s["seq_lens"], s["cu_tokens"], s["dims"], s["nodes"], masks=s["masks"],
                                       workspace=s["workspace"])
        return api.decode_tree(s["q"], s["ckv_pool"], s["kr_pool"], s["block_table"], s["seq_lens"],
                               s["cu_tokens"], s["dims"], s["nodes"], masks=s["masks"], workspace=s["workspace"])
    if s["op"] == "plan":
        p = api.step_plan(s["cached_lens"], s["new_lens"], s["free_pages"], s["free_head"], s["block_table"],
                          s["num_tokens"], parents=s["parents"], max_nodes=s["new"] if s["tree"] else 0)
        return [s["block_table"], p.seq_lens, p.cu_tokens, p.seq_ids, p.positions, p.slots, p.free_head, p.masks]
    if s["op"] == "rotary":
        return api.rotary(s["x"], s["positions"], s["inv_freq"], mscale=s["mscale"], layout=s["layout"],
                          offset=s["offset"], out=s["out"], k=s["k"], k_out=s["k_out"])
    if s["cache"] == "e4m3":
        api.append_kv_slots_fp8(s["ckv_new"], s["kr_new"], s["slots"], s["ckv_pool"], s["scales"], s["kr_pool"],
                                s["dims"], positions=s["positions"], inv_freq=s["inv_freq"], mscale=s["mscale"],
                                layout=s["layout"])
        return [s["ckv_pool"].view(torch.float8_e4m3fn), s["kr_pool"], s["scales"]]
    api.append_kv_slots(s["ckv_new"], s["kr_new"], s["slots"], s["ckv_pool"], s["kr_pool"], s["dims"],
                        positions=s["positions"], inv_freq=s["inv_freq"], mscale=s["mscale"], layout=s["layout"])
    return [s["ckv_pool"], s["kr_pool"]]


# ------------------------------------------------------------------ the plain forms

def _cache_rows(s, dtype):
    """Every sequence's cached [c_KV] and [k_R] rows, padded to the table's width: [B, Lpad, d]."""
    pages = s["block_table"].long().clamp(min=0)
    c = s["ckv_pool"][pages]
    if s["cache"] == "e4m3":   # the cached value is value(code) * scale, rounded to bf16
        c = (c.view(torch.float8_e4m3fn).float() * s["scales"][pages][..., None]).bfloat16()
    B = pages.shape[0]
    return c.to(dtype).view(B, -1, c.shape[-1]), s["kr_pool"][pages].to(dtype).view(B, c.shape[1] * PAGE, -1)


def _tree(s):
    cu, lens, n, H = s["cu_tokens"].long(), s["seq_lens"].long(), s["nodes"], s["heads"]
    c, k = _cache_rows(s, torch.float32)
    B, Lp, dc = c.shape
    count = cu[1:] - cu[:-1]
    node = torch.arange(n, device="cuda")
    at = (cu[:-1, None] + node).clamp(max=s["q"].shape[0] - 1)          # [B, n]
    q = s["q"][at].float().view(B, n * H, -1)
    score = q @ torch.cat([c, k], -1).transpose(1, 2) * s["scale"]      # [B, n H, Lp]
    j = torch.arange(Lp, device="cuda")[None] - (lens - count)[:, None]  # drafted node held by a cache row
    word = s["masks"][at].gather(2, (j.clamp(0, n - 1) // 32)[:, None].expand(B, n, Lp).long())
    bit = (word >> (j.clamp(0, n - 1) % 32)[:, None].int()) & 1
    seen = (j < 0)[:, None] | ((j < count[:, None])[:, None] & (bit == 1))
    score = score.view(B, n, H, Lp).masked_fill_(~seen[:, :, None], -math.inf).view(B, n * H, Lp)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ c / total.clamp(min=1e-38)).view(B, n, H, dc)
    lse = (top + total.log()).view(B, n, H)
    live = node[None] < count[:, None]
    return o[live].bfloat16(), lse[live]


def _plan(s):
    T, free, table = s["num_tokens"], s["free_pages"].long(), s["block_table"]
    c, n = s["cached_lens"].long(), s["new_lens"].long()
    lens = c + n
    cu = torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])
    p0 = (c + PAGE - 1) // PAGE
    fresh = (lens + PAGE - 1) // PAGE - p0
    first = s["free_head"].long() + torch.cumsum(fresh, 0) - fresh
    col = torch.arange(table.shape[1], device="cuda")[None] - p0[:, None]
    take = (col >= 0) & (col < fresh[:, None])
    table.copy_(torch.where(take, free[(first[:, None] + col).clamp(0, free.numel() - 1)].int(), table))
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = t < cu[-1]
    bb = b.clamp(max=c.numel() - 1)
    i = t - cu[bb]
    at = c[bb] + i
    page = table[bb, (at // PAGE).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live, page * PAGE + at % PAGE, torch.full_like(at, -1))
    masks, depth = None, i
    if s["parents"] is not None:
        w = (s["new"] + 31) // 32
        start = cu[bb]
        seen = torch.zeros(T, w * 32, dtype=torch.bool, device="cuda")
        seen[t[live], i[live]] = True
        jump = torch.where(live, s["parents"].long(), torch.full_like(t, -1))
        for _ in range(max(1, math.ceil(math.log2(max(2, s["new"]))))):
            alive = jump >= 0
            up = start + jump.clamp(min=0)
            up = torch.where(alive, up, t)
            seen = seen | (seen[up] & alive[:, None])
            jump = torch.where(alive, jump[up], jump)
        masks, depth = _pack(seen), seen.sum(-1) - 1
    none = torch.full_like(b, -1)
    return [table, lens.int(), cu.int(), torch.where(live, b, none).int(),
            torch.where(live, c[bb] + depth, none).int(), slots, (s["free_head"] + fresh.sum()).int(), masks]


def _turn(x, s, dtype, rot, offset):
    """x [T, heads, width] with channels offset .. offset + rot turned, in `dtype`."""
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["mscale"]).to(dtype), (angle.sin() * s["mscale"]).to(dtype)
    r = x[..., offset:offset + rot].to(dtype)
    y = x.to(dtype).clone()
    if s["layout"] == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y[..., offset:offset + rot] = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        y[..., offset:offset + rot] = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return y


def _rotary(s):
    return [_turn(s[k], s, torch.float32, s["rot"], s["offset"]).to(s[k].dtype) for k in ("x", "k")]


def _append(s):
    live = s["slots"] >= 0
    at = s["slots"][live]
    dr = s["kr_new"].shape[1]
    k = _turn(s["kr_new"][:, None], s, torch.float32, dr, 0)[:, 0].bfloat16()
    s["kr_pool"].view(-1, dr)[at] = k[live]
    c = s["ckv_new"][live]
    if s["cache"] == "bf16":
        s["ckv_pool"].view(-1, c.shape[1])[at] = c
        return [s["ckv_pool"], s["kr_pool"]]
    x = c.float()
    top = x.abs().amax(-1, keepdim=True)
    codes = (x * (448.0 / top)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    s["ckv_pool"].view(-1, c.shape[1])[at] = codes.view(torch.uint8)
    s["scales"].view(-1)[at] = (top / 448.0)[:, 0]
    return [s["ckv_pool"].view(torch.float8_e4m3fn), s["kr_pool"], s["scales"]]


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree, "plan": _plan, "rotary": _rotary, "append": _append}[state["op"]](state)


def work(case):
    if case["op"] == "tree":
        B, H, n, L, dc = (case[k] for k in ("batch", "heads", "nodes", "length", "dc"))
        dr = 64 if dc == 512 else 8
        if case["ragged"]:   # means of the drawn lengths and node counts
            n, L = (n + 1) / 2, (max(n, L // 32) + L) / 2
        rows = B * n * H
        token = dc * 2 if case["cache"] == "bf16" else dc + 4
        return {"bytes": B * L * (token + dr * 2) + rows * ((dc + dr) * 2 + dc * 2 + 4),
                "flops": rows * (L - n / 2) * 2 * (2 * dc + dr)}
    if case["op"] == "plan":
        B, T = case["batch"], case["batch"] * case["new"] / 2
        words = (case["new"] + 31) // 32 if case["tree"] else 0
        return {"bytes": B * 16 + (T / PAGE + B) * 8 + T * (16 + (4 * words + 4 if case["tree"] else 0)), "flops": 0}
    if case["op"] == "rotary":
        size = 4 if case["dtype"] == "float32" else 2
        n = case["tokens"] * (case["heads"] + 1)
        return {"bytes": 2 * n * case["width"] * size + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    dc = case["dc"]
    dr = 64 if dc == 512 else 8
    written = dc * 2 if case["cache"] == "bf16" else dc + 4
    return {"bytes": case["tokens"] * (dc * 2 + written + 4 * dr + 12), "flops": 3 * case["tokens"] * dr}


# ------------------------------------------------------------------ the definitions in 64 bits

def _turn64(x, s, rot, offset):
    """The rotation as a complex product, in 64 bits."""
    y = x.double()
    phase = torch.polar(torch.full_like(s["inv_freq"], s["mscale"]).expand(x.shape[0], -1),
                        s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    r = y[..., offset:offset + rot]
    if s["layout"] == "half":
        z = torch.complex(r[..., :rot // 2].contiguous(), r[..., rot // 2:].contiguous()) * phase
        t = torch.cat([z.real, z.imag], -1)
    else:
        t = torch.view_as_real(torch.view_as_complex(r.contiguous().unflatten(-1, (-1, 2))) * phase).flatten(-2)
    return torch.cat([y[..., :offset], t, y[..., offset + rot:]], -1)


def exact(case, seed):
    if case["op"] == "plan":
        return None   # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return [_turn64(s[k], s, s["rot"], s["offset"]) for k in ("x", "k")]
    if case["op"] == "append":
        live = s["slots"] >= 0
        dr = s["kr_new"].shape[1]
        k = s["kr_pool"].double()
        k.view(-1, dr)[s["slots"][live]] = _turn64(s["kr_new"][:, None], s, dr, 0)[:, 0][live]
        if case["cache"] == "bf16":
            c = s["ckv_pool"].double()
            c.view(-1, case["dc"])[s["slots"][live]] = s["ckv_new"][live].double()
            return [c, k]
        scales = s["scales"].double()
        scales.view(-1)[s["slots"][live]] = s["ckv_new"][live].double().abs().amax(-1) / 448
        return [None, k, scales]   # the codes are the definition's own 8-bit rounding
    cu, lens = s["cu_tokens"].tolist(), s["seq_lens"].tolist()
    outs, lses = [], []
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        pages = s["block_table"][b, :(L + PAGE - 1) // PAGE].long()
        c = s["ckv_pool"][pages].flatten(0, 1)[:L]
        if case["cache"] == "e4m3":
            c = (c.view(torch.float8_e4m3fn).float() * s["scales"][pages].flatten()[:L, None]).bfloat16()
        c, k = c.double(), s["kr_pool"][pages].flatten(0, 1)[:L].double()
        for i in range(n):   # one node at a time
            q = s["q"][cu[b] + i].double()
            j = torch.arange(n, device="cuda")
            bits = (s["masks"][cu[b] + i].long()[j // 32] >> (j % 32)) & 1
            seen = torch.cat([torch.ones(L - n, dtype=torch.bool, device="cuda"), bits == 1])
            x = (q[:, :c.shape[1]] @ c.T + q[:, c.shape[1]:] @ k.T) * s["scale"]
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            lse = torch.logsumexp(x, -1)
            outs.append(torch.exp(x - lse[:, None]) @ c)
            lses.append(lse)
    return torch.stack(outs), torch.stack(lses)
