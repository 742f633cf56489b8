"""The packed step's plan, rotary positions, cache write by slot map, and all of them together with
tree attention, against their plain forms."""
import math

import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu
PAGE = 64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}   # half of fp16's smallest step


@pytest.fixture(scope="module")
def api():
    from mla_latent_kv_18_b200 import api as _api
    assert torch.cuda.is_available()
    return _api


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ the plan

def _plan_case(seed, B, new, cached, tree, pad):
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(0, new + 1, (B,), generator=g).tolist()
    c = torch.randint(0, cached + 1, (B,), generator=g).tolist()
    if B > 2:
        c[1], n[2] = 0, 0
    T = sum(n) + pad
    width = (cached + new + PAGE - 1) // PAGE + 1
    table = torch.randint(1000, 2000, (B, width), generator=g, dtype=torch.int32)
    free = (5000 + torch.randperm(sum(n) // PAGE + B + 4, generator=g)).tolist()
    parents = None
    if tree:
        parents = []
        for k in n:
            parents += [int(torch.randint(-1, i, (1,), generator=g)) if i else -3 for i in range(k)]
        parents += [9] * pad
    return c, n, free, table, T, parents


@pytest.mark.parametrize("B,new,cached,tree,pad", [
    (1, 1, 0, False, 0), (1, 1, 63, True, 7), (3, 70, 200, False, 1), (5, 256, 1000, True, 3), (4, 0, 90, False, 2),
    (64, 8, 4000, True, 0), (513, 5, 300, True, 11), (600, 200, 300, False, 5), (2000, 3, 64, False, 0)])
def test_plan(api, B, new, cached, tree, pad):
    c, n, free, table, T, parents = _plan_case(B + new, B, new, cached, tree, pad)
    got_table = table.cuda()
    nodes = max(1, new) if tree else 0
    p = api.step_plan(_i32(c), _i32(n), _i32(free), _i32([2]), got_table, T,
                      parents=None if parents is None else _i32(parents), max_nodes=nodes)
    torch.cuda.synchronize()
    assert api.get_device_error() == 0
    want = ref.plan(c, n, free, 2, table, T, parents, nodes)
    assert torch.equal(got_table.cpu(), table)
    for k in ("seq_lens", "cu_tokens", "seq_ids", "positions", "slots", "free_head"):
        assert getattr(p, k).tolist() == want[k], k
    if tree:
        assert torch.equal(p.masks.cpu(), want["masks"])
    else:
        assert p.masks is None


def test_plan_largest_batch_and_empty_ones(api):
    B = api.STEP_MAX_BATCH
    c = [b % 130 for b in range(B)]
    n = [b % 3 for b in range(B)]
    table = torch.arange(B * 4, dtype=torch.int32).view(B, 4)
    free = list(range(100000, 100000 + B))
    got = table.cuda()
    p = api.step_plan(_i32(c), _i32(n), _i32(free), _i32([0]), got, sum(n))
    want = ref.plan(c, n, free, 0, table, sum(n))
    assert torch.equal(got.cpu(), table) and p.slots.tolist() == want["slots"] and p.cu_tokens.tolist() == want["cu_tokens"]
    # no request, and no token
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    p = api.step_plan(e, e, e, _i32([0]), e.view(0, 3), 5)
    assert p.cu_tokens.tolist() == [0] and p.slots.tolist() == [-1] * 5 and p.seq_ids.tolist() == [-1] * 5
    p = api.step_plan(_i32([7]), _i32([0]), e, _i32([0]), _i32([[3, 4]]), 0)
    assert p.seq_lens.tolist() == [7] and p.cu_tokens.tolist() == [0, 0] and p.free_head.tolist() == [0]
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def test_plan_bad_data_is_reported(api):
    def err():
        torch.cuda.synchronize()
        assert api.get_device_error() == 4
        assert api.get_device_error() == 0
    one = lambda c, n, free, head, T, width=4, **kw: api.step_plan(  # noqa: E731
        _i32(c), _i32(n), _i32(free), _i32([head]), torch.full((len(c), width), 50, dtype=torch.int32, device="cuda"), T, **kw)
    # lengths that do not fit: planned with no new tokens, the others as ever
    for c, n in ((-1, 2), (5, -2), (250, 7), (2 ** 31 - 1, 2 ** 31 - 1), (300, 0)):
        p = one([10, c, 20], [3, n, 4], [7, 8], 0, 16)
        err()
        assert p.cu_tokens.tolist() == [0, 3, 3, 7] and p.slots.tolist()[3:7] == [50 * 64 + 20 + i for i in range(4)]
        assert p.seq_lens.tolist() == [13, min(max(c, 0), 256), 24]
    # the free list runs out: no page, no slot
    p = one([60, 0], [8, 100], [9], 0, 108)
    err()
    assert p.slots.tolist()[:8] == [50 * 64 + 60 + i for i in range(4)] + [9 * 64 + i for i in range(4)]
    assert p.slots.tolist()[8:] == [-1] * 100 and p.free_head.tolist() == [1]
    for head in (-1, 5):
        one([0], [1], [9], head, 1)
        err()
    # more tokens than rows
    p = one([0], [5], [9], 0, 3)
    err()
    assert p.slots.tolist() == [576, 577, 578] and p.cu_tokens.tolist() == [0, 5]
    # parents that do not come before, and more nodes than masks hold
    p = one([0], [3], [9], 0, 3, parents=_i32([0, 2, 1]), max_nodes=3)
    err()
    assert p.masks[:, 0].tolist() == [1, 2, 6] and p.positions.tolist() == [0, 0, 1]
    p = one([0], [40], [9], 0, 40, parents=_i32(list(range(-1, 39))), max_nodes=32)
    err()
    assert p.masks[39, 0].item() == -1 and p.positions.tolist() == list(range(40))
    # an old table entry without a page
    p = api.step_plan(_i32([3]), _i32([2]), _i32([9]), _i32([0]), _i32([[-1, -1]]), 2)
    err()
    assert p.slots.tolist() == [-1, -1]


# ------------------------------------------------------------------ rotary positions

def _turn_check(got, x, pos, f, m, layout, offset, inverse=False, rows=None):
    want, bound = ref.rotary(x, pos, f, m, layout, offset, inverse)
    bound = bound + HALF_STEP[x.dtype] * (want.abs() + bound) + TINY[x.dtype]
    off = (got.double() - want).abs()
    live = pos >= 0 if rows is None else rows
    assert (off[live] <= bound[live]).all(), ((off - bound)[live]).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,width,rot,offset", [(1, 16, 64, 64, 0), (37, 128, 192, 64, 128), (5, 3, 18, 18, 0),
                                                  (130, 1, 64, 64, 0), (2, 7, 69, 8, 61), (9, 2, 80, 64, 8),
                                                  (3, 5, 2, 2, 0), (2, 1, 4100, 4096, 4)])
def test_rotary(api, dtype, layout, T, H, width, rot, offset):
    g = torch.Generator("cuda").manual_seed(T + H)
    x = torch.randn(T, H, width, generator=g, device="cuda").to(dtype)
    k = torch.randn(T, 2, width, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 200000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, m = api.rope_frequencies(rot, scaling="yarn", factor=16.0, device="cuda")
    y, yk = api.rotary(x, pos, f, m, layout, offset, k=k)
    _turn_check(y, x, pos, f, m, layout, offset)
    _turn_check(yk, k, pos, f, m, layout, offset)
    assert torch.equal(y[..., :offset], x[..., :offset]) and torch.equal(y[..., offset + rot:], x[..., offset + rot:])
    # in place, the same bits
    z = x.clone()
    assert api.rotary(z, pos, f, m, layout, offset, out=z) is z and torch.equal(z, y)
    # the inverse is the transpose: its value, and <R x, w> = <x, R^T w> as a gradient has it
    w = torch.randn(T, H, width, generator=g, device="cuda").to(dtype)
    _turn_check(api.rotary(w, pos, f, m, layout, offset, inverse=True), w, pos, f, m, layout, offset, True)
    assert api.get_device_error() == 0


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_gradient_by_differences(api, layout):
    """The inverse turn of the output's gradient is the gradient: against central differences,
    which are exact for a linear map but for rounding (fp32: 2^-24 of sums of 12 values, over 2h = 2)."""
    T, H, W = 3, 2, 6
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(T, H, W, generator=g, device="cuda")
    w = torch.randn(T, H, W, generator=g, device="cuda")
    pos, (f, m) = _i32([5, 0, 90000]), api.rope_frequencies(6, device="cuda", scaling="yarn", factor=4.0)
    grad = api.rotary(w, pos, f, m, layout, inverse=True)
    loss = lambda v: (api.rotary(v, pos, f, m, layout).double() * w.double()).sum()  # noqa: E731
    for t in range(T):
        for h in range(H):
            for c in range(W):
                d = torch.zeros_like(x)
                d[t, h, c] = 1.0
                num = (loss(x + d) - loss(x - d)) / 2
                assert abs(num - grad[t, h, c].double()) <= 1e-5


def test_rotary_strides_skips_and_far_positions(api):
    g = torch.Generator("cuda").manual_seed(0)
    big = torch.randn(11, 5, 4, 200, generator=g, device="cuda").bfloat16()
    pos = _i32([0, -1, 5, 2 ** 31 - 1, 77, -2 ** 31, 1, 2, 3, 4, 1 << 20])
    f, m = api.rope_frequencies(64, device="cuda")
    for x in (big[:, 1, :, 3:67], big[:, :, 2, 8:72], big.transpose(1, 2)[:, 1, :, :64], big[:, 0, :1, 100:164]):
        for layout in ("interleaved", "half"):
            y = api.rotary(x, pos, f, m, layout)
            _turn_check(y, x, pos, f, m, layout, 0)
            assert (y[1] == 0).all() and (y[5] == 0).all()
            before = big.clone()
            api.rotary(x, pos, f, m, layout, out=x)     # in place in a view: nothing else moves
            assert torch.equal(x[pos >= 0], y[pos >= 0])
            x.copy_(before[0].new_zeros(()).expand_as(x))
            moved = big != before
            x_mask = torch.zeros_like(big, dtype=torch.bool)
            x_mask.as_strided(x.shape, x.stride(), x.storage_offset()).fill_(True)
            assert not (moved & ~x_mask).any()
            big.copy_(before)


def test_rotary_agrees_with_the_absorbed_query_rope(api):
    """Plain frequencies, interleaved: the rotation mla_absorb_q_rope and mla_append_kv apply, within
    one rounding of each (both are within the bound of the same fp64 value)."""
    T, H = 9, 4
    g = torch.Generator("cuda").manual_seed(1)
    q_r = torch.randn(T, H, 64, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 60000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, m = api.rope_frequencies(64, device="cuda")
    dims = api.make_dims(H, 1, 128, 512, 64, 128)
    q = api.absorb_q_rope(torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda"), q_r,
                          torch.zeros(H, 128, 512, dtype=torch.bfloat16, device="cuda"), dims, pos)
    _turn_check(api.rotary(q_r, pos, f, m), q_r, pos, f, m, "interleaved", 0)
    _turn_check(q[..., 512:], q_r, pos, f, m, "interleaved", 0)


# ------------------------------------------------------------------ the cache write

@pytest.mark.parametrize("dc,fp8", [(512, False), (64, False), (512, True)])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T", [1, 7, 200])
def test_append_slots(api, dc, fp8, layout, T):
    dr = 64 if dc == 512 else 8
    g = torch.Generator("cuda").manual_seed(T)
    both = torch.randn(T, dc + dr + 8, generator=g, device="cuda").bfloat16()
    ckv_new, kr_new = both[:, :dc], both[:, dc:dc + dr]
    pages = 9
    slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:T].contiguous()
    if T > 2:
        slots[1] = -1
    pos = torch.randint(0, 150000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, m = api.rope_frequencies(dr, scaling="linear", factor=2.0, device="cuda")
    dims = api.make_dims(1, 1, 128, dc, dr, 128)
    pool = torch.randn(pages, PAGE, dc + dr, generator=g, device="cuda").bfloat16()
    kr = pool[..., dc:]
    live = slots >= 0
    at = slots[live]
    rest = torch.ones(pages * PAGE, dtype=torch.bool, device="cuda")
    rest[at] = False
    before = pool.clone().view(pages * PAGE, -1)
    if fp8:
        codes, scales = api.alloc_fp8_cache(pages, dc, "cuda")
        codes.fill_(3)
        api.append_kv_slots_fp8(ckv_new, kr_new, slots, codes, scales, kr, dims, pos, f, m, layout)
        # the rows of the write by positions, which the oracle's tests hold
        c2, s2 = api.alloc_fp8_cache(pages, dc, "cuda")
        kr2 = torch.zeros(pages, PAGE, dr, dtype=torch.bfloat16, device="cuda")
        table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
        api.append_kv_fp8(ckv_new[live].contiguous(), kr_new[live].contiguous(), torch.zeros_like(at).int(), at.int(),
                          c2, s2, kr2, table, dims, theta=0.0)
        assert torch.equal(codes.view(-1, dc)[at], c2.view(-1, dc)[at])
        assert torch.equal(scales.view(-1)[at], s2.view(-1)[at])
        assert (codes.view(-1, dc)[rest] == 3).all() and (scales.view(-1)[rest] == 0).all()
    else:
        api.append_kv_slots(ckv_new, kr_new, slots, pool[..., :dc], kr, dims, pos, f, m, layout)
        assert torch.equal(pool[..., :dc].reshape(-1, dc)[at], ckv_new[live])
    torch.cuda.synchronize()
    assert api.get_device_error() == 0
    got = pool.view(pages * PAGE, -1)
    assert torch.equal(got[rest], before[rest])
    _turn_check(got[at][:, None, dc:], kr_new[live][:, None], pos[live], f, m, layout, 0)
    # without positions the key is copied
    if not fp8:
        api.append_kv_slots(ckv_new, kr_new, slots, pool[..., :dc], kr, dims)
        assert torch.equal(kr.reshape(-1, dr)[at], kr_new[live])


def test_append_slots_bad_slots_are_skipped(api):
    dims = api.make_dims(1, 1, 128, 512, 64, 128)
    c, k = torch.ones(6, 512, device="cuda").bfloat16(), torch.ones(6, 64, device="cuda").bfloat16()
    pool, kr = torch.zeros(2, 64, 512, device="cuda").bfloat16(), torch.zeros(2, 64, 64, device="cuda").bfloat16()
    for bad in (-2, 128, 2 ** 40, -2 ** 62):
        slots = torch.tensor([5, bad, -1, 127, -1, 0], device="cuda")
        pool.zero_()
        kr.zero_()
        api.append_kv_slots(c, k, slots, pool, kr, dims)
        torch.cuda.synchronize()
        assert api.get_device_error() == 4
        written = pool.view(128, 512).sum(1).nonzero()[:, 0].tolist()
        assert written == [0, 5, 127] == kr.view(128, 64).sum(1).nonzero()[:, 0].tolist()
    # a negative position turns as 0, and says so
    f, m = api.rope_frequencies(64, device="cuda")
    api.append_kv_slots(c, k, torch.arange(6, device="cuda"), pool, kr, dims, _i32([-1] * 6), f, m)
    torch.cuda.synchronize()
    assert api.get_device_error() == 4 and (kr.view(128, 64)[:6] == 1).all()


def test_single_rows_empty_calls_and_whole_numbers(api):
    """One token, whose strides say nothing; no token; sizes as numpy's integers."""
    import numpy as np
    dims = api.make_dims(1, 1, 128, 512, 64, 128)
    f, m = api.rope_frequencies(64, device="cuda")
    g = torch.Generator("cuda").manual_seed(2)
    c, k = (torch.randn(n, 1, generator=g, device="cuda").bfloat16().as_strided((1, n), (1, 1)) for n in (512, 64))
    pool, kr = torch.zeros(2, 64, 512, device="cuda").bfloat16(), torch.zeros(2, 64, 64, device="cuda").bfloat16()
    api.append_kv_slots(c, k, torch.tensor([70], device="cuda"), pool, kr, dims, _i32([3]), f, m)
    assert torch.equal(pool[1, 6], c[0]) and (pool[0] == 0).all()
    _turn_check(kr[1, 6][None, None], k[:, None], _i32([3]), f, m, "interleaved", 0)
    x = k.as_strided((1, 1, 64), (1, 3, 1))
    _turn_check(api.rotary(x, _i32([3]), f, m), x, _i32([3]), f, m, "interleaved", 0)
    # broadcast inputs: every token's row is the same one
    x = torch.randn(1, 2, 64, generator=g, device="cuda").bfloat16().expand(5, 2, 64)
    _turn_check(api.rotary(x, _i32([0, 1, 2, 3, 4]), f, m), x, _i32([0, 1, 2, 3, 4]), f, m, "interleaved", 0)
    # nothing to do
    before = pool.clone()
    api.append_kv_slots(c[:0], k[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), pool, kr, dims, _i32([]), f, m)
    assert api.rotary(x[:0], _i32([]), f, m).shape == (0, 2, 64)
    assert api.rotary(x[:, :0], _i32([0] * 5), f, m).shape == (5, 0, 64)
    assert torch.equal(pool, before)
    table = _i32([[4, -1]])
    p = api.step_plan(_i32([60]), _i32([6]), _i32([9]), _i32([0]), table, np.int64(6), _i32(list(range(-1, 5))),
                      np.int32(8))
    assert p.slots.tolist() == [4 * 64 + 60 + i for i in range(4)] + [9 * 64, 9 * 64 + 1] and table.tolist() == [[4, 9]]
    with pytest.raises(Exception, match="whole number"):
        api.step_plan(_i32([60]), _i32([6]), _i32([9]), _i32([0]), table, 6.0)
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


# ------------------------------------------------------------------ a step, as it is used

@pytest.mark.parametrize("fp8", [False, True])
def test_steps_together(api, fp8):
    """Prompts, then two turns of draft trees on top of them, through the calls a server
    makes, the step captured once and replayed: against fp64 attention over the tokens themselves."""
    B, H, dn, dc, dr, dv = 3, 16, 128, 512, 64, 128
    g = torch.Generator("cuda").manual_seed(9)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    w_uk, w_uv = rnd(H, dn, dc, std=dc ** -0.5), rnd(H, dc, dv, std=dc ** -0.5)
    dims = api.make_dims(H, 1, dn, dc, dr, dv)
    pages, T, nodes = 24, 96, 64
    kr = torch.zeros(pages, PAGE, dr, dtype=torch.bfloat16, device="cuda")
    ckv = torch.zeros(pages, PAGE, dc, dtype=torch.bfloat16, device="cuda")
    codes, scales = api.alloc_fp8_cache(pages, dc, "cuda")
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").int()
    f, m = api.rope_frequencies(dr, scaling="yarn", factor=8.0, device="cuda")
    cached, new, head = _i32([0] * B), _i32([0] * B), _i32([0])
    parents = torch.zeros(T, dtype=torch.int32, device="cuda")
    plan = api.alloc_step_plan(B, T, "cuda", nodes)
    q_c, q_r, kv = rnd(T, H, dn), rnd(T, H, dr), rnd(T, dc + dr)
    q_rot = torch.zeros_like(q_r)
    ws = api.alloc_tree_workspace(dims, "cuda")
    out, lse = torch.zeros(T, H, dv, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")

    def step():
        api.step_plan(cached, new, free, head, table, T, parents=parents, max_nodes=nodes, out=plan)
        api.rotary(q_r, plan.positions, f, m, out=q_rot)
        append = (kv[:, :dc], kv[:, dc:], plan.slots)
        if fp8:
            api.append_kv_slots_fp8(*append, codes, scales, kr, dims, plan.positions, f, m)
        else:
            api.append_kv_slots(*append, ckv, kr, dims, plan.positions, f, m)
        o, l = api.tree_attend(q_c, q_rot, codes if fp8 else ckv, kr, table, plan.seq_lens, plan.cu_tokens, w_uk, w_uv,
                               nodes, masks=plan.masks, scales=scales if fp8 else None, workspace=ws)
        out.copy_(o)
        lse.copy_(l)

    step()                      # an idle step: nothing new
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    history = [[] for _ in range(B)]   # per request: (latent, key, position) of accepted tokens
    want_scale = 1 / math.sqrt(dn + dr)
    for turn, counts in enumerate(([40, 1, 55], [0, 9, 33], [12, 0, 64])):
        for t in (q_c, q_r, kv):
            t.copy_(rnd(*t.shape))
        par = []
        for n in counts:
            if turn == 0:
                par += list(range(-1, n - 1))
            else:
                par += [int(torch.randint(-1, i, (1,))) if i else -1 for i in range(n)]
        cached.copy_(_i32([len(h) for h in history]))
        new.copy_(_i32(counts))
        parents.fill_(7)
        parents[:len(par)] = _i32(par)
        graph.replay()
        torch.cuda.synchronize()
        assert api.get_device_error() == 0
        at = 0
        for b, n in enumerate(counts):
            if n == 0:
                continue
            seen = ref.ancestors(par[at:at + n])
            pos = len(history[b]) + seen.sum(1).int().cuda() - 1
            assert plan.positions[at:at + n].tolist() == pos.tolist()
            c = kv[at:at + n, :dc].clone()   # (the step's own buffers are reused next turn)
            if fp8:
                amax = c.float().abs().amax(-1, keepdim=True)
                code = (c.float() * (448.0 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
                c = (code.float() * (amax / 448.0)).bfloat16()
            k = ref.rotary(kv[at:at + n, None, dc:], pos, f, m, "interleaved", 0)[0][:, 0]
            turned = ref.rotary(q_r[at:at + n], pos, f, m, "interleaved", 0)[0]
            old = history[b]
            C = torch.cat([torch.stack([h[0] for h in old])] + [c]) if old else c
            K = torch.cat([torch.stack([h[1] for h in old])] + [k]) if old else k
            q_lat = torch.einsum("thd,hdc->thc", q_c[at:at + n].double(), w_uk.double())
            q = torch.cat([q_lat, turned], -1)
            full = torch.cat([torch.ones(n, len(old), dtype=torch.bool), seen], 1)
            o, l, A, _ = ref.tree_attention(q, C, K, want_scale, full)
            w = w_uv.double()
            y = torch.einsum("thc,hcd->thd", o, w)
            # q, the turned query and the turned key are rounded to bf16 (2^-8 of each value): a score is
            # off by at most 2 * 2^-8 of the sum of its terms' magnitudes, far less than that in
            # total; measured against the rounded operands the kernels are held tightly elsewhere,
            # here the bound is the whole chain's: weights, latent result and output on top
            size = torch.stack([(q[i].abs() @ torch.cat([C, K], -1).double().abs().T * want_scale).amax(-1)
                                for i in range(n)])
            ds = (2.0 ** -7) * size
            bound = torch.einsum("thc,hcd->thd", (2 * ds[..., None] + 3 * 2.0 ** -8) * A, w.abs()) + 2.0 ** -8 * y.abs()
            assert ((out[at:at + n].double() - y).abs() <= bound).all()
            assert (((lse[at:at + n].double() - l).abs()) <= ds + 1e-4).all()
            # and in the mean: independent roundings add as squares, so 2 % of the norm is generous
            # against 2^-8 per factor and far below what one wrong token or angle would give
            rel = (out[at:at + n].double() - y).norm() / y.norm()
            assert rel <= 0.02, rel
            # accept the deepest path; its tokens are rewritten at their final places next turn
            if turn == 0:
                history[b] = [(c[i], k[i]) for i in range(n)]
            at += n
        head.copy_(plan.free_head if turn == 0 else head)


@pytest.mark.parametrize("nodes", [1, 8, 31, 32, 33, 100, 200])
def test_plan_masks_hold_max_nodes_bits(api, nodes):
    """A request with more tokens than max_nodes: reported, and no bit beyond max_nodes in any mask."""
    g = torch.Generator().manual_seed(nodes)
    n = [nodes, nodes + 20, 3]
    par = [[int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(k)] for k in (n[0], n[1], min(3, nodes))]
    par[2] += [-1] * (3 - len(par[2]))
    par[1][nodes:] = range(nodes - 1, nodes + 19)      # a chain across the border
    T = sum(n)
    p = api.step_plan(_i32([5, 0, 60]), _i32(n), _i32(list(range(10, 40))), _i32([0]),
                      torch.full((3, 8), 3, dtype=torch.int32, device="cuda"), T, parents=_i32(sum(par, [])), max_nodes=nodes)
    torch.cuda.synchronize()
    assert api.get_device_error() == 4
    at = 0
    for c, k, q in zip((5, 0, 60), n, par):
        seen = ref.ancestors(q)
        want = torch.zeros(k, nodes, dtype=torch.bool)
        want[:, :min(k, nodes)] = seen[:, :nodes]
        assert torch.equal(p.masks[at:at + k].cpu(), ref.pack(want, nodes))
        assert p.positions[at:at + k].tolist() == (c + seen.sum(1) - 1).tolist()
        at += k


def test_plan_walks_end(api):
    """A chain far longer than any tree: the walk up ends after TREE_MAX_NODES ancestors, and the call reports it."""
    n = 3000
    p = api.step_plan(_i32([100]), _i32([n]), _i32(list(range(60))), _i32([0]),
                      torch.full((1, 60), 3, dtype=torch.int32, device="cuda"), n, parents=_i32(list(range(-1, n - 1))),
                      max_nodes=8)
    torch.cuda.synchronize()
    assert api.get_device_error() == 4
    assert p.positions.tolist() == [100 + min(i, api.TREE_MAX_NODES) for i in range(n)]
    for i in (0, 3, 7, 8, 255):
        assert p.masks[i, 0].item() == (1 << min(i + 1, 8)) - 1


# ------------------------------------------------------------------ what the calls write, and autograd

def _writes(api):
    """Every call with the tensors that it writes: (name, call, written tensors)."""
    g = torch.Generator("cuda").manual_seed(3)
    T, H, pages = 6, 16, 3
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    dims = api.make_dims(H, 1, 128, 512, 64, 128)
    f, m = api.rope_frequencies(64, device="cuda")
    pos, slots = _i32(list(range(T))), torch.arange(T, device="cuda")
    x, k, y, ky = rnd(T, H, 64), rnd(T, 2, 64), rnd(T, H, 64), rnd(T, 2, 64)
    ckv, kr, kr8 = rnd(pages, PAGE, 512), rnd(pages, PAGE, 64), rnd(pages, PAGE, 64)
    codes, scales = api.alloc_fp8_cache(pages, 512, "cuda")
    c_new, k_new, q = rnd(T, 512), rnd(T, 64), rnd(T, H, 576)
    o, lse = rnd(T, H, 512), torch.zeros(T, H, device="cuda")
    table, plan = _i32([[0, 1]]), api.alloc_step_plan(1, T, "cuda", 8)
    return [
        ("plan", lambda: api.step_plan(_i32([0]), _i32([T]), _i32([2]), _i32([0]), table, T, _i32([-1] * T), 8, out=plan),
         [table, *plan]),
        ("rotary", lambda: api.rotary(x, pos, f, m, out=x), [x]),
        ("rotary of two", lambda: api.rotary(x, pos, f, m, out=y, k=k, k_out=ky), [y, ky]),
        ("append", lambda: api.append_kv_slots(c_new, k_new, slots, ckv, kr, dims, pos, f, m), [ckv, kr]),
        ("append e4m3", lambda: api.append_kv_slots_fp8(c_new, k_new, slots, codes, scales, kr8, dims, pos, f, m),
         [codes, scales, kr8]),
        ("tree", lambda: api.decode_tree(q, ckv, kr, _i32([[0, 1]]), _i32([T]), _i32([0, T]), dims, 8, o_lat=o,
                                         lse_out=lse), [o, lse]),
    ]


def test_versions_move_with_what_is_written(api):
    """As after an operation of torch in place, so that autograd notices a saved tensor that has changed."""
    for name, call, written in _writes(api):
        before = [t._version for t in written]
        call()
        assert all(t._version > v for t, v in zip(written, before)), name
    w = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
    x = torch.ones(4, 2, 64, device="cuda")
    loss = (w * x).sum()
    f, m = api.rope_frequencies(64, device="cuda")
    api.rotary(x, _i32([1, 2, 3, 4]), f, m, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # a refused call has written nothing
    v = x._version
    with pytest.raises(RuntimeError, match="MLA_ERR_INVALID_ARG"):
        api.rotary(x, _i32([1, 2, 3, 4]), f, math.inf, out=x)
    assert x._version == v
    # tensors of inference mode have no version
    with torch.inference_mode():
        z = torch.ones(4, 2, 64, device="cuda")
        api.rotary(z, _i32([1, 2, 3, 4]), f, m, out=z)
    api.rotary(z, _i32([1, 2, 3, 4]), f, m, out=z)
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def test_outputs_that_require_grad_are_refused(api):
    """Autograd does not see these writes: a tensor that it tracks is written with gradients off only."""
    for name, call, written in _writes(api):
        for t in written:
            if not t.is_floating_point():
                continue
            t.requires_grad_(True)
            with pytest.raises(RuntimeError, match="requires grad"):
                call()
            with torch.no_grad():
                call()
            with torch.inference_mode():
                call()
            t.requires_grad_(False)
    # inputs may require one: the outputs take no part in autograd
    f, m = api.rope_frequencies(64, device="cuda")
    x = torch.ones(4, 2, 64, device="cuda", requires_grad=True)
    assert not api.rotary(x, _i32([1, 2, 3, 4]), f, m).requires_grad
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


# ------------------------------------------------------------------ refusals of tensors that do not fit

def _fitting(api, call):
    """Keyword arguments of a call that fits."""
    T, H, B, pages = 7, 16, 2, 4
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    dims = api.make_dims(H, 1, 128, 512, 64, 128)
    freq = torch.zeros(32, dtype=torch.float64, device="cuda")
    pools = dict(ckv_pool=bf(pages, 64, 512), kr_pool=bf(pages, 64, 64), dims=dims)
    codes = dict(ckv8_pool=torch.zeros(pages, 64, 512, dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros(pages, 64, device="cuda"), kr_pool=bf(pages, 64, 64), dims=dims)
    if call == "step_plan":
        return dict(cached_lens=i32(B), new_lens=i32(B), free_pages=i32(5), free_head=i32(1), block_table=i32(B, 4),
                    num_tokens=T, parents=i32(T), max_nodes=8, out=api.alloc_step_plan(B, T, "cuda", 8))
    if call == "rotary":
        return dict(x=bf(T, H, 64), positions=i32(T), inv_freq=freq, out=bf(T, H, 64), k=bf(T, 2, 64), k_out=bf(T, 2, 64))
    if call.startswith("append"):
        return dict(ckv_new=bf(T, 512), kr_new=bf(T, 64), slots=torch.full((T,), -1, device="cuda"), positions=i32(T),
                    inv_freq=freq, **(codes if call.endswith("fp8") else pools))
    tree = dict(block_table=i32(B, 4), seq_lens=i32(B), cu_tokens=i32(B + 1), max_nodes=8, masks=i32(T, 1))
    if call == "tree_attend":
        del pools["dims"]
        return dict(q_c=bf(T, H, 128), q_r=bf(T, H, 64), w_uk=bf(H, 128, 512), w_uv=bf(H, 512, 128), **pools, **tree)
    return dict(q=bf(T, H, 576), workspace=api.alloc_tree_workspace(dims, "cuda"), o_lat=bf(T, H, 512),
                lse_out=torch.zeros(T, H, device="cuda"), **tree, **(codes if call.endswith("fp8") else pools))


def _piece(t, **kw):
    return t._replace(**kw)


_BF, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
_WRONG = {
    "step_plan": [
        (dict(cached_lens=lambda t: t[:1]), r"cached_lens and new_lens \[B\]"),
        (dict(new_lens=lambda t: t.repeat(2)), r"cached_lens and new_lens \[B\]"),
        (dict(new_lens=lambda t: t.long()), "new_lens is a contiguous Int"),
        (dict(cached_lens=lambda t: t.cpu()), "cached_lens is a contiguous Int"),
        (dict(free_pages=lambda t: t.float()), "free_pages is a contiguous Int"),
        (dict(free_head=lambda t: t.repeat(2)), "one free_head"),
        (dict(block_table=lambda t: t.view(-1)), r"block_table \[B, max_pages\]"),
        (dict(block_table=lambda t: t.repeat(1, 2)[:, ::2]), "block_table is a contiguous Int"),
        (dict(block_table=lambda t: t[:, :0]), "mla_step_plan"),
        (dict(parents=lambda t: t[:-1]), r"parents \[num_tokens\]"),
        (dict(num_tokens=lambda t: t + 1), r"parents \[num_tokens\]"),
        (dict(num_tokens=lambda t: -1), "num_tokens is a whole number"),
        (dict(max_nodes=lambda t: 0), "max_nodes is a whole number"),
        (dict(max_nodes=lambda t: 257), "max_nodes is a whole number"),
        (dict(max_nodes=lambda t: 33), "out of other sizes"),
        (dict(out=lambda t: t[:6]), "out is a StepPlan"),
        (dict(out=lambda t: _piece(t, seq_lens=t.seq_lens[:1])), "out of other sizes"),
        (dict(out=lambda t: _piece(t, cu_tokens=t.cu_tokens[:2])), "out of other sizes"),
        (dict(out=lambda t: _piece(t, positions=t.positions[:6])), "out of other sizes"),
        (dict(out=lambda t: _piece(t, slots=t.slots.int())), "out is a contiguous Long"),
        (dict(out=lambda t: _piece(t, masks=t.masks.view(1, -1))), "out of other sizes"),
        (dict(out=lambda t: _piece(t, masks=None)), "out is a tensor"),
    ],
    "rotary": [
        (dict(x=lambda t: t.double()), "x is bf16, fp16 or fp32"),
        (dict(x=lambda t: t[0]), r"x \[T, heads, width\]"),
        (dict(positions=lambda t: t[:-1]), r"positions \[T\]"),
        (dict(positions=lambda t: t.long()), "positions is a contiguous Int"),
        (dict(inv_freq=lambda t: t.float()), "inv_freq is a contiguous Double"),
        (dict(inv_freq=lambda t: t.repeat(2)), "mla_rotary"),      # 128 channels of heads of 64
        (dict(inv_freq=lambda t: t[:0]), "mla_rotary"),
        (dict(inv_freq=lambda t: t.view(2, 16)), r"inv_freq \[rot / 2\]"),
        (dict(out=lambda t: t[:1]), "out of the same shape"),
        (dict(out=lambda t: t.float()), "tensors of one type"),
        (dict(out=lambda t: t.cpu()), "out of the same shape"),
        (dict(out=lambda t: t[:1].expand(7, 16, 64)), "mla_rotary"),
        (dict(k=lambda t: t[:3]), "tensors of one type, tokens and width"),
        (dict(k=lambda t: t[..., :32]), "tensors of one type, tokens and width"),
        (dict(k_out=lambda t: t[:, :1]), "out of the same shape"),
        (dict(layout=lambda t: "neox"), "layout is"),
        (dict(offset=lambda t: 2), "mla_rotary"),
        (dict(offset=lambda t: -1), "offset is a whole number"),
        (dict(mscale=lambda t: "one"), "mscale is a number"),
    ],
    "append_kv_slots": [
        (dict(ckv_new=lambda t: t[:, :256]), r"ckv_new \[T, d_c\]"),
        (dict(ckv_new=lambda t: t.half()), r"ckv_new \[T, d_c\]"),
        (dict(kr_new=lambda t: t[:6]), r"kr_new \[T, d_R\]"),
        (dict(kr_new=lambda t: t.t().contiguous().t()), r"kr_new \[T, d_R\]"),
        (dict(kr_new=lambda t: t.cpu()), r"kr_new \[T, d_R\]"),
        (dict(ckv_new=lambda t: t[:1].expand(7, 512)), "mla_append_kv_slots"),
        (dict(slots=lambda t: t.int()), "slots is a contiguous Long"),
        (dict(slots=lambda t: t[:6]), r"slots \[T\]"),
        (dict(positions=lambda t: t[:6]), r"positions \[T\]"),
        (dict(inv_freq=lambda t: t[:16]), r"inv_freq \[d_R / 2\]"),
        (dict(inv_freq=lambda t: None), r"inv_freq \[d_R / 2\]"),
        (dict(ckv_pool=lambda t: t[:, :32]), "pools"),
        (dict(ckv_pool=lambda t: t[..., :256]), "pools"),
        (dict(ckv_pool=lambda t: t[:3]), "pools"),
        (dict(ckv_pool=lambda t: t.view(torch.uint8)), "pools"),
        (dict(kr_pool=lambda t: t.transpose(1, 2)), "pools"),
        (dict(kr_pool=lambda t: t.cpu()), "pools"),
        (dict(ckv_pool=lambda t: t[:1].expand(4, 64, 512)), "mla_append_kv_slots"),   # pages on top of each other
        (dict(layout=lambda t: 1), "layout is"),
        (dict(dims=lambda t: None), "dims are make_dims'"),
    ],
    "append_kv_slots_fp8": [
        (dict(scales=lambda t: t[:3]), r"scales \[pages, 64\]"),
        (dict(scales=lambda t: t.double()), "scales is a contiguous Float"),
        (dict(scales=lambda t: None), r"scales \[pages, 64\]"),
        (dict(ckv8_pool=lambda t: t.view(_BF)), "pools"),
    ],
    "decode_tree": [
        (dict(q=lambda t: t[..., :512].contiguous()), r"q \[T, H, d_c \+ d_R\]"),
        (dict(q=lambda t: t[:, :8].contiguous()), r"q \[T, H, d_c \+ d_R\]"),
        (dict(q=lambda t: t[:, :8]), "q is a contiguous BFloat16"),
        (dict(q=lambda t: t.float()), "q is a contiguous BFloat16"),
        (dict(q=lambda t: t.cpu()), "q is on a CUDA device"),
        (dict(masks=lambda t: t[:-1]), r"masks \[T, ceil"),
        (dict(masks=lambda t: t.repeat(1, 2)), r"masks \[T, ceil"),
        (dict(max_nodes=lambda t: 33), r"masks \[T, ceil"),
        (dict(max_nodes=lambda t: 0), "max_nodes is a whole number"),
        (dict(max_nodes=lambda t: 257), "max_nodes is a whole number"),
        (dict(seq_lens=lambda t: t[:1]), r"seq_lens \[B\]"),
        (dict(seq_lens=lambda t: t.long()), "seq_lens is a contiguous Int"),
        (dict(cu_tokens=lambda t: t[:2]), r"cu_tokens \[B \+ 1\]"),
        (dict(block_table=lambda t: t[:1]), r"seq_lens \[B\]"),
        (dict(block_table=lambda t: t[:, :0]), "mla_decode_tree"),
        (dict(block_table=lambda t: t.t()), "block_table is a contiguous Int"),
        (dict(ckv_pool=lambda t: t[:, :32]), "pools"),
        (dict(kr_pool=lambda t: t[:3]), "pools"),
        (dict(kr_pool=lambda t: t[..., :32]), "pools"),
        (dict(ckv_pool=lambda t: t[:0], kr_pool=lambda t: t[:0]), "mla_decode_tree"),
        (dict(workspace=lambda t: t[:-256]), "mla_decode_tree"),
        (dict(workspace=lambda t: t[16:]), "mla_decode_tree"),
        (dict(workspace=lambda t: t.view(_F32)), "workspace is a contiguous Byte"),
        (dict(num_parts=lambda t: 1000), "mla_decode_tree"),      # more than the workspace holds
        (dict(num_parts=lambda t: 0), "num_parts is a whole number"),
        (dict(o_lat=lambda t: t[:6]), r"o_lat \[T, H, d_c\]"),
        (dict(o_lat=lambda t: t.half()), "o_lat is a contiguous BFloat16"),
        (dict(lse_out=lambda t: t[:6]), r"lse_out \[T, H\]"),
        (dict(lse_out=lambda t: t.bfloat16()), "lse_out is a contiguous Float"),
        (dict(dims=lambda t: 5), "dims are make_dims'"),
    ],
    "decode_tree_fp8": [
        (dict(scales=lambda t: t[:3]), r"scales \[pages, 64\]"),
        (dict(scales=lambda t: None), r"scales \[pages, 64\]"),
        (dict(scales=lambda t: torch.zeros(257, device="cuda")[1:].view(4, 64)), "mla_decode_tree_fp8"),
        (dict(ckv8_pool=lambda t: t[..., :256]), "pools"),
    ],
    "tree_attend": [
        (dict(q_c=lambda t: t.float()), "tree_attend: contiguous bf16"),
        (dict(q_r=lambda t: t[:6]), "tree_attend: contiguous bf16"),
        (dict(w_uk=lambda t: t[:8]), "tree_attend: contiguous bf16"),
        (dict(w_uv=lambda t: t.transpose(1, 2)), "tree_attend: contiguous bf16"),
        (dict(w_uv=lambda t: t.cpu()), "tree_attend: contiguous bf16"),
        (dict(masks=lambda t: t[:6]), r"masks \[T, ceil"),
        (dict(ckv_pool=lambda t: t[..., :256]), "pools"),
    ],
}


@pytest.mark.parametrize("call", _WRONG)
def test_wrong_tensors_are_refused(api, call):
    """Each argument wrong by itself, on the GPU and told by its message (the call that fits runs): sizes, types,
    devices and strides that would otherwise become accesses out of range."""
    from mla_latent_kv_18_b200._binding import MLAError
    getattr(api, call)(**_fitting(api, call))
    for change, message in _WRONG[call]:
        kw = _fitting(api, call)
        for name, f in change.items():
            kw[name] = f(kw.get(name))
        with pytest.raises(MLAError, match=message):
            getattr(api, call)(**kw)
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


# ------------------------------------------------------------------ drafts accepted in part

def test_turns_with_drafts_accepted_in_part(api):
    """Turns of draft trees of which a path is accepted. Accepted tokens that already lie at their places stay
    (the request's cached length grows over them); the others of the path are written again, first in the
    next step, as a chain before its drafts. Pages past the cached length go back to the free list before the
    next plan, which overwrites their entries: no page is lost, and none has two owners."""
    B, H, dc, dr, nodes, pages = 3, 16, 512, 64, 96, 21
    g, host = torch.Generator("cuda").manual_seed(5), torch.Generator().manual_seed(5)
    draw = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=host))  # noqa: E731
    dims, scale = api.make_dims(H, 1, 128, dc, dr, 128), 1 / math.sqrt(192)
    f, m = api.rope_frequencies(dr, device="cuda")
    ckv = torch.zeros(pages, PAGE, dc, dtype=torch.bfloat16, device="cuda")
    kr = torch.zeros(pages, PAGE, dr, dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, 7), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=host).tolist()
    history = [[] for _ in range(B)]   # accepted tokens: rows [c | k], the key not turned
    cached, given_back, again = [0] * B, set(), 0
    for turn in range(9):
        pending = [h[c:] for h, c in zip(history, cached)]
        drafts = [draw(1, 40) if turn else (50, 3, 90)[b] for b in range(B)]
        new = [len(p) + n for p, n in zip(pending, drafts)]
        parents, rows = [], []
        for p, n in zip(pending, drafts):
            chain = list(range(-1, len(p) - 1))
            own = [len(p) + (draw(-1, i - 1) if turn else i - 1) for i in range(n)]   # len(p) - 1: follows the context
            parents += chain + own
            rows += p + list(torch.randn(n, dc + dr, generator=g, device="cuda").bfloat16())
        kv = torch.stack(rows)
        T = sum(new)
        p = api.step_plan(_i32(cached), _i32(new), _i32(free), _i32([0]), table, T, _i32(parents), nodes + 40)
        api.append_kv_slots(kv[:, :dc], kv[:, dc:], p.slots, ckv, kr, dims, p.positions, f, m)
        q = torch.randn(T, H, dc + dr, generator=g, device="cuda").bfloat16()
        o, lse = api.decode_tree(q, ckv, kr, table, p.seq_lens, p.cu_tokens, dims, nodes + 40, masks=p.masks)
        torch.cuda.synchronize()
        assert api.get_device_error() == 0
        head = p.free_head.item()
        again += len(given_back & set(free[:head]))
        free = free[head:]
        at = 0
        for b, n in enumerate(new):
            seen = ref.ancestors(parents[at:at + n])
            old = torch.stack(history[b][:cached[b]] or [kv[0]])[:cached[b]]
            c = torch.cat([old, kv[at:at + n]])
            pos = torch.cat([torch.arange(cached[b]), cached[b] + seen.sum(1) - 1]).int().cuda()
            assert p.positions[at:at + n].tolist() == pos[cached[b]:].tolist()
            # the cached keys: the fp64 turn rounded to bf16 is within one step of the kernel's, so the reference
            # reads them from the cache, whose turn is tested by itself, and only checks that they are these tokens'
            where = table[b].long().repeat_interleave(PAGE)[:cached[b] + n] * PAGE + torch.arange(cached[b] + n, device="cuda") % PAGE
            assert torch.equal(ckv.view(-1, dc)[where], c[:, :dc])
            k = kr.view(-1, dr)[where]
            _turn_check(k[:, None], c[:, None, dc:], pos, f, m, "interleaved", 0)
            full = torch.cat([torch.ones(n, cached[b], dtype=torch.bool), seen], 1)
            ref.check_tree(o[at:at + n], lse[at:at + n], ref.tree_attention(q[at:at + n], c[:, :dc], k, scale, full), len(c))
            # accept a path (in the first turn the whole chain)
            node = draw(len(pending[b]) - 1, n - 1) if turn else n - 1
            path = seen[node].nonzero()[:, 0].tolist() if node >= 0 else []
            history[b] = history[b][:cached[b]] + [kv[at + i] for i in path]
            stay = 0
            while stay < len(path) and path[stay] == stay:
                stay += 1
            end = (cached[b] + n + PAGE - 1) // PAGE
            cached[b] += stay
            at += n
            back = range((cached[b] + PAGE - 1) // PAGE, end)
            returned = [int(table[b, i]) for i in back]
            free, given_back = returned + free, given_back | set(returned)   # the next plan takes them first
            for i in back:
                table[b, i] = -1
        owned = [int(v) for v in table.view(-1) if v >= 0]
        assert sorted(owned + free) == list(range(pages))
    assert again > 0          # pages have come round
