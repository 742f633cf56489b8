"""Tree attention over the paged latent cache (mla_decode_tree) against its plain fp64 form."""
import math

import pytest
import torch

from step_reference import ancestors, check_tree, pack, tree_attention

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def api():
    from mla_latent_kv_18_b200 import api as _api
    assert torch.cuda.is_available()
    return _api


def _bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


class Step:
    """A packed step: caches, queries, and per-sequence truth values of who sees what."""

    def __init__(self, api, heads, counts, lens, dc=512, seed=0, kind="tree", pad=0, max_nodes=None, fused_pool=False,
                 fp8=False, extra_pages=3):
        g = torch.Generator("cuda").manual_seed(seed)
        h = torch.Generator().manual_seed(seed)
        self.api, self.H, self.dc, self.dr = api, heads, dc, (64 if dc == 512 else 8)
        self.counts, self.lens, self.fp8 = counts, lens, fp8
        B, n = len(lens), max([1] + counts)
        self.max_nodes = max_nodes or n
        self.dims = api.make_dims(heads, 1, 128 if dc == 512 else 120, dc, self.dr, 128)
        self.scale = 1.0 / math.sqrt((128 if dc == 512 else 120) + self.dr)
        need = [(L + PAGE - 1) // PAGE for L in lens]
        pages = sum(need) + extra_pages
        perm = torch.randperm(pages, generator=h).tolist()
        self.table = torch.full((B, max(1, max(need)) + 1), -1, dtype=torch.int32)
        for b, k in enumerate(need):
            for p in range(k):
                self.table[b, p] = perm.pop()
        if fused_pool:   # both pools as views of one [pages, 64, dc + dr] tensor
            both = _bf16(g, pages, PAGE, dc + self.dr)
            self.ckv, self.kr = both[..., :dc], both[..., dc:]
        else:
            self.ckv, self.kr = _bf16(g, pages, PAGE, dc), _bf16(g, pages, PAGE, self.dr)
        if fp8:
            x = torch.randn(pages, PAGE, dc, generator=g, device="cuda")
            self.scales = (x.abs().amax(-1) / 448).contiguous()
            self.codes = (x / self.scales[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            self.refresh()
        self.T = sum(counts) + pad
        dn = 128 if dc == 512 else 120
        self.q = torch.cat([_bf16(g, self.T, heads, dc, std=math.sqrt(dn / dc)), _bf16(g, self.T, heads, self.dr)], -1)
        self.seen = []   # per sequence [n, n]
        for c in counts:
            if kind == "chain":
                par = list(range(-1, c - 1))
            else:
                par = [int(torch.randint(-1, i, (1,), generator=h)) if i else -1 for i in range(c)]
            self.seen.append(ancestors(par))
        self.cu = torch.tensor([0] + counts).cumsum(0).to("cuda", torch.int32)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.block_table = self.table.cuda()

    def refresh(self):
        """The bf16 values the E4M3 cache stands for."""
        self.ckv = (self.codes.view(torch.float8_e4m3fn).float() * self.scales[..., None]).bfloat16()

    def masks(self):
        m = torch.zeros(self.T, (self.max_nodes + 31) // 32, dtype=torch.int32)
        at = 0
        for s in self.seen:
            m[at:at + len(s)] = pack(s, self.max_nodes)
            at += len(s)
        return m.cuda()

    def run(self, masks="own", **kw):
        m = self.masks() if isinstance(masks, str) else masks
        if self.fp8:
            return self.api.decode_tree_fp8(self.q, self.codes, self.scales, self.kr, self.block_table, self.seq_lens,
                                            self.cu, self.dims, self.max_nodes, masks=m, **kw)
        return self.api.decode_tree(self.q, self.ckv, self.kr, self.block_table, self.seq_lens, self.cu, self.dims,
                                    self.max_nodes, masks=m, **kw)

    def reference(self, b):
        L, n = self.lens[b], self.counts[b]
        pages = self.block_table[b, :(L + PAGE - 1) // PAGE].long()
        c, k = self.ckv[pages].flatten(0, 1)[:L], self.kr[pages].flatten(0, 1)[:L]
        seen = torch.cat([torch.ones(n, L - n, dtype=torch.bool), self.seen[b]], 1)
        at = sum(self.counts[:b])
        return tree_attention(self.q[at:at + n], c, k, self.scale, seen), slice(at, at + n)

    def check(self, o, lse, which=None):
        torch.cuda.synchronize()
        assert self.api.get_device_error() == 0
        for b in range(len(self.lens)) if which is None else which:
            if self.counts[b] == 0:
                continue
            ref, at = self.reference(b)
            check_tree(o[at], lse[at], ref, self.lens[b])


CASES = {
    "one token of one": dict(heads=128, counts=[1], lens=[1]),
    "context of zero": dict(heads=16, counts=[5, 64, 1], lens=[5, 64, 1]),
    "one head": dict(heads=1, counts=[3, 1], lens=[70, 129]),
    "rows straddle nodes": dict(heads=24, counts=[7, 13, 1], lens=[200, 64, 65]),
    "odd heads": dict(heads=5, counts=[33, 2], lens=[63, 1000]),
    "full rows": dict(heads=128, counts=[4, 1, 9], lens=[130, 700, 4097]),
    "idle sequences": dict(heads=16, counts=[0, 4, 0, 0, 3, 0], lens=[100, 77, 0, 640, 3, 0]),
    "trees past a page": dict(heads=16, counts=[100, 65, 31], lens=[163, 65, 96]),
    "largest tree": dict(heads=8, counts=[256, 255], lens=[256, 700]),
    "many sequences": dict(heads=32, counts=[1 + b % 5 for b in range(70)], lens=[5 + 37 * b for b in range(70)]),
    "long": dict(heads=16, counts=[8], lens=[20000]),
}


@pytest.mark.parametrize("dc", [512, 64])
@pytest.mark.parametrize("name", CASES)
def test_tree(api, name, dc):
    s = Step(api, dc=dc, seed=len(name), **CASES[name])
    s.check(*s.run())


@pytest.mark.parametrize("name", ["one token of one", "rows straddle nodes", "full rows", "trees past a page",
                                  "idle sequences", "long"])
def test_tree_e4m3(api, name):
    s = Step(api, fp8=True, seed=3, **CASES[name])
    s.check(*s.run())


@pytest.mark.parametrize("dc", [512, 64])
@pytest.mark.parametrize("parts", [1, 2, 3, 7, 74, 148, 400])
def test_tree_partition_counts(api, parts, dc):
    """Items shared by several partitions, partitions of several items, idle partitions."""
    s = Step(api, heads=48, counts=[9, 1, 0, 30], lens=[3000, 10, 64, 777], dc=dc, seed=parts)
    o, lse = s.run(num_parts=parts)
    s.check(o, lse)
    again = s.run(num_parts=parts)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("parts", [2, 3, 5, 11, 74])
def test_tree_blocks_that_start_inside_a_sequence(api, fp8, parts):
    """Several row blocks of long sequences: partitions whose segments start at any tile and wrap around,
    over the drafted tokens and the end of the sequence too."""
    s = Step(api, heads=128, counts=[9, 2, 12], lens=[3001, 777, 2100], seed=parts, fp8=fp8)
    o, lse = s.run(num_parts=parts)
    s.check(o, lse)
    again = s.run(num_parts=parts)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dc", [512, 64])
def test_tree_chain_is_the_chain_mask(api, dc):
    s = Step(api, heads=24, counts=[6, 1, 40], lens=[500, 64, 41], dc=dc, kind="chain")
    o, lse = s.run()
    s.check(o, lse)
    c = s.run(masks=None)
    assert torch.equal(o, c[0]) and torch.equal(lse, c[1])


@pytest.mark.parametrize("dc,heads", [(512, 64), (64, 32)])
def test_tree_of_two_agrees_with_the_causal_pair_decode(api, dc, heads):
    """A chain of two tokens is the two-query decode: the same sums, split and merged elsewhere."""
    s = Step(api, heads=heads, counts=[2] * 5, lens=[300, 2, 64, 65, 5000], dc=dc, kind="chain")
    o, lse = s.run(masks=None)
    d2 = api.make_dims(heads, 2, 128 if dc == 512 else 120, dc, s.dr, 128)
    parts = api.num_parts_for(d2, 100, "cuda")
    q = s.q.view(5, 2 * heads, -1)
    ws = api.decode_splitkv(q, s.ckv, s.kr, s.block_table, s.seq_lens, d2, parts)
    o2, lse2 = api.combine(ws, s.seq_lens, s.block_table.shape[1], d2, parts)
    s.check(o, lse)
    s.check(o2.reshape(o.shape), lse2.reshape(lse.shape))


@pytest.mark.parametrize("dc", [512, 64])
def test_tree_rows_that_see_nothing(api, dc):
    """No context and an empty mask: 0 and -inf; the others are as ever."""
    s = Step(api, heads=20, counts=[8, 6, 70], lens=[8, 900, 70], dc=dc)
    s.seen[0][2] = False
    s.seen[0][7] = False
    s.seen[1][:] = False      # sees the context alone
    s.seen[2][:] = False
    s.seen[2][69, 64] = True  # one row, one token of the second page
    s.check(*s.run())


@pytest.mark.parametrize("dc,fp8", [(512, False), (64, False), (512, True)])
@pytest.mark.parametrize("parts", [1, 5, None])
def test_tree_nothing_unseen_leaks(api, dc, fp8, parts):
    """NaN and infinities past the sequences' ends and in drafted tokens that rows do not see
    stay away from those rows; rows that see a NaN are NaN."""
    s = Step(api, heads=40, counts=[12, 70, 3], lens=[780, 130, 3], dc=dc, fp8=fp8, seed=5)
    clean = s.run(num_parts=parts)
    s.check(*clean)
    bad = {0: [3, 9], 1: [0, 64, 69], 2: [1]}
    nan, inf = float("nan"), float("inf")
    for b, L in enumerate(s.lens):
        ctx = L - s.counts[b]
        for j, i in enumerate(bad[b]):
            s.seen[b][:, i] = False   # ... and every row stops seeing these
            page, row = int(s.table[b, (ctx + i) // PAGE]), (ctx + i) % PAGE
            if fp8:
                s.codes[page, row, 7 + 300 * (j % 2)] = 0x7F   # the NaN code
                s.scales[page, row] = [0.01, inf, nan][j % 3]
            else:
                s.ckv[page, row, j::3] = [nan, inf, -inf][j % 3]
                s.ckv[page, row, dc - 1] = inf
            s.kr[page, row] = [inf, nan, -inf][j % 3]
        used = L % PAGE
        if used:
            page = int(s.table[b, L // PAGE])
            s.kr[page, used:] = nan
            if fp8:
                s.codes[page, used:] = 0xFF
                s.scales[page, used:] = inf
            else:
                s.ckv[page, used:] = nan
    if fp8:
        s.refresh()
    o, lse = s.run(num_parts=parts)
    s.check(o, lse)
    # a row that does see one is NaN, and no other changes
    s.seen[0][5, 3] = True
    o2, lse2 = s.run(num_parts=parts)
    torch.cuda.synchronize()
    assert torch.isnan(o2[5]).all() and torch.isnan(lse2[5]).all()
    keep = torch.arange(o.shape[0], device="cuda") != 5
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])


def test_tree_non_finite_queries_stay_in_their_rows(api):
    for dc in (512, 64):
        s = Step(api, heads=24, counts=[9, 4], lens=[200, 9], dc=dc)
        o, lse = s.run()
        s.q[3, 5] = float("nan")
        s.q[11, :, 2] = float("inf")
        o2, lse2 = s.run()
        torch.cuda.synchronize()
        keep = torch.ones(13, 24, dtype=torch.bool, device="cuda")
        keep[3, 5] = False
        keep[11] = False
        assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])
        assert torch.isnan(o2[3, 5]).all() and torch.isnan(lse2[3, 5])


@pytest.mark.parametrize("dc", [512, 64])
def test_tree_padded_batch_leaves_rows_behind_alone(api, dc):
    s = Step(api, heads=16, counts=[3, 0, 11], lens=[40, 1, 600], dc=dc, pad=5, max_nodes=64)
    o = torch.full((s.T, 16, dc), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T, 16), 7.0, device="cuda")
    s.q[-5:] = float("nan")
    s.run(o_lat=o, lse_out=lse)
    s.check(o[:-5], lse[:-5])
    assert (o[-5:] == 7).all() and (lse[-5:] == 7).all()


@pytest.mark.parametrize("dc", [512, 64])
def test_tree_views_of_one_pool(api, dc):
    s = Step(api, heads=16, counts=[5, 9], lens=[100, 333], dc=dc, fused_pool=True)
    s.check(*s.run())


def test_tree_large_scores(api):
    """Scores of some thousands: the running maximum moves by more than any threshold."""
    for dc in (512, 64):
        s = Step(api, heads=16, counts=[4, 20], lens=[500, 90], dc=dc)
        s.q *= 64
        s.check(*s.run())


def test_tree_offsets_past_32_bits(api):
    """Pages beyond 2^31 cache elements, and query rows and outputs beyond 2^31 elements."""
    s = Step(api, heads=16, counts=[6, 2], lens=[150, 64])
    pages = (1 << 31) // (64 * 512) + 7
    ckv = torch.zeros(pages, 64, 512, dtype=torch.bfloat16, device="cuda")
    kr = torch.zeros(pages, 64, 64, dtype=torch.bfloat16, device="cuda")
    old = s.block_table[s.block_table >= 0].long()
    new = pages - 1 - torch.arange(old.numel(), device="cuda")
    ckv[new], kr[new] = s.ckv[old], s.kr[old]
    o, lse = s.run()
    s.block_table[s.block_table >= 0] = new.int()
    s.ckv, s.kr = ckv, kr
    o2, lse2 = s.run()
    s.check(o2, lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    del ckv, kr, s
    B = (1 << 31) // (256 * 128 * 512) + 3
    s = Step(api, heads=128, counts=[256] * B, lens=[256 + b % 3 for b in range(B)], kind="chain")
    o, lse = s.run(masks=None)
    s.check(o, lse, which=[0, B - 2, B - 1])


def test_tree_bad_data_is_reported_and_skipped(api):
    """Lengths, token counts and page ids that do not fit: the device error, the other sequences right."""
    def fresh():
        return Step(api, heads=16, counts=[4, 5, 3], lens=[100, 80, 30])
    for what in ("short", "long", "negative", "wide", "past the end", "backwards", "page", "negative page"):
        s = fresh()
        ok = [0, 2]
        if what == "short":
            s.seq_lens[1] = 4
        elif what == "long":
            s.seq_lens[1] = s.block_table.shape[1] * 64 + 1
        elif what == "negative":
            s.seq_lens[1] = -7
        elif what == "wide":
            s.max_nodes = 4
            s.seen = [m[:, :4] for m in s.seen]
        elif what == "past the end":
            s.cu[3] = s.T + 1
            ok = [0, 1]
        elif what == "backwards":
            s.cu[2] = 2
            s.cu[3] = 2   # sequence 1: 4 .. 2, sequence 2: 2 .. 2
            ok = [0]
        elif what == "page":
            s.block_table[1, 0] = s.ckv.shape[0]
        else:
            s.block_table[1, 1] = -1
        o, lse = s.run()
        torch.cuda.synchronize()
        assert api.get_device_error() == 4, what
        assert api.get_device_error() == 0
        for b in ok:
            ref, at = s.reference(b)
            check_tree(o[at], lse[at], ref, s.lens[b])


@pytest.mark.parametrize("dc", [512, 64])
def test_tree_with_offsets_that_turn_back_is_not_run(api, dc):
    """Sequences that overlap, with more tokens together than q holds: the device error, nothing written."""
    s = Step(api, heads=16, counts=[40] + [0] * 79, lens=[64] * 80, dc=dc)
    s.cu = torch.tensor([40 * (b & 1) for b in range(81)], dtype=torch.int32, device="cuda")   # 40 x [0, 40)
    o = torch.full((s.T, 16, dc), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T, 16), 7.0, device="cuda")
    s.run(o_lat=o, lse_out=lse)
    torch.cuda.synchronize()
    assert api.get_device_error() == 4
    assert (o == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("dc", [512, 64])
def test_tree_without_tokens_or_sequences(api, dc):
    s = Step(api, heads=16, counts=[3], lens=[70], dc=dc)
    masks, kw = s.masks(), dict(max_nodes=s.max_nodes, dims=s.dims)
    i32 = dict(dtype=torch.int32, device="cuda")
    o, lse = api.decode_tree(s.q[:0], s.ckv, s.kr, s.block_table, s.seq_lens, torch.zeros(2, **i32), masks=masks[:0], **kw)
    assert o.shape == (0, 16, dc) and lse.shape == (0, 16)
    o = torch.full((s.T, 16, dc), 7.0, dtype=torch.bfloat16, device="cuda")
    api.decode_tree(s.q, s.ckv, s.kr, s.block_table[:0], s.seq_lens[:0], torch.zeros(1, **i32), masks=masks, o_lat=o, **kw)
    api.decode_tree(s.q, s.ckv, s.kr, s.block_table, s.seq_lens, torch.zeros(2, **i32), masks=masks, o_lat=o, **kw)
    assert (o == 7).all()
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def test_tree_captured_replayed_and_on_two_streams(api):
    """A captured step replayed on new lengths; two streams at once, each with its workspace."""
    a = Step(api, heads=64, counts=[6, 1, 9], lens=[900, 10, 300], seed=1)
    masks = a.masks()
    ws = api.alloc_tree_workspace(a.dims, "cuda")
    o = torch.empty(a.T, 64, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(a.T, 64, device="cuda")
    a.run(masks=masks, workspace=ws, o_lat=o, lse_out=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(masks=masks, workspace=ws, o_lat=o, lse_out=lse)
    a.lens = [333, 64, 12]
    a.seq_lens.copy_(torch.tensor(a.lens, dtype=torch.int32))
    o.zero_()
    graph.replay()
    a.check(o, lse)
    b = Step(api, heads=128, counts=[5] * 8, lens=[2000] * 8, seed=2)
    want_a, want_b = a.run(), b.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got.append((a.run(stream=streams[0]), b.run(stream=streams[1])))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], want_a[0]) and torch.equal(y[0], want_b[0])
        assert torch.equal(x[1], want_a[1]) and torch.equal(y[1], want_b[1])
    assert api.get_device_error() == 0


@pytest.mark.parametrize("dc,heads,fp8", [(512, 16, False), (512, 128, False), (64, 32, False), (512, 24, True)])
def test_tree_attend(api, dc, heads, fp8):
    """Both projections around the tree decode against fp64, in a padded step with a sequence that is skipped:
    rows that no sequence owns are 0 and -inf, whatever the memory held before."""
    s = Step(api, heads=heads, counts=[5, 4, 0, 9], lens=[300, 90, 64, 1100], dc=dc, pad=6, fp8=fp8, seed=heads)
    g = torch.Generator("cuda").manual_seed(7)
    dn, dv = (128 if dc == 512 else 120), 128
    q_c, q_r = _bf16(g, s.T, heads, dn), _bf16(g, s.T, heads, s.dr)
    q_c[-6:] = float("nan")           # rows behind the last sequence hold anything
    w_uk, w_uv = _bf16(g, heads, dn, dc, std=dc ** -0.5), _bf16(g, heads, dc, dv, std=dc ** -0.5)
    s.seq_lens[1] = -1                # does not fit: skipped
    masks, ws = s.masks(), api.alloc_tree_workspace(s.dims, "cuda")
    for shape, dtype in (((s.T, heads, dc), torch.bfloat16), ((s.T, heads), torch.float32)):
        junk = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(6)]
        del junk                      # what freshly allocated outputs may hold
    out, lse = api.tree_attend(q_c, q_r, s.codes if fp8 else s.ckv, s.kr, s.block_table, s.seq_lens, s.cu, w_uk, w_uv,
                               s.max_nodes, masks=masks, scales=s.scales if fp8 else None, workspace=ws)
    torch.cuda.synchronize()
    assert api.get_device_error() == 4
    assert out.shape == (s.T, heads, dv) and lse.shape == (s.T, heads)
    for rows in (slice(5, 9), slice(s.T - 6, s.T)):
        assert (out[rows] == 0).all() and (lse[rows] == -math.inf).all()
    for b in (0, 3):
        L, n, at = s.lens[b], s.counts[b], sum(s.counts[:b])
        pages = s.block_table[b, :(L + PAGE - 1) // PAGE].long()
        c, k = s.ckv[pages].flatten(0, 1)[:L], s.kr[pages].flatten(0, 1)[:L]
        q = torch.cat([torch.einsum("thd,hdc->thc", q_c[at:at + n].double(), w_uk.double()), q_r[at:at + n].double()], -1)
        seen = torch.cat([torch.ones(n, L - n, dtype=torch.bool), s.seen[b]], 1)
        o, l, A, size = tree_attention(q, c, k, s.scale, seen)
        w = w_uv.double()
        y = torch.einsum("thc,hcd->thd", o, w)
        # the absorbed query is rounded to bf16 (2^-8 of each value, so at most that of the sum of a score's
        # terms' magnitudes; 2^-9 more covers the fp32 sums): a weight is off by twice that; the weights, the
        # latent result and the output are rounded to bf16 as well
        ds = (2.0 ** -8 + 2.0 ** -9) * size
        bound = torch.einsum("thc,hcd->thd", (2 * ds[..., None] + 3 * 2.0 ** -8) * A, w.abs()) + 2.0 ** -8 * y.abs()
        got = out[at:at + n].double()
        assert ((got - y).abs() <= bound).all()
        assert ((lse[at:at + n].double() - l).abs() <= ds + 1e-4).all()
        assert (got - y).norm() / y.norm() <= 0.02     # independent roundings add as squares


@pytest.mark.parametrize("dc", [512, 64])
def test_tree_attend_into_given_outputs(api, dc):
    """The same bits as in outputs of its own; rows that no sequence owns keep what the buffers held, and the
    projection is made from it."""
    s = Step(api, heads=16, counts=[7, 2], lens=[400, 33], dc=dc, pad=3)
    g = torch.Generator("cuda").manual_seed(1)
    dn = 128 if dc == 512 else 120
    args = (_bf16(g, s.T, 16, dn), _bf16(g, s.T, 16, s.dr), s.ckv, s.kr, s.block_table, s.seq_lens, s.cu,
            _bf16(g, 16, dn, dc, std=dc ** -0.5), _bf16(g, 16, dc, 128, std=dc ** -0.5), s.max_nodes)
    masks = s.masks()
    want, want_lse = api.tree_attend(*args, masks=masks)
    o = torch.ones(s.T, 16, dc, dtype=torch.bfloat16, device="cuda")
    lse, out = torch.full((s.T, 16), 5.0, device="cuda"), torch.empty(s.T, 16, 128, dtype=torch.bfloat16, device="cuda")
    got, got_lse = api.tree_attend(*args, masks=masks, o_lat=o, lse_out=lse, out=out)
    assert got is out and got_lse is lse
    assert torch.equal(out[:-3], want[:-3]) and torch.equal(lse[:-3], want_lse[:-3])
    assert (o[-3:] == 1).all() and (lse[-3:] == 5).all() and (out[-3:] != 0).any()
    o.zero_()
    assert api.tree_attend(*args, masks=masks, o_lat=o, lse_out=lse, out=out)[0] is out and torch.equal(out, want)
    for bad in (dict(out=out[:-1]), dict(out=out.float()), dict(o_lat=o[:-1]), dict(lse_out=lse.double())):
        with pytest.raises(RuntimeError, match="MLA_ERR_INVALID_ARG"):
            api.tree_attend(*args, masks=masks, **bad)
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


def test_tree_attend_and_autograd(api):
    """The outputs that it is given, as those of the other calls: versions move, and none may require grad."""
    s = Step(api, heads=16, counts=[3], lens=[70], dc=64)
    g = torch.Generator("cuda").manual_seed(1)
    args = (_bf16(g, 3, 16, 120), _bf16(g, 3, 16, 8), s.ckv, s.kr, s.block_table, s.seq_lens, s.cu,
            _bf16(g, 16, 120, 64), _bf16(g, 16, 64, 128), s.max_nodes)
    kw = dict(o_lat=_bf16(g, 3, 16, 64), lse_out=torch.zeros(3, 16, device="cuda"), out=_bf16(g, 3, 16, 128))
    for t in args[-3:-1]:
        t.requires_grad_(True)        # weights may; the result takes no part in autograd
    before = {k: t._version for k, t in kw.items()}
    assert not any(t.requires_grad for t in api.tree_attend(*args, **kw))
    assert all(t._version > before[k] for k, t in kw.items())
    for k, t in kw.items():
        t.requires_grad_(True)
        with pytest.raises(RuntimeError, match="requires grad"):
            api.tree_attend(*args, **kw)
        with torch.no_grad():
            api.tree_attend(*args, **kw)
        t.requires_grad_(False)
    torch.cuda.synchronize()
    assert api.get_device_error() == 0


@pytest.mark.parametrize("dc,fp8", [(512, False), (64, False), (512, True)])
def test_tree_in_the_mean(api, dc, fp8):
    """What bounds per element cannot see: a loss that goes one way. The weights and the result are rounded to
    bf16 (rms at most 2^-8 / sqrt(3) of each value, independently: sqrt(2/3) 2^-8 of the norm together; a tenth more
    covers the fp32 sums), and roundings to nearest have no direction: the result's projection on the exact one is 1
    but for the mean of at least 10^4 of them (2^-8 / 100), a hundredth of what truncation would take."""
    s = Step(api, heads=32, counts=[16, 9, 30], lens=[2000, 4097, 600], dc=dc, fp8=fp8, seed=11)
    o, lse = s.run()
    torch.cuda.synchronize()
    assert api.get_device_error() == 0
    for b in range(3):
        (ro, rl, _, _), at = s.reference(b)
        got = o[at].double()
        assert (got - ro).norm() / ro.norm() <= 1.1 * math.sqrt(2 / 3) * 2.0 ** -8
        assert abs((got * ro).sum() / (ro * ro).sum() - 1) <= 2.0 ** -8 / 100
        assert abs((lse[at].double() - rl).mean()) <= 2.0 ** -16
