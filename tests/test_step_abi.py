"""Host side of the packed-step operators (include/mla_step.h), without a GPU: refusals before
anything is launched, sizing helpers and the rotary frequencies."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

from mla_latent_kv_18_b200 import build as mla_build

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def b():
    mla_build.build()
    from mla_latent_kv_18_b200 import _binding
    return _binding


@pytest.fixture(scope="module")
def api(b):
    from mla_latent_kv_18_b200 import api as _api
    return _api


def _dims(b, **kw):
    d = dict(num_heads=16, n_q=1, d_nope=128, d_latent=512, d_rope=64, d_v=128, page_size=64, softmax_scale=0.0)
    d.update(kw)
    return b.MLADims(**d)


P = 4096   # a pointer that is never followed: every call here is refused on the host


def _tree(b, fp8=False, **kw):
    a = dict(dims=_dims(b), q=P, T=8, ckv=b.MLAPool(P, 64 * 512, 512), scales=P, kr=b.MLAPool(P, 64 * 64, 64), pages=4,
             table=P, max_pages=4, lens=P, cu=P, B=2, masks=P, nodes=8, parts=4, ws=P, ws_bytes=None, o=P, lse=P)
    a.update(kw)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = b.lib.mla_tree_workspace_bytes(a["dims"], max(1, a["parts"])) if a["dims"] else 0
    head = [a["dims"], a["q"], a["T"], a["ckv"]] + ([a["scales"]] if fp8 else [])
    rest = [a[k] for k in ("kr", "pages", "table", "max_pages", "lens", "cu", "B", "masks", "nodes", "parts", "ws",
                           "ws_bytes", "o", "lse")]
    return (b.lib.mla_decode_tree_fp8 if fp8 else b.lib.mla_decode_tree)(*head, *rest, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID),
    (dict(ws=None), INVALID), (dict(o=None), INVALID), (dict(q=P + 8), INVALID), (dict(ws=P + 16), INVALID),
    (dict(o=P + 4), INVALID), (dict(lse=P + 2), INVALID), (dict(masks=P + 1), INVALID), (dict(T=-1), INVALID),
    (dict(B=-1), INVALID), (dict(parts=0), INVALID), (dict(nodes=0), INVALID), (dict(nodes=257), INVALID),
    (dict(max_pages=0), INVALID), (dict(pages=0), INVALID), (dict(ws_bytes=100), INVALID),
    (dict(dims=None), INVALID), (dict(T=1 << 28), UNSUPPORTED), (dict(max_pages=1 << 30), UNSUPPORTED),
])
def test_tree_refusals(b, kw, status):
    assert _tree(b, **kw) == status


def test_tree_refuses_tables_past_31_bits(b):
    assert _tree(b, T=1, B=1, max_pages=(1 << 25) - 1) == UNSUPPORTED
    assert _tree(b, T=1, B=1, max_pages=1 << 27) == UNSUPPORTED


def test_tree_refuses_bad_pools_and_dims(b):
    assert _tree(b, ckv=b.MLAPool(P + 2, 64 * 512, 512)) == INVALID
    assert _tree(b, ckv=b.MLAPool(P, 64 * 512, 256)) == INVALID
    assert _tree(b, kr=b.MLAPool(P, 64 * 64, 60)) == INVALID
    for kw in (dict(d_latent=256), dict(page_size=32), dict(num_heads=129)):
        assert _tree(b, dims=_dims(b, **kw), ws_bytes=1 << 40) == UNSUPPORTED
    assert _tree(b, fp8=True, scales=None, ckv=b.MLAPool(P, 64 * 512, 512)) == INVALID
    assert _tree(b, fp8=True, ckv=b.MLAPool(P, 64 * 512, 500)) == INVALID
    small = _dims(b, d_latent=64, d_rope=8, d_nope=120)
    assert _tree(b, fp8=True, dims=small, ckv=b.MLAPool(P, 64 * 64, 64), kr=b.MLAPool(P, 64 * 8, 8)) == UNSUPPORTED


def test_tree_nothing_to_do_is_ok(b):
    assert _tree(b, B=0) == 0 and _tree(b, T=0) == 0


def test_tree_sizing(b):
    d = _dims(b)
    assert b.lib.mla_tree_num_parts(d, 148) == 74
    assert b.lib.mla_tree_num_parts(_dims(b, d_latent=64, d_rope=8, n_q=999), 148) == 148
    assert b.lib.mla_tree_num_parts(_dims(b, num_heads=129), 148) == 0
    assert b.lib.mla_tree_workspace_bytes(d, 74) == 2 * 74 * 128 * 513 * 4 + 74 * 16
    assert b.lib.mla_tree_workspace_bytes(d, 0) == 0


def _plan(b, **kw):
    a = dict(cached=P, new=2 * P, B=2, free=3 * P, num_free=10, head=4 * P, table=5 * P, max_pages=4, parents=6 * P,
             nodes=8, T=8, seq_lens=7 * P, cu=8 * P, ids=9 * P, pos=10 * P, slots=11 * P, masks=12 * P, head_out=13 * P)
    a.update(kw)
    return b.lib.mla_step_plan(*[a[k] for k in ("cached", "new", "B", "free", "num_free", "head", "table", "max_pages",
                                                "parents", "nodes", "T", "seq_lens", "cu", "ids", "pos", "slots",
                                                "masks", "head_out")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(cached=None), INVALID), (dict(new=None), INVALID), (dict(head=None), INVALID), (dict(table=None), INVALID),
    (dict(free=None), INVALID), (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(masks=None), INVALID),
    (dict(head_out=4 * P), INVALID), (dict(seq_lens=P), INVALID), (dict(seq_lens=2 * P), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(max_pages=0), INVALID), (dict(nodes=0), INVALID),
    (dict(nodes=257), INVALID), (dict(slots=11 * P + 4), INVALID), (dict(B=16385), UNSUPPORTED),
])
def test_plan_refusals(b, kw, status):
    assert _plan(b, **kw) == status


def _rot(b, x=None, y=None, dtype=0, T=4, width=64, offset=0, rot=64, pos=P, freq=P, mscale=1.0, layout=0, inverse=0,
         **kw):
    t = dict(src=P, out=P, in_token=1024, in_head=64, out_token=1024, out_head=64, heads=16)
    t.update(kw)
    return b.lib.mla_rotary(x or b.MLARotaryTensor(**t), y, dtype, T, width, offset, rot, pos, freq, mscale, layout,
                            inverse, None)


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=7), dict(rot=66), dict(offset=-1), dict(offset=2), dict(width=0), dict(dtype=3),
    dict(layout=2), dict(pos=None), dict(freq=None), dict(mscale=math.inf), dict(src=None), dict(out=None),
    dict(src=P + 1, out=P + 1), dict(out_token=512), dict(heads=-1), dict(heads=65537), dict(T=-1),
    dict(rot=4098, width=5000), dict(freq=P + 4)])
def test_rotary_refusals(b, kw):
    assert _rot(b, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(out_token=0), dict(out_head=0), dict(src=2 * P, out_token=0)])
def test_rotary_refuses_outputs_that_fall_together(b, kw):
    assert _rot(b, **kw) == INVALID
    y = b.MLARotaryTensor(src=P, out=2 * P, in_token=0, in_head=0, out_token=64, out_head=0, heads=2)
    assert _rot(b, y=y) == INVALID


def test_rotary_refuses_rows_too_wide(b):
    assert _rot(b, heads=1024, width=32768, rot=64) == UNSUPPORTED


def test_rotary_nothing_to_do_is_ok(b):
    assert _rot(b, T=0) == 0 and _rot(b, heads=0) == 0


def _append(b, fp8=False, **kw):
    a = dict(dims=_dims(b), ckv=P, ckv_stride=512, kr=P, kr_stride=64, slots=P, pos=P, freq=P, mscale=1.0, layout=0,
             T=4, pool=b.MLAPool(P, 64 * 512, 512), scales=P, krpool=b.MLAPool(P, 64 * 64, 64), pages=4)
    a.update(kw)
    args = [a[k] for k in ("dims", "ckv", "ckv_stride", "kr", "kr_stride", "slots", "pos", "freq", "mscale", "layout",
                           "T", "pool")] + ([a["scales"]] if fp8 else []) + [a["krpool"], a["pages"], None]
    return (b.lib.mla_append_kv_slots_fp8 if fp8 else b.lib.mla_append_kv_slots)(*args)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [
    dict(ckv=None), dict(kr=None), dict(slots=None), dict(freq=None), dict(ckv=P + 8), dict(ckv_stride=510),
    dict(ckv_stride=256), dict(kr_stride=32), dict(layout=5), dict(T=-1), dict(pages=0), dict(slots=P + 4),
    dict(mscale=math.nan), dict(dims=None), dict(pool=None), dict(krpool=None)])
def test_append_refusals(b, fp8, kw):
    assert _append(b, fp8, **kw) == INVALID
    assert _append(b, fp8, T=0) == 0


def test_append_refuses_other_pages(b):
    assert _append(b, dims=_dims(b, page_size=32)) == UNSUPPORTED
    assert _append(b, True, scales=None) == INVALID


# ------------------------------------------------------------------ frequencies

def _want(rot, theta, scaling, s, trained, fast, slow):
    out = []
    base = theta * s ** (rot / (rot - 2)) if scaling == "ntk" else theta
    n = lambda beta: rot * math.log(trained / (2 * math.pi * beta)) / (2 * math.log(theta))  # noqa: E731
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= s
        if scaling == "yarn":
            lo, hi = max(math.floor(n(fast)), 0), min(math.ceil(n(slow)), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = r * f / s + (1 - r) * f
        out.append(f)
    return out, (0.1 * math.log(s) + 1 if scaling == "yarn" and s > 1 else 1.0)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,theta,s,trained", [(64, 10000.0, 40.0, 4096), (8, 10000.0, 1.0, 2048),
                                                 (18, 5e5, 8.0, 8192), (4, 1.5, 2.0, 64)])
def test_rope_frequencies(api, scaling, rot, theta, s, trained):
    f, m = api.rope_frequencies(rot, theta, scaling, s, trained)
    want, wm = _want(rot, theta, scaling, s, trained, 32.0, 1.0)
    # a power, a division and a blend in fp64: a few units of 2^-53 times the exponent's size
    assert torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=2.0 ** -45, atol=0)
    assert abs(m - wm) <= 2.0 ** -50


def test_yarn_keeps_fast_pairs_and_stretches_slow_ones(api):
    plain, _ = api.rope_frequencies(64)
    yarn, m = api.rope_frequencies(64, scaling="yarn", factor=40.0, original_max=4096)
    assert torch.equal(yarn[:8], plain[:8]) and m > 1
    assert torch.allclose(yarn[-4:], plain[-4:] / 40, rtol=1e-14)


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(theta=1.0), dict(theta=math.inf),
                                dict(factor=0.5), dict(factor=math.nan), dict(scaling="longrope"),
                                dict(rot_dim=2, scaling="ntk"), dict(scaling="yarn", original_max=0),
                                dict(scaling="yarn", beta_fast=0.0), dict(scaling="yarn", beta_slow=math.inf)])
def test_rope_frequencies_refusals(api, b, kw):
    a = dict(rot_dim=64, theta=10000.0, scaling="none", factor=2.0)
    a.update(kw)
    with pytest.raises(b.MLAError):
        api.rope_frequencies(**a)


def test_python_entry_points_refuse_cpu_tensors_and_wrong_shapes(api, b):
    dims = _dims(b)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(b.MLAError):
        api.step_plan(i32(2), i32(2), i32(4), i32(1), i32(2, 4), 8)
    with pytest.raises(b.MLAError):
        api.step_plan(i32(3), i32(2), i32(4), i32(1), i32(2, 4), 8)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    for kw in (dict(), dict(layout="neox"), dict(out=x[:1])):
        with pytest.raises(b.MLAError):
            api.rotary(x, i32(2), f, **kw)
    with pytest.raises(b.MLAError):
        api.rotary(x.double(), i32(2), f)
    q = torch.zeros(8, 16, 576, dtype=torch.bfloat16)
    ckv, kr = torch.zeros(4, 64, 512, dtype=torch.bfloat16), torch.zeros(4, 64, 64, dtype=torch.bfloat16)
    for kw in (dict(), dict(masks=i32(8, 2)), dict(masks=i32(7, 1))):
        with pytest.raises(b.MLAError):
            api.decode_tree(q, ckv, kr, i32(2, 4), i32(2), i32(3), dims, 8, **kw)
    with pytest.raises(b.MLAError):
        api.append_kv_slots(ckv[0], kr[0], torch.zeros(64, dtype=torch.int64), ckv, kr, dims)
    with pytest.raises(b.MLAError):
        api.append_kv_slots(ckv[0], kr[0], i32(64), ckv, kr, dims)


def test_streams_of_another_device_are_refused(api, b):
    """`stream` has to be one of the tensors' device (the check comes before anything else)."""
    class Stream:
        device = torch.device("cuda", 1)
    s, x = Stream(), torch.zeros(2, 4, 64)
    i32 = torch.zeros(2, 4, dtype=torch.int32)
    for call in (lambda: api.rotary(x, i32, x, stream=s),
                 lambda: api.step_plan(i32, i32, i32, i32, i32, 8, stream=s),
                 lambda: api.append_kv_slots(x, x, i32, x, x, None, stream=s),
                 lambda: api.append_kv_slots_fp8(x, x, i32, x, x, x, None, stream=s),
                 lambda: api.decode_tree(x, x, x, i32, i32, i32, None, 8, stream=s),
                 lambda: api.decode_tree_fp8(x, x, x, x, i32, i32, i32, None, 8, stream=s),
                 lambda: api.tree_attend(x, x, x, x, i32, i32, i32, x, x, 8, stream=s)):
        with pytest.raises(b.MLAError, match="stream of cuda:1, tensors on cpu"):
            call()


def test_tree_attend_refuses_cpu_tensors(api, b):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(b.MLAError):
        api.tree_attend(z(8, 16, 128), z(8, 16, 64), z(4, 64, 512), z(4, 64, 64), i32(2, 4), i32(2), i32(3),
                        z(16, 128, 512), z(16, 512, 128), 8)


def test_rotary_tensor_struct_matches_the_header(b):
    assert ctypes.sizeof(b.MLARotaryTensor) == 56


def test_the_other_calls_run_without_the_compiled_binding(b):
    """A library without its binding of the packed-step calls: they fail loudly, decode and prefill are there."""
    code = """
import sys
sys.modules['mla_latent_kv_18_b200._step'] = None    # an import of it fails
import torch
from mla_latent_kv_18_b200 import api
d = api.make_dims(16, 1, 128, 512, 64, 128)
assert api.workspace_bytes(d, 2, 4) > 0 and api.route(1, 16) == "absorb" and api._b.lib.mla_tree_num_parts(d, 148) == 74
assert api.rope_frequencies(8)[1] == 1.0
z = torch.zeros(2, 2, 8)
calls = (lambda: api.step_plan(z, z, z, z, z, 8), lambda: api.rotary(z, z, z),
         lambda: api.append_kv_slots(z, z, z, z, z, d), lambda: api.append_kv_slots_fp8(z, z, z, z, z, z, d),
         lambda: api.decode_tree(z, z, z, z, z, z, d, 8), lambda: api.decode_tree_fp8(z, z, z, z, z, z, z, d, 8))
for call in calls:
    try:
        call()
    except ImportError as e:
        assert "_step.so" in str(e) and "mla_latent_kv_18_b200.build" in str(e), e
    else:
        raise AssertionError("ran")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)
