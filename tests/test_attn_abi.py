"""The attention entry points without a GPU: refusals of bad arguments on
the host, before any CUDA call (fake addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import gated_deltanet_speculative_gb300 as gdn
from gated_deltanet_speculative_gb300 import _binding as B

A16, MIS = 0x10000, 0x10002
R = ctypes.byref


def parts(**over):
    d = B.c_attn_dims(24, 4, 256, 64, 0, 0, 0, 0.0625, 1.0, 0.0, 1e-6)
    w = B.c_attn_weights(A16, A16, A16)
    c = B.c_attn_cache(A16, A16, None, None)
    g = B.c_pages(A16, A16, A16, A16, A16, 4, 32, 100, 16)
    r = B.c_attn_rows(A16, A16, A16, A16, 6144, 256, 1024, 256, 1024, 256)
    for k, v in over.items():
        hit = [x for x in (d, w, c, g, r) if hasattr(x, k)]
        assert hit, k
        for x in hit[:1]:
            setattr(x, k, v)
    return d, w, c, g, r


def step(d, w, c, g, r, slot=A16, n=2, q=A16, out=A16, ws=A16, ws_bytes=1 << 40):
    return gdn.load().gdn_attn_step(R(d), R(c), R(g), slot, n, q, out, ws, ws_bytes, None)


def prep(d, w, c, g, r, pos=A16, place=A16, n=2):
    return gdn.load().gdn_attn_prep(R(d), R(w), R(c), R(g), R(r), pos, place, n, None)


@pytest.mark.parametrize("field,value", [
    ("n_q_heads", 0), ("n_q_heads", 23), ("n_q_heads", 4 * 17), ("n_kv_heads", 0), ("d_head", 96), ("d_head", 512),
    ("d_rot", 8), ("d_rot", 272), ("d_rot", -16), ("rot_style", 2), ("act_type", 2), ("kv_type", 1), ("kv_type", 3),
    ("scale", float("inf")), ("rot_gain", float("nan")), ("norm_offset", float("inf")), ("eps", -1.0),
    ("page_size", 8), ("page_size", 48), ("page_size", 2048), ("n_slots", 0), ("max_pages", 0), ("n_pages", 0),
    ("n_pages", 1 << 27), ("max_pages", 1 << 27)])
def test_bad_geometry_is_einval(field, value):
    p = parts(**{field: value})
    assert step(*p) == -1
    if field not in ("n_slots", "max_pages"):
        assert prep(*p) == -1
    if field not in ("n_slots", "max_pages", "n_pages", "page_size"):
        return
    g = p[3]
    assert gdn.load().gdn_pages_plan(R(g), A16, A16, None, 2, 4, A16, A16, None) == -1
    assert gdn.load().gdn_pages_release(R(g), A16, 2, None) == -1


def test_bad_counts_are_einval():
    lib = gdn.load()
    p = parts()
    d, w, c, g, r = p
    for n in (0, -1, 65536):
        assert step(*p, n=n) == -1
        assert lib.gdn_pages_plan(R(g), A16, A16, None, n, 4, A16, A16, None) == -1
        assert lib.gdn_pages_commit(R(g), A16, A16, None, A16, n, 4, None) == -1
        assert lib.gdn_pages_release(R(g), A16, n, None) == -1
        assert lib.gdn_attn_commit(R(d), R(c), R(g), A16, A16, A16, A16, n, 4, None) == -1
        assert lib.gdn_attn_workspace_size(R(d), R(g), n, 4) == 0
    assert lib.gdn_attn_window(R(d), R(c), R(g), A16, A16, 2, 0, A16, A16, A16, 1 << 40, None) == -1
    assert prep(*p, n=0) == -1
    assert prep(*parts(q_row=6140)) == -1
    assert prep(*parts(v_head=-8)) == -1
    assert step(*parts(k_scale=A16)) == -1     # scales belong to 8-bit caches


def test_missing_pointers_are_enull():
    lib = gdn.load()
    p = parts()
    d, w, c, g, r = p
    assert step(*p, slot=None) == -2 and step(*p, q=None) == -2 and step(*p, out=None) == -2
    for f in ("block_table", "kv_len", "k", "v"):
        over = parts()
        setattr(over[2] if f in ("k", "v") else over[3], f, None)
        assert step(*over) == -2
    for f in ("n_held", "free_pages", "n_free"):
        g2 = parts(**{f: None})[3]
        assert lib.gdn_pages_plan(R(g2), A16, A16, None, 2, 4, A16, A16, None) == -2
        assert lib.gdn_pages_release(R(g2), A16, 2, None) == -2
    assert prep(*p, pos=None) == -2 and prep(*p, place=None) == -2
    assert prep(*parts(q_out=None)) == -2 and prep(*parts(inv_freq=None)) == -2
    assert lib.gdn_attn_window(R(d), R(c), R(g), A16, None, 2, 4, A16, A16, A16, 1 << 40, None) == -2
    assert lib.gdn_attn_tree(R(d), R(c), R(g), A16, A16, None, 2, 4, A16, A16, A16, 1 << 40, None) == -2
    assert lib.gdn_attn_commit(R(d), R(c), R(g), A16, A16, None, A16, 2, 4, None) == -2
    assert lib.gdn_attn_commit(R(d), R(c), R(g), A16, A16, A16, None, 2, 4, None) == -2
    assert lib.gdn_pages_commit(R(g), A16, A16, None, None, 2, 4, None) == -2
    assert lib.gdn_pages_plan(R(g), A16, A16, None, 2, 4, None, A16, None) == -2
    assert lib.gdn_attn_step(None, R(c), R(g), A16, 2, A16, A16, A16, 1 << 40, None) == -2
    assert lib.gdn_attn_step(R(d), None, R(g), A16, 2, A16, A16, A16, 1 << 40, None) == -2
    assert lib.gdn_attn_step(R(d), R(c), None, A16, 2, A16, A16, A16, 1 << 40, None) == -2


def test_misaligned_pointers_are_ealign():
    lib = gdn.load()
    p = parts()
    d, w, c, g, r = p
    assert step(*p, q=A16 + 8) == -3 and step(*p, out=MIS) == -3 and step(*p, slot=MIS) == -3
    assert step(*p, ws=A16 + 8) == -3
    for f in ("k_norm", "inv_freq", "q_out"):
        assert prep(*parts(**{f: MIS})) == -3
    assert prep(*p, pos=MIS) == -3
    assert step(*parts(block_table=MIS)) == -3
    assert lib.gdn_pages_plan(R(g), A16, MIS, None, 2, 4, A16, A16, None) == -3
    assert lib.gdn_attn_tree(R(d), R(c), R(g), A16, A16, MIS, 2, 4, A16, A16, A16, 1 << 40, None) == -3
    assert lib.gdn_attn_commit(R(d), R(c), R(g), A16, A16, A16, MIS, 2, 4, None) == -3


def test_workspace_is_checked():
    p = parts()
    need = gdn.load().gdn_attn_workspace_size(R(p[0]), R(p[3]), 2, 2)
    assert need > 0
    assert step(*p, ws=None) == -5
    assert step(*p, ws_bytes=need - 1) == -5


def test_attn_dims_refuse_unknown_layouts_and_types():
    with pytest.raises(ValueError):
        gdn.AttnDims(8, 2, 128, rot="spiral")
    d = gdn.AttnDims(8, 2, 128)
    with pytest.raises(TypeError):
        d.c(torch.float32)
    with pytest.raises(TypeError):
        d.c(torch.bfloat16, torch.int8)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    d = gdn.AttnDims(8, 2, 128)
    z = torch.zeros(2, dtype=torch.int32)
    pages = {"block_table": torch.zeros(2, 4, dtype=torch.int32), "kv_len": z, "n_held": z, "free_pages": z,
             "n_free": z[:1], "page_size": 16}
    with pytest.raises(ValueError):
        gdn.pages_plan(pages, z, torch.zeros(3, dtype=torch.int32), z, z)
    with pytest.raises(ValueError):
        B._strided(torch.zeros(2, 8, 128).transpose(1, 2), "q", torch.float32, (2, 128, 8))
    with pytest.raises(TypeError):
        B._attn_cache(d, {"k": torch.zeros(2, 2, 16, 128), "v": None}, 2, 16)


@pytest.mark.parametrize("d_rot", [16, 64, 128])
def test_inv_freq_schemes(d_rot):
    import math
    half = d_rot // 2
    plain = gdn.attn_inv_freq(d_rot, 10000.0, device="cpu")
    assert plain.dtype is torch.float64 and plain.shape == (half,)
    assert plain[0] == 1.0
    assert abs(float(plain[1]) - 10000.0 ** (-2.0 / d_rot)) < 1e-15
    assert torch.equal(gdn.attn_inv_freq(d_rot, factor=4.0, device="cpu"), plain / 4)
    ntk = gdn.attn_inv_freq(d_rot, ntk=8.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(plain[-1] / ntk[-1]) - 8.0) < 1e-9
    yarn = gdn.attn_inv_freq(d_rot, yarn=(16.0, 4096, 32, 1), device="cpu")
    assert torch.all(yarn <= plain) and torch.all(yarn >= plain / 16)
    turns = plain * 4096 / (2 * math.pi)
    inside = torch.arange(half)
    lo = max(math.floor(d_rot * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000.0))), 0)
    hi = min(math.ceil(d_rot * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000.0))), half - 1)
    assert torch.equal(yarn[inside <= lo], plain[inside <= lo])
    assert torch.allclose(yarn[inside >= hi], plain[inside >= hi] / 16, rtol=1e-12)
    assert torch.all(turns[inside < lo] > 32) and torch.all(turns[inside > hi] < 1)


def test_the_count_of_held_pages_is_needed_where_tokens_are_looked_up():
    lib = gdn.load()
    d, w, c, g, r = p = parts(n_held=None)
    assert step(*p) == -2
    assert lib.gdn_attn_commit(R(d), R(c), R(g), A16, A16, A16, A16, 2, 4, None) == -2
    assert lib.gdn_pages_commit(R(g), A16, A16, None, A16, 2, 4, None) == -2
    p = parts(n_held=MIS)
    assert step(*p) == -3


def test_the_wait_limit_hook_bounds_its_polls():
    lib = gdn.load()
    assert lib.gdn_debug_attn_wait_limit((1 << 20) + 1) == -1
    assert lib.gdn_debug_attn_wait_limit(5) == 0 and lib.gdn_debug_attn_wait_limit(1 << 20) == 0


@pytest.mark.parametrize("d_rot,base,trained,fast,slow", [(64, 10000.0, 131072, 32, 1), (128, 10000.0, 1 << 20, 32, 1),
                                                          (64, 10000.0, 4096, 32, 1), (64, 1e6, 32768, 32, 1),
                                                          (16, 500.0, 131072, 64, 2)])
def test_yarn_divides_only_pairs_that_turn_too_seldom(d_rot, base, trained, fast, slow):
    """A pair that turns r times within the trained length is divided by the factor as the ramp between the pairs of
    `fast` and `slow` turns says; one that turns more than `slow` times is never divided by all of it."""
    import math
    by = 4.0
    plain = base ** (-2.0 * torch.arange(d_rot // 2, dtype=torch.float64) / d_rot)
    yarn = gdn.attn_inv_freq(d_rot, base, yarn=(by, trained, fast, slow), device="cpu")
    turns = plain * trained / (2 * math.pi)
    # the pair that turns r times: base^(-2i/d_rot) trained / 2 pi = r
    at = [d_rot / 2 * math.log(trained / (2 * math.pi * r)) / math.log(base) for r in (fast, slow)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d_rot - 1)
    for i in range(d_rot // 2):
        share = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        want = float(plain[i]) * ((1 - share) + share / by)
        assert abs(float(yarn[i]) - want) < 1e-12 * want
        if turns[i] > slow and hi < d_rot - 1 and at[1] != math.ceil(at[1]):
            assert yarn[i] > plain[i] / by * (1 + 1e-9)


def test_the_workspace_does_not_grow_with_the_table_where_the_pool_is_small():
    size = lambda **over: gdn.load().gdn_attn_workspace_size(R(parts()[0]), R(parts(**over)[3]), 16, 256)  # noqa: E731
    narrow = size(max_pages=512, n_pages=2000)
    assert narrow == size(max_pages=1 << 16, n_pages=2000) > 0
    assert size(max_pages=1 << 16, n_pages=1 << 20) > 20 * narrow
    # 16 streams of a million tokens each, 24 heads on 4 of 256: pieces of 96 columns, 1032 a key head and stream
    assert size(max_pages=1 << 16, n_pages=1 << 20) < 1.01 * (96 * 1024 + 1024) * (4 * 16 * 1040 + 160 * 7)
