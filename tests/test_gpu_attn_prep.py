"""attn_prep against its definition in 64 bits: norms, both rotation layouts,
part of the head, far positions, both row types, both cache types, strided
inputs, rows without a place."""
import numpy as np
import pytest
import torch

import gated_deltanet_speculative_gb300 as gdn

from attn_harness import E4M3, check, half_step, prep_ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def inputs(R, hq, hkv, d, act, seed, gate=False):
    g = torch.Generator().manual_seed(seed)
    per_q = 2 if gate else 1     # q's heads may stand between those of an output gate
    x = torch.randn((R, (per_q * hq + 2 * hkv) * d), generator=g).to(act)
    q, k, v = x.split([per_q * hq * d, hkv * d, hkv * d], 1)
    q = q.view(R, hq, per_q * d)[..., :d]
    return x, q, k.view(R, hkv, d), v.view(R, hkv, d), g


def run(R=5, hq=6, hkv=2, d=128, d_rot=None, style="half", act=BF, kv=None, page=16, far=5000, norm="both",
        offset=0.0, gain=1.0, scales=True, seed=1, gate=False, in_place=False, skip=(), lowest=0):
    kv = kv or act
    d_rot = d if d_rot is None else d_rot
    x, q, k, v, g = inputs(R, hq, hkv, d, act, seed, gate)
    w = {n: (torch.randn((d,), generator=g) * 0.2 + 1 - offset).to(act) if norm in ("both", n[0]) else None
         for n in ("q_norm", "k_norm")}
    inv = gdn.attn_inv_freq(d_rot, 1e6, device="cpu") if d_rot else torch.zeros(0, dtype=torch.float64)
    pos = torch.randint(lowest, far, (R,), generator=g).to(torch.int32)
    n_pages = -(-R // page) + 1
    place = torch.randperm(n_pages * page, generator=g)[:R].to(torch.int32)
    for r in skip:
        place[r] = -1
    ks = vs = None
    if kv is E4M3 and scales:
        ks, vs = torch.rand((hkv,), generator=g) * 0.1 + 0.02, torch.rand((hkv,), generator=g) + 0.1
    xc = x.cuda()
    per_q = 2 if gate else 1
    qc, kc, vc = xc.split([per_q * hq * d, hkv * d, hkv * d], 1)
    qc = qc.view(R, hq, per_q * d)[..., :d]
    if in_place:
        qc = qc.contiguous()
    rows = {"q": qc, "k": kc.view(R, hkv, d), "v": vc.view(R, hkv, d),
            "q_out": qc if in_place else torch.full((R, hq, d), float("nan"), dtype=act, device="cuda")}
    cache = {n: torch.zeros((n_pages, hkv, page, d), device="cuda").to(kv) for n in ("k", "v")}
    if ks is not None:
        cache["k_scale"], cache["v_scale"] = ks.cuda(), vs.cuda()
    dims = gdn.AttnDims(hq, hkv, d, d_rot=d_rot, rot=style, norm_offset=offset, rot_gain=gain)
    wc = {n: None if t is None else t.cuda() for n, t in w.items()}
    wc["inv_freq"] = inv.cuda()
    gdn.attn_prep(dims, wc, cache, rows, pos.cuda(), place.cuda())
    assert gdn.get_device_error() == 0
    arithmetic = (d + 40) * 2.0 ** -24
    ref, size = prep_ref(q, w["q_norm"], pos, inv, style, gain, offset)
    check(rows["q_out"], ref, arithmetic * size, act, "q")
    for name, t, weight, sc in (("k", k, w["k_norm"], ks), ("v", v, None, vs)):
        ref, size = prep_ref(t, weight, pos, inv if name == "k" else torch.zeros(0, dtype=torch.float64), style, gain, offset)
        if sc is not None:
            ref, size = ref / sc.double()[:, None], size / sc.double()[:, None]
        if kv is E4M3:
            ref = ref.clamp(-448, 448)
        got = cache[name].float().cpu().transpose(1, 2).reshape(-1, hkv, d)
        there = torch.zeros(n_pages * page, dtype=torch.bool)
        keep = place >= 0
        there[place[keep].long()] = True
        assert not got[~there].any(), f"{name}: written outside its rows' places"
        check(got[place[keep].long()], ref[keep], arithmetic * size[keep], kv, name)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("act,kv", [(BF, BF), (HF, HF), (BF, E4M3), (HF, E4M3)])
def test_prep(d, style, act, kv):
    run(d=d, style=style, act=act, kv=kv)


@pytest.mark.parametrize("d,d_rot", [(64, 0), (64, 16), (64, 48), (128, 32), (128, 112), (256, 64), (256, 16), (256, 240)])
@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_part_of_the_head(d, d_rot, style):
    run(d=d, d_rot=d_rot, style=style)


def test_far_and_negative_positions():
    run(far=2 ** 31 - 1, lowest=2 ** 31 - 4000, act=HF)
    run(far=0, lowest=-3000, act=HF, style="interleaved")
    run(far=1, lowest=0)


@pytest.mark.parametrize("norm", ["both", "q", "k", "none"])
def test_norms_left_out(norm):
    run(norm=norm)


def test_offset_gain_and_no_scales():
    run(offset=1.0, gain=1.2)
    run(kv=E4M3, scales=False)


@pytest.mark.parametrize("R,page", [(1, 16), (2, 1024), (1000, 64), (33, 16)])
def test_row_counts(R, page):
    run(R=R, page=page, hq=3, hkv=1)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 1), (5, 5), (64, 8)])
def test_head_counts(hq, hkv):
    run(hq=hq, hkv=hkv, d=64)


def test_strided_and_in_place_queries():
    run(gate=True)
    run(in_place=True)


def test_rows_without_a_place():
    run(R=6, skip=(0, 3))


def test_place_out_of_range_is_refused():
    R, hq, hkv, d = 3, 2, 1, 64
    x, q, k, v, g = inputs(R, hq, hkv, d, BF, 3)
    cache = {n: torch.zeros((1, hkv, 16, d), dtype=BF, device="cuda") for n in ("k", "v")}
    rows = {"q": q.contiguous().cuda(), "k": k.contiguous().cuda(), "v": v.contiguous().cuda(),
            "q_out": torch.full((R, hq, d), float("nan"), dtype=BF, device="cuda")}
    dims = gdn.AttnDims(hq, hkv, d, d_rot=0)
    gdn.attn_prep(dims, {}, cache, rows, torch.zeros(R, dtype=torch.int32, device="cuda"),
                  torch.tensor([16, -2, 4], dtype=torch.int32, device="cuda"))
    assert gdn.get_device_error() == 64
    assert torch.equal(rows["q_out"], rows["q"])
    got = cache["v"][0, 0]
    assert torch.equal(got[4], rows["v"][2, 0]) and not got[:4].any() and not got[5:].any()


def test_nan_and_infinity_stay_what_they_are():
    R, hq, hkv, d = 2, 1, 1, 64
    x, q, k, v, g = inputs(R, hq, hkv, d, BF, 4)
    v = v.clone()
    v[0, 0, 3], v[0, 0, 5], v[0, 0, 6] = float("nan"), float("inf"), -float("inf")
    for kv in (BF, E4M3):
        cache = {n: torch.zeros((1, hkv, 16, d), device="cuda").to(kv) for n in ("k", "v")}
        rows = {"q": q.contiguous().cuda(), "k": k.contiguous().cuda(), "v": v.cuda(),
                "q_out": torch.empty((R, hq, d), dtype=BF, device="cuda")}
        gdn.attn_prep(gdn.AttnDims(hq, hkv, d, d_rot=0), {}, cache, rows,
                      torch.zeros(R, dtype=torch.int32, device="cuda"),
                      torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
        got = cache["v"].float()[0, 0, 0]
        assert torch.isnan(got[3])
        top = 448.0 if kv is E4M3 else float("inf")
        assert got[5] == top and got[6] == -top
    assert gdn.get_device_error() == 0


def test_prepared_call_in_a_graph():
    R, hq, hkv, d = 4, 4, 2, 128
    x, q, k, v, g = inputs(R, hq, hkv, d, BF, 5)
    dims = gdn.AttnDims(hq, hkv, d)
    w = {"q_norm": torch.ones(d, dtype=BF, device="cuda"), "k_norm": None, "inv_freq": gdn.attn_inv_freq(d)}
    pos = torch.arange(R, dtype=torch.int32, device="cuda")
    out = []
    for graph in (False, True):
        cache = {n: torch.zeros((1, hkv, 16, d), dtype=BF, device="cuda") for n in ("k", "v")}
        rows = {"q": q.contiguous().cuda(), "k": k.contiguous().cuda(), "v": v.contiguous().cuda(),
                "q_out": torch.zeros((R, hq, d), dtype=BF, device="cuda")}
        call = gdn.prepare(gdn.attn_prep, dims, w, cache, rows, pos, pos)
        if graph:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                call()
            gr.replay()
        else:
            call()
        torch.cuda.synchronize()
        out.append((rows["q_out"], cache["k"], cache["v"]))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_a_page_of_more_than_two_to_the_31_elements():
    """Key heads whose place in their page passes 31 bits (8-bit cache, one page of 2.1 GB each for k and v)."""
    R, heads, d, page = 2, 8200, 256, 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((R, heads, d), generator=g, device="cuda").to(BF) for _ in range(3))
    cache = {n: torch.zeros((1, heads, page, d), dtype=torch.uint8, device="cuda").view(E4M3) for n in ("k", "v")}
    place = torch.tensor([3, 1023], dtype=torch.int32, device="cuda")
    gdn.attn_prep(gdn.AttnDims(heads, heads, d, d_rot=0), {}, cache, {"q": q, "k": k, "v": v, "q_out": torch.empty_like(q)},
                  torch.zeros(R, dtype=torch.int32, device="cuda"), place)
    assert gdn.get_device_error() == 0
    for name, x in (("k", k), ("v", v)):
        raw = cache[name].view(torch.uint8)[0]
        want = x.float().to(E4M3).view(torch.uint8)
        for r, at in enumerate(place.tolist()):
            assert torch.equal(raw[:, at], want[r]), name
            raw[:, at] = 0
        assert not raw.any(), name


def test_far_angles_to_the_last_bits():
    """Near the last position, where a pair is almost back at its start: the sine is then far smaller than what an
    angle made of 53 bits would be off by."""
    from fractions import Fraction
    import math
    half, d = 32, 64
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    rng = np.random.default_rng(7)
    inv = np.sort(rng.uniform(0.05, 1.0, half))[::-1].copy()
    p = np.arange(2 ** 31 - 65536, 2 ** 31, dtype=np.uint64)
    pos, want = [], []
    for f in inv.tolist():
        turn = int(Fraction(f) / (2 * pi) * 2 ** 64) % 2 ** 64
        off = (p * np.uint64(turn)).astype(np.int64)          # of a whole turn, 2^-64 of it each
        at = int(p[np.argmin(np.abs(off.astype(np.float64)))])
        part = Fraction(f) * at / (2 * pi)
        part -= round(part)
        pos.append(at)
        want.append(math.sin(float(2 * pi * part)))
    x = torch.zeros((half, 1, d), dtype=BF, device="cuda")
    x[..., :half] = 1.0                                       # (1, 0) turns to (cos, sin)
    rows = {"q": x, "k": x, "v": x, "q_out": torch.empty_like(x)}
    cache = {n: torch.zeros((1, 1, 64, d), dtype=BF, device="cuda") for n in ("k", "v")}
    gdn.attn_prep(gdn.AttnDims(1, 1, d), {"inv_freq": torch.from_numpy(inv).cuda()}, cache, rows,
                  torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.arange(half, dtype=torch.int32, device="cuda"))
    assert gdn.get_device_error() == 0
    got = torch.diagonal(rows["q_out"][:, 0, half:]).double().cpu()
    want = torch.tensor(want, dtype=torch.float64)
    # bf16's half step, the turn's 2^-64 and its upper 32 bits, and some 2^-21 of fp32
    bound = want.abs() * (half_step(BF) + 2.0 ** -20) + 2 * math.pi * (2.0 ** -33 + 2.0 ** -32)
    far = (got - want).abs()
    assert (far <= bound).all(), f"{float((far / bound).max()):.3g} times the bound"
