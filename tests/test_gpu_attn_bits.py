"""How many bits of a weight and of a query reach the attention's results, on
inputs where the results' own rounding does not hide it.

A query is one element (1) and the scale 1, so a score is one element of a
key and exact; a weight is then off by its parts' rounding (PART), by the
score's two products with rounded constants and the exponential (some 2^-20
for scores up to 4) and by the products' 32-bit sums (2^-22 of the sum of
magnitudes): REST = 2^-18 covers the last three.  The values of the heavy tokens
cancel in pairs, so that a result is far smaller than what it is a sum of.
"""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_gb300 as gdn

from attn_harness import E4M3, Pool, half_step

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TYPES = [(BF, BF), (HF, HF), (BF, E4M3), (HF, E4M3)]
REST = 2.0 ** -18


def part(act, kv):
    """Half a step of the parts that a weight is held in, and its error at least, relative to the largest weight."""
    if kv is E4M3:
        return 2.0 ** -13
    return 2.0 ** -16 if act is BF else 2.0 ** -20


def attend(pool, q, k, v, rows, scale=1.0, **scales):
    dims = gdn.AttnDims(q.shape[1], k.shape[1], q.shape[2], scale=scale)
    pages, dev = pool.dev(), lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    cache = {"k": k.cuda(), "v": v.cuda()} | {n: t.cuda() for n, t in scales.items()}
    out = torch.full(q.shape, -77.0, dtype=q.dtype, device="cuda")
    ws = torch.empty(gdn.attn_workspace_size(dims, pages, pool.S, q.shape[0]), dtype=torch.uint8, device="cuda")
    if rows == 1:
        gdn.attn_step(dims, cache, pages, dev(pool.slot), q.cuda(), out, ws)
    else:
        gdn.attn_window(dims, cache, pages, dev(pool.slot), dev(pool.row_ptr), q.cuda(), out, ws)
    assert gdn.get_device_error() == 0
    return out.double().cpu()


def place(pool, token, shape, kv, fill=0.0):
    """A pool that holds token[j] ([tokens, d]) at stream 0's tokens."""
    x = torch.full(shape, fill)
    at = pool.tokens(0)[: token.shape[0]]
    x[at // pool.page_size, 0, at % pool.page_size] = token.float()
    return x.to(kv)


@pytest.mark.parametrize("rows", [1, 3])   # the step kernel; with 16 heads of 3 rows the window kernel
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("act,kv", TYPES)
def test_weights_keep_their_bits(act, kv, d, rows):
    tokens, heavy, G = 333, 24, 16
    pool = Pool([tokens], [rows], 16)
    g = torch.Generator().manual_seed(d + rows)
    score = torch.full((tokens + rows,), -24.0)
    at = torch.randperm(tokens, generator=g)[:heavy]
    score[at] = torch.rand((heavy,), generator=g) * 3
    score = score.to(kv).double()
    q = torch.zeros((rows, G, d))
    q[..., 0] = 1.0
    keys = torch.zeros((tokens + rows, d), dtype=torch.float64)
    keys[:, 0] = score
    p = torch.exp(score)
    values = torch.zeros((tokens + rows, d), dtype=torch.float64)
    for e in range(d):   # (rounding the second value leaves a result of half a step of it)
        a, b = at[torch.randperm(heavy, generator=g)[:2]]
        values[a, e] = 1.0
        values[b, e] = float((-p[a] / p[b]).to(kv))
    shape = (pool.n_pages, 1, 16, d)
    out = attend(pool, q.to(act), place(pool, keys, shape, kv), place(pool, values, shape, kv), rows)
    for i in range(rows):
        w = p[: tokens + i + 1] / p[: tokens + i + 1].sum()
        ref, size = w @ values[: tokens + i + 1], w @ values[: tokens + i + 1].abs()
        bound = (part(act, kv) + REST) * size
        bound = bound + half_step(act) * (ref.abs() + bound) + (2.0 ** -25 if act is HF else 0.0)
        far = (out[i] - ref).abs()
        assert (far <= bound).all(), f"row {i}: {float((far / bound).max()):.3g} times the bound"


# over an 8-bit cache: (weights' and queries' errors at the least) relative to the power of two above the largest
# weight of a tile, and to the largest element of a query
LEAST = {1: (2.0 ** -26, 2.0 ** -21), 3: (2.0 ** -22, 2.0 ** -21)}


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("act", [BF, HF])
def test_small_weights_reach_the_sum(act, rows):
    """One key with nearly all the weight and a value of 0, and 126 with 2^-18 of it each and values that agree."""
    tokens, G, d = 127, 16, 64
    pool = Pool([tokens], [rows], 16)
    q = torch.zeros((rows, G, d))
    q[..., 0] = 1.5781   # times -8: 2^-18.2
    q = q.to(act)
    keys, values = torch.zeros((tokens + rows, d)), torch.zeros((tokens + rows, d))
    keys[1:, 0] = -8.0
    values[1:tokens] = torch.linspace(0.5, 2.0, d).to(E4M3).float()
    shape = (pool.n_pages, 1, 16, d)
    out = attend(pool, q, place(pool, keys, shape, E4M3), place(pool, values, shape, E4M3), rows)
    for i in range(rows):
        score = keys[: tokens + i + 1, 0].double() * q[0, 0, 0].double()
        w = torch.exp(score) / torch.exp(score).sum()
        ref = w @ values[: tokens + i + 1].double()
        bound = (2.0 ** -13 + REST) * ref + LEAST[rows][0] * values.double().sum(0)
        bound = bound + half_step(act) * (ref + bound) + (2.0 ** -25 if act is HF else 0.0)
        far = (out[i] - ref).abs()
        assert (far <= bound).all(), f"row {i}: {float((far / bound).max()):.3g} times the bound"


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("act", [BF, HF])
def test_small_elements_of_a_query_reach_the_scores(act, rows):
    """A query with one large element that meets zeros, and small ones (2^-17.4 of it) that decide."""
    tokens, G, d, large = 40, 16, 64, 1024.0
    pool = Pool([tokens], [rows], 16)
    small = torch.tensor(0.75 * 2.0 ** -10 * 8).to(act)
    q = torch.full((rows, G, d), float(small)).to(act)
    q[..., 0] = large
    g = torch.Generator().manual_seed(3)
    keys = torch.randint(-4, 5, (tokens + rows, 1), generator=g).float().expand(-1, d).clone()
    keys[:, 0] = 0.0
    values = torch.randn((tokens + rows, d), generator=g).to(E4M3).float()
    shape = (pool.n_pages, 1, 16, d)
    out = attend(pool, q, place(pool, keys, shape, E4M3), place(pool, values, shape, E4M3), rows)
    for i in range(rows):
        k, v = keys[: tokens + i + 1].double(), values[: tokens + i + 1].double()
        score = k @ q[0, 0].double()
        w = torch.softmax(score, 0)
        off = LEAST[rows][1] * large * float(k.abs().sum(1).max()) + 2.0 ** -22 * float((k.abs() @ q[0, 0].double().abs()).max())
        ref = w @ v
        bound = (2 * off + 2.0 ** -13 + REST) * (w @ v.abs())
        bound = bound + half_step(act) * (ref.abs() + bound)
        far = (out[i] - ref).abs()
        assert (far <= bound).all(), f"row {i}: {float((far / bound).max()):.3g} times the bound"


@pytest.mark.parametrize("rows,G", [(1, 4), (1, 16), (16, 8)])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("act", [BF, HF])
def test_infinite_committed_values_are_infinite_results(act, d, rows, G):
    """A weight is not 0, so an infinite value of a token that all rows see makes its element an infinity of that sign;
    both signs make it no number."""
    tokens = 500
    pool = Pool([tokens], [rows], 16)
    g = torch.Generator().manual_seed(d)
    shape = (pool.n_pages, 1, 16, d)
    q, k = torch.randn((rows, G, d), generator=g).to(act), torch.randn((tokens + rows, d), generator=g).to(act)
    v = torch.randn((tokens + rows, d), generator=g).to(act)
    clean = attend(pool, q, place(pool, k, shape, act), place(pool, v, shape, act), rows, scale=0.25)
    inf = float("inf")
    v[3, 1] = v[200, 2] = v[499, 2] = v[130, 4] = inf
    v[7, 3] = v[130, 5] = v[400, 4] = -inf
    out = attend(pool, q, place(pool, k, shape, act), place(pool, v, shape, act), rows, scale=0.25)
    # (an fp16 weight below 2^-39 of the largest of its 128 tokens may be 0)
    score = torch.einsum("rgd,td->rgt", q.double(), k.double()) * 0.25
    for e, at, sign in ((1, [3], inf), (2, [200, 499], inf), (3, [7], -inf), (5, [130], -inf)):
        held = torch.ones((rows, G), dtype=torch.bool)
        for t in at if act is HF else []:
            tile = score[..., t // 128 * 128:min(t // 128 * 128 + 128, tokens)]
            held &= score[..., t] - tile.amax(-1) > -38 * np.log(2.0)
        assert (out[..., e][held] == sign).all() and held.any() and not out[..., e].isfinite().any()
    assert out[..., 4].isnan().all()
    rest = [e for e in range(d) if e not in (1, 2, 3, 4, 5)]
    assert torch.equal(out[..., rest], clean[..., rest])
