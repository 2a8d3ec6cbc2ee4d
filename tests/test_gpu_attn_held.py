"""A slot's table row may name pages that are no longer the slot's (entries behind
n_held stay as they were): no call reads, moves or counts tokens there."""
import numpy as np
import pytest
import torch

import gated_deltanet_speculative_gb300 as gdn

pytestmark = pytest.mark.gpu
INT = dict(dtype=torch.int32, device="cuda")
PAGES = 64


def dev(x):
    return torch.tensor(np.asarray(x), **INT)


class Reused:
    """Slot 0 gave its 5 pages back, slot 1 took all 8 there are, and slot 0 is used again with none left."""

    def __init__(self, hq=4, hkv=2, d=64):
        self.pages = {"block_table": torch.full((2, 8), -1, **INT), "kv_len": torch.zeros(2, **INT), "n_held": torch.zeros(2, **INT),
                      "free_pages": torch.arange(8, **INT), "n_free": torch.full((1,), 8, **INT), "page_size": 16}
        self.dims = gdn.AttnDims(hq, hkv, d)
        g = torch.Generator().manual_seed(1)
        self.cache = {n: torch.randn((8, hkv, 16, d), generator=g).to(torch.bfloat16).cuda() for n in ("k", "v")}
        self.row = lambda n: torch.randn((n, hq, d), generator=g).to(torch.bfloat16).cuda()
        assert self.plan([0], [70]) == 0
        gdn.pages_release(self.pages, dev([0]))
        assert self.plan([1], [120]) == 0
        gdn.pages_commit(self.pages, dev([1]), dev([0, 120]), dev([119]), n_rows=120)
        assert gdn.get_device_error() == 0 and int(self.pages["n_free"]) == 0
        assert (self.pages["block_table"][0, :5] >= 0).all()   # pages of slot 1 now

    def plan(self, slots, rows, parent=None):
        n = int(sum(rows))
        pos, self.place = torch.full((n,), -9, **INT), torch.full((n,), -9, **INT)
        gdn.pages_plan(self.pages, dev(slots), dev(np.concatenate([[0], np.cumsum(rows)])), pos, self.place, parent=parent)
        return gdn.get_device_error()


def test_a_reused_slot_without_pages_is_refused():
    r = Reused()
    slots, ptr, parent, keep = dev([0, 1]), dev([0, 4, 8]), dev([-1, 0, 0, 2] * 2), dev([3, -1])
    assert r.plan([0, 1], [4, 4], parent) == PAGES
    assert r.place[:4].tolist() == [-1] * 4 and (r.place[4:] >= 0).all()
    before = {n: t.clone() for n, t in r.cache.items()}
    q = r.row(8)
    ws = torch.empty(gdn.attn_workspace_size(r.dims, r.pages, 2, 8), dtype=torch.uint8, device="cuda")
    for tree in (False, True):
        out = torch.full_like(q, -77.0)
        if tree:
            gdn.attn_tree(r.dims, r.cache, r.pages, slots, ptr, parent, q, out, ws)
        else:
            gdn.attn_window(r.dims, r.cache, r.pages, slots, ptr, q, out, ws)
        assert gdn.get_device_error() == PAGES
        assert (out[:4] == -77.0).all() and torch.isfinite(out[4:]).all() and (out[4:] != -77.0).all()
    out = torch.full_like(q[:2], -77.0)
    gdn.attn_step(r.dims, r.cache, r.pages, slots, q[:2], out, ws)
    assert gdn.get_device_error() == PAGES and (out[0] == -77.0).all() and (out[1] != -77.0).any()
    gdn.attn_commit(r.dims, r.cache, r.pages, slots, ptr, parent, keep)
    assert gdn.get_device_error() == PAGES
    assert all(torch.equal(t, before[n]) for n, t in r.cache.items())
    for p in (parent, None):
        gdn.pages_commit(r.pages, slots, ptr, keep, n_rows=8, parent=p)
        assert gdn.get_device_error() == PAGES
        assert r.pages["kv_len"].tolist() == [0, 120]


@pytest.mark.parametrize("held", [-1, 9, 7])
def test_a_count_of_held_pages_out_of_range_or_too_small_is_refused(held):
    r = Reused()
    r.pages["n_held"][1] = held
    q = r.row(1)
    out = torch.full_like(q, -77.0)
    ws = torch.empty(gdn.attn_workspace_size(r.dims, r.pages, 1, 1), dtype=torch.uint8, device="cuda")
    gdn.attn_step(r.dims, r.cache, r.pages, dev([1]), q, out, ws)
    assert gdn.get_device_error() == PAGES and (out == -77.0).all()
    gdn.pages_commit(r.pages, dev([1]), dev([0, 1]), dev([0]), n_rows=1)
    assert gdn.get_device_error() == PAGES and int(r.pages["kv_len"][1]) == 120
