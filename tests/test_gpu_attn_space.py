"""The attention calls' workspace: it grows with the pool's tokens, not with the table's
width, is enough however the tokens are divided, and tables that share pages say so."""
import numpy as np
import pytest
import torch

import gated_deltanet_speculative_gb300 as gdn

from test_gpu_attn import BF, E4M3, Round, dev

pytestmark = pytest.mark.gpu
SPACE = 128


def wide(pages, width):
    """The same streams in a table with room for `width` pages a row."""
    table = torch.full((pages["block_table"].shape[0], width), -1, dtype=torch.int32, device="cuda")
    table[:, : pages["block_table"].shape[1]] = pages["block_table"]
    return pages | {"block_table": table}


@pytest.mark.parametrize("lengths,rows", [([40000, 3, 200, 700], [16, 1, 9, 16]), ([5000] * 9, [16] * 9), ([1] * 200, [3] * 200),
                                          ([511, 512, 513, 8191, 8192, 8193, 1023, 1024] * 2, [1] * 16),
                                          ([60000], [1]), ([100] * 33 + [30000], [1] * 34)])
@pytest.mark.parametrize("hq", [1, 12, 16])
def test_a_wide_table_costs_nothing(lengths, rows, hq):
    r = Round(lengths, rows, d=64, hq=hq, hkv=1, page=64, step=max(rows) == 1)
    want, pages = r.run(), r.pool.dev()
    pages_wide = wide(pages, 1 << 14)   # a million tokens a row
    S, R = r.pool.S, r.q.shape[0]
    size = gdn.attn_workspace_size(r.dims, pages_wide, S, R)
    slot = 16 * hq * (64 * 4 + 16)      # an upper bound of a piece, a row of a table of a million tokens being 1032 of them
    tokens = r.pool.n_pages * 64
    assert size <= (1 << 20) + slot * ((16 if hq > 8 else 2) * (2 * S + tokens // 512 + 1) + 160 * 7)
    assert torch.equal(r.run(pages=pages_wide), want)
    r.check(want, streams=range(0, S, 17))


@pytest.mark.parametrize("kv", [BF, E4M3])
@pytest.mark.parametrize("rows", [1, 8])
def test_tables_that_share_pages_need_to_say_so(kv, rows):
    """24 streams with the same 20000 tokens in the same pages, and rows' pages of their own."""
    S, tokens, page = 24, 20000, 16
    r = Round([tokens] + [16] * (S - 1), [rows] * S, d=64, hq=2, hkv=1, kv=kv, page=page, step=rows == 1)
    p = r.pool
    common = tokens // page   # (20000 is a multiple of 16)
    wide_rows = np.full((p.n_slots, common + 2), -1, np.int32)
    for s in range(S):
        wide_rows[p.slot[s], :common] = p.block_table[p.slot[0], :common]
        wide_rows[p.slot[s], common] = p.block_table[p.slot[s], 1 if s else common]
    p.block_table, p.max_pages = wide_rows, common + 2
    p.lengths = [tokens] * S
    p.kv_len[p.slot], p.n_held[p.slot] = tokens, common + 1
    pages = p.dev()
    R = r.q.shape[0]
    few = gdn.attn_workspace_size(r.dims, pages, S, R)
    enough = gdn.attn_workspace_size(r.dims, pages, S, R, n_pages=S * (common + 1))
    assert few < enough
    out = r.run(check_error=SPACE, pages=pages, workspace=torch.empty(few, dtype=torch.uint8, device="cuda"))
    assert (out == -77.0).all()
    out = r.run(pages=pages, workspace=torch.empty(enough, dtype=torch.uint8, device="cuda"))
    r.check(out, streams=(0, 1, S - 1))
