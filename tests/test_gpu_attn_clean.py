"""What stands behind a stream's last token (NaN here) is taken out of its last
tile once the tile is there, however late it comes: items of several tiles in
one run, heads of 256 elements (two pieces a tile, four to six places for
them), caches that come from memory."""
import pytest
import torch

from test_gpu_attn import BF, HF, E4M3, Round

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,rows", [(256, 8, 1), (256, 32, 1), (256, 16, 16), (256, 12, 16), (256, 4, 16), (128, 16, 16)])
@pytest.mark.parametrize("act,kv", [(BF, BF), (HF, HF), (BF, E4M3)])
def test_last_tiles_that_come_late(act, kv, d, hq, rows):
    r = Round([700, 90, 3, 1500, 385, 257] * 40, [rows] * 240, d=d, act=act, kv=kv, hq=hq, hkv=2, page=64, step=rows == 1)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")   # twice the L2
    first = None
    for i in range(12):
        flush.fill_(i)
        out = r.run()
        first = out if first is None else first
        assert torch.isfinite(out).all() and torch.equal(out, first)
    r.check(first, streams=range(0, 240, 17))
